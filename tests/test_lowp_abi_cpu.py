"""The 8-bit and mixture-of-experts entry points on the host: refusals,
argument positions and quick returns, with no GPU work (made-up addresses;
calls that could reach a launch run with the GPUs hidden)."""
import ctypes

import pytest

import fp32_gemm_tile_amd as fg

from test_abi_cpu import run_without_gpu


def quant(type=0, block=0, M=4, N=4, X=16, ldx=4, Q=16, ldq=16, S=16, lds=4, QT=0, ldqt=0, ST=0,
          ldst=0):
    return fg.fg_quantize_fp8(type, block, M, N, X, ldx, Q, ldq, S, lds, QT, ldqt, ST, ldst)


@pytest.mark.parametrize("kw,bad", [
    (dict(type=2), 1), (dict(type=-1), 1), (dict(block=2), 2), (dict(M=-1), 3), (dict(N=-1), 4),
    (dict(X=0), 5), (dict(X=18), 5), (dict(type=1, X=17), 5), (dict(ldx=3), 6), (dict(Q=0), 7),
    (dict(Q=24), 7), (dict(ldq=20), 8), (dict(N=20, ldx=20, ldq=16), 8), (dict(S=0), 9),
    (dict(S=18), 9), (dict(lds=3), 10), (dict(QT=24, ldqt=16, ST=16, ldst=4), 11),
    (dict(QT=16, ldqt=8, ST=16, ldst=4), 12), (dict(M=20, lds=20, QT=16, ldqt=16, ST=16, ldst=4), 12),
    (dict(QT=16, ldqt=16, ST=0, ldst=4), 13), (dict(QT=16, ldqt=16, ST=16, ldst=3), 14),
    (dict(block=1, M=300, lds=2), 10),
])
def test_quantize_refusals(kw, bad):
    assert quant(**kw) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


def test_quantize_quick_returns_and_limits():
    assert quant(M=0) == fg.FG_OK and quant(N=0) == fg.FG_OK
    assert quant(ldq=fg.FG_MAX_LD + 16) == fg.FG_ERR_UNSUPPORTED
    assert quant(M=(1 << 30) + 1, lds=1 << 31) == fg.FG_ERR_UNSUPPORTED
    run_without_gpu("""
st = fg.fg_quantize_fp8(0, 1, 300, 4, 16, 4, 16, 16, 16, 3)
assert st in NO_DEVICE, st
st = fg.fg_quantize_fp8(1, 0, 1, 4, 18, 4, 0, 0, 0, 0, 16, 16, 16, 4)
assert st in NO_DEVICE, st
""")


def gemm(M=4, N=4, K=4, alpha=1.0, A=16, lda=16, SA=16, ldsa=4, B=16, ldb=16, SB=16, ldsb=4,
         block=0, beta=0.0, C=16, ldc=4, tc=0, ws=0, wb=0):
    return fg.fg_gemm_fp8(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, block, beta, C, ldc,
                          tc, ws, wb)


@pytest.mark.parametrize("kw,bad", [
    (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(A=0), 5), (dict(A=24), 5),
    (dict(lda=24), 6), (dict(K=20), 6), (dict(SA=0), 7), (dict(ldsa=3), 8), (dict(B=0), 9),
    (dict(B=8), 9), (dict(ldb=8), 10), (dict(SB=0), 11), (dict(ldsb=3), 12), (dict(block=2), 13),
    (dict(C=0), 15), (dict(C=18), 15), (dict(ldc=3), 16), (dict(tc=2), 17), (dict(ws=24), 18),
    (dict(block=1, N=300, ldc=300, ldsb=2), 12),
])
def test_gemm_refusals(kw, bad):
    assert gemm(**kw) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


def test_gemm_quick_returns_and_limits():
    assert gemm(M=0, A=0, C=0) == fg.FG_OK and gemm(N=0, B=0, C=0) == fg.FG_OK
    assert gemm(K=0, A=0, B=0, SA=0, SB=0, beta=1.0) == fg.FG_OK
    assert gemm(alpha=0.0, A=0, B=0, SA=0, SB=0, beta=1.0) == fg.FG_OK
    assert gemm(lda=fg.FG_MAX_LD + 16) == fg.FG_ERR_UNSUPPORTED
    assert gemm(ldc=fg.FG_MAX_LD + 4) == fg.FG_ERR_UNSUPPORTED
    assert fg.fg_gemm_fp8_workspace_size(0, 4, 4) == 0
    assert fg.fg_gemm_fp8_workspace_size(1, 1 << 31, 4) == 0
    for M, N, K in ((1, 1024, 1024), (33, 200, 8192), (517, 2047, 3001), (8192, 8192, 8192)):
        assert fg.fg_gemm_fp8_workspace_size(M, N, K) % (4 * M * N) == 0
    run_without_gpu("""
for kw in (dict(K=0, beta=0.5), dict(alpha=0.0), dict()):
    K, alpha, beta = kw.get("K", 4), kw.get("alpha", 1.0), kw.get("beta", 0.0)
    st = fg.fg_gemm_fp8(4, 4, K, alpha, 16, 16, 16, 4, 16, 16, 16, 4, 0, beta, 16, 4, 0)
    assert st in NO_DEVICE, (kw, st)
""")


def layer(T=2, E=4, k=2, H=32, I=16, ty=0, wt=0, act=3, ren=1, x=16, ldx=32, gate=None, up=None,
          down=None, router=16, ldr=32, rt=0, ids=16, w=16, out=16, ldo=32):
    m = lambda r, c: fg.fg_experts(16, c, r * c, 16, 1, 1)
    return fg.fg_moe_layer(T, E, k, H, I, ty, wt, act, ren, x or None, ldx, gate or m(I, H),
                           up or m(I, H), down or m(H, I), router or None, ldr, rt, ids or None,
                           w or None, out or None, ldo)


E = fg.fg_experts


@pytest.mark.parametrize("kw,bad", [
    (dict(T=-1), 1), (dict(T=65), 1), (dict(E=0), 2), (dict(E=513), 2), (dict(k=0), 3),
    (dict(k=5), 3), (dict(E=64, k=17), 3), (dict(H=0), 4), (dict(I=0), 5), (dict(ty=2), 6),
    (dict(wt=3), 7), (dict(act=4), 8), (dict(act=-1), 8), (dict(ren=2), 9), (dict(x=0), 10),
    (dict(x=18), 10), (dict(ldx=31), 11), (dict(gate=E(0, 32, 512, 0, 0, 0)), 12),
    (dict(gate=E(16, 31, 512, 0, 0, 0)), 12), (dict(gate=E(24, 32, 512, 0, 0, 0)), 12),
    (dict(up=E(16, 33, 528, 0, 0, 0)), 13), (dict(up=E(16, 32, 514, 0, 0, 0)), 13),
    (dict(down=E(16, 16, -16, 0, 0, 0)), 14), (dict(wt=2, down=E(16, 16, 512, 0, 1, 1)), 14),
    (dict(wt=2, H=256, ldx=256, ldo=256, ldr=256, down=E(16, 16, 4096, 16, 1, 1)), 14),
    (dict(router=18), 15), (dict(ldr=31), 16), (dict(rt=2), 17), (dict(ids=0), 18),
    (dict(w=0), 19), (dict(out=0), 20), (dict(out=18), 20), (dict(ldo=31), 21),
])
def test_moe_refusals(kw, bad):
    assert fg.fg_moe(layer(**kw), 16, 1 << 30) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


def test_moe_workspace_and_quick_returns():
    need = fg.fg_moe_workspace_size(2, 2, 4, 32, 16)
    assert need > 0
    assert fg.fg_moe(layer(), 0, 1 << 30) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 22
    assert fg.fg_moe(layer(), 24, 1 << 30) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 22
    assert fg.fg_moe(layer(), 16, need - 1) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 23
    assert fg.fg_moe(None, 16, need) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_moe(layer(T=0, x=0, ids=0, w=0, out=0), 0, 0) == fg.FG_OK
    assert fg.fg_moe_workspace_size(65, 2, 4, 32, 16) == 0
    assert fg.fg_moe_workspace_size(2, 5, 4, 32, 16) == 0
    big = fg.FG_MAX_LD + 16
    assert fg.fg_moe(layer(gate=E(16, big, 16 * big, 0, 0, 0)), 16, need) == fg.FG_ERR_UNSUPPORTED
    assert ctypes.sizeof(fg.fg_experts) == 48


def test_moe_valid_call_stops_at_the_device_check():
    run_without_gpu("""
m = lambda r, c: fg.fg_experts(16, c, r * c, None, 0, 0)
l = fg.fg_moe_layer(2, 4, 2, 32, 16, 0, 0, 3, 1, 16, 32, m(16, 32), m(16, 32), m(32, 16), None, 0,
                    0, 16, 16, 16, 32)
st = fg.fg_moe(l, 16, fg.fg_moe_workspace_size(2, 2, 4, 32, 16))
assert st in NO_DEVICE, st
""")


def test_torch_layer_checks_need_no_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        fg.quantize_fp8(x)
    with pytest.raises(ValueError, match="GPU"):
        fg.gemm_fp8(None, None, None, None, x)
    with pytest.raises(ValueError, match="GPU"):
        fg.moe(x, None, None, None, None, None, None)
    q, s = fg.empty_fp8(5, 130, "tile", device="cpu")
    assert q.shape == (5, 130) and q.stride() == (144, 1) and s.shape == (2, 1)
    q, s = fg.empty_fp8(5, 130, device="cpu")
    assert s.shape == (2, 5)
