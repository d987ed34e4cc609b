"""Quantisation to block-scaled e4m3 and the product of two such matrices, on
the GPU, against the binary64 oracle (oracle/lowp.py)."""
import numpy as np
import pytest

import fp32_gemm_tile_amd as fg
from oracle import lowp

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fg.load_library()
    yield
    torch.cuda.synchronize()


def codes_buffer(rows, cols, fill=0xAA, extra=0):
    """Device bytes [rows, wide] with rows at multiples of 16, and the view of
    the codes."""
    import torch
    wide = -(-max(1, cols) // 16) * 16 + extra
    base = torch.full((rows, wide), fill, dtype=torch.uint8, device="cuda")
    return base, base[:, :cols]


def device_codes(codes, extra=16):
    """Codes on the device; everything else in their rows is NaN codes."""
    import torch
    base, view = codes_buffer(*codes.shape, fill=NAN_CODE, extra=extra)
    view.copy_(torch.from_numpy(codes))
    return view


def device_scales(s, extra=3):
    import torch
    base = torch.full((s.shape[0], s.shape[1] + extra), float("nan"), device="cuda")
    view = base[:, :s.shape[1]]
    view.copy_(torch.from_numpy(s))
    return view


def make_x(rng, R, C, dtype, pad=0):
    """(device view with row stride C + pad, the same values as float32)."""
    import torch
    x = rng.standard_normal((R, C + pad)).astype(np.float32) * np.exp(
        2 * rng.standard_normal((1, C + pad))).astype(np.float32)
    t = torch.from_numpy(x).to("cuda").to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return t[:, :C], t[:, :C].float().cpu().numpy()


def check_quant(x_dev, x, block, ways=("n", "t")):
    import torch
    R, C = x.shape
    tall = 1 if block == "row" else 128
    bufs, args = {}, []
    for way, r, c in (("n", R, C), ("t", C, R)):
        if way in ways:
            base, q = codes_buffer(r, c, extra=16)
            s = torch.full((lowp.cdiv(c, 128), lowp.cdiv(r, tall) + 2), -1.0, device="cuda")
            bufs[way] = (base, q, s)
            args += [q, s[:, :lowp.cdiv(r, tall)]]
        else:
            args += [None, None]
    print("  quantize", R, C, x_dev.dtype, x_dev.stride(0), block, ways, flush=True)
    fg.quantize_fp8(x_dev, *args, block=block)
    torch.cuda.synchronize()
    for way, (base, q, s) in bufs.items():
        want, ws = lowp.quantize(x if way == "n" else x.T, tall)
        np.testing.assert_array_equal(s[:, :ws.shape[1]].cpu().numpy(), ws)
        assert (s[:, ws.shape[1]:] == -1).all()
        got = q.cpu().numpy()
        nan = (want & 0x7F) == NAN_CODE
        np.testing.assert_array_equal((got & 0x7F) == NAN_CODE, nan)
        np.testing.assert_array_equal(got[~nan], want[~nan])
        assert (base[:, q.shape[1]:] == 0xAA).all()      # bytes past the codes


SIZES = [(1, 1), (1, 128), (1, 4096), (5, 130), (127, 129), (128, 128), (300, 257), (33, 1000),
         (257, 64), (640, 384)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ways", ["n", "t", "nt"])
def test_quantize_bit_exact(block, dtype, ways):
    rng = np.random.default_rng(1)
    for R, C in SIZES:
        x_dev, x = make_x(rng, R, C, dtype, pad=0 if R % 2 else 5)
        check_quant(x_dev, x, block, ways)


@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_special_values(block):
    """NaN and infinities, a block of zeros, values of the smallest and the
    largest size, negative zero."""
    import torch
    rng = np.random.default_rng(2)
    x = rng.standard_normal((260, 390)).astype(np.float32)
    x[0, 3], x[1, 200], x[2, 380] = np.nan, np.inf, -np.inf
    x[3, :] = 0
    x[:, 7] = -0.0
    x[130:258, 128:256] = 0
    x[4] *= np.float32(1e-38)
    x[5, :128] = np.float32(1e-45)
    x[6, 256:384] = np.float32(3.4e38)
    x[7, :128], x[8] = np.nan, np.inf
    x[9, 128:140] = 3e38
    check_quant(torch.from_numpy(x).cuda(), x, block)


def test_quantize_next_to_the_middle_of_two_codes():
    """x = s * middle where that is exact, and one unit in the last place to
    either side, for scales whose significand is short and long."""
    import torch
    mid = (lowp.MAGNITUDES[1:] + lowp.MAGNITUDES[:-1]) / 2
    rows = []
    for top in (448.0, 448.0 * 1.25, 448.0 * (1 + 2.0 ** -12), 3.0e-36, 1.0, 7.7e30, 0.3333):
        s = max(np.float32(np.float32(top) / 448.0), np.float32(2.0 ** -126))
        v = (mid * np.float64(s)).astype(np.float32)
        for w in (v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf)), -v):
            rows.append(np.concatenate([w, [np.float32(top), 0]]).astype(np.float32))
    x = np.stack(rows)
    assert x.shape[1] == 128
    check_quant(torch.from_numpy(x).cuda(), x, "row")


def test_quantize_every_bfloat16():
    import torch
    bits = np.arange(65536, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80].reshape(-1, 128)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    xf = x.float().cpu().numpy()
    check_quant(x, xf, "row", "n")
    rng = np.random.default_rng(5)
    mixed = xf.reshape(-1)[rng.permutation(xf.size)].reshape(xf.shape)
    check_quant(torch.from_numpy(mixed).cuda().to(torch.bfloat16), mixed, "row", "n")


# ---- product -----------------------------------------------------------------

def make_operand(rng, R, C, tall, spread=1.0):
    x = rng.standard_normal((R, C)).astype(np.float32) * np.exp(
        spread * rng.standard_normal((1, C))).astype(np.float32)
    return lowp.quantize(x, tall)


def run_gemm(A, SA, B, SB, tall, out="f32", alpha=1.0, beta=0.0, C0=None, ws="full", pad=0,
             offset=0):
    """C as float32, from fg.gemm_fp8, with guard columns checked."""
    import torch
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    dt = torch.float32 if out == "f32" else torch.bfloat16
    flat = torch.full((M * (N + pad) + offset + 8,), float("nan"), dtype=dt, device="cuda")
    base = flat[offset:offset + M * (N + pad)].view(M, N + pad)
    base.fill_(7.0)
    C = base[:, :N]
    C.copy_(torch.from_numpy(C0)) if C0 is not None else C.fill_(float("nan"))
    need = fg.fg_gemm_fp8_workspace_size(M, N, K)
    w = None
    if ws == "full" and need:
        w = torch.full((need // 4 + 4,), float("nan"), device="cuda")[:need // 4]
    elif ws == "half" and need:
        w = torch.full((max(4, need // 8),), float("nan"), device="cuda")
    print("  gemm", M, N, K, tall, out, alpha, beta, ws, pad, offset, flush=True)
    fg.gemm_fp8(device_codes(A), device_scales(SA), device_codes(B), device_scales(SB), C,
                alpha=alpha, beta=beta, workspace=w)
    torch.cuda.synchronize()
    if pad:
        assert (base[:, N:] == 7.0).all()
    assert torch.isnan(flat[offset + M * (N + pad):]).all()
    return C.float().cpu().numpy()


def check_gemm(A, SA, B, SB, tall, out="f32", alpha=1.0, beta=0.0, C0=None, **kw):
    import torch
    if C0 is not None and out == "bf16":
        C0 = torch.from_numpy(C0).to(torch.bfloat16).float().numpy()
    got = run_gemm(A, SA, B, SB, tall, out, alpha, beta, C0, **kw)
    want, bound = lowp.product(A, SA, B, SB, tall, alpha, beta,
                               C0.astype(np.float64) if C0 is not None else None,
                               narrow=out == "bf16")
    if out == "bf16":
        bound = bound + lowp.bf16_half_step(np.abs(want) + bound)
    err = np.abs(got - want)
    assert (err <= bound).all(), (float((err / np.maximum(bound, 1e-300)).max()),
                                  np.argwhere(~(err <= bound))[:5])
    return got


GEMM_SIZES = [(1, 1, 1), (3, 5, 7), (1, 130, 128), (2, 1024, 1024), (17, 33, 129), (16, 300, 515),
              (33, 64, 2048), (64, 64, 64), (63, 257, 4100), (65, 129, 257), (129, 257, 1000),
              (200, 300, 640), (300, 520, 272)]


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm_against_oracle(tall, out):
    rng = np.random.default_rng(10)
    for n, (M, N, K) in enumerate(GEMM_SIZES):
        A, SA = make_operand(rng, M, K, 1)
        B, SB = make_operand(rng, N, K, tall)
        beta = (0.0, 0.5, 1.0)[n % 3]
        C0 = rng.standard_normal((M, N)).astype(np.float32) if beta else None
        check_gemm(A, SA, B, SB, tall, out, alpha=(1.0, -1.5)[n % 2], beta=beta, C0=C0,
                   ws=("full", "none", "half")[n % 3], pad=(0, 4, 3)[n % 3], offset=n % 2)


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("M,N,K", [(700, 900, 1100), (2100, 2050, 384), (40, 4100, 1500)])
def test_gemm_larger(M, N, K, tall):
    rng = np.random.default_rng(M)
    A, SA = make_operand(rng, M, K, 1)
    B, SB = make_operand(rng, N, K, tall)
    check_gemm(A, SA, B, SB, tall)
    check_gemm(A, SA, B, SB, tall, "bf16", beta=1.0,
               C0=rng.standard_normal((M, N)).astype(np.float32))


@pytest.mark.parametrize("M", [1, 16, 40, 64, 200, 600])
def test_gemm_integers_are_exact(M):
    """Small integers and power-of-two scales: every sum is exact, so every
    split and order gives the same bits."""
    rng = np.random.default_rng(M)
    N, K = 333, 1700
    ints = lowp.nearest_codes(np.arange(-8, 9).astype(np.float64))
    A, B = rng.choice(ints, (M, K)), rng.choice(ints, (N, K))
    for tall in (1, 128):
        SA = 2.0 ** rng.integers(-1, 2, (lowp.cdiv(K, 128), M)).astype(np.float32)
        SB = 2.0 ** rng.integers(-1, 2, (lowp.cdiv(K, 128), lowp.cdiv(N, tall))).astype(np.float32)
        want = lowp.stands_for(A, SA, 1) @ lowp.stands_for(B, SB, tall).T
        got = run_gemm(A, SA, B, SB, tall)
        np.testing.assert_array_equal(got, want)


def test_gemm_all_codes_and_wide_sums():
    """Products of every pair of finite codes, and sums in which large terms
    cancel and leave small ones (a sum that lost low bits would show)."""
    codes = np.array([c for c in range(256) if c & 0x7F != NAN_CODE], np.uint8)
    A = codes[:, None].copy()
    one = np.ones((1, codes.size), np.float32)
    v = lowp.values(codes)
    np.testing.assert_array_equal(run_gemm(A, one, A, one, 1), np.outer(v, v))
    rng = np.random.default_rng(12)
    K = 128
    A = np.zeros((64, K), np.uint8)
    B = np.zeros((64, K), np.uint8)
    big, small = lowp.nearest_codes(np.array([448.0, 2.0 ** -3]))
    A[:, 0], A[:, 1], B[:, 0], B[:, 1] = big, big | 0x80, big, big
    A[:, 2:], B[:, 2:] = small, small
    one = np.ones((1, 64), np.float32)
    for _ in range(3):
        perm = rng.permutation(K)
        got = run_gemm(A[:, perm], one, B[:, perm], one, 1)
        # 126 products of 2^-6 beside +-200704: a binary32 sum can be off by
        # one unit of 2^18 * 2^-23 for each of 128 additions
        assert np.abs(got - 126 * 2.0 ** -6).max() <= 128 * 2.0 ** -5


def test_gemm_nan_codes_reach_their_row_and_column_only():
    rng = np.random.default_rng(13)
    for M in (20, 150):
        A, SA = make_operand(rng, M, 300, 1)
        B, SB = make_operand(rng, 140, 300, 128)
        A[3, 299] = NAN_CODE
        B[139, 0] = 0xFF
        got = run_gemm(A, SA, B, SB, 128)
        nan = np.zeros(got.shape, bool)
        nan[3], nan[:, 139] = True, True
        np.testing.assert_array_equal(np.isnan(got), nan)


def test_gemm_scaling_only():
    """K == 0 or alpha == 0: C = beta * C, A and B not read, NaN in C not read
    when beta == 0."""
    import torch
    for dt in (torch.float32, torch.bfloat16):
        C = torch.full((5, 7), 3.0, dtype=dt, device="cuda")
        e, s = fg.empty_fp8(5, 0)
        f, t = fg.empty_fp8(7, 0)
        fg.gemm_fp8(e, s, f, t, C, beta=0.5)
        assert (C == 1.5).all()
        C[0, 0] = float("nan")
        fg.gemm_fp8(e, s, f, t, C)
        assert (C == 0).all()


@pytest.mark.parametrize("M,N,K", [(8, 512, 4096), (100, 300, 5000), (700, 700, 700)])
def test_gemm_repeats_and_streams(M, N, K):
    """Repeated calls give identical bits, on another stream too."""
    import torch
    rng = np.random.default_rng(14)
    A, SA = make_operand(rng, M, K, 1)
    B, SB = make_operand(rng, N, K, 128)
    a, sa, b, sb = device_codes(A), device_scales(SA), device_codes(B), device_scales(SB)
    need = fg.fg_gemm_fp8_workspace_size(M, N, K)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    first = fg.gemm_fp8(a, sa, b, sb, torch.empty(M, N, device="cuda"), workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        C = torch.empty(M, N, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        fg.gemm_fp8(a, sa, b, sb, C, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(C, first)


def test_linear_layer_forward_and_backward():
    """The three products of a linear layer on one quantisation of each
    operand (both orders in one pass), against the formulas in binary64 and
    against differences of the (linear) binary64 forward product; captured
    into a graph and replayed on new values."""
    import torch
    rng = np.random.default_rng(15)
    T, I, O = 200, 330, 270
    X = torch.from_numpy(rng.standard_normal((T, I)).astype(np.float32)).cuda()
    W = torch.from_numpy((rng.standard_normal((O, I)) * I ** -0.5).astype(np.float32)).cuda()
    G = torch.from_numpy(rng.standard_normal((T, O)).astype(np.float32)).cuda().to(torch.bfloat16)
    q = {}
    for name, t, block in (("X", X, "row"), ("W", W, "tile"), ("G", G, "row")):
        q[name] = fg.empty_fp8(*t.shape, block) + fg.empty_fp8(t.shape[1], t.shape[0], block)
    Y = torch.empty(T, O, dtype=torch.bfloat16, device="cuda")
    dX = torch.empty(T, I, device="cuda")
    dW = torch.zeros(O, I, device="cuda")
    need = max(fg.fg_gemm_fp8_workspace_size(*s) for s in ((T, O, I), (T, I, O), (O, I, T)))
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")

    def step():
        for name, t, block in (("X", X, "row"), ("W", W, "tile"), ("G", G, "row")):
            fg.quantize_fp8(t, *q[name], block=block)
        fg.gemm_fp8(*q["X"][:2], *q["W"][:2], Y, workspace=ws)              # X W^T
        fg.gemm_fp8(*q["G"][:2], *q["W"][2:], dX, workspace=ws)             # G W
        fg.gemm_fp8(*q["G"][2:], *q["X"][2:], dW, beta=1.0, workspace=ws)   # dW += G^T X

    def check(base):
        n = lambda t: t.float().cpu().numpy()
        xq, xs = lowp.quantize(n(X), 1)
        wq, wsc = lowp.quantize(n(W), 128)
        gq, gs = lowp.quantize(n(G), 1)
        wtq, wts = lowp.quantize(n(W).T, 128)
        gtq, gts = lowp.quantize(n(G).T, 1)
        xtq, xts = lowp.quantize(n(X).T, 1)
        y, b = lowp.product(xq, xs, wq, wsc, 128, narrow=True)
        assert (np.abs(n(Y) - y) <= b + lowp.bf16_half_step(np.abs(y) + b)).all()
        dx, b = lowp.product(gq, gs, wtq, wts, 128)
        assert (np.abs(n(dX) - dx) <= b).all()
        dw, b = lowp.product(gtq, gts, xtq, xts, 1, beta=1.0, C=base)
        assert (np.abs(n(dW) - dw) <= b).all()
        # differences: f(X) = <G, X W^T> for the values the codes stand for
        g64, w64 = lowp.stands_for(gq, gs, 1), lowp.stands_for(wq, wsc, 128)
        x64, v = lowp.stands_for(xq, xs, 1), rng.standard_normal((T, I))
        f = lambda x: float((g64 * (x @ w64.T)).sum())
        diff = (f(x64 + v) - f(x64 - v)) / 2
        # (dX's operand is W's transposed codes: the same values, W is by tiles)
        dxn, b = lowp.product(gq, gs, wtq, wts, 128)
        assert abs((n(dX) * v).sum() - diff) <= (b * np.abs(v)).sum() + 1e-9 * abs(diff)

    step()
    torch.cuda.synchronize()
    check(np.zeros((O, I)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(3):
        X.normal_()
        G.normal_()
        dW.normal_()
        base = dW.cpu().numpy().astype(np.float64)
        graph.replay()
        torch.cuda.synchronize()
        check(base)


def test_torch_wrappers_refuse():
    import torch
    X = torch.zeros(4, 8, device="cuda")
    q, s = fg.empty_fp8(4, 8)
    with pytest.raises(TypeError):
        fg.quantize_fp8(X.double(), q, s)
    with pytest.raises(ValueError):
        fg.quantize_fp8(X, q[:3], s)
    with pytest.raises(ValueError):
        fg.quantize_fp8(X, q, s[:, :3])
    with pytest.raises(TypeError):
        fg.quantize_fp8(X, q, s.double())
    with pytest.raises(fg.FgError):
        fg.quantize_fp8(X, torch.zeros(4, 8, dtype=torch.uint8, device="cuda"), s)
    with pytest.raises(ValueError):
        fg.quantize_fp8(X, q.cpu(), s)
    C = torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError):
        fg.gemm_fp8(q, s, q[:3], s, C)
    with pytest.raises(ValueError):
        fg.gemm_fp8(q, s, q, s[:, :2], C)
    with pytest.raises(TypeError):
        fg.gemm_fp8(q.float(), s, q, s, C)
    with pytest.raises(TypeError):
        fg.gemm_fp8(q, s, q, s, C.half())
