"""The gated block's and the 4-bit products' entry points on the host: refusals,
argument positions and quick returns, with no GPU work (made-up addresses; calls
that could reach a launch run with the GPUs hidden)."""
import ctypes
import os

import pytest

import fp32_gemm_tile_amd as fg

from test_abi_cpu import declared_functions, run_without_gpu

BIG = fg.FG_MAX_LD + 16


def block(T=3, H=16, I=8, ty=0, act=3, x=16, ldx=16, gate=16, ldgate=16, up=16, ldup=16, save=0,
          g=16, ldg=16, u=16, ldu=16, sg=16, ldsg=3, su=16, ldsu=3, h=16, ldh=8):
    p = lambda v: v or None  # noqa: E731
    return fg.fg_gated_block(T, H, I, ty, act, p(x), ldx, p(gate), ldgate, p(up), ldup, save, p(g),
                             ldg, p(u), ldu, p(sg), ldsg, p(su), ldsu, p(h), ldh)


def grads(dh=16, lddh=8, dx=16, lddx=16, dgate=16, lddgate=16, dup=16, lddup=16, beta=0.0):
    p = lambda v: v or None  # noqa: E731
    return fg.fg_gated_grads(p(dh), lddh, p(dx), lddx, p(dgate), lddgate, p(dup), lddup, beta)


SHARED = [
    (dict(T=-1), 1), (dict(H=-1), 2), (dict(I=-1), 3), (dict(ty=2), 4), (dict(ty=-1), 4),
    (dict(act=4), 5), (dict(act=-1), 5), (dict(x=0), 6), (dict(x=20), 6), (dict(ldx=15), 7),
    (dict(ldx=18), 7), (dict(ty=1, ldx=20), 7), (dict(gate=0), 8), (dict(gate=24), 8),
    (dict(ldgate=12), 9), (dict(ldgate=17), 9), (dict(up=0), 10), (dict(up=8), 10),
    (dict(ldup=12), 11), (dict(save=3), 12), (dict(save=-1), 12), (dict(save=1, g=0), 13),
    (dict(save=1, g=18), 13), (dict(save=2, g=24), 13), (dict(save=1, ldg=7), 14),
    (dict(save=2, ldg=24), 14), (dict(save=1, u=0), 15), (dict(save=1, ldu=7), 16),
    (dict(save=2, sg=0), 17), (dict(save=2, sg=18), 17), (dict(save=2, ldsg=2), 18),
    (dict(save=2, su=0), 19), (dict(save=2, ldsu=2), 20), (dict(h=18), 21), (dict(ldh=7), 22),
]


@pytest.mark.parametrize("kw,bad", SHARED + [(dict(h=0), 21)])
def test_gated_refusals(kw, bad):
    assert fg.fg_gated(block(**kw)) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


@pytest.mark.parametrize("kw,bad", SHARED)
def test_gated_backward_refusals(kw, bad):
    kw = dict(dict(save=1), **kw)
    assert fg.fg_gated_backward(block(**kw), grads(), 16, 1 << 20) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


@pytest.mark.parametrize("kw,bad", [
    (dict(dh=0), 23), (dict(dh=18), 23), (dict(lddh=7), 24), (dict(dx=18), 25), (dict(lddx=15), 26),
    (dict(dgate=18), 27), (dict(dgate=0), 27), (dict(lddgate=15), 28), (dict(dup=0), 29),
    (dict(dup=18), 29), (dict(lddup=15), 30),
])
def test_gradients_refusals(kw, bad):
    assert fg.fg_gated_backward(block(save=1), grads(**kw), 16, 1 << 20) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


def test_gated_workspaces_limits_and_quick_returns():
    assert fg.fg_gated(None) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 1
    assert fg.fg_gated_backward(None, grads()) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_gated_backward(block(save=1), None) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 23
    assert fg.fg_gated(block(), 24, 100) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 23
    assert fg.fg_gated_backward(block(save=0), grads(), 16, 1 << 20) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 12
    need = fg.fg_gated_backward_min_workspace_size(3, 8, 0)
    assert need == 2 * 3 * 128 * 4
    for ws in (0, 24):
        assert fg.fg_gated_backward(block(save=1), grads(), ws, need) == fg.FG_ERR_INVALID_ARG
        assert fg.fg_last_bad_arg() == 32
    assert fg.fg_gated_backward(block(save=1), grads(), 16, need - 1) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 33
    for kw in (dict(ldx=BIG), dict(ldgate=BIG), dict(ldup=BIG), dict(ldh=BIG), dict(save=1, ldg=BIG),
               dict(save=1, ldu=BIG), dict(T=(1 << 30) + 1), dict(I=1 << 31, ldh=1 << 31)):
        assert fg.fg_gated(block(**kw)) == fg.FG_ERR_UNSUPPORTED, kw
    for kw in (dict(lddh=BIG), dict(lddx=BIG), dict(lddgate=BIG), dict(lddup=BIG)):
        assert fg.fg_gated_backward(block(save=1), grads(**kw), 16, 1 << 30) == fg.FG_ERR_UNSUPPORTED
    assert fg.fg_gated(block(T=0, x=0, h=0)) == fg.FG_OK
    assert fg.fg_gated(block(I=0, gate=0, up=0, h=0)) == fg.FG_OK
    none = dict(dx=0, dgate=0, dup=0)
    assert fg.fg_gated_backward(block(save=1, h=0, x=0, gate=0, up=0), grads(**none), 16, need) == fg.FG_OK
    assert fg.fg_gated_backward(block(T=0, save=1, x=0, g=0, u=0, h=0), grads(dh=0, dx=0, beta=1.0)) == fg.FG_OK
    assert fg.fg_gated_backward(block(H=0, save=1, h=0), grads(), 16, need) == fg.FG_OK
    assert fg.fg_gated_workspace_size(-1, 4, 4, 0) == 0 and fg.fg_gated_workspace_size(4, 4, 4, 2) == 0
    assert fg.fg_gated_backward_workspace_size(4, 4, 1 << 31, 1) == 0
    for ty in (0, 1):
        for T, H, I in ((1, 2048, 1408), (200, 2048, 1408), (4096, 4096, 8192)):
            assert (fg.fg_gated_backward_workspace_size(T, H, I, ty)
                    >= fg.fg_gated_backward_min_workspace_size(T, I, ty) > 0)


def test_gated_valid_calls_stop_at_the_device_check():
    run_without_gpu("""
import sys
sys.path.insert(0, "tests")
from test_gated_abi_cpu import block, grads, weights, int4, gated4
for ty in (0, 1):
    for T in (3, 100):
        for save in (0, 1, 2):
            for H in (16, 0):
                b = block(T=T, H=H, ty=ty, save=save, ldsg=T, ldsu=T)
                assert fg.fg_gated(b) in NO_DEVICE
                if save and H:
                    assert fg.fg_gated_backward(b, grads(), 16, 1 << 20) in NO_DEVICE
    b = block(T=0, ty=ty, save=1)
    assert fg.fg_gated_backward(b, grads(beta=0.5)) in NO_DEVICE
assert int4() in NO_DEVICE and gated4() in NO_DEVICE and int4(K=0, x=0) in NO_DEVICE
""")


def test_tile_hooks():
    for product, ty, some in ((0, 0, True), (0, 1, True), (1, 1, True), (2, 1, True), (1, 0, True), (2, 0, True),
                              (3, 1, False), (0, 2, False)):
        assert (len(fg.fg_gated_tiles(product, ty)) > 0) == some
    r, c, lib = ctypes.c_int32(), ctypes.c_int32(), fg.load_library()
    ref = ctypes.byref
    for args, bad in (((3, 1, 0, ref(r), ref(c)), 1), ((1, 2, 0, ref(r), ref(c)), 2),
                      ((0, 1, 99, ref(r), ref(c)), 3), ((0, 1, 0, None, ref(c)), 4),
                      ((0, 1, 0, ref(r), None), 5)):
        assert lib.fg_gated_tile(*args) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == bad
    for args, bad in (((-1, 1, 1, 1, 1), 1), ((2, 2, 1, 1, 1), 2), ((0, 1, 0, 1, 1), 3),
                      ((0, 1, 1, 0, 1), 4), ((0, 1, 1, 1, 0), 5)):
        with pytest.raises(fg.FgError) as e:
            fg.fg_select_gated(*args)
        assert e.value.bad_arg == bad
    for args, bad in (((3, 1, 0, 1), 1), ((1, 2, 0, 1), 2), ((0, 1, 99, 1), 3), ((0, 1, -2, 1), 3),
                      ((0, 1, 0, 17), 4), ((0, 1, 0, -1), 4)):
        assert fg.fg_set_gated_tile(*args) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == bad
    assert fg.fg_select_gated(0, 1, 4, 4096, 4096) == (-1, 1)
    try:
        assert fg.fg_set_gated_tile(0, 1, 1, 2) == fg.FG_OK
        assert fg.fg_select_gated(0, 1, 4, 4096, 4096, 1 << 30) == (1, 2)
        assert fg.fg_select_gated(0, 1, 4, 4096, 4096, 0) == (1, 1)
    finally:
        assert fg.fg_set_gated_tile(0, 1) == fg.FG_OK
    assert fg.fg_select_gated(0, 1, 4, 4096, 4096) == (-1, 1)


def test_every_tile_is_chosen_somewhere():
    """No tile that no size would choose."""
    for product, ty in ((0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (2, 1)):
        chosen = set()
        for T in (1, 65, 100, 130, 200, 300, 517, 1025, 2048, 4096, 8192):
            for H in (64, 300, 1024, 2048, 4096, 8192):
                for I in (64, 300, 1408, 2048, 4096, 8192):
                    for ws in (0, 1 << 28):
                        chosen.add(fg.fg_select_gated(product, ty, T, H, I, ws)[0])
        assert chosen - {-1} == set(range(len(fg.fg_gated_tiles(product, ty)))), (product, ty, chosen)


def weights(q=16, ldq=16, s=16, lds=8, z=0, ldz=0):
    return fg.fg_int4(q or None, ldq, s or None, lds, z or None, ldz)


def int4(T=3, N=8, K=16, group=32, ty=0, st=0, x=16, ldx=16, w=None, out=16, ldo=8):
    return fg.fg_gemm_int4(T, N, K, group, ty, st, x, ldx, w or weights(), out, ldo)


def gated4(T=3, N=8, K=16, group=32, ty=0, st=0, x=16, ldx=16, w=None, up=None, act=3, out=16, ldo=8):
    return fg.fg_gated_int4(T, N, K, group, ty, st, x, ldx, w or weights(), up or weights(), act,
                            out, ldo)


INT4 = [
    (dict(T=-1), 1), (dict(T=65), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(group=16), 4),
    (dict(group=0), 4), (dict(group=256), 4), (dict(ty=2), 5), (dict(st=2), 6), (dict(x=0), 7),
    (dict(x=24), 7), (dict(ldx=15), 8), (dict(ldx=18), 8), (dict(w=weights(q=0)), 9),
    (dict(w=weights(q=24)), 9), (dict(w=weights(ldq=24)), 9), (dict(K=64, ldx=64, w=weights(ldq=16)), 9),
    (dict(w=weights(s=0)), 9), (dict(w=weights(s=18)), 9), (dict(st=1, w=weights(s=17)), 9),
    (dict(w=weights(lds=7)), 9), (dict(w=weights(z=16, ldz=7)), 9), (dict(out=0), 12),
    (dict(out=18), 12), (dict(ldo=7), 13),
]


@pytest.mark.parametrize("kw,bad", INT4)
def test_int4_refusals(kw, bad):
    for call in (int4, gated4):
        assert call(**kw) == fg.FG_ERR_INVALID_ARG
        assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


@pytest.mark.parametrize("kw,bad", [(dict(up=weights(q=0)), 10), (dict(up=weights(lds=7)), 10),
                                    (dict(act=4), 11), (dict(act=-1), 11)])
def test_gated_int4_refusals(kw, bad):
    assert gated4(**kw) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == bad and fg.fg_last_error()


def test_int4_limits_and_quick_returns():
    assert fg.fg_gemm_int4(3, 8, 16, 32, 0, 0, 16, 16, None, 16, 8) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 9
    assert fg.fg_gated_int4(3, 8, 16, 32, 0, 0, 16, 16, weights(), None, 3, 16, 8) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 10
    assert int4(T=0, x=0, out=0) == fg.FG_OK and int4(N=0, w=weights(q=0, s=0), out=0) == fg.FG_OK
    assert int4(ldx=BIG) == fg.FG_ERR_UNSUPPORTED and int4(w=weights(ldq=BIG)) == fg.FG_ERR_UNSUPPORTED
    assert int4(ldo=BIG) == fg.FG_ERR_UNSUPPORTED
    # scales and zero points of 2 GiB: one group and two, 4 bytes, 2 and 1
    for K, st, lds, ldz in ((16, 0, 1 << 29, 0), (64, 0, 1 << 28, 0), (16, 1, 1 << 30, 0),
                            (64, 0, 8, 1 << 30)):
        w = weights(s=16, lds=lds, z=16 if ldz else 0, ldz=ldz, ldq=32)
        assert int4(K=K, ldx=64, st=st, w=w) == fg.FG_ERR_UNSUPPORTED and fg.fg_last_bad_arg() == 9


def test_new_headers_declare_what_the_library_exports():
    lib = fg.load_library()
    here = os.path.dirname(os.path.abspath(__file__))
    import re
    for name in ("fp32gemm_gated.h", "fp32gemm_int4.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(here, "..", "include", name)).read(), flags=re.S)
        names = set(re.findall(r"\b(fg_[a-z_0-9]+)\s*\(", text))
        assert names
        for n in names:
            assert hasattr(lib, n), n
    assert declared_functions()


def test_headers_are_plain_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "t.c"
    src.write_text('#include "fp32gemm_gated.h"\n#include "fp32gemm_int4.h"\n'
                   "int main(void){return sizeof(fg_gated_block) == 0;}\n")
    inc = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", inc, str(src)],
                   check=True)


def test_torch_layer_checks_need_no_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    for call in (lambda: fg.gated(x, x, x, x), lambda: fg.gated_backward(x, x, x, x, (x, x)),
                 lambda: fg.gemm_int4(x, (x, x, None), x),
                 lambda: fg.gated_int4(x, (x, x, None), (x, x, None), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
