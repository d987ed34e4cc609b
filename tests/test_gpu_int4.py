"""Products with 4-bit weights on the GPU against the binary64 oracle."""
import numpy as np
import pytest

import fp32_gemm_tile_amd as fg
from oracle import gated as og

from test_gpu_gated import aligned, dtype_of, guarded, near, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fg.load_library()
    yield
    torch.cuda.synchronize()


class Weights:
    def __init__(self, rng, N, K, group, st, zeros, pad=0):
        import torch
        half, groups = (K + 1) // 2, -(-K // group)
        self.codes = rng.integers(0, 256, (N, half)).astype(np.uint8)
        base = torch.full((N, -(-half // 16) * 16 + 16 * pad), 0xFF, dtype=torch.uint8, device="cuda")
        base[:, :half] = torch.from_numpy(self.codes).cuda()
        s = torch.full((groups, N + pad), float("nan"), dtype=dtype_of(st), device="cuda")
        s[:, :N] = torch.from_numpy(np.exp(0.3 * rng.standard_normal((groups, N))) * max(K, 1) ** -0.5).cuda()
        z = None
        if zeros:
            z = torch.from_numpy(rng.integers(0, 16, (groups, N + pad)).astype(np.uint8)).cuda()[:, :N]
        self.t = (base[:, :half], s[:, :N], z)
        self.v, self.most = og.int4_weights(self.codes, s[:, :N].double().cpu().numpy(),
                                            None if z is None else z.cpu().numpy(), K, group)


def check(T, N, K, group, ty, st, zeros, gated, pad=0, act="silu", seed=0):
    import torch
    rng = np.random.default_rng(seed + T + N + K)
    bf16 = ty == "bf16"
    x = aligned(rng.standard_normal((T, K)) * np.exp(0.5 * rng.standard_normal((1, K))), ty, pad)
    w = [Weights(rng, N, K, group, st, zeros, pad) for _ in range(2 if gated else 1)]
    out, base = guarded(T, N, ty)
    print("  int4", T, N, K, group, ty, st, zeros, gated, pad, act, flush=True)
    if gated:
        fg.gated_int4(x, w[0].t, w[1].t, out, group=group, activation=act)
    else:
        fg.gemm_int4(x, w[0].t, out, group=group)
    torch.cuda.synchronize()
    untouched(base, T, N)
    xv = x.double().cpu().numpy()
    if not gated:
        near(out, *og.int4_product(xv, w[0].v, w[0].most, bf16, group), "out")
        return out
    (g, eg), (u, eu) = (og.int4_product(xv, v.v, v.most, bf16, group, rounded=False) for v in w)
    a = og.act(g, act)
    ea = 1.13 * eg + og.act_error(g, a, act)
    h = a * u
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 4 * og.U * np.abs(h)
    near(out, h, eh + og.half_step(np.abs(h) + eh, bf16), "h")
    return out


SIZES = [(1, 16, 128), (1, 1, 1), (1, 5, 31), (2, 17, 33), (3, 64, 129), (5, 33, 257), (16, 48, 320),
         (17, 20, 100), (31, 100, 640), (33, 65, 96), (64, 130, 390), (1, 200, 4100), (4, 7, 2000)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_products(T, N, K, ty, group):
    check(T, N, K, group, ty, "f32", True, False)
    check(T, N, K, group, ty, "bf16", False, True)


@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_strides_and_activations(ty):
    for act in ("none", "relu", "gelu", "silu"):
        check(7, 37, 200, 64, ty, "bf16", True, True, pad=5, act=act)
    check(40, 37, 200, 32, ty, "f32", True, False, pad=3)
    check(6, 3, 77, 32, ty, "bf16", True, False, pad=1)


@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_many_rows_of_weights(ty):
    """As many rows of W as change how many of them a workgroup has."""
    for T, N, K, gated in ((1, 8200, 130, False), (4, 8193, 100, False), (3, 4099, 260, False),
                           (2, 8200, 70, True), (16, 8200, 40, False), (20, 8193, 33, True)):
        check(T, N, K, 32, ty, "f32", True, gated)


def test_long_rows():
    """Rows so far apart that offsets pass 32 bits: the bits of compact ones."""
    import torch
    rng = np.random.default_rng(9)
    N, K, group, far = 2100, 96, 32, 1 << 21
    w = Weights(rng, N, K, group, "f32", True)
    q = torch.empty(N, far, dtype=torch.uint8, device="cuda")[:, :K // 2]
    q.copy_(w.t[0])
    for T, ty in ((3, "bf16"), (16, "f32"), (64, "f32")):
        x = aligned(rng.standard_normal((T, K)), ty)
        xf = torch.empty(T, far, dtype=x.dtype, device="cuda")[:, :K]
        xf.copy_(x)
        out = torch.empty(T, N, dtype=x.dtype, device="cuda")
        of = torch.empty(T, far, dtype=x.dtype, device="cuda")[:, :N]
        fg.gemm_int4(x, w.t, out, group=group)
        fg.gemm_int4(xf, (q, *w.t[1:]), of, group=group)
        assert torch.equal(out, of)


def test_every_code_times_one():
    """One column at a time: each code minus its zero point, exactly."""
    import torch
    for group in (32, 64, 128):
        N, K = 16, 256
        codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
        for n in range(N):
            codes[n] = n | (15 - n) << 4
        z = torch.randint(0, 256, (K // group, N), dtype=torch.uint8, device="cuda")
        s = torch.ones(K // group, N, device="cuda")
        for ty in ("f32", "bf16"):
            x = torch.zeros(64, K, dtype=dtype_of(ty), device="cuda")
            cols = torch.randperm(K)[:64]
            x[torch.arange(64), cols] = 1.0
            out = torch.empty(64, N, dtype=dtype_of(ty), device="cuda")
            fg.gemm_int4(x, (codes, s, z), out, group=group)
            n = torch.arange(N)
            q = torch.where(cols[:, None] % 2 == 0, n[None, :], 15 - n[None, :]).double()
            want = q - z.cpu()[cols // group].double()
            assert torch.equal(out.double().cpu(), want)


def test_infinities_nan_and_large_values():
    """x that is infinite, NaN or next to the largest value touches its own row of out
    only, as the formula in 64 bits says."""
    import torch
    rng = np.random.default_rng(4)
    T, N, K, group = 9, 40, 300, 64
    for ty in ("f32", "bf16"):
        w = Weights(rng, N, K, group, "f32", True)
        x = torch.from_numpy(rng.standard_normal((T, K))).cuda().to(dtype_of(ty))
        top = torch.finfo(dtype_of(ty)).max
        x[1, 4] = float("inf")
        x[2, 200] = float("nan")
        x[3, 7], x[3, 290] = float("inf"), -float("inf")
        x[4, :3] = top
        x[5] = 0
        x[6, 9] = -top
        w.t[1][:, 5] = 0.0
        x = aligned(x.double().cpu().numpy(), ty)
        w.v, w.most = og.int4_weights(w.codes, w.t[1].double().cpu().numpy(), w.t[2].cpu().numpy(), K, group)
        out = torch.empty(T, N, dtype=dtype_of(ty), device="cuda")
        fg.gemm_int4(x, w.t, out, group=group)
        xv = x.double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            y, e = og.int4_product(xv, w.v, w.most, ty == "bf16", group)
        got = out.double().cpu().numpy()
        for t in range(T):
            fine = np.isfinite(y[t]) & (np.abs(y[t]) < 0.5 * top)
            with np.errstate(invalid="ignore"):
                assert (np.abs(got[t] - y[t]) <= e[t])[fine].all(), t
            huge = np.isfinite(y[t]) & (np.abs(y[t]) > 2.0 * top)
            assert np.isinf(got[t][huge]).all()
            assert (np.isnan(got[t]) == np.isnan(y[t]))[~huge].all(), t
            inf = np.isinf(y[t])
            assert (got[t][inf] == y[t][inf]).all(), t


@pytest.mark.parametrize("T", [2, 4, 16, 24, 50])
def test_infinities_in_every_variant(T):
    """The same where x has other numbers of rows: an infinity, two of them, a NaN."""
    import torch
    rng = np.random.default_rng(T)
    N, K, group = 21, 290, 32
    for ty in ("f32", "bf16"):
        w = Weights(rng, N, K, group, "bf16", True)
        x = rng.standard_normal((T, K))
        special = [{4: np.inf}, {7: np.inf, 289: -np.inf}, {200: np.nan}, {288: -np.inf}]
        for i, at in enumerate(special[:max(1, T // 2)]):
            for col, v in at.items():
                x[T - 1 - i, col] = v
        x = aligned(x, ty)
        out = torch.empty(T, N, dtype=dtype_of(ty), device="cuda")
        fg.gemm_int4(x, w.t, out, group=group)
        with np.errstate(invalid="ignore", over="ignore"):
            y, e = og.int4_product(x.double().cpu().numpy(), w.v, w.most, ty == "bf16", group)
        got = out.double().cpu().numpy()
        fine = np.isfinite(y)
        with np.errstate(invalid="ignore"):
            assert (np.abs(got - y) <= e)[fine].all()
        assert (np.isnan(got) == np.isnan(y)).all()
        assert (got == y)[np.isinf(y)].all()


def test_empty_sizes():
    import torch
    out = torch.full((3, 8), 7.0, device="cuda")
    codes = torch.empty(8, 0, dtype=torch.uint8, device="cuda")
    s = torch.empty(0, 8, device="cuda")
    fg.gemm_int4(torch.empty(3, 0, device="cuda"), (codes, s, None), out)
    assert not out.any()
    fg.gemm_int4(torch.empty(0, 0, device="cuda"), (codes, s, None), out[:0])


def test_a_served_block_eagerly_and_captured():
    """gate and up, then down, on 4-bit weights: a decode step, captured and replayed
    with eager calls between, equal bits."""
    import torch
    rng = np.random.default_rng(6)
    T, H, I, group = 4, 256, 384, 64
    gate, up = (Weights(rng, I, H, group, "bf16", True) for _ in range(2))
    down = Weights(rng, H, I, group, "bf16", False)
    x = torch.from_numpy(rng.standard_normal((T, H))).cuda().bfloat16()
    h, y = (torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for n in (I, H))

    def step():
        fg.gated_int4(x, gate.t, up.t, h, group=group)
        fg.gemm_int4(h, down.t, y, group=group)

    step()
    torch.cuda.synchronize()
    first = y.clone()
    near(y, *og.int4_product(h.double().cpu().numpy(), down.v, down.most, True, group), "down")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, y)
        step()
        torch.cuda.synchronize()


def test_wrong_tensors_are_refused():
    import torch
    rng = np.random.default_rng(1)
    w = Weights(rng, 8, 64, 32, "f32", True)
    x, out = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 8, device="cuda")
    q, s, z = w.t
    for bad in ((q[:4], s, z), (q, s[:1], z), (q, s, z[:1]), (q, s.t().contiguous().t(), z)):
        with pytest.raises(ValueError):
            fg.gemm_int4(x, bad, out, group=32)
    for group in (0, 48, -32):
        with pytest.raises(ValueError):
            fg.gemm_int4(x, w.t, out, group=group)
    with pytest.raises(TypeError):
        fg.gemm_int4(x, (q.float(), s, z), out, group=32)
    with pytest.raises(TypeError):
        fg.gemm_int4(x, (q, s.half(), z), out, group=32)
    with pytest.raises(TypeError):
        fg.gemm_int4(x, w.t, out.bfloat16(), group=32)
    with pytest.raises(TypeError):
        fg.gated_int4(x, w.t, (q, s.bfloat16(), z), out, group=32)
    with pytest.raises(fg.FgError):
        fg.gemm_int4(torch.zeros(65, 64, device="cuda"), w.t, torch.zeros(65, 8, device="cuda"), group=32)
    with pytest.raises(fg.FgError):
        fg.gemm_int4(torch.zeros(2, 65, device="cuda")[:, 1:], w.t, out, group=32)
