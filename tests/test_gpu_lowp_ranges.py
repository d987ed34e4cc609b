"""The 8-bit and mixture-of-experts calls at the ends of their ranges: results
from one to many tiles, long sums, largest layers, rows further apart than 32
bits reach, two calls at once, a whole step captured into one graph."""
import numpy as np
import pytest

import fp32_gemm_tile_amd as fg
from oracle import lowp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fg.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def integers(g, rows, cols, tall):
    """Codes of integers -8 .. 8, scales 1/2, 1 or 2, and the values (float64)."""
    import torch
    v = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda")
    q, s = fg.empty_fp8(rows, cols, "row" if tall == 1 else "tile")
    q.copy_(v.float().to(torch.float8_e4m3fn))
    s.copy_(2.0 ** torch.randint(-1, 2, s.shape, generator=g, device="cuda").float())
    wide = s.repeat_interleave(128, 0)[:cols].repeat_interleave(tall, 1)[:, :rows]
    return q, s, v.double() * wide.t().double()


# One row to many tiles of every height and width, with partial ones, sums of
# two to 157 blocks, small results of long sums.
SIZES = [(1, 33, 130), (1, 33, 20000), (130, 33, 20000), (2050, 33, 130), (4100, 33, 520),
         (4100, 33, 2060), (257, 33, 20000), (2500, 1030, 130), (161, 3010, 1030),
         (700, 3010, 130), (515, 2050, 300), (1030, 33, 20000), (3000, 515, 300),
         (2050, 130, 20000), (2050, 2050, 130), (700, 3010, 520), (1030, 515, 20000),
         (2500, 4100, 130), (1500, 2050, 300), (3000, 70, 20000), (257, 2050, 20000),
         (3000, 4100, 300), (3000, 2050, 8200), (161, 3010, 20000), (3000, 4100, 2060)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_products_of_integers_are_exact(M, N, K):
    """Products of at most 2^8 in quarters, and sums of them that stay far below
    2^22: exact in binary32 whatever the tile, split and order; bfloat16 C is
    the nearest."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 7 * K)
    A, SA, a = integers(g, M, K, 1)
    for tall in (1, 128):
        B, SB, b = integers(g, N, K, tall)
        want = a @ b.t()
        assert want.abs().max() < 2 ** 20
        for dt in (torch.float32, torch.bfloat16):
            need = fg.fg_gemm_fp8_workspace_size(M, N, K)
            ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
            base = torch.full((M, N + 1), 7.0, dtype=dt, device="cuda")
            print("  product", M, N, K, tall, dt, need, flush=True)
            fg.gemm_fp8(A, SA, B, SB, base[:, :N], workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(base[:, :N], want.to(dt)) and (base[:, N] == 7.0).all()
            C0 = torch.randint(-64, 65, (M, N), generator=g, device="cuda").to(dt)
            C = C0.clone()
            fg.gemm_fp8(A, SA, B, SB, C, alpha=-2.0, beta=4.0, workspace=ws)
            # (sum and product with beta are exact in binary32: one rounding to C)
            assert torch.equal(C, (-2.0 * want + 4.0 * C0.double()).to(dt))


def test_rows_beyond_32_bits():
    """Row pitches at the limit, so that the last row starts past 2^32 bytes."""
    import torch
    ld, M, N = fg.FG_MAX_LD, 2100, 70
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, N, generator=g, device="cuda")
    far = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").as_strided((M, N), (ld, 1))
    far.copy_(x)
    near = far.contiguous()
    q0, s0 = fg.empty_fp8(M, N)
    t0, u0 = fg.empty_fp8(N, M)
    fg.quantize_fp8(near, q0, s0, t0, u0)
    q1 = torch.empty(M * ld, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q1 = q1.as_strided((M, N), (ld, 1))
    t1, u1 = fg.empty_fp8(N, M)
    fg.quantize_fp8(far, q1, s0.zero_(), t1, u1)
    torch.cuda.synchronize()
    assert torch.equal(q1.contiguous().view(torch.uint8), q0.contiguous().view(torch.uint8))
    assert torch.equal(t1.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))
    assert torch.equal(u0, u1)
    B, SB, _ = integers(g, 40, N, 1)
    want = fg.gemm_fp8(q0, s0, B, SB, torch.empty(M, 40, device="cuda"))
    C = torch.empty(M * ld // 2, device="cuda").as_strided((M // 2, 40), (ld, 1))
    fg.gemm_fp8(q1[M // 2:], s0[:, M // 2:].contiguous(), B, SB, C)
    assert torch.equal(C, want[M // 2:])


def test_more_rows_than_small_tiles_reach():
    """So many rows that a grid of the smallest tiles would have 2^32 threads."""
    import torch
    M, N, K = (1 << 27) + 5, 8, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    A, SA, B, SB, b = (torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"),
                       torch.ones(1, M, device="cuda")) + integers(g, N, K, 1)
    some = torch.randint(-8, 9, (4096, K), generator=g, device="cuda").float()
    A.view(torch.uint8)[:] = some[0].to(torch.float8_e4m3fn).view(torch.uint8)
    A[-4096:] = some.to(torch.float8_e4m3fn)
    C = fg.gemm_fp8(A, SA, B, SB, torch.empty(M, N, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(C[-4096:], (some.double() @ b.t()).float())
    first = (some[0].double() @ b.t()).float()
    assert (C[:-4096] == first).all()


class Experts:
    """Random experts of small integers / 8 (exact in every type)."""

    def __init__(self, rng, E, H, I, dt):
        import torch
        self.E, self.H, self.I = E, H, I
        self.v = [rng.integers(-3, 4, (E, R, C)).astype(np.float64) / 8
                  for R, C in ((I, H), (I, H), (H, I))]
        self.t = []
        for v in self.v:
            E_, R, C = v.shape
            base = torch.zeros(E_, R, -(-C // 16) * 16, dtype=dt, device="cuda")
            base[:, :, :C].copy_(torch.from_numpy(v).cuda().float())
            self.t.append(base[:, :, :C])
        one = lambda R, C: torch.ones(E, lowp.cdiv(C, 128), lowp.cdiv(R, 128), device="cuda")
        self.scales = ((one(I, H), one(I, H), one(H, I))
                       if dt == torch.float8_e4m3fn else None)


def check(L, x, ids, w, out, act="silu"):
    import torch
    bf16 = x.dtype == torch.bfloat16
    want, bound = lowp.layer(x.double().cpu().numpy(), *L.v, ids.cpu().numpy(),
                             w.double().cpu().numpy(), act, h_bits=16 if bf16 else 24)
    if bf16:
        bound = bound + lowp.bf16_half_step(np.abs(want) + bound)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("wt", ["float8_e4m3fn", "bfloat16", "float32"])
def test_largest_layers(wt, xt):
    """The most tokens, experts and slots, with all of a token's slots filled by
    different experts and by one; many rows of output; a long sum."""
    import torch
    rng = np.random.default_rng(31)
    dt, xdt = getattr(torch, wt), {"f32": torch.float32, "bf16": torch.bfloat16}[xt]
    for T, E, k, H, I in ((64, 512, 16, 64, 40), (64, 500, 16, 48, 17), (64, 16, 16, 4200, 48),
                          (3, 4, 2, 40, 4200), (2, 3, 1, 8, 20000), (64, 2, 2, 16, 33)):
        L = Experts(rng, E, H, I, dt)
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().to(xdt)
        ws = torch.full((fg.fg_moe_workspace_size(T, k, E, H, I),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        router = torch.from_numpy((rng.standard_normal((E, H)) * H ** -0.5)
                                  .astype(np.float32)).cuda()
        ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        out = torch.empty(T, H, dtype=xdt, device="cuda")
        print("  layer", T, E, k, H, I, wt, xt, flush=True)
        fg.moe(x, *L.t, ids, w, out, router=router, scales=L.scales, workspace=ws)
        want_ids, _ = lowp.route(x.double().cpu().numpy(), router.double().cpu().numpy(), k, True)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        check(L, x, ids, w, out)
        ids.copy_(torch.arange(T * k, device="cuda").view(T, k) % E)
        fg.moe(x, *L.t, ids, w, out, scales=L.scales, workspace=ws)
        check(L, x, ids, w, out)
        ids.fill_(E - 1)
        fg.moe(x, *L.t, ids, w, out, scales=L.scales, workspace=ws)
        check(L, x, ids, w, out)


@pytest.mark.parametrize("E,k", [(3, 3), (40, 7), (64, 16), (100, 16), (128, 5), (300, 16), (512, 8)])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 64])
def test_router_order(E, k, T):
    """Equal logits, logits equal in their upper 32 bits, infinite and NaN ones,
    against a stable sort in binary64."""
    import torch
    rng = np.random.default_rng(E + T)
    H = 8
    L = Experts(rng, E, H, 8, torch.bfloat16)
    x = torch.zeros(T, H, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -40
    if T > 1:
        x[1::3, 0] = -1.0
        x[T - 1] = 0.0                                   # all of its logits equal
    router = torch.zeros(E, H, device="cuda")
    router[:, 0] = torch.from_numpy(rng.integers(-2, 3, E).astype(np.float32))
    router[:, 1] = torch.from_numpy(rng.integers(-1, 2, E).astype(np.float32))
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    out = torch.empty(T, H, device="cuda")
    for special in (False, True):
        if special:
            router[E // 2, 0], router[E - 1, 0] = float("nan"), float("-inf")
            x[T - 1, 0] = 1.0                            # (0 * inf is NaN)
        fg.moe(x, *L.t, ids, w, out, router=router)
        logits = x.double().cpu().numpy() @ router.double().cpu().numpy().T
        order = np.where(np.isnan(logits), -np.inf, logits)
        want = np.argsort(-order, axis=1, kind="stable")[:, :k]
        np.testing.assert_array_equal(ids.cpu().numpy(), want)
        chosen = np.take_along_axis(logits, want, 1)
        top = chosen[:, :1]
        with np.errstate(invalid="ignore"):
            e = np.exp(chosen - top)
            weights = e / e.sum(1, keepdims=True)
        # (differences below 8, exp, a sum of at most 16 and a division)
        np.testing.assert_allclose(w.cpu().numpy(), weights, rtol=40 * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("wt", ["bfloat16", "float32"])
def test_largest_and_infinite_values(wt):
    """binary32 x and h between the largest bfloat16 and infinity stay finite;
    infinities and NaN reach their own token only."""
    import torch
    top, tiny = float(np.finfo(np.float32).max), 2.0 ** -120
    H, I, dt = 20, 18, getattr(torch, wt)
    gate, up, down = (torch.zeros(1, I, 32, dtype=dt, device="cuda")[:, :, :H],
                      torch.zeros(1, I, 32, dtype=dt, device="cuda")[:, :, :H],
                      torch.zeros(1, H, 32, dtype=dt, device="cuda")[:, :, :I])
    gate[0, 0, 0], gate[0, 1, 1] = tiny, 1.0
    up[0, 0, 0], up[0, 1, 2] = tiny, 1.0
    down[0, 0, 0], down[0, 1, 1], down[0, 2, 0] = 1.0, tiny, -1.0
    x = torch.zeros(4, H, device="cuda")
    x[0, 0] = -top                       # h[0] = (top tiny)^2
    x[1, 1], x[1, 2] = 1.0, top          # h[1] = top
    x[2, 0] = float("inf")
    x[3, 5] = float("nan")
    ids, w = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    out = fg.moe(x, gate, up, down, ids, w, torch.empty(4, H, device="cuda"), activation="none")
    out = out.double().cpu().numpy()
    a, b = (top * tiny) ** 2, top * tiny
    # (roundings of g, u, g * u and the sums: a few of 2^-24 each)
    np.testing.assert_allclose(out[0, :3], [a, 0.0, -a], rtol=2.0 ** -20)
    np.testing.assert_allclose(out[1, :3], [0.0, b, 0.0], rtol=2.0 ** -20)
    assert (out[:2, 3:] == 0).all() and np.isnan(out[3]).all()
    assert not np.isfinite(out[2, 0])


def test_experts_beyond_32_bits():
    """Experts further apart than 2^32 bytes."""
    import torch
    rng = np.random.default_rng(32)
    E, H, I, stride = 3, 96, 40, (1 << 31) + 8
    L = Experts(rng, E, H, I, torch.bfloat16)
    far = []
    for t in L.t:
        store = torch.empty(2 * stride + t.stride(0), dtype=torch.bfloat16, device="cuda")
        f = store.as_strided(t.shape, (stride,) + t.stride()[1:])
        f.copy_(t)
        far.append(f)
    x = torch.from_numpy(rng.standard_normal((5, H)).astype(np.float32)).cuda()
    ids = torch.tensor([[0, 2], [2, 1], [1, 0], [2, 2], [0, 1]], dtype=torch.int32, device="cuda")
    w = torch.rand(5, 2, device="cuda")
    out = fg.moe(x, *L.t, ids, w, torch.empty(5, H, device="cuda"))
    got = fg.moe(x, *far, ids, w, torch.empty(5, H, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    check(L, x, ids, w, got)


def test_two_calls_at_once():
    """Layers and split products on two streams, each with its own workspace."""
    import torch
    rng = np.random.default_rng(33)
    L = Experts(rng, 24, 1024, 512, torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(5)
    A, SA, _ = integers(g, 130, 20000, 1)
    B, SB, _ = integers(g, 33, 20000, 128)
    need = fg.fg_gemm_fp8_workspace_size(130, 33, 20000)
    assert need > 0
    T, k = 20, 4
    router = torch.from_numpy((rng.standard_normal((24, 1024)) / 32).astype(np.float32)).cuda()
    xs = [torch.randn(T, 1024, generator=g, device="cuda") for _ in range(2)]

    def state():
        e = lambda *s, **kw: torch.empty(*s, device="cuda", **kw)
        return dict(ids=e(T, k, dtype=torch.int32), w=e(T, k), out=e(T, 1024), C=e(130, 33),
                    ws=e(fg.fg_moe_workspace_size(T, k, 24, 1024, 512), dtype=torch.uint8),
                    wg=e(need, dtype=torch.uint8))

    def step(x, s, stream=None):
        fg.moe(x, *L.t, s["ids"], s["w"], s["out"], router=router, scales=L.scales,
               workspace=s["ws"], stream=stream)
        fg.gemm_fp8(A, SA, B, SB, s["C"], workspace=s["wg"], stream=stream)

    alone = [state(), state()]
    for x, s in zip(xs, alone):
        step(x, s)
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream(), torch.cuda.Stream()], [state(), state()]
    torch.cuda.synchronize()
    for _ in range(8):
        for x, s, st in zip(xs, both, streams):
            step(x, s, st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for n in ("ids", "w", "out", "C"):
            assert torch.equal(a[n], b[n]), n


def test_quantise_product_and_layer_in_one_graph():
    """A captured step (quantise both ways, split product, weight gradient added
    to C, layer of one token and of several) replayed on new values equals the
    eager one, with eager work between the replays."""
    import torch
    rng = np.random.default_rng(34)
    g = torch.Generator(device="cuda").manual_seed(6)
    L = Experts(rng, 12, 512, 256, torch.bfloat16)
    router = torch.from_numpy((rng.standard_normal((12, 512)) / 22).astype(np.float32)).cuda()
    X = torch.randn(20000, 130, generator=g, device="cuda")
    Y = torch.randn(20000, 33, generator=g, device="cuda")
    x = torch.randn(7, 512, generator=g, device="cuda").to(torch.bfloat16)
    need = fg.fg_gemm_fp8_workspace_size(130, 33, 20000)

    def buffers():
        e = lambda *s, **kw: torch.empty(*s, device="cuda", **kw)
        s = dict(C=torch.zeros(130, 33, device="cuda"), wg=e(need, dtype=torch.uint8),
                 ws=e(fg.fg_moe_workspace_size(7, 3, 12, 512, 256), dtype=torch.uint8),
                 ids=e(7, 3, dtype=torch.int32), w=e(7, 3), out=e(7, 512, dtype=torch.bfloat16),
                 ids1=e(1, 3, dtype=torch.int32), w1=e(1, 3), out1=e(1, 512, dtype=torch.bfloat16))
        s["X"], s["Y"] = fg.empty_fp8(130, 20000), fg.empty_fp8(33, 20000)
        return s

    def step(s):
        fg.quantize_fp8(X, None, None, *s["X"])
        fg.quantize_fp8(Y, None, None, *s["Y"])
        fg.gemm_fp8(*s["X"], *s["Y"], s["C"], beta=1.0, workspace=s["wg"])
        fg.moe(x, *L.t, s["ids"], s["w"], s["out"], router=router, workspace=s["ws"])
        fg.moe(s["out"][:1], *L.t, s["ids1"], s["w1"], s["out1"], router=router, workspace=s["ws"])

    a, b = buffers(), buffers()
    step(b)
    torch.cuda.synchronize()
    b["C"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    a["C"].zero_()
    for n in range(3):
        X.copy_(torch.randn(20000, 130, generator=g, device="cuda") * (n + 1))
        x.copy_(torch.randn(7, 512, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        for key in ("C", "ids", "w", "out", "ids1", "w1", "out1"):
            assert torch.equal(a[key], b[key]), (n, key)
        check(L, x, b["ids"], b["w"], b["out"])


def test_overlapping_scales_are_refused():
    """Scales of several blocks in one row of memory (a broadcast tensor)."""
    import torch
    X = torch.zeros(40, 300, device="cuda")
    q, s = fg.empty_fp8(40, 300)
    same = torch.ones(1, 40, device="cuda").expand(3, 40)
    C = torch.zeros(40, 40, device="cuda")
    with pytest.raises(fg.FgError):
        fg.quantize_fp8(X, q, same)
    fg.quantize_fp8(X, q, s)
    for sa, sb in ((same, s), (s, same)):
        with pytest.raises(fg.FgError):
            fg.gemm_fp8(q, sa, q, sb, C)
    fg.gemm_fp8(q, same.contiguous(), q, s, C)
    torch.cuda.synchronize()


def test_nothing_to_do():
    """Empty matrices and no tokens: accepted, nothing written."""
    import torch
    for M, N in ((0, 5), (5, 0), (0, 0)):
        q, s = fg.empty_fp8(M, N)
        fg.quantize_fp8(torch.empty(M, N, device="cuda"), q, s)
        B, SB = fg.empty_fp8(4, N)
        C = torch.full((M, 4), 3.0, device="cuda")
        fg.gemm_fp8(q, s, B, SB, C)
        assert (C == 0).all()
    L = Experts(np.random.default_rng(35), 2, 16, 16, torch.float32)
    e = torch.empty(0, 2, device="cuda")
    out = fg.moe(torch.empty(0, 16, device="cuda"), *L.t, e.int(), e,
                 torch.empty(0, 16, device="cuda"))
    assert out.shape == (0, 16)
