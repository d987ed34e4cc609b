"""The mixture-of-experts layer on the GPU against the binary64 oracle."""
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


class Layer:
    """Random weights in the tensors fg.moe takes and in binary64. Padding of
    every row is NaN (codes or values)."""

    def __init__(self, rng, E, H, I, wt, extra=0):
        import torch
        self.E, self.H, self.I, self.wt = E, H, I, wt
        self.t, self.s, self.v = [], [], []
        for R, C in ((I, H), (I, H), (H, I)):
            w = (rng.standard_normal((E, R, C)) * C ** -0.5).astype(np.float32)
            if wt == "e4m3":
                per = 16
                q = [lowp.quantize(m, 128) for m in w]
                codes = np.stack([c for c, _ in q])
                sc = np.stack([s for _, s in q])
                base = torch.full((E, R, -(-C // per) * per + extra * per), 0x7F,
                                  dtype=torch.uint8, device="cuda")
                base[:, :, :C] = torch.from_numpy(codes).cuda()
                self.s.append(torch.from_numpy(sc).cuda())
                self.v.append(np.stack([lowp.stands_for(c, s, 128) for c, s in q]))
            else:
                dt = torch.float32 if wt == "f32" else torch.bfloat16
                per = 4 if wt == "f32" else 8
                base = torch.full((E, R, -(-C // per) * per + extra * per), float("nan"), dtype=dt,
                                  device="cuda")
                base[:, :, :C] = torch.from_numpy(w).cuda().to(dt)
                self.v.append(base[:, :, :C].double().cpu().numpy())
            self.t.append(base[:, :, :C])
        self.scales = tuple(self.s) if wt == "e4m3" else None


def tokens(rng, T, H, xt, pad=0):
    import torch
    x = torch.from_numpy(rng.standard_normal((T, H + pad)).astype(np.float32)).cuda()
    return x.to(torch.float32 if xt == "f32" else torch.bfloat16)[:, :H]


def run(L, x, ids, w, router=None, renorm=True, act="silu", ws=None, pad=0, stream=None):
    import torch
    T, k = ids.shape
    if ws is None:
        ws = torch.full((fg.fg_moe_workspace_size(T, k, L.E, L.H, L.I),), 0xFF, dtype=torch.uint8,
                        device="cuda")     # NaN wherever it is read unwritten
    base = torch.full((T, L.H + pad), 7.0, dtype=x.dtype, device="cuda")
    out = base[:, :L.H]
    print("  moe", T, L.E, k, L.H, L.I, x.dtype, L.wt, router is not None, renorm, act, flush=True)
    fg.moe(x, *L.t, ids, w, out, router=router, renormalize=renorm, scales=L.scales,
           activation=act, workspace=ws, stream=stream)
    if stream is None:
        torch.cuda.synchronize()
        assert (base[:, L.H:] == 7.0).all()
    return out


def check(L, x, ids, w, out, act="silu"):
    import torch
    bf16 = x.dtype == torch.bfloat16
    want, bound = lowp.layer(x.double().cpu().numpy(), *L.v, ids.cpu().numpy(),
                             w.double().cpu().numpy(), act, h_bits=16 if bf16 else 24)
    if bf16:
        bound = bound + lowp.bf16_half_step(np.abs(want) + bound)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


CASES = [  # T, E, k, H, I
    (1, 1, 1, 1, 1), (1, 8, 2, 256, 128), (2, 5, 3, 130, 33), (3, 64, 6, 100, 50),
    (17, 8, 2, 384, 160), (40, 4, 4, 257, 129), (64, 3, 2, 64, 48), (5, 512, 16, 40, 24),
]


@pytest.mark.parametrize("wt", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_layer_with_router(wt, xt):
    import torch
    rng = np.random.default_rng(21)
    for n, (T, E, k, H, I) in enumerate(CASES):
        L = Layer(rng, E, H, I, wt, extra=n % 2)
        x = tokens(rng, T, H, xt, pad=(0, 3)[n % 2])
        rt = torch.float32 if n % 3 else torch.bfloat16
        router = torch.from_numpy((rng.standard_normal((E, H + n % 2)) * H ** -0.5)
                                  .astype(np.float32)).cuda().to(rt)[:, :H]
        ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), float("nan"), device="cuda")
        renorm = n % 2 == 0
        out = run(L, x, ids, w, router, renorm, pad=n % 4)
        want_ids, want_w = lowp.route(x.double().cpu().numpy(), router.double().cpu().numpy(), k,
                                      renorm)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        # exp of a difference rounded to binary32 (|difference| * 2^-24), a sum
        # of at most 512 terms and one division
        spread = 40.0
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=(spread / 2 + 520 + 8) * 2.0 ** -23,
                                   atol=2.0 ** -126)
        check(L, x, ids, w, out)


@pytest.mark.parametrize("wt", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_layer_with_given_routing(wt, act):
    """Empty slots, tokens with none filled, ids out of range, one expert twice
    in a token, one expert for every token."""
    import torch
    rng = np.random.default_rng(22)
    for T, E, k, H, I, xt in ((1, 3, 2, 64, 32, "f32"), (6, 4, 3, 136, 72, "bf16"),
                              (64, 6, 4, 200, 144, "f32")):
        L = Layer(rng, E, H, I, wt)
        x = tokens(rng, T, H, xt)
        ids = torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).cuda()
        w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        check(L, x, ids, w, run(L, x, ids, w, act=act), act)
        ids[0] = -1                       # nothing for token 0
        if T > 1:
            ids[1], ids[2, 0] = E + 5, -7  # out of range
            ids[3] = 1                    # the same expert in every slot
            w[2, 0] = float("nan")        # an empty slot's weight is not used
        out = run(L, x, ids, w, act=act)
        assert (out[0] == 0).all()
        w2 = torch.where((ids >= 0) & (ids < E), w, torch.zeros_like(w))
        check(L, x, ids, w2, out, act)
        ids.fill_(2)
        check(L, x, ids, w2, run(L, x, ids, w2, act=act), act)
        ids.fill_(-1)
        assert (run(L, x, ids, w, act=act) == 0).all()


def test_router_ties_nans_and_near_logits():
    """Equal logits go to the lowest expert; a NaN logit ranks last; logits
    that differ by less than binary32 holds keep their order."""
    import torch
    rng = np.random.default_rng(23)
    E, H, k = 130, 64, 5
    L = Layer(rng, E, H, 16, "bf16")
    x = torch.ones(2, H, device="cuda")
    router = torch.zeros(E, H, device="cuda")
    ids = torch.empty(2, k, dtype=torch.int32, device="cuda")
    w = torch.empty(2, k, device="cuda")
    run(L, x, ids, w, router)
    assert (ids.cpu().numpy() == np.arange(k)).all()
    router[:, 0] = 1000.0
    router[77, 1] = 2.0 ** -20      # 1000 + 2^-20 is 1000 in binary32
    router[100, 1] = 2.0 ** -19
    run(L, x, ids, w, router)
    assert (ids.cpu().numpy() == [100, 77, 0, 1, 2]).all()
    router[100, 3] = float("nan")
    run(L, x, ids, w, router)
    assert (ids.cpu().numpy() == [77, 0, 1, 2, 3]).all()
    x[1, 5] = float("nan")
    out = run(L, x, ids, w, router)
    assert (ids[1].cpu().numpy() == np.arange(k)).all() and torch.isnan(w[1]).all()
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()


def test_repeats_streams_graph():
    """Identical bits from repeated calls and on another stream; a captured
    call replayed on new tokens equals the eager one."""
    import torch
    rng = np.random.default_rng(24)
    T, E, k, H, I = 9, 16, 4, 512, 256
    L = Layer(rng, E, H, I, "e4m3")
    x = tokens(rng, T, H, "bf16")
    router = torch.from_numpy((rng.standard_normal((E, H)) * H ** -0.5).astype(np.float32)).cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    need = fg.fg_moe_workspace_size(T, k, E, H, I)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    first = run(L, x, ids, w, router, ws=ws).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = run(L, x, ids, w, router, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    gout = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        fg.moe(x, *L.t, ids, w, gout, router=router, scales=L.scales, workspace=ws)
    for n in range(3):
        x.copy_(tokens(rng, T, H, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = gout.clone()
        i2, w2 = torch.empty_like(ids), torch.empty_like(w)
        eager = run(L, x, i2, w2, router)
        assert torch.equal(got, eager) and torch.equal(ids, i2) and torch.equal(w, w2)
        check(L, x, i2, w2, eager)


def test_quantised_experts_end_to_end():
    """Weights quantised by the library (128 x 128 blocks), used by the layer:
    the result is that of the values the codes stand for."""
    import torch
    rng = np.random.default_rng(25)
    T, E, k, H, I = 4, 6, 2, 300, 200
    tens, scales, vals = [], [], []
    for R, C in ((I, H), (I, H), (H, I)):
        w = torch.from_numpy((rng.standard_normal((E, R, C)) * C ** -0.5).astype(np.float32)).cuda()
        q = torch.empty(E, R, -(-C // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")[:, :, :C]
        s = torch.empty(E, -(-C // 128), -(-R // 128), device="cuda")
        for e in range(E):
            fg.quantize_fp8(w[e], q[e], s[e], block="tile")
        tens.append(q)
        scales.append(s)
        vals.append(np.stack([lowp.stands_for(q[e].view(torch.uint8).cpu().numpy(),
                                              s[e].cpu().numpy(), 128) for e in range(E)]))
    x = tokens(rng, T, H, "f32")
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    out = fg.moe(x, *tens, ids, w, torch.empty(T, H, device="cuda"), scales=tuple(scales))
    want, bound = lowp.layer(x.double().cpu().numpy(), *vals, ids.cpu().numpy(),
                             w.double().cpu().numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


def test_moe_wrapper_refuses():
    import torch
    rng = np.random.default_rng(26)
    L = Layer(rng, 4, 32, 16, "bf16")
    x = tokens(rng, 2, 32, "f32")
    ids = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 2, device="cuda")
    out = torch.zeros(2, 32, device="cuda")
    ok = lambda **kw: fg.moe(*[kw.get(n, v) for n, v in (
        ("x", x), ("gate", L.t[0]), ("up", L.t[1]), ("down", L.t[2]), ("ids", ids), ("w", w),
        ("out", out))], **{n: v for n, v in kw.items() if n in ("router", "scales", "workspace")})
    ok()
    for bad in (dict(out=out.bfloat16()), dict(ids=ids.long()), dict(w=w.double()),
                dict(w=w[:, :1]), dict(up=L.t[1][:3]), dict(down=L.t[0]),
                dict(router=torch.zeros(4, 31, device="cuda")), dict(ids=ids.t().t()[:1])):
        with pytest.raises((ValueError, TypeError)):
            ok(**bad)
    with pytest.raises(TypeError):
        ok(up=L.t[1].float())
    with pytest.raises(fg.FgError):
        ok(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
