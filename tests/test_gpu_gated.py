"""The gated feed-forward block on the GPU against the binary64 oracle."""
import itertools

import numpy as np
import pytest

import fp32_gemm_tile_amd as fg
from oracle import gated as og
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


def dtype_of(ty):
    import torch
    return torch.float32 if ty == "f32" else torch.bfloat16


def aligned(v, ty, extra=0):
    """v on the GPU, rows at multiples of 16 bytes (and `extra` such pieces more),
    NaN in the padding."""
    import torch
    per = 4 if ty == "f32" else 8
    R, C = v.shape
    base = torch.full((R, (-(-C // per) + extra) * per), float("nan"), dtype=dtype_of(ty), device="cuda")
    base[:, :C] = torch.from_numpy(np.ascontiguousarray(v)).cuda().to(base.dtype)
    return base[:, :C]


def guarded(R, C, ty, pad=3):
    """(R x C view of any alignment, its base) filled with 7."""
    import torch
    base = torch.full((R + 2, C + pad), 7.0, dtype=dtype_of(ty), device="cuda")
    return base[1:R + 1, 1:C + 1], base


def untouched(base, R, C):
    import torch
    ring = torch.ones_like(base, dtype=torch.bool)
    ring[1:R + 1, 1:C + 1] = False
    assert (base[ring] == 7.0).all()


def near(got, want, bound, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4],
                           want[bad][:4], bound[bad][:4])


class Case:
    def __init__(self, T, H, I, ty, seed=0, extra=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.ty, self.bf16 = T, H, I, ty, ty == "bf16"
        self.x = aligned(rng.standard_normal((T, H)) * spread, ty, extra)
        self.gate = aligned(rng.standard_normal((I, H)) * max(H, 1) ** -0.5, ty, extra)
        self.up = aligned(rng.standard_normal((I, H)) * max(H, 1) ** -0.5, ty, extra)
        self.rng = rng
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.v = f(self.x), f(self.gate), f(self.up)

    def workspace(self, n):
        import torch
        return torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN where read unwritten

    def forward(self, save="none", act="silu", ws=1 << 22, stream=None):
        """h and what was kept, checked."""
        import torch
        T, I, ty = self.T, self.I, self.ty
        h, hb = guarded(T, I, ty)
        saved, bases = None, []
        if save == "same":
            (g, gb), (u, ub) = guarded(T, I, ty), guarded(T, I, ty)
            saved, bases = (g, u), [gb, ub]
        elif save == "e4m3":
            saved = fg.empty_fp8(T, I) + fg.empty_fp8(T, I)
            for t in saved:
                t.view(torch.uint8).fill_(0x55) if t.dtype != torch.float32 else t.fill_(7.0)
        print("  gated", T, self.H, I, ty, save, act, ws, flush=True)
        fg.gated(self.x, self.gate, self.up, h, activation=act, saved=saved,
                 workspace=self.workspace(ws) if ws else None, stream=stream)
        torch.cuda.synchronize()
        for b in [hb] + bases:
            untouched(b, T, I)
        (vh, eh), (vg, eg), (vu, eu) = og.forward(*self.v, act, self.bf16)
        near(h, vh, eh, "h")
        if save == "same":
            near(saved[0], vg, eg, "G")
            near(saved[1], vu, eu, "U")
        elif save == "e4m3" and I:
            for codes, scales, v in ((saved[0], saved[1], vg), (saved[2], saved[3], vu)):
                self.check_codes(codes, scales, v)
        return h, saved

    def check_codes(self, codes, scales, v):
        _, e = og.products(*(self.v[:1] + (self.v[1],))) if v is None else (None, None)
        x = np.abs(self.v[0])
        e = (self.H + 16) * og.U * (x @ np.maximum(np.abs(self.v[1]), np.abs(self.v[2])).T)
        s = scales.double().cpu().numpy()
        T, I = v.shape
        for b in range(-(-I // 128)):
            blk, eb = v[:, 128 * b:128 * b + 128], e[:, 128 * b:128 * b + 128]
            most, em = np.abs(blk).max(1), eb.max(1)
            want = np.maximum(most / 448, 2.0 ** -126)
            assert (np.abs(s[b] - want) <= em / 448 + 2 * og.U * want).all()
            got = lowp.values(codes.view(__import__("torch").uint8).cpu().numpy()[:, 128 * b:128 * b + 128]) \
                * s[b][:, None]
            # half a step: 2^-4 relative, or half of 2^-9 scales for the smallest codes
            tol = eb * (1 + 2.0 ** -4) + np.maximum(np.abs(blk) * 2.0 ** -4, s[b][:, None] * 2.0 ** -10) * (1 + 2.0 ** -20)
            assert (np.abs(got - blk) <= tol).all()

    def kept(self, save):
        """(tensors as gated saves them, their binary64 values)."""
        import torch
        T, I, ty = self.T, self.I, self.ty
        v = [self.rng.standard_normal((T, I)) * 1.5 for _ in range(2)]
        if save == "same":
            out = []
            for a in v:
                t, _ = guarded(T, I, ty)
                t.copy_(torch.from_numpy(a))
                out.append(t)
            return tuple(out), [t.double().cpu().numpy() for t in out]
        out, vals = [], []
        for a in v:
            c, s = lowp.quantize(a.astype(np.float32), 1)
            q, sc = fg.empty_fp8(T, I)
            base = q.as_strided((T, q.stride(0)), (q.stride(0), 1)) if T else q
            base.view(torch.uint8).fill_(0x7F)     # NaN codes in the padding
            q.view(torch.uint8).copy_(torch.from_numpy(c))
            sc.copy_(torch.from_numpy(s))
            out += [q, sc]
            vals.append(lowp.stands_for(c, s, 1))
        return tuple(out), vals

    def backward(self, save="same", act="silu", beta=0.0, more_ws=1 << 22, parts=("dx", "dw", "h"),
                 stream=None):
        import torch
        T, H, I, ty = self.T, self.H, self.I, self.ty
        saved, (g, u) = self.kept(save)
        dh, _ = guarded(T, I, ty)
        dh.copy_(torch.from_numpy(self.rng.standard_normal((T, I))))
        new = {"dx": guarded(T, H, ty), "dgate": guarded(I, H, ty), "dup": guarded(I, H, ty),
               "h": guarded(T, I, ty)}
        old = {}
        for k in ("dgate", "dup"):
            if beta:
                new[k][0].copy_(torch.from_numpy(self.rng.standard_normal((I, H))))
            else:
                new[k][0].fill_(float("nan"))      # not read
            old[k] = new[k][0].double().cpu().numpy() if beta else 0.0
        need = fg.fg_gated_backward_min_workspace_size(T, I, int(self.bf16))
        print("  gated_backward", T, H, I, ty, save, act, beta, more_ws, parts, flush=True)
        want_w = "dw" in parts
        fg.gated_backward(dh, self.x, self.gate, self.up, saved,
                          new["dx"][0] if "dx" in parts else None,
                          new["dgate"][0] if want_w else None, new["dup"][0] if want_w else None,
                          new["h"][0] if "h" in parts else None, beta=beta, activation=act,
                          workspace=self.workspace(need + more_ws), stream=stream)
        torch.cuda.synchronize()
        want = og.backward(dh.double().cpu().numpy(), *self.v, g, u, act, self.bf16, beta,
                           old["dgate"], old["dup"])
        shapes = {"dx": (T, H), "dgate": (I, H), "dup": (I, H), "h": (T, I)}
        done = [k for k in want if k in parts or (want_w and k in ("dgate", "dup"))]
        for k in done:
            near(new[k][0], *want[k], k)
        for k in want:
            untouched(new[k][1], *shapes[k])
        return {k: new[k][0] for k in done}


FEW = [(1, 64, 16), (1, 1, 1), (2, 7, 5), (5, 33, 127), (16, 130, 40), (17, 100, 33), (32, 257, 64),
       (33, 64, 129), (48, 31, 17), (64, 300, 50)]
MANY = [(65, 64, 128), (70, 1, 3), (100, 33, 129), (129, 100, 260), (200, 300, 127), (300, 65, 64)]


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", FEW + MANY)
def test_forward(T, H, I, ty):
    c = Case(T, H, I, ty, seed=T + H + I)
    for save, act in (("none", "silu"), ("same", "gelu"), ("e4m3", "silu")):
        c.forward(save, act)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T", [9, 90])
def test_forward_every_activation_and_stride(ty, T):
    for act in ("none", "relu", "gelu", "silu"):
        Case(T, 70, 45, ty, seed=T, extra=3).forward("same", act)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_forward_every_tile(ty):
    """Whatever the library would choose: every tile, alone and with slices."""
    code = int(ty == "bf16")
    c = Case(150, 300, 330, ty, seed=8)
    few = Case(3, 300, 140, ty, seed=9)
    try:
        for tile, slices in itertools.product(range(len(fg.fg_gated_tiles(0, code))), (1, 2, 4)):
            assert fg.fg_set_gated_tile(0, code, tile, slices) == fg.FG_OK
            for save in ("none", "same", "e4m3"):
                c.forward(save)
                few.forward(save, "gelu")
    finally:
        fg.fg_set_gated_tile(0, code)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", FEW + MANY)
def test_backward(T, H, I, ty):
    c = Case(T, H, I, ty, seed=T + H + I)
    c.backward("same", "silu", 0.0)
    c.backward("e4m3", "gelu", 0.5)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_backward_every_activation_and_part(ty):
    c = Case(90, 70, 45, ty, seed=5, extra=2)
    for act in ("none", "relu", "gelu", "silu"):
        c.backward("same", act, 1.0, more_ws=0)
    for parts in (("dx",), ("dw",), ("h",), ("dx", "h"), ("dx", "dw")):
        c.backward("e4m3", "silu", 0.0, parts=parts)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("product", [1, 2])
def test_backward_every_tile(product, ty):
    code = int(ty == "bf16")
    c = Case(150, 330, 300, ty, seed=8)
    try:
        for tile, slices in itertools.product(range(len(fg.fg_gated_tiles(product, code))), (1, 2, 3, 4)):
            assert fg.fg_set_gated_tile(product, code, tile, slices) == fg.FG_OK
            c.backward("same", "silu", 0.0)
            c.backward("e4m3", "gelu", -1.5)
    finally:
        fg.fg_set_gated_tile(product, code)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_gate_and_up_of_different_strides(ty):
    import torch
    for T, H, I in ((7, 70, 45), (150, 330, 300)):
        c = Case(T, H, I, ty, seed=6)
        wide = torch.full((I, (H + 47) // 8 * 8), float("nan"), dtype=c.up.dtype, device="cuda")
        at = wide[:, 8:8 + H]
        at.copy_(c.up)
        c.up = at
        code = int(ty == "bf16")
        try:
            for tile, slices in ((-1, 0), (0, 2), (1, 1), (2, 4)):
                for product in (0, 1):
                    fg.fg_set_gated_tile(product, code, tile, slices)
                c.forward("same")
                c.backward("same", parts=("dx",))
        finally:
            for product in (0, 1):
                fg.fg_set_gated_tile(product, code)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", [(130, 1000, 1500), (33, 999, 1501), (300, 2048, 1408), (517, 1100, 900)])
def test_all_gradients_in_one_launch(T, H, I, ty):
    """Sizes at which dx is in the launch of dgate and dup, with slices and without."""
    if ty == "bf16" and T < 517:   # (the condition in bfloat16)
        assert fg.fg_select_gated(2, 1, T, H, I, 0) == (1, 1)
    c = Case(T, H, I, ty, seed=T, extra=1)
    c.backward("same", "silu", 0.0, more_ws=0)
    c.backward("e4m3", "gelu", 1.0, more_ws=1 << 25)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_as_many_rows_of_weights_as_change_the_kernel(ty):
    for T, I in ((3, 2500), (9, 2500), (16, 4100), (17, 2500)):
        c = Case(T, 70, I, ty, seed=I, extra=1)
        c.forward("same")
        c.forward("none", "gelu", ws=0)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 12, 40, 150])
def test_a_token_touches_its_own_row_only(ty, T):
    """Infinities and NaN in two tokens: the other rows' bits are what they were."""
    import torch
    c = Case(T, 130, 300, ty, seed=T)
    bad = [1, T - 1]
    good = [t for t in range(T) if t not in bad]

    def run():
        h, g, u = (torch.empty(T, 300, dtype=c.x.dtype, device="cuda") for _ in range(3))
        fg.gated(c.x, c.gate, c.up, h, saved=(g, u), workspace=c.workspace(1 << 20))
        dx = torch.empty(T, 130, dtype=c.x.dtype, device="cuda")
        fg.gated_backward(h, c.x, c.gate, c.up, (g, u), dx=dx)
        return h, g, u, dx

    before = run()
    c.x[1, 129] = float("inf")
    c.x[T - 1, 0] = float("nan")
    after = run()
    for a, b in zip(before, after):
        assert torch.equal(a[good], b[good])
    for t in after[:3]:
        assert torch.isnan(t[T - 1]).all()
    assert not torch.isfinite(after[1][1]).any()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T", [8, 300])
@pytest.mark.parametrize("ws", [0, 1 << 24])
def test_codes_beside_infinities_and_nan(ty, T, ws):
    """A block's scale and its other codes are those it has with zeros in the place of sums
    that are infinite or NaN, whose codes are NaN."""
    import torch
    c = Case(T, 130, 300, ty, seed=T)

    def run():
        saved = fg.empty_fp8(T, 300) + fg.empty_fp8(T, 300)
        h = torch.empty(T, 300, dtype=c.x.dtype, device="cuda")
        fg.gated(c.x, c.gate, c.up, h, saved=saved, workspace=c.workspace(ws) if ws else None)
        return [t.view(torch.uint8) if t.element_size() == 1 else t for t in saved]

    bad = [5, 64, 200]
    c.gate[bad] = 0
    clean = run()
    c.gate[5, 3], c.gate[64, 129], c.gate[200, 0] = float("inf"), -float("inf"), float("nan")
    dirty = run()
    good = [n for n in range(300) if n not in bad]
    assert torch.equal(clean[0][:, good], dirty[0][:, good])
    for a, b in zip(clean[1:], dirty[1:]):
        assert torch.equal(a, b)
    assert ((dirty[0][:, bad] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_long_rows(ty):
    """Rows so far apart that offsets pass 32 bits: the bits of compact ones."""
    import torch
    T, H, I, far = 1100, 40, 48, 1 << 21
    c = Case(T, H, I, ty, seed=3)

    def apart(t):
        out = torch.empty(t.shape[0], far, dtype=t.dtype, device="cuda")[:, :t.shape[1]]
        out.copy_(t)
        return out

    def run(place):
        x, gate, up = place(c.x), place(c.gate), place(c.up)
        h, g, u = (place(torch.zeros(T, I, dtype=x.dtype, device="cuda")) for _ in range(3))
        ws = c.workspace(1 << 24)
        fg.gated(x, gate, up, h, saved=(g, u), workspace=ws)
        few = place(torch.zeros(4, I, dtype=x.dtype, device="cuda"))
        fg.gated(x[:4], gate, up, few)
        dx = place(torch.zeros(T, H, dtype=x.dtype, device="cuda"))
        dg, du = (place(torch.ones(I, H, dtype=x.dtype, device="cuda")) for _ in range(2))
        fg.gated_backward(h, x, gate, up, (g, u), dx, dg, du, beta=0.5, workspace=ws)
        return [t.contiguous() for t in (h, g, u, few, dx, dg, du)]

    compact = run(lambda t: t)
    for a, b in zip(compact, run(apart)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_empty_sizes(ty):
    import torch
    dt = dtype_of(ty)
    z = lambda *s: torch.full(s, 3.0, dtype=dt, device="cuda")  # noqa: E731
    fg.gated(z(0, 8), z(8, 8), z(8, 8), z(0, 8))
    fg.gated(z(4, 8), z(0, 8), z(0, 8), z(4, 0))
    # no hidden size: empty sums
    for T in (4, 80):
        h, g, u = z(T, 8), z(T, 8), z(T, 8)
        fg.gated(z(T, 0), z(8, 0), z(8, 0), h, saved=(g, u))
        assert not h.any() and not g.any() and not u.any()
        q = fg.empty_fp8(T, 8) + fg.empty_fp8(T, 8)
        fg.gated(z(T, 0), z(8, 0), z(8, 0), h, saved=q)
        assert (q[1] == 2.0 ** -126).all() and not q[2].float().any()
    # no tokens: the weights' gradients are beta times what was there
    dg, du = z(8, 16), z(8, 16)
    fg.gated_backward(z(0, 8), z(0, 16), z(8, 16), z(8, 16), (z(0, 8), z(0, 8)), z(0, 16), dg, du, beta=0.5)
    assert (dg == 1.5).all() and (du == 1.5).all()
    fg.gated_backward(z(0, 8), z(0, 16), z(8, 16), z(8, 16), (z(0, 8), z(0, 8)), None, dg, du)
    assert not dg.any() and not du.any()
    # no inner size: dx is an empty sum
    dx = z(5, 16)
    fg.gated_backward(z(5, 0), z(5, 16), z(0, 16), z(0, 16), (z(5, 0), z(5, 0)), dx, z(0, 16), z(0, 16))
    assert not dx.any()


def test_codes_of_exact_sums():
    """Whole numbers: sums are exact, so codes and scales are the oracle's, bit for bit,
    with NaN and infinities as NaN codes outside the scale."""
    import torch
    rng = np.random.default_rng(1)
    T, H, I = 140, 48, 300
    c = Case(T, H, I, "bf16")
    for t in (c.x, c.gate, c.up):
        t.copy_(torch.from_numpy(rng.integers(-3, 4, tuple(t.shape)).astype(np.float32)))
    c.x[3, 5] = float("inf")
    c.x[7, 1] = float("nan")
    c.x[9].zero_()
    x, gate, up = (t.double().cpu().numpy() for t in (c.x, c.gate, c.up))
    with np.errstate(invalid="ignore"):
        want = [lowp.quantize((x @ w.T).astype(np.float32), 1) for w in (gate, up)]
    code = 1
    try:
        for tile in [-1] + list(range(len(fg.fg_gated_tiles(0, code)))):
            for slices in (1, 2):
                fg.fg_set_gated_tile(0, code, tile, slices)
                saved = fg.empty_fp8(T, I) + fg.empty_fp8(T, I)
                h = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
                fg.gated(c.x, c.gate, c.up, h, saved=saved, workspace=c.workspace(1 << 22))
                for k, (codes, scales) in enumerate(want):
                    got = saved[2 * k].view(torch.uint8).cpu().numpy()
                    nan = (codes & 0x7F) == 0x7F
                    assert ((got & 0x7F == 0x7F) == nan).all()
                    zero = ~nan & ((codes & 0x7F) == 0)      # (of either sign)
                    assert ((got & 0x7F)[zero] == 0).all()
                    assert (got == codes)[~nan & ~zero].all()
                    assert (saved[2 * k + 1].cpu().numpy() == scales).all()
    finally:
        fg.fg_set_gated_tile(0, code)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_at_the_activation_s_ends(ty, act):
    """Far from 0 and at the infinities: act' is 0 or 1, nothing becomes NaN."""
    import torch
    dt = dtype_of(ty)
    g = torch.tensor([[-float("inf"), -1e30, -200.0, -90.0, 0.0, 90.0, 200.0, 1e30, float("inf")]],
                     dtype=dt, device="cuda")
    one = torch.ones_like(g)
    I = g.shape[1]
    x = torch.ones(1, 8, dtype=dt, device="cuda")
    w = torch.zeros(I, 8, dtype=dt, device="cuda")
    dgate, dup = torch.empty_like(w), torch.empty_like(w)
    fg.gated_backward(one, x, w, w, (g, one), None, dgate, dup, activation=act)
    assert dgate[:, 0].tolist() == [0, 0, 0, 0, 0.5, 1, 1, 1, 1]
    got = dup[:, 0].tolist()
    assert got[4:] == g[0].tolist()[4:] and all(abs(v) < 1e-30 for v in got[1:4])


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_gradients_against_differences(ty):
    """The whole block, forward twice per direction, in the direction of its gradient."""
    import torch
    c = Case(70, 96, 128, "f32", seed=3)
    rng = np.random.default_rng(7)
    dh = torch.from_numpy(rng.standard_normal((c.T, c.I)).astype(np.float32)).cuda()
    mats = [c.x, c.gate, c.up]
    if ty == "bf16":
        mats = [m.bfloat16().contiguous() for m in mats]
    dt = mats[0].dtype
    h, g, u = (torch.empty(c.T, c.I, dtype=dt, device="cuda") for _ in range(3))
    fg.gated(*mats, h, saved=(g, u))
    d = [torch.empty(m.shape, dtype=dt, device="cuda") for m in mats]
    fg.gated_backward(dh.to(dt), *mats, (g, u), *d, out=h)

    def loss(ms):
        hh, _, _ = og.forward(*(m.double().cpu().numpy() for m in ms), "silu", False)
        return float((dh.to(dt).double().cpu().numpy() * hh[0]).sum())

    for k in range(3):
        way = [m.double() for m in mats]
        step = d[k].double()
        eps = 1e-4 / step.norm()
        lo, hi = list(way), list(way)
        hi[k], lo[k] = way[k] + eps * step, way[k] - eps * step
        slope = (loss(hi) - loss(lo)) / (2 * float(eps))
        # the gradient's length along itself; errors of its elements are roundings (bf16:
        # 2^-8 of each of the two it passes, and of G and U), which mostly cancel
        want = float((step * step).sum())
        assert slope == pytest.approx(want, rel=4 * 2.0 ** -8 if ty == "bf16" else 1e-4)


def test_a_training_step_and_a_captured_one():
    """Forward with an 8-bit checkpoint, a plain product, the gradients: eagerly and
    captured; another stream, replays with eager work between, equal bits."""
    import torch
    T, H, I = 130, 96, 200
    c = Case(T, H, I, "bf16", seed=2)
    rng = np.random.default_rng(2)
    saved = fg.empty_fp8(T, I) + fg.empty_fp8(T, I)
    out = {n: torch.empty(s, dtype=torch.bfloat16, device="cuda")
           for n, s in (("h", (T, I)), ("dx", (T, H)), ("dgate", (I, H)), ("dup", (I, H)), ("h2", (T, I)))}
    dh = torch.from_numpy(rng.standard_normal((T, I))).cuda().bfloat16()
    wf = c.workspace(fg.fg_gated_workspace_size(T, H, I, 1))
    wb = c.workspace(fg.fg_gated_backward_workspace_size(T, H, I, 1))

    def step():
        fg.gated(c.x, c.gate, c.up, out["h"], saved=saved, workspace=wf)
        fg.gated_backward(dh, c.x, c.gate, c.up, saved, out["dx"], out["dgate"], out["dup"],
                          out=out["h2"], workspace=wb)

    def everything():
        return [t.clone() for t in list(out.values()) + [s.view(torch.uint8) if s.dtype != torch.float32 else s
                                                         for s in saved]]

    step()
    torch.cuda.synchronize()
    first = everything()
    g = [lowp.stands_for(saved[k].view(torch.uint8).cpu().numpy(), saved[k + 1].cpu().numpy(), 1) for k in (0, 2)]
    want = og.backward(dh.double().cpu().numpy(), *c.v, *g, "silu", True)
    for k, t in (("dx", "dx"), ("dgate", "dgate"), ("dup", "dup"), ("h", "h2")):
        near(out[t], *want[k], k)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        for s in saved:
            s.view(torch.uint8).fill_(0x11)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, everything()):
            assert torch.equal(a, b)
        c.x.mul_(1.0)
        step()
        torch.cuda.synchronize()


def test_two_streams_and_repeated_calls_give_equal_bits():
    import torch
    for T in (20, 150):
        c = Case(T, 128, 256, "bf16", seed=T)
        outs = []
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for k in range(4):
            h = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
            torch.cuda.synchronize()
            fg.gated(c.x, c.gate, c.up, h, workspace=c.workspace(1 << 20), stream=streams[k % 2])
            outs.append(h)
        torch.cuda.synchronize()
        for h in outs[1:]:
            assert torch.equal(outs[0], h)


def test_wrong_tensors_are_refused():
    import torch
    c = Case(4, 16, 8, "bf16")
    h = torch.empty(4, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        fg.gated(c.x, c.gate.float(), c.up, h)
    with pytest.raises(ValueError):
        fg.gated(c.x, c.gate, c.up[:4], h)
    with pytest.raises(ValueError):
        fg.gated(c.x, c.gate, c.up, h.t())
    with pytest.raises(ValueError):
        fg.gated(c.x, c.gate, c.up, h, saved=(h,))
    with pytest.raises(fg.FgError):
        fg.gated(c.x, torch.zeros(8, 17, dtype=torch.bfloat16, device="cuda")[:, 1:], c.up, h)
    with pytest.raises(ValueError):
        fg.gated(c.x, c.gate, c.up, h, activation="tanh")
    with pytest.raises(fg.FgError):
        fg.gated_backward(h, c.x, c.gate, c.up, (h, h), dgate=torch.empty_like(c.gate))
    with pytest.raises(fg.FgError):
        fg.gated_backward(h, c.x, c.gate, c.up, (h, h), dx=torch.empty_like(c.x), workspace=h[:1])
