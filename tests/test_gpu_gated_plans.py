"""The gated block's tiles with the slices that were asked for, against the binary64 oracle."""
import pytest

import fp32_gemm_tile_amd as fg

from test_gpu_gated import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fg.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("product,T,H,I", [(0, 40, 2040, 140), (1, 40, 130, 2040), (2, 2040, 72, 60)])
def test_every_tile_in_as_many_slices_as_asked_for(product, T, H, I, ty):
    code, ws = int(ty == "bf16"), 1 << 22
    c = Case(T, H, I, ty, seed=product)
    try:
        for tile in range(len(fg.fg_gated_tiles(product, code))):
            for slices in (2, 5, 8, 16):
                assert fg.fg_set_gated_tile(product, code, tile, slices) == fg.FG_OK
                assert fg.fg_select_gated(product, code, T, H, I, ws) == (tile, slices)
                if product == 0:
                    c.forward("same", ws=ws)
                    c.forward("e4m3", "gelu", ws=ws)
                else:
                    c.backward("same", beta=0.5, more_ws=ws, parts=("dx",) if product == 1 else ("dw",))
    finally:
        fg.fg_set_gated_tile(product, code)


@pytest.mark.parametrize("ty,T,H,I,alone,sliced", [
    ("f32", 517, 1001, 299, (64, 1), (64, 1)), ("f32", 333, 2047, 301, (64, 1), (64, 2)),
    ("f32", 130, 1000, 1500, None, (64, 8)), ("f32", 65, 1000, 2047, None, (64, 12)),
    ("bf16", 33, 999, 1501, (32, 1), (32, 1)), ("bf16", 130, 1000, 1500, (32, 1), (32, 1)),
    ("bf16", 300, 2047, 901, (64, 1), (64, 1))])
def test_the_launch_of_all_gradients(ty, T, H, I, alone, sliced):
    """dx beside dgate and dup, in one slice and in several: (rows of dx's tile, slices) with and
    without room for partial sums, None: two launches."""
    code = int(ty == "bf16")
    c = Case(T, H, I, ty, seed=T, extra=1)
    for more, want in ((0, alone), (1 << 25, sliced)):
        tile, slices = fg.fg_select_gated_pair(code, T, H, I, more)
        assert (None if tile < 0 else (fg.fg_gated_tiles(1, code)[tile][0], slices)) == want
        c.backward("same", "silu", 0.0, more_ws=more)
        c.backward("e4m3", "gelu", 1.0, more_ws=more)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_activations_of_the_infinities(ty, act):
    """G = -inf, +inf and NaN: h forward (weights streamed and tiles) and again backward, and
    the gradients, as the formulas say."""
    import torch
    inf, nan = float("inf"), float("nan")
    dt = torch.float32 if ty == "f32" else torch.bfloat16
    below = nan if act in ("silu", "gelu") else 0.0 if act == "relu" else -inf
    want = torch.tensor([below, inf, nan, 0.0], dtype=torch.float64)
    slope = torch.tensor([1.0 if act == "none" else 0.0, 1.0, 1.0 if act == "none" else nan,
                          {"silu": 0.5, "gelu": 0.5, "relu": 0.0, "none": 1.0}[act]], dtype=torch.float64)
    same = lambda a, b: torch.equal(torch.nan_to_num(a.double().cpu(), nan=7.0), torch.nan_to_num(b, nan=7.0))  # noqa: E731
    for T in (1, 40):
        x = torch.ones(T, 8, dtype=dt, device="cuda")
        gate, up = torch.zeros(4, 8, dtype=dt, device="cuda"), torch.zeros(4, 8, dtype=dt, device="cuda")
        gate[0, 0], gate[1, 0], gate[2, 0], up[:, 0] = -inf, inf, nan, 1.0
        h, g, u, again = (torch.empty(T, 4, dtype=dt, device="cuda") for _ in range(4))
        fg.gated(x, gate, up, h, activation=act, saved=(g, u))
        one = torch.ones_like(h)
        dgate, dup = torch.empty_like(gate), torch.empty_like(up)
        fg.gated_backward(one, x, gate, up, (g, u), None, dgate, dup, out=again, activation=act)
        for t in range(T):
            assert same(h[t], want) and same(again[t], want)
        assert same(dgate[:, 1], slope * T) and same(dup[:, 1], want * T)


def test_dx_in_binary32_adds_two_sums():
    """dG gate is 2^24 and dU up 256 times 2^-3: whole beside each other, lost in one running
    sum. Every tile, in one slice and in several, and the launch of all gradients."""
    import torch
    I = 256

    def run(T, H, all_three):
        x, ones = torch.zeros(T, H, device="cuda"), torch.ones(T, I, device="cuda")
        gate, up = torch.full((I, H), 2.0 ** 24 / I, device="cuda"), torch.full((I, H), 2.0 ** -3, device="cuda")
        dx = torch.empty(T, H, device="cuda")
        dw = [torch.empty_like(gate) for _ in range(2)] if all_three else [None, None]
        fg.gated_backward(ones, x, gate, up, (ones, ones), dx, *dw, activation="none")
        assert (dx == 2.0 ** 24 + 32).all()

    try:
        for tile in range(len(fg.fg_gated_tiles(1, 0))):
            for slices in (1, 2, 3):
                assert fg.fg_set_gated_tile(1, 0, tile, slices) == fg.FG_OK
                run(70, 40, False)
    finally:
        fg.fg_set_gated_tile(1, 0)
    assert fg.fg_select_gated_pair(0, 517, 1000, I, 0)[0] >= 0
    run(517, 1000, True)
