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
