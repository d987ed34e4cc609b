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
