"""Which kernels the gated block runs, as the tuning hooks tell it: host only."""
import pytest

import fp32_gemm_tile_amd as fg

BIG = 1 << 40   # bytes of workspace
# sizes (T, H, I) whose sums, by product, are of 16384 terms
LONG = {0: (150, 16384, 300), 1: (150, 330, 16384), 2: (16384, 330, 300)}


@pytest.mark.parametrize("product,ty", [(p, t) for p in (0, 1, 2) for t in (0, 1)])
def test_a_forced_number_of_slices_is_what_runs(product, ty):
    try:
        for tile in range(len(fg.fg_gated_tiles(product, ty))):
            for n in range(1, 17):
                assert fg.fg_set_gated_tile(product, ty, tile, n) == fg.FG_OK
                assert fg.fg_select_gated(product, ty, *LONG[product], BIG) == (tile, n)
        for n in range(1, 17):
            assert fg.fg_set_gated_tile(product, ty, -1, n) == fg.FG_OK
            assert fg.fg_select_gated(product, ty, *LONG[product], BIG)[1] == n
    finally:
        fg.fg_set_gated_tile(product, ty)


def test_forced_slices_that_do_not_fit():
    """Eight steps (512 columns of bfloat16 by 128 bytes): the most slices below the forced
    number that are as many parts of them; and as many as the workspace holds."""
    parts = {1: 1, 2: 2, 3: 3, 4: 4, 5: 4, 6: 4, 7: 4}
    try:
        for n in range(1, 17):
            assert fg.fg_set_gated_tile(0, 1, 4, n) == fg.FG_OK
            assert fg.fg_select_gated(0, 1, 32, 512, 8192, BIG) == (4, parts.get(n, 8))
            slices = 32 * 8192 * 4 * 2   # bytes of one slice's sums of G and U
            for room in (1, 3, 4, 7):
                assert fg.fg_select_gated(0, 1, 32, 512, 8192, room * slices) == (4, parts[min(n, room)])
    finally:
        fg.fg_set_gated_tile(0, 1)


def test_larger_numbers_of_slices_are_considered():
    """32 steps do not divide into 12 parts, but into 16."""
    assert fg.fg_select_gated(1, 1, 20, 512, 2047, BIG) == (4, 16)
    assert fg.fg_select_gated(1, 0, 20, 2048, 1024, BIG) == (3, 16)
