"""Which kernels the gated block runs, as the tuning hooks tell it: host only."""
import ctypes

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


@pytest.mark.parametrize("T,H,I", [(300, 256, 8192), (200, 512, 8192), (64, 512, 8192), (100, 512, 4096),
                                   (17, 1024, 4096)])
def test_a_long_sum_of_few_tiles_is_not_beside_the_weights_gradients(T, H, I):
    """dx in bfloat16 is one slice in the launch of dgate and dup; 53 us against 27 for
    64 x 512 x 8192 in two launches, where it has sixteen."""
    assert fg.fg_select_gated(1, 1, T, H, I, BIG)[1] > 1
    assert fg.fg_select_gated_pair(1, T, H, I, BIG) == (-1, 0)


def test_short_sums_are():
    """Sizes at which one launch is quicker: 200 x 2048 x 1408 21 us, 27 in two."""
    for T, H, I in ((64, 2048, 1408), (200, 2048, 1408), (300, 2048, 1408), (200, 4096, 512), (300, 1024, 4096)):
        tile, slices = fg.fg_select_gated_pair(1, T, H, I, BIG)
        assert slices == 1 and fg.fg_gated_tiles(1, 1)[tile] in ((32, 64), (64, 64))


def test_the_pair_s_arguments():
    for args, bad in (((2, 1, 1, 1), 1), ((0, 0, 1, 1), 2), ((0, 1, 0, 1), 3), ((0, 1, 1, 0), 4)):
        with pytest.raises(fg.FgError) as e:
            fg.fg_select_gated_pair(*args)
        assert e.value.bad_arg == bad
    lib, out = fg.load_library(), ctypes.c_int32()
    ref = ctypes.byref(out)
    for args, bad in (((None, ref), 6), ((ref, None), 7)):
        assert lib.fg_select_gated_pair(0, 1, 1, 1, 0, *args) == fg.FG_ERR_INVALID_ARG
        assert fg.fg_last_bad_arg() == bad
    try:   # a set tile or number of slices is run in launches of their own
        for product, tile, slices in ((1, 3, 0), (2, 1, 0), (1, -1, 1)):
            assert fg.fg_set_gated_tile(product, 1, tile, slices) == fg.FG_OK
            assert fg.fg_select_gated_pair(1, 200, 2048, 1408, BIG) == (-1, 0)
            assert fg.fg_set_gated_tile(product, 1) == fg.FG_OK
    finally:
        for product in (1, 2):
            fg.fg_set_gated_tile(product, 1)


def test_no_workspace_beyond_the_reported_one_changes_a_plan():
    for T in (17, 64, 65, 100, 130, 300, 517, 1025):
        for H in (64, 300, 1000, 1536, 4096):
            for I in (48, 300, 1408, 2047, 8192):
                for ty in (0, 1):
                    room = fg.fg_gated_workspace_size(T, H, I, ty)
                    assert fg.fg_select_gated(0, ty, T, H, I, room) == fg.fg_select_gated(0, ty, T, H, I, BIG)
                    room = (fg.fg_gated_backward_workspace_size(T, H, I, ty)
                            - fg.fg_gated_backward_min_workspace_size(T, I, ty))
                    pair = fg.fg_select_gated_pair(ty, T, H, I, BIG)
                    assert fg.fg_select_gated_pair(ty, T, H, I, room) == pair, (T, H, I, ty)
                    for product in (1, 2):
                        assert (fg.fg_select_gated(product, ty, T, H, I, room)
                                == fg.fg_select_gated(product, ty, T, H, I, BIG))
