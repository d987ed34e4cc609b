"""The choice of the 8-bit product's tiles and slices, on the host."""
import pytest

import fp32_gemm_tile_amd as fg


@pytest.fixture(autouse=True)
def _chosen_by_the_library():
    yield
    assert fg.fg_set_fp8_tile(-1) == fg.FG_OK


def test_tiles():
    tiles = fg.fg_fp8_tiles()
    assert len(tiles) >= 4 and all(m % 16 == 0 and n % 32 == 0 for m, n in tiles)
    lib = fg.load_library()
    assert lib.fg_fp8_tile(-1, None, None) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 1
    assert lib.fg_fp8_tile(len(tiles), None, None) == fg.FG_ERR_INVALID_ARG
    assert lib.fg_fp8_tile(0, None, None) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 2
    for tile in (-2, len(tiles)):
        assert fg.fg_set_fp8_tile(tile) == fg.FG_ERR_INVALID_ARG and fg.fg_last_bad_arg() == 1


def test_selection_refusals():
    for bad, sizes in ((1, (0, 4, 4)), (2, (4, -1, 4)), (3, (4, 4, 0))):
        with pytest.raises(fg.FgError) as e:
            fg.fg_select_fp8(*sizes)
        assert e.value.status == fg.FG_ERR_INVALID_ARG and e.value.bad_arg == bad
    for sizes in ((1 << 31, 4, 4), (4, 4, fg.FG_MAX_LD + 1), (1 << 30, 1 << 30, 4)):
        with pytest.raises(fg.FgError) as e:
            fg.fg_select_fp8(*sizes)
        assert e.value.status == fg.FG_ERR_UNSUPPORTED
    lib = fg.load_library()
    assert lib.fg_select_fp8(4, 4, 4, 0, None, None) == fg.FG_ERR_INVALID_ARG
    assert fg.fg_last_bad_arg() == 5


def test_slices_need_their_workspace():
    split = 0
    for tile in [-1] + list(range(len(fg.fg_fp8_tiles()))):
        assert fg.fg_set_fp8_tile(tile) == fg.FG_OK
        for M, N, K in ((1, 33, 130), (130, 33, 20000), (256, 256, 65536), (517, 2047, 3001)):
            need = fg.fg_gemm_fp8_workspace_size(M, N, K)
            chosen, slices = fg.fg_select_fp8(M, N, K, need)
            assert tile in (-1, chosen) and need == (4 * slices * M * N if slices > 1 else 0)
            assert fg.fg_select_fp8(M, N, K)[1] == 1
            if need:
                assert fg.fg_select_fp8(M, N, K, need - 1)[1] < slices
                split += 1
    assert split > 0


def test_every_tile_is_chosen_somewhere():
    """No tile is built that no call reaches."""
    sizes = [(1, 8192, 8192), (32, 8192, 8192), (64, 8192, 8192), (517, 2047, 3001),
             (2048, 1024, 1024), (600, 4096, 4096), (2048, 2048, 2048), (4096, 4096, 4096)]
    sizes += [(M, N, K) for M in (64, 128, 256, 512, 1024) for N in (512, 1000, 2048)
              for K in (256, 1024, 4096)]
    chosen = {fg.fg_select_fp8(*s, fg.fg_gemm_fp8_workspace_size(*s))[0] for s in sizes}
    assert chosen == set(range(len(fg.fg_fp8_tiles())))
