"""Products with 4-bit weights where columns of x differ much in size."""
import numpy as np
import pytest

import fp32_gemm_tile_amd as fg

from test_gpu_int4 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fg.load_library()
    yield
    torch.cuda.synchronize()


def weights(rng, N, K, group, zeros, columns):
    """Codes, whole scales that are powers of two, zero points; the codes of `columns` are their
    zero points. (on the GPU, values in binary64)"""
    import torch
    groups = -(-K // group)
    z = rng.integers(0, 16, (groups, N)) if zeros else np.full((groups, N), 8)
    q = rng.integers(0, 16, (N, K + K % 2))
    at = np.arange(K) // group
    for c in columns:
        q[:, c] = z[at[c]]
    s = 2.0 ** rng.integers(-1, 3, (groups, N))
    w = (q[:, :K] - z[at].T) * s[at].T
    half = -(-K // 32) * 16
    codes = torch.zeros(N, half, dtype=torch.uint8, device="cuda")[:, :(K + 1) // 2]
    codes.copy_(torch.from_numpy((q[:, ::2] | q[:, 1::2] << 4).astype(np.uint8)))
    return (codes, torch.from_numpy(s.astype(np.float32)).cuda(),
            torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None), w


@pytest.mark.parametrize("T", [1, 4, 16, 24, 50])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
def test_large_columns_at_their_zero_point_leave_no_error(T, group, zeros):
    """Whole numbers in binary32: every sum of (q - z) x is exact, those of q x are not
    where a column is 2^21 + 1 (15 times that has 25 bits)."""
    import torch
    rng = np.random.default_rng(T + group)
    for N, K in ((40, 300), (8200, 160)):
        big = [3, 77, 150]
        x = rng.integers(-3, 4, (T, K)).astype(np.float32)
        x[:, big] = rng.choice([-1, 1], (T, 3)) * (2.0 ** 21 + 1)
        xg = torch.zeros(T, -(-K // 4) * 4, device="cuda")[:, :K]
        xg.copy_(torch.from_numpy(x))
        (wg, vg), (wu, vu) = (weights(rng, N, K, group, zeros, big) for _ in range(2))
        out = torch.empty(T, N, device="cuda")
        print("  int4", T, N, K, group, zeros, flush=True)
        fg.gemm_int4(xg, wg, out, group=group)
        want = x.astype(np.float64) @ vg.T
        assert np.array_equal(out.double().cpu().numpy(), want)
        fg.gated_int4(xg, wg, wu, out, group=group, activation="none")
        both = want * (x.astype(np.float64) @ vu.T)     # (one rounding)
        assert (np.abs(out.double().cpu().numpy() - both) <= 2.0 ** -24 * np.abs(both)).all()


@pytest.mark.parametrize("T", [2, 9, 30, 64])
def test_small_values_of_x(T):
    """Binary32 x as three bfloat16 terms: exact above 2^-109, below it off by less than
    2^-133 an element, and 0 is 0."""
    import torch
    rng = np.random.default_rng(T)
    N, K, group = 33, 64, 32
    w, v = weights(rng, N, K, group, True, [])
    for e in (-80, -109, -115, -126):
        x = (rng.standard_normal((T, K)) * 2.0 ** e).astype(np.float32)
        x[:, 5] = 0
        out = torch.empty(T, N, device="cuda")
        fg.gemm_int4(torch.from_numpy(x).cuda(), w, out, group=group)
        size = np.abs(v).sum(1)
        want = x.astype(np.float64) @ v.T
        # K + 26 roundings of a binary32 sum, each also of at most half of 2^-149
        bound = (K + 26) * (2.0 ** -23 * (np.abs(x).astype(np.float64) @ np.abs(v).T) + 2.0 ** -149) + 2.0 ** -133 * size
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all(), e


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 13, 27, 64])
def test_both_numbers_of_rows_of_a_workgroup(T, ty):
    """4096 rows of W are 256 workgroups of 16; 4100 have 32 each where that is quicker."""
    for N in (4096, 4100):
        for gated in (False, True):
            check(T, N, 200, 64, ty, "bf16", True, gated, pad=1)
