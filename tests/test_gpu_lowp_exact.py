"""The 8-bit product and the mixture-of-experts layer where a sum's low bits,
a factor's range or an infinite operand decides the result."""
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


# ---- product -----------------------------------------------------------------

def on_device(codes, scales):
    """Codes in rows of whole 16 bytes, and scales, on the device."""
    import torch
    q = torch.zeros(codes.shape[0], -(-codes.shape[1] // 16) * 16, dtype=torch.uint8, device="cuda")
    q[:, :codes.shape[1]] = torch.from_numpy(codes).cuda()
    return q[:, :codes.shape[1]], torch.from_numpy(scales).cuda()


def product(A, SA, B, SB, dt, C=None, **kw):
    import torch
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    if C is None:
        C = torch.empty(M, N, dtype=dt, device="cuda")
    ws = torch.empty(max(16, fg.fg_gemm_fp8_workspace_size(M, N, K)), dtype=torch.uint8,
                     device="cuda")
    print("  product", M, N, K, tuple(SB.shape), dt, kw, flush=True)
    fg.gemm_fp8(*on_device(A, SA), *on_device(B, SB), C, workspace=ws, **kw)
    torch.cuda.synchronize()
    return C


def cancelling(rng, M, N, K, tall):
    """Codes whose blocks hold 448 * 448 and -448 * 448 beside products of
    integers -8 .. 8, unit scales, and the exact product."""
    ints = lowp.nearest_codes(np.arange(-8, 9).astype(np.float64))
    A, B = rng.choice(ints, (M, K)), rng.choice(ints, (N, K))
    top, bottom = lowp.nearest_codes(np.array([448.0, -448.0]))
    for k in range(0, K - 1, 128):
        i, j = k + rng.permutation(min(128, K - k))[:2]
        A[:, i], A[:, j], B[:, i], B[:, j] = top, top, top, bottom
    SA = np.ones((lowp.cdiv(K, 128), M), np.float32)
    SB = np.ones((lowp.cdiv(K, 128), lowp.cdiv(N, tall)), np.float32)
    return A, SA, B, SB, lowp.values(A) @ lowp.values(B).T


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("M,N,K", [(1, 33, 128), (20, 100, 130), (64, 257, 1000), (130, 130, 300),
                                   (300, 520, 640), (1100, 1030, 256), (2100, 2050, 200)])
def test_block_sums_keep_what_large_products_leave(M, N, K, tall):
    """Products of integers of which two per block are +-448^2: every partial
    sum is an integer below 2^24 and so exact in binary32, whatever the order; C
    is that sum, or the bfloat16 nearest to it."""
    import torch
    A, SA, B, SB, want = cancelling(np.random.default_rng(M + N + K), M, N, K, tall)
    want = torch.from_numpy(want)
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(product(A, SA, B, SB, dt).cpu(), want.to(dt))


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_small_products_beside_large_ones(out):
    """Sums of 126 products of 4 beside two of +-448^2: the bound of a binary32
    sum (4: a unit in the last place of 2^18 for each of 128 additions) is far
    below the 504 that a sum without the small products would lose."""
    import torch
    K, dt = 128, torch.float32 if out == "f32" else torch.bfloat16
    rng = np.random.default_rng(41)
    big, two = lowp.nearest_codes(np.array([448.0, 2.0]))
    for M, N in ((1, 40), (64, 64), (200, 300), (700, 600)):
        A, B = np.full((M, K), two), np.full((N, K), two)
        A[:, 0], A[:, 1], B[:, 0], B[:, 1] = big, big | 0x80, big, big
        perm = rng.permutation(K)
        C = product(A[:, perm], np.ones((1, M), np.float32), B[:, perm],
                    np.ones((1, N), np.float32), dt).double()
        # (504 is a bfloat16; numbers next to it are 2 apart)
        assert (C - 504.0).abs().max().item() <= 128 * 2.0 ** -5 + (1.0 if out == "bf16" else 0.0)


# ---- layer -------------------------------------------------------------------

WEIGHTS = {"e4m3": "float8_e4m3fn", "bf16": "bfloat16", "f32": "float32"}


def experts(values, wt, scale=1.0):
    """[1, R, C] weights (times 1 / scale, which the codes' scales undo) and, for
    codes, their scales."""
    import torch
    R, C = values.shape
    t = torch.zeros(1, R, -(-C // 16) * 16, dtype=getattr(torch, WEIGHTS[wt]), device="cuda")
    t[0, :, :C] = torch.from_numpy(values / scale).float().to(t.dtype).cuda()
    s = torch.full((1, lowp.cdiv(C, 128), lowp.cdiv(R, 128)), scale, device="cuda")
    return t[:, :, :C], s


def one_expert(x, gate, up, down, wt, scale=1.0, act="none", weight=1.0):
    """The layer with one expert, which every token chooses."""
    import torch
    T = x.shape[0]
    (g, sg), (u, su), (d, sd) = (experts(v, wt, scale if wt == "e4m3" else 1.0)
                                 for v in (gate, up, down))
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), weight, device="cuda")
    print("  layer", T, gate.shape, wt, x.dtype, act, flush=True)
    out = fg.moe(x, g, u, d, ids, w, torch.empty(T, down.shape[0], dtype=x.dtype, device="cuda"),
                 scales=(sg, su, sd) if wt == "e4m3" else None, activation=act)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


@pytest.mark.parametrize("wt", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_h_keeps_its_bits(T, xt, wt):
    """h[0] = (1 + 2^-12)(1 + 2^-10) and h[1] = 1 + 2^-10 + 2^-12 are binary32
    numbers whose difference is 2^-22, exact through every sum."""
    import torch
    H, I = 24, 20
    x = torch.zeros(T, H, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -12
    gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
    gate[0, [0, 2]], up[0, [0, 1]] = 1.0, 1.0
    gate[1, 0], up[1, [0, 1, 2]] = 1.0, 1.0
    down[3, 0], down[3, 1], down[4, 1] = 1.0, -1.0, 2.0
    out = one_expert(x.to(getattr(torch, xt)), gate, up, down, wt)
    assert (out[:, 3] == 2.0 ** -22).all()
    assert (np.abs(out[:, 4] - 2.0) < 2.0 ** -7).all() and (out[:, 5:] == 0).all()


@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 6, 64])
@pytest.mark.parametrize("H,I", [(300, 40), (210, 3000)])
def test_codes_of_scaled_weights_reach_the_largest_values(H, I, T, xt):
    """A weight of 1 held as code 256 with scale 2^-8: x and h up to the largest
    number of their type stay finite, and cancel, though 256 x does not."""
    import torch
    dt = getattr(torch, xt)
    top = float(torch.finfo(dt).max)
    x = torch.zeros(T, H, device="cuda", dtype=dt)
    x[:, 0], x[:, 1], x[:, 2], x[:, 200] = top, -top, 2.0 ** -100, 0.5
    gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
    gate[0, 0], up[0, 2] = 1.0, 1.0                       # h[0] = top 2^-100
    gate[1, [0, 1, 200]], up[1, 200] = 1.0, 1.0           # h[1] = (top - top + 0.5) 0.5
    gate[2, 1], up[2, 200] = 1.0, 1.0                  # h[2] = -top / 2
    gate[3, 200], up[3, 0] = 1.0, 1.0                     # h[3] = top / 2
    gate[I - 1], up[I - 1] = gate[3], up[3]               # h[I - 1] = top / 2
    down[0, 0], down[1, 1], down[2, 2], down[3, [2, 3]] = 1.0, 1.0, 1.0, 1.0
    down[4, 1], down[H - 1, I - 1] = 0.5, 1.0
    out = one_expert(x, gate, up, down, "e4m3", scale=2.0 ** -8)
    want = np.array([top * 2.0 ** -100, 0.25, -top / 2, 0.0, 0.125])
    # (products by powers of two, sums that cancel exactly: every step is exact)
    np.testing.assert_array_equal(out[:, :5], np.tile(want, (T, 1)))
    assert (out[:, 5:H - 1] == 0).all() and (out[:, H - 1] == top / 2).all()


def test_codes_beside_scales_of_any_size():
    """Large weights on small tokens and small weights on large ones: the
    result, not code * x, decides what is finite."""
    import torch
    H, I = 140, 33
    for e in (-126, -60, 0, 60, 119):
        x = torch.zeros(5, H, device="cuda")
        x[:, 0], x[:, 130] = 2.0 ** min(127, 8 - e), 1.0
        gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
        gate[0, 0] = 2.0 ** e * 256
        g, sg = experts(gate, "e4m3", 2.0 ** e)
        up[0, 130] = 1.0
        u, su = experts(up, "e4m3")
        down[0, 0] = 1.0
        d, sd = experts(down, "e4m3")
        ids = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
        out = fg.moe(x, g, u, d, ids, torch.ones(5, 1, device="cuda"),
                     torch.empty(5, H, device="cuda"), scales=(sg, su, sd), activation="none")
        assert (out[:, 0].double() == 2.0 ** (e + 8 + min(127, 8 - e))).all(), e


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_scales_whose_product_leaves_binary32(out, tall):
    """Factors SA * SB below the smallest and above the largest binary32 number,
    with results that are inside: rows, columns and blocks of K of many sizes."""
    import torch
    dt = torch.float32 if out == "f32" else torch.bfloat16
    rng = np.random.default_rng(43)
    for M, N, K in ((1, 70, 300), (40, 200, 300), (130, 150, 128), (300, 700, 200)):
        A, _ = lowp.quantize(rng.standard_normal((M, K)).astype(np.float32), 1)
        B, _ = lowp.quantize(rng.standard_normal((N, K)).astype(np.float32), 1)
        A[:, 5], B[:, 5] = 0x38, 0x38                        # (a product of 1 at least)
        kb = lowp.cdiv(K, 128)
        for lo, hi in ((-126, -100), (-70, -56), (100, 110), (50, 70), (-126, 120)):
            e = rng.uniform(lo, hi, (kb, M))
            SA = (2.0 ** e).astype(np.float32)
            # results from 2^-120 to 2^100, some lost altogether
            f = rng.uniform(-150, 90, (kb, lowp.cdiv(N, tall))) - (lo + hi) / 2
            SB = (2.0 ** np.clip(f, -126, 127)).astype(np.float32)
            got = product(A, SA, B, SB, dt).double().cpu().numpy()
            want, bound = lowp.product(A, SA, B, SB, tall)
            bound = bound + (2 * K + 8) * 2.0 ** -149
            limit = float(torch.finfo(dt).max)
            if out == "bf16":
                bound = bound + lowp.bf16_half_step(np.abs(want) + bound)
            # (a partial sum may pass the largest number where the terms' sizes do)
            terms = np.abs(lowp.stands_for(A, SA, 1)) @ np.abs(lowp.stands_for(B, SB, tall)).T
            inside = terms < limit / 2
            assert inside.mean() > 0.2
            err = np.abs(got - want)
            assert (err <= bound)[inside].all(), (M, N, K, lo, hi)
            over = np.abs(want) - bound > 2 * limit
            assert not np.isfinite(got[over]).any()


def test_scales_of_blocks_without_codes():
    """Codes of zeros with scales at the ends: they add nothing, also where the
    scales' product is infinite or lost."""
    import torch
    rng = np.random.default_rng(44)
    ints = lowp.nearest_codes(np.arange(-8, 9).astype(np.float64))
    for M, N, K in ((3, 40, 400), (150, 260, 400)):
        A, B = rng.choice(ints, (M, K)), rng.choice(ints, (N, K))
        A[M // 2, :256] = 0
        B[N // 2:, 128:256] = 0
        SA, SB = np.ones((4, M), np.float32), np.ones((4, N), np.float32)
        SA[:2, M // 2] = 2.0 ** 127, 2.0 ** -126
        SB[1, N // 2:] = 2.0 ** 120
        SB[0, 1], SA[1, 0] = 2.0 ** 6, 2.0 ** 10
        want = lowp.stands_for(A, SA, 1) @ lowp.stands_for(B, SB, 1).T
        got = product(A, SA, B, SB, torch.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).float())


@pytest.mark.parametrize("tall", [1, 128])
def test_infinite_scales(tall):
    """An infinite scale makes its own rows or columns infinite, also in the last
    block of K, past which groups of waves have no block."""
    import torch
    one = 0x38                                               # the code of 1
    for M, N, K in ((1, 40, 300), (70, 300, 130), (300, 300, 300)):
        A, B = np.full((M, K), one, np.uint8), np.full((N, K), one, np.uint8)
        kb = lowp.cdiv(K, 128)
        SA, SB = np.ones((kb, M), np.float32), np.ones((kb, lowp.cdiv(N, tall)), np.float32)
        SB[kb - 1, 0] = np.inf
        SA[0, M - 1] = -np.inf if M > 1 else 1.0
        got = product(A, SA, B, SB, torch.float32).cpu().numpy()
        columns = min(tall, N)
        assert (got[:M - 1, :columns] == np.inf).all() and (got[:M - 1, columns:] == K).all()
        if M > 1:
            assert np.isnan(got[M - 1, :columns]).all() and (got[M - 1, columns:] == -np.inf).all()
        else:
            assert (got[0, :columns] == np.inf).all() and (got[0, columns:] == K).all()


@pytest.mark.parametrize("wt", ["bf16", "f32"])
@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 9])
def test_infinite_weights(T, xt, wt):
    """An infinite weight times a finite value is infinite, times 0 NaN, and
    reaches its own row of the matrix only."""
    import torch
    H, I = 40, 24
    x = torch.zeros(T, H, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 0.5, 1.0 + 2.0 ** -20
    gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
    gate[0, 0], up[0, 1] = np.inf, -2.0                 # h[0] = -inf
    gate[1, 2], up[1, 0] = 1.0, 1.0                     # h[1] = x[2]
    gate[2, 1], up[2, 3] = 1.0, np.inf                  # h[2] = 0.5 * (inf * 0) = NaN
    down[0, 0], down[1, 1] = 1.0, -np.inf
    down[2, 1], down[3, 2] = 1.0, 1.0
    xx = x.to(getattr(torch, xt))
    out = one_expert(xx, gate, up, down, wt)
    # every row of `down` meets h[0] = -inf and h[2] = NaN: all NaN
    assert np.isnan(out).all()
    gate[0, 0], up[2, 3] = 1.0, 1.0                     # h[0] = -1, h[2] = 0
    out = one_expert(xx, gate, up, down, wt)
    assert (out[:, 0] == -1).all() and (out[:, 1] == -np.inf).all()
    np.testing.assert_array_equal(out[:, 2], xx[:, 2].double().cpu().numpy())
    assert (out[:, 3:] == 0).all()
    gate[0, 0] = np.inf                                 # h[0] = -inf alone, out all of it
    out = one_expert(xx, gate[:1], up[:1], np.full((H, 1), 0.5), wt)
    assert (out == -np.inf).all()


# ---- every tile of the product -------------------------------------------------

@pytest.fixture
def forced():
    yield fg.fg_set_fp8_tile
    assert fg.fg_set_fp8_tile(-1) == fg.FG_OK


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("tall", [1, 128])
def test_every_tile_gives_exact_integers(tall, out, forced):
    """Each tile kernel, whatever the library would choose: whole and partial
    tiles, sums of one block to 71 with a partial last one, slices of K, C as it
    is and scaled into."""
    import torch
    dt = torch.float32 if out == "f32" else torch.bfloat16
    rng = np.random.default_rng(45)
    slices = set()
    for tile, (m, n) in enumerate(fg.fg_fp8_tiles()):
        assert forced(tile) == fg.FG_OK
        for M, N, K in ((1, 5, 130), (m + 3, 2 * n + 1, 300), (2 * m, n, 128), (m - 1, n - 1, 1700),
                        (m + 1, n + 2, 9000)):
            need = fg.fg_gemm_fp8_workspace_size(M, N, K)
            chosen, used = fg.fg_select_fp8(M, N, K, need)
            assert chosen == tile
            slices.add(used)
            A, SA, B, SB, want = cancelling(rng, M, N, K, tall)
            want = torch.from_numpy(want)
            print("  tile", tile, (m, n), "slices", used, flush=True)
            assert torch.equal(product(A, SA, B, SB, dt).cpu(), want.to(dt))
            C0 = torch.from_numpy(rng.integers(-64, 65, (M, N)).astype(np.float32)).to(dt)
            C = product(A, SA, B, SB, dt, C0.cuda(), alpha=-2.0, beta=4.0)
            assert torch.equal(C.cpu(), (-2.0 * want + 4.0 * C0.double()).to(dt))
    assert 1 in slices and max(slices) > 1


def test_every_tile_takes_its_sums_again(forced):
    """Factors that overflow in some rows and some blocks of K, in every tile."""
    import torch
    rng = np.random.default_rng(46)
    ints = lowp.nearest_codes(np.arange(-8, 9).astype(np.float64))
    for tile, (m, n) in enumerate(fg.fg_fp8_tiles()):
        assert forced(tile) == fg.FG_OK
        for M, N, K, tall in ((m + 5, n + 9, 700, 1), (2 * m, n + 1, 700, 128)):
            A, B = rng.choice(ints, (M, K)), rng.choice(ints, (N, K))
            SA = np.ones((lowp.cdiv(K, 128), M), np.float32)
            SB = np.ones((lowp.cdiv(K, 128), lowp.cdiv(N, tall)), np.float32)
            A[3], SA[:, 3] = 0, 2.0 ** 127          # a row of zeros
            SB[2], SA[2] = 2.0 ** 125, 2.0 ** -120  # a block of factors 2^5
            want = lowp.stands_for(A, SA, 1) @ lowp.stands_for(B, SB, tall).T
            got = product(A, SA, B, SB, torch.float32)
            assert torch.equal(got.cpu(), torch.from_numpy(want).float())


@pytest.mark.parametrize("wt", ["e4m3", "bf16", "f32"])
def test_small_values_keep_their_bits(wt):
    """x and h down to 2^-109 hold 24 bits (their last terms are bfloat16 numbers
    below the normal ones)."""
    import torch
    H, I = 24, 20
    for e in (-80, -100, -105, -109):
        small = 2.0 ** e * (1 + 2.0 ** -11 + 2.0 ** -23)
        x = torch.zeros(3, H, device="cuda")
        x[:, 0], x[:, 1] = small, 1.0
        gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
        gate[2, 0], up[2, 1], down[4, 2] = 1.0, 1.0, -2.0
        out = one_expert(x, gate, up, down, wt)
        assert (out[:, 4] == -2.0 * small).all(), e
