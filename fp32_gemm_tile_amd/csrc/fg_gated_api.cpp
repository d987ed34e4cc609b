// Host side of include/fp32gemm_gated.h and include/fp32gemm_int4.h: argument
// validation, quick returns, the choice of kernel and launches on the caller's
// stream.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/fp32gemm_gated.h"
#include "../../include/fp32gemm_int4.h"
#include "../../include/fp32gemm_tune.h"
#include "fg_gated_kernels.h"
#include "fg_host.h"

using fg::cdiv;
using fg::check_device;
using fg::clear_error;
using fg::fail;

namespace {

constexpr int64_t kMaxDim = 1ll << 30;  // as fg_sgemm

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t round_up(int64_t v, int64_t a) { return cdiv(v, a) * a; }
int64_t type_size(int t) { return t == FG_TYPE_F32 ? 4 : 2; }

fg_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(FG_ERR_HIP, 0, "%s: %s", what, hipGetErrorString(e));
    return FG_OK;
}

// A matrix of rows x cols elements of `size` bytes. align: of its rows.
fg_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size,
                       int64_t align, int arg, const char* name) {
    if (rows > 0 && cols > 0 && !p) return fail(FG_ERR_INVALID_ARG, arg, "%s is NULL", name);
    if (!aligned(p, (uintptr_t)align))
        return fail(FG_ERR_INVALID_ARG, arg, "%s is not %lld-byte aligned", name, (long long)align);
    if (ld < std::max<int64_t>(1, cols))
        return fail(FG_ERR_INVALID_ARG, arg + 1, "leading dimension of %s: %lld < %lld", name,
                    (long long)ld, (long long)cols);
    if (ld * size % align)
        return fail(FG_ERR_INVALID_ARG, arg + 1, "rows of %s must start at multiples of %lld bytes",
                    name, (long long)align);
    if (ld > FG_MAX_LD)
        return fail(FG_ERR_UNSUPPORTED, arg + 1, "leading dimension of %s above FG_MAX_LD", name);
    return FG_OK;
}

fg_status check_block_scales(const float* s, int64_t ld, int64_t rows, int arg, const char* name) {
    if (rows > 0 && !s) return fail(FG_ERR_INVALID_ARG, arg, "%s is NULL", name);
    if (!aligned(s, 4)) return fail(FG_ERR_INVALID_ARG, arg, "%s is not 4-byte aligned", name);
    if (ld < std::max<int64_t>(1, rows))
        return fail(FG_ERR_INVALID_ARG, arg + 1, "leading dimension of %s: %lld < %lld", name,
                    (long long)ld, (long long)rows);
    return FG_OK;
}

// ---- choice of the tile --------------------------------------------------------

// Tile and slices that every call of a product and type runs (-1, 0: the cheapest).
struct Forced {
    std::atomic<int> tile{-1}, slices{0};
};
Forced g_forced[3][2];

bool known_product(int op, int type) {
    return op >= fg::GATED_FORWARD && op <= fg::GATED_DW && (type == FG_TYPE_BF16 || type == FG_TYPE_F32);
}

struct Plan {
    int shape;
    int64_t steps, per, splits;
    double us;   // by estimate
};

// Rows and columns of the result, length of its sum, matrices of the result (times
// which the partial sums are written) and of the sum.
struct Sizes {
    int64_t M, N, K;
    int results, terms;
};
Sizes sizes_of(int op, int64_t T, int64_t H, int64_t I) {
    if (op == fg::GATED_FORWARD) return {T, I, H, 2, 1};
    if (op == fg::GATED_DX) return {T, H, I, 1, 2};
    return {I, H, T, 2, 1};
}

constexpr double kCUs = 256, kFinish = 4;                // us, of the kernel that joins slices
constexpr double kPartial = 4e6;                         // bytes per us, of their sums
constexpr int64_t kSlices[] = {1, 2, 3, 4, 6, 8, 12, 16};

// The cheapest by estimate: rounds of as many workgroups as run together, the last of
// which may have one to a CU; slices of the sum cost a kernel and their partial sums'
// way to memory and back. codes: a block of 128 columns has to be in one workgroup,
// or in the kernel that joins slices. (A number of slices by which the steps do not
// divide into as many parts is none; a larger one may be.) A forced number: that many,
// or the most below it that the steps and the workspace have.
Plan plan_tiles(int op, bool bf16, bool codes, const Sizes& z, size_t ws_bytes) {
    constexpr double kMaxTiles = 1 << 23;         // of 512 threads: a grid has fewer than 2^32
    Forced& forced = g_forced[op][bf16];
    const int only = forced.tile.load(), asked = forced.slices.load();
    const double slice = (double)z.M * (double)z.N * 4 * z.results;
    Plan best{-1, 0, 0, 1, 0};
    for (int pass = 0; pass < 2 && best.shape < 0; ++pass) {   // (1: the forced tile cannot)
        for (int s = 0; s < fg::gated_num_shapes(op, bf16); ++s) {
            const fg::GatedShape sh = fg::gated_shape(op, bf16, s);
            if (pass == 0 && only >= 0 && s != only) continue;
            const double tiles = (double)cdiv(z.M, sh.bm) * (double)cdiv(z.N, sh.bn) *
                                 (op == fg::GATED_DW ? 2 : 1);
            if (tiles >= kMaxTiles) continue;
            const int64_t steps = cdiv(z.K * (bf16 ? 2 : 4), sh.kb) * z.terms;
            auto fits = [&](int64_t n) {
                return cdiv(steps, cdiv(steps, n)) == n && (n == 1 || (double)n * slice <= (double)ws_bytes) &&
                       !(n == 1 && codes && sh.bn % 128);
            };
            auto consider = [&](int64_t n) {
                const int64_t per = cdiv(steps, n);
                const double slots = kCUs * sh.per_cu, full = std::floor(tiles * (double)n / slots);
                const double rest = tiles * (double)n - full * slots;
                double us = full * (sh.start_us + (double)per * sh.full_us);
                if (rest > 0)
                    us += sh.start_us + (double)per * (rest <= kCUs ? sh.step_us : sh.full_us);
                if (n > 1) us += kFinish + 2 * (double)n * slice / kPartial;
                const bool better = pass == 0 && asked > 0 && n != best.splits ? n > best.splits : us < best.us;
                if (best.shape < 0 || better) best = Plan{s, steps, per, n, us};
            };
            if (pass == 0 && asked > 0) {
                int64_t n = asked;
                while (n > 0 && !fits(n)) --n;
                if (n > 0) consider(n);
            } else {
                for (const int64_t n : kSlices)
                    if (fits(n)) consider(n);
            }
        }
        if (only < 0) break;
    }
    return best;
}

// Forward products that stream the weights instead of tiling the result.
bool streams_weights(bool bf16, int save, int64_t T) {
    return T <= fg::kRowsMaxTokens && save != FG_SAVE_E4M3 && g_forced[0][bf16].tile.load() < 0;
}

size_t partial_bytes(int op, bool bf16, int64_t T, int64_t H, int64_t I) {
    if (op == fg::GATED_FORWARD && streams_weights(bf16, FG_SAVE_NONE, T) && T > 0) {
        // (also enough for FG_SAVE_E4M3, whose choice of tiles is narrower)
        const Sizes z = sizes_of(op, T, H, I);
        const int64_t n = plan_tiles(op, bf16, true, z, (size_t)-1 / 2).splits;
        return n > 1 ? (size_t)(n * z.M * z.N) * 4 * (size_t)z.results : 0;
    }
    const Sizes z = sizes_of(op, T, H, I);
    size_t most = 0;
    for (int codes = 0; codes < (op == fg::GATED_FORWARD ? 2 : 1); ++codes) {
        const int64_t n = plan_tiles(op, bf16, codes != 0, z, (size_t)-1 / 2).splits;
        if (n > 1) most = std::max(most, (size_t)(n * z.M * z.N) * 4 * (size_t)z.results);
    }
    return most;
}

bool sizes_ok(int64_t T, int64_t H, int64_t I) {
    return T >= 0 && H >= 0 && I >= 0 && T <= kMaxDim && H <= kMaxDim && I <= kMaxDim;
}

// ---- the block's arguments -------------------------------------------------------

fg_status check_block(const fg_gated_block& b, bool backward, bool need_x, bool need_w) {
    if (b.tokens < 0) return fail(FG_ERR_INVALID_ARG, 1, "tokens < 0");
    if (b.hidden < 0) return fail(FG_ERR_INVALID_ARG, 2, "hidden < 0");
    if (b.inner < 0) return fail(FG_ERR_INVALID_ARG, 3, "inner < 0");
    if (b.type != FG_TYPE_F32 && b.type != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 4, "type must be FG_TYPE_F32 or FG_TYPE_BF16");
    if (b.activation < FG_ACT_NONE || b.activation > FG_ACT_SILU)
        return fail(FG_ERR_INVALID_ARG, 5, "unknown activation %d", b.activation);
    if (b.save < FG_SAVE_NONE || b.save > FG_SAVE_E4M3 || (backward && b.save == FG_SAVE_NONE))
        return fail(FG_ERR_INVALID_ARG, 12, backward ? "save=%d: the gradients need G and U"
                                                      : "unknown save=%d", b.save);
    const int64_t T = b.tokens, H = b.hidden, I = b.inner, size = type_size(b.type);
    fg_status st;
    if (need_x && (st = check_matrix(b.x, b.ldx, T, H, size, 16, 6, "x")) != FG_OK) return st;
    if (need_w && (st = check_matrix(b.gate, b.ldgate, I, H, size, 16, 8, "gate")) != FG_OK) return st;
    if (need_w && (st = check_matrix(b.up, b.ldup, I, H, size, 16, 10, "up")) != FG_OK) return st;
    if (b.save != FG_SAVE_NONE) {
        const bool codes = b.save == FG_SAVE_E4M3;
        const int64_t es = codes ? 1 : size, align = codes ? 16 : size;
        if ((st = check_matrix(b.g, b.ldg, T, I, es, align, 13, "g")) != FG_OK) return st;
        if ((st = check_matrix(b.u, b.ldu, T, I, es, align, 15, "u")) != FG_OK) return st;
        if (codes && I > 0) {
            if ((st = check_block_scales(b.sg, b.ldsg, T, 17, "sg")) != FG_OK) return st;
            if ((st = check_block_scales(b.su, b.ldsu, T, 19, "su")) != FG_OK) return st;
        }
    }
    if (!backward || b.h)
        if ((st = check_matrix(b.h, b.ldh, T, I, size, size, 21, "h")) != FG_OK) return st;
    return FG_OK;
}

fg_status check_limits(const fg_gated_block& b) {
    if (!sizes_ok(b.tokens, b.hidden, b.inner))
        return fail(FG_ERR_UNSUPPORTED, 0, "tokens, hidden and inner are limited to 2^30");
    return FG_OK;
}

void fill_saved(const fg_gated_block& b, void* (&saved)[2], int64_t (&ld)[2]) {
    saved[0] = b.g;
    saved[1] = b.u;
    ld[0] = b.ldg;
    ld[1] = b.ldu;
}

// dG and dU: rows of whole steps of any tile that reads them along their rows, with zeros
// at their ends (what a step reads of the next row would meet zeros of gate and up, and may
// be NaN).
int64_t grad_ld(int64_t I) { return round_up(I, fg::kGradRow); }
size_t grad_bytes(int64_t T, int64_t I, int type) {
    return (size_t)round_up(T * grad_ld(I) * type_size(type), 256);
}

void set_plan(const Sizes& z, const Plan& plan, fg::GatedTileParams& p) {
    p.M = (int32_t)z.M;
    p.N = (int32_t)z.N;
    p.K = (int32_t)z.K;
    p.steps = (int32_t)plan.steps;
    p.per_split = (int32_t)plan.per;
    p.splits = (int32_t)plan.splits;
}

// dx (px) beside dgate and dup (pw) in one launch, where that is cheaper by estimate than
// the plans they have; px.shape -1: apart.
//
// binary32: tiles of 64 x 128, two to a CU, which take the next as they end: the mean of what
// the CUs get, and not less than seven tenths of the longest (alone on its CU it is faster).
// 1025 tokens, 1536 x 2047: 246 us, apart 278; 517, 2047 x 3001: 243 and 264; 1000, 1000 x
// 3000: 221 and 227; 700, 2048 x 1408: 150 and 162.
// bfloat16: dx's smallest tiles beside tiles of 128 x 128, as long as they do not fill the CUs
// by themselves. dx is one slice there, so its sum has to end before two launches, of which
// the second costs 2 us, would have: a step takes 1.35 times what it does alone. 64 tokens, 2048 x
// 1408: 16 us, apart 22; 200: 21 and 27; 300: 22 and 32; 200, 1024 x 4096 33 and 36; 200, 2048 x
// 5632 51 and 67. Longer sums of few tiles (not taken): 300, 256 x 8192 55 and 37; 64, 512 x
// 8192 53 and 27; 17, 512 x 4096 29 and 18. (Of 52 sizes three are chosen wrongly, by up to 9 %.)
void plan_pair(bool bf16, const Sizes& zx, const Sizes& zw, size_t ws_bytes, Plan& px, Plan& pw) {
    for (int op : {fg::GATED_DX, fg::GATED_DW})
        if (g_forced[op][bf16].tile.load() >= 0 || g_forced[op][bf16].slices.load() > 0) {
            px.shape = -1;
            return;
        }
    if (bf16) {
        const double apart = px.us + pw.us + 2;
        px.shape = pw.shape == fg::kPairDw && pw.splits == 1 ? fg::gated_pair(zx.M, zx.N, zw.M) : -1;
        if (px.shape < 0) return;
        const fg::GatedShape x = fg::gated_shape(fg::GATED_DX, true, px.shape);
        px.steps = px.per = cdiv(zx.K * 2, x.kb) * zx.terms;
        px.splits = 1;
        if (x.start_us + 1.35 * (double)px.steps * x.step_us >= apart) px.shape = -1;
        return;
    }
    const fg::GatedShape x = fg::gated_shape(fg::GATED_DX, false, fg::kPairDxF32);
    const fg::GatedShape w = fg::gated_shape(fg::GATED_DW, false, fg::kPairDwF32);
    const double apart = px.us + pw.us;
    const double nx = (double)cdiv(zx.M, x.bm) * (double)cdiv(zx.N, x.bn);
    const double nw = (double)cdiv(zw.M, w.bm) * (double)cdiv(zw.N, w.bn) * 2;
    const int64_t steps = cdiv(zx.K * 4, x.kb) * zx.terms, steps_w = cdiv(zw.K * 4, w.kb);
    const double each_w = w.start_us + (double)steps_w * w.full_us, slots = kCUs * x.per_cu;
    const double slice = (double)zx.M * (double)zx.N * 4;
    px.shape = -1;
    px.us = 0.95 * apart;   // (the estimates' error)
    if (nx * 16 + nw >= (double)(1 << 22)) return;
    for (const int64_t n : kSlices) {
        const int64_t per = cdiv(steps, n);
        if (cdiv(steps, per) != n || (n > 1 && (double)n * slice > (double)ws_bytes)) continue;
        const double each = x.start_us + (double)per * x.full_us;
        double us = std::max((nx * (double)n * each + nw * each_w) / slots, 0.7 * std::max(each, each_w));
        if (n > 1) us += kFinish + 2 * (double)n * slice / kPartial;
        if (us < px.us) px = Plan{fg::kPairDxF32, steps, per, n, us};
    }
    pw = Plan{fg::kPairDwF32, steps_w, steps_w, 1, 0};
}

// dx's part of the one launch that a call which wants all gradients makes; shape -1: it
// makes two. pw: that of dgate and dup.
Plan plan_gradients(bool bf16, const Sizes& zx, const Sizes& zw, size_t ws_bytes, Plan& pw) {
    Plan px = plan_tiles(fg::GATED_DX, bf16, false, zx, ws_bytes);
    pw = plan_tiles(fg::GATED_DW, bf16, false, zw, ws_bytes);
    if (pw.shape < 0) px.shape = -1;
    if (px.shape >= 0) plan_pair(bf16, zx, zw, ws_bytes, px, pw);
    return px;
}

// One product of tiles, with its finish. p: everything but sizes, steps, slices and ws.
fg_status run_tiles(int op, bool bf16, bool codes, const Sizes& z, fg::GatedTileParams& p,
                    void* ws, size_t ws_bytes, hipStream_t stream) {
    if (z.K == 0) {   // empty sums
        set_plan(z, Plan{0, 0, 0, 0, 0}, p);
        return launched(fg::launch_gated_finish(op, bf16, p, stream), "gated block kernel");
    }
    const Plan plan = plan_tiles(op, bf16, codes, z, ws ? ws_bytes : 0);
    if (plan.shape < 0) return fail(FG_ERR_UNSUPPORTED, 0, "2^23 or more output tiles");
    set_plan(z, plan, p);
    p.ws = static_cast<float*>(ws);
    fg_status st = launched(fg::launch_gated_tile(op, bf16, plan.shape, p, stream), "gated block kernel");
    if (st == FG_OK && p.splits > 1)
        st = launched(fg::launch_gated_finish(op, bf16, p, stream), "gated block's reduction kernel");
    return st;
}

}  // namespace

extern "C" {

int32_t fg_gated_num_tiles(int32_t product, int32_t type) {
    return known_product(product, type) ? fg::gated_num_shapes(product, type == FG_TYPE_BF16) : 0;
}

fg_status fg_gated_tile(int32_t product, int32_t type, int32_t tile, int32_t* rows,
                        int32_t* columns) {
    clear_error();
    if (product < 0 || product > fg::GATED_DW)
        return fail(FG_ERR_INVALID_ARG, 1, "unknown product %d", product);
    if (!known_product(product, type)) return fail(FG_ERR_INVALID_ARG, 2, "no tiles for type %d", type);
    if (tile < 0 || tile >= fg_gated_num_tiles(product, type))
        return fail(FG_ERR_INVALID_ARG, 3, "no tile %d", tile);
    if (!rows) return fail(FG_ERR_INVALID_ARG, 4, "rows is NULL");
    if (!columns) return fail(FG_ERR_INVALID_ARG, 5, "columns is NULL");
    const fg::GatedShape s = fg::gated_shape(product, type == FG_TYPE_BF16, tile);
    *rows = s.bm;
    *columns = s.bn;
    return FG_OK;
}

fg_status fg_select_gated(int32_t product, int32_t type, int64_t T, int64_t H, int64_t I,
                          size_t workspace_bytes, int32_t* tile, int32_t* slices) {
    clear_error();
    if (product < 0 || product > fg::GATED_DW)
        return fail(FG_ERR_INVALID_ARG, 1, "unknown product %d", product);
    if (!known_product(product, type)) return fail(FG_ERR_INVALID_ARG, 2, "no tiles for type %d", type);
    if (T <= 0) return fail(FG_ERR_INVALID_ARG, 3, "T < 1");
    if (H <= 0) return fail(FG_ERR_INVALID_ARG, 4, "H < 1");
    if (I <= 0) return fail(FG_ERR_INVALID_ARG, 5, "I < 1");
    if (!tile) return fail(FG_ERR_INVALID_ARG, 7, "tile is NULL");
    if (!slices) return fail(FG_ERR_INVALID_ARG, 8, "slices is NULL");
    if (!sizes_ok(T, H, I))
        return fail(FG_ERR_UNSUPPORTED, 0, "tokens, hidden and inner are limited to 2^30");
    const bool bf16 = type == FG_TYPE_BF16;
    if (product == fg::GATED_FORWARD && streams_weights(bf16, FG_SAVE_NONE, T)) {
        *tile = -1;
        *slices = 1;
        return FG_OK;
    }
    const Plan plan = plan_tiles(product, bf16, false, sizes_of(product, T, H, I), workspace_bytes);
    if (plan.shape < 0) return fail(FG_ERR_UNSUPPORTED, 0, "2^23 or more output tiles");
    *tile = plan.shape;
    *slices = (int32_t)plan.splits;
    return FG_OK;
}

fg_status fg_select_gated_pair(int32_t type, int64_t T, int64_t H, int64_t I,
                               size_t workspace_bytes, int32_t* tile, int32_t* slices) {
    clear_error();
    if (!known_product(fg::GATED_DX, type)) return fail(FG_ERR_INVALID_ARG, 1, "no tiles for type %d", type);
    if (T <= 0) return fail(FG_ERR_INVALID_ARG, 2, "T < 1");
    if (H <= 0) return fail(FG_ERR_INVALID_ARG, 3, "H < 1");
    if (I <= 0) return fail(FG_ERR_INVALID_ARG, 4, "I < 1");
    if (!tile) return fail(FG_ERR_INVALID_ARG, 6, "tile is NULL");
    if (!slices) return fail(FG_ERR_INVALID_ARG, 7, "slices is NULL");
    if (!sizes_ok(T, H, I))
        return fail(FG_ERR_UNSUPPORTED, 0, "tokens, hidden and inner are limited to 2^30");
    Plan pw;
    const Plan px = plan_gradients(type == FG_TYPE_BF16, sizes_of(fg::GATED_DX, T, H, I),
                                   sizes_of(fg::GATED_DW, T, H, I), workspace_bytes, pw);
    *tile = px.shape;
    *slices = px.shape < 0 ? 0 : (int32_t)px.splits;
    return FG_OK;
}

fg_status fg_set_gated_tile(int32_t product, int32_t type, int32_t tile, int32_t slices) {
    clear_error();
    if (product < 0 || product > fg::GATED_DW)
        return fail(FG_ERR_INVALID_ARG, 1, "unknown product %d", product);
    if (!known_product(product, type)) return fail(FG_ERR_INVALID_ARG, 2, "no tiles for type %d", type);
    if (tile < -1 || tile >= fg_gated_num_tiles(product, type))
        return fail(FG_ERR_INVALID_ARG, 3, "no tile %d", tile);
    if (slices < 0 || slices > 16) return fail(FG_ERR_INVALID_ARG, 4, "slices outside 0 .. 16");
    g_forced[product][type].tile.store(tile);
    g_forced[product][type].slices.store(slices);
    return FG_OK;
}

size_t fg_gated_workspace_size(int64_t tokens, int64_t hidden, int64_t inner, int32_t type) {
    if (!sizes_ok(tokens, hidden, inner) || (type != FG_TYPE_F32 && type != FG_TYPE_BF16)) return 0;
    if (tokens == 0 || hidden == 0 || inner == 0) return 0;
    return partial_bytes(fg::GATED_FORWARD, type == FG_TYPE_BF16, tokens, hidden, inner);
}

size_t fg_gated_backward_min_workspace_size(int64_t tokens, int64_t inner, int32_t type) {
    if (!sizes_ok(tokens, 0, inner) || (type != FG_TYPE_F32 && type != FG_TYPE_BF16)) return 0;
    return 2 * grad_bytes(tokens, inner, type);
}

size_t fg_gated_backward_workspace_size(int64_t tokens, int64_t hidden, int64_t inner,
                                        int32_t type) {
    if (!sizes_ok(tokens, hidden, inner)) return 0;
    size_t n = fg_gated_backward_min_workspace_size(tokens, inner, type);
    const bool bf16 = type == FG_TYPE_BF16;
    if (n > 0 && hidden > 0) {
        Plan pw;   // (dx's slices in one launch may be more than it has in its own)
        const Plan px = plan_gradients(bf16, sizes_of(fg::GATED_DX, tokens, hidden, inner),
                                       sizes_of(fg::GATED_DW, tokens, hidden, inner), (size_t)-1 / 2, pw);
        n += std::max({partial_bytes(fg::GATED_DX, bf16, tokens, hidden, inner),
                       partial_bytes(fg::GATED_DW, bf16, tokens, hidden, inner),
                       px.shape >= 0 && px.splits > 1 ? (size_t)(px.splits * tokens * hidden) * 4 : (size_t)0});
    }
    return n;
}

fg_status fg_gated(const fg_gated_block* block, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
    clear_error();
    if (!block) return fail(FG_ERR_INVALID_ARG, 1, "block is NULL");
    const fg_gated_block& b = *block;
    fg_status st;
    if ((st = check_block(b, false, true, true)) != FG_OK) return st;
    if (workspace && !aligned(workspace, 16))
        return fail(FG_ERR_INVALID_ARG, 23, "workspace is not 16-byte aligned");
    if ((st = check_limits(b)) != FG_OK) return st;
    if (b.tokens == 0 || b.inner == 0) return FG_OK;
    if ((st = check_device()) != FG_OK) return st;
    const bool bf16 = b.type == FG_TYPE_BF16;
    if (b.hidden > 0 && streams_weights(bf16, b.save, b.tokens)) {
        fg::RowsParams p;
        memset(&p, 0, sizeof p);
        p.T = (int32_t)b.tokens;
        p.N = (int32_t)b.inner;
        p.K = (int32_t)b.hidden;
        p.x_bf16 = bf16;
        p.act = b.activation;
        p.matrices = 2;
        p.x = b.x;
        p.ldx = b.ldx;
        p.w[0].w = static_cast<const uint8_t*>(b.gate);
        p.w[0].ld = b.ldgate * type_size(b.type);
        p.w[1].w = static_cast<const uint8_t*>(b.up);
        p.w[1].ld = b.ldup * type_size(b.type);
        p.out = b.h;
        p.ldo = b.ldh;
        if (b.save == FG_SAVE_SAME) fill_saved(b, p.save, p.ld_save);
        return launched(fg::launch_rows(p, stream), "few-row kernel");
    }
    fg::GatedTileParams p;
    memset(&p, 0, sizeof p);
    p.A[0] = b.x;
    p.lda = b.ldx;
    p.B[0] = b.gate;
    p.B[1] = b.up;
    p.ldb[0] = b.ldgate;
    p.ldb[1] = b.ldup;
    p.C[0] = b.h;
    p.ldc[0] = b.ldh;
    p.act = b.activation;
    p.save = b.save;
    fill_saved(b, p.saved, p.ld_saved);
    p.scales[0] = b.sg;
    p.scales[1] = b.su;
    p.ld_scales[0] = b.ldsg;
    p.ld_scales[1] = b.ldsu;
    return run_tiles(fg::GATED_FORWARD, bf16, b.save == FG_SAVE_E4M3,
                     sizes_of(fg::GATED_FORWARD, b.tokens, b.hidden, b.inner), p, workspace,
                     workspace_bytes, stream);
}

fg_status fg_gated_backward(const fg_gated_block* block, const fg_gated_grads* grads,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    if (!block) return fail(FG_ERR_INVALID_ARG, 1, "block is NULL");
    if (!grads) return fail(FG_ERR_INVALID_ARG, 23, "grads is NULL");
    const fg_gated_block& b = *block;
    const fg_gated_grads& d = *grads;
    fg_status st;
    if ((st = check_block(b, true, d.dgate != nullptr, d.dx != nullptr)) != FG_OK) return st;
    const int64_t T = b.tokens, H = b.hidden, I = b.inner, size = type_size(b.type);
    if ((st = check_matrix(d.dh, d.lddh, T, I, size, size, 23, "dh")) != FG_OK) return st;
    if (d.dx && (st = check_matrix(d.dx, d.lddx, T, H, size, size, 25, "dx")) != FG_OK) return st;
    if (d.dgate) {
        if ((st = check_matrix(d.dgate, d.lddgate, I, H, size, size, 27, "dgate")) != FG_OK) return st;
        if (!d.dup) return fail(FG_ERR_INVALID_ARG, 29, "dgate is given and dup is not");
        if ((st = check_matrix(d.dup, d.lddup, I, H, size, size, 29, "dup")) != FG_OK) return st;
    } else if (d.dup) {
        return fail(FG_ERR_INVALID_ARG, 27, "dup is given and dgate is not");
    }
    if ((st = check_limits(b)) != FG_OK) return st;
    // (the workspace's rows are read as a matrix's)
    if (grad_ld(I) > FG_MAX_LD) return fail(FG_ERR_UNSUPPORTED, 3, "inner above FG_MAX_LD");
    const size_t each = grad_bytes(T, I, b.type);
    if (each > 0 && (!workspace || !aligned(workspace, 16)))
        return fail(FG_ERR_INVALID_ARG, 32, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < 2 * each)
        return fail(FG_ERR_INVALID_ARG, 33, "workspace of %zu bytes, need %zu", workspace_bytes, 2 * each);
    const bool bf16 = b.type == FG_TYPE_BF16;
    const bool want_dx = d.dx && T > 0 && H > 0, want_dw = d.dgate && I > 0 && H > 0;
    const bool want_grad = T > 0 && I > 0 && (b.h || want_dx || want_dw);
    if (!want_grad && !want_dx && !(want_dw && d.beta != 1.f)) return FG_OK;
    if ((st = check_device()) != FG_OK) return st;

    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    void *dg = ws, *du = ws ? ws + each : nullptr;
    const int64_t ldd = std::max<int64_t>(fg::kGradRow, grad_ld(I));
    if (want_grad) {
        fg::GatedGradParams p;
        memset(&p, 0, sizeof p);
        p.T = (int32_t)T;
        p.I = (int32_t)I;
        p.act = b.activation;
        p.save = b.save;
        p.dh = d.dh;
        p.lddh = d.lddh;
        p.saved[0] = b.g;
        p.saved[1] = b.u;
        p.ld_saved[0] = b.ldg;
        p.ld_saved[1] = b.ldu;
        p.scales[0] = b.sg;
        p.scales[1] = b.su;
        p.ld_scales[0] = b.ldsg;
        p.ld_scales[1] = b.ldsu;
        p.dg = dg;
        p.du = du;
        p.ld_d = ldd;
        p.h = b.h;
        p.ldh = b.ldh;
        st = launched(fg::launch_gated_grad(bf16, p, stream), "activation's gradient kernel");
        if (st != FG_OK) return st;
    }
    void* const more = ws ? ws + 2 * each : nullptr;
    const size_t more_bytes = workspace_bytes - 2 * each;
    fg::GatedTileParams x, w;
    memset(&x, 0, sizeof x);
    x.A[0] = dg;
    x.A[1] = du;
    x.lda = ldd;
    x.B[0] = b.gate;
    x.B[1] = b.up;
    x.ldb[0] = b.ldgate;
    x.ldb[1] = b.ldup;
    x.C[0] = d.dx;
    x.ldc[0] = d.lddx;
    memset(&w, 0, sizeof w);
    w.A[0] = dg;
    w.A[1] = du;
    w.lda = ldd;
    w.B[0] = b.x;
    w.ldb[0] = b.ldx;
    w.C[0] = d.dgate;
    w.C[1] = d.dup;
    w.ldc[0] = d.lddgate;
    w.ldc[1] = d.lddup;
    w.beta = d.beta;
    const Sizes zx = sizes_of(fg::GATED_DX, T, H, I), zw = sizes_of(fg::GATED_DW, T, H, I);
    if (want_dx && want_dw && I > 0) {
        Plan pw;
        const Plan px = plan_gradients(bf16, zx, zw, more_bytes, pw);
        if (px.shape >= 0) {
            set_plan(zx, px, x);
            set_plan(zw, pw, w);
            x.ws = static_cast<float*>(more);
            st = launched(fg::launch_gated_pair(bf16, px.shape, x, w, stream), "gated block's gradient kernel");
            if (st == FG_OK && px.splits > 1)
                st = launched(fg::launch_gated_finish(fg::GATED_DX, bf16, x, stream),
                              "gated block's reduction kernel");
            return st;
        }
    }
    if (want_dx) st = run_tiles(fg::GATED_DX, bf16, false, zx, x, more, more_bytes, stream);
    if (st == FG_OK && want_dw && !(T == 0 && d.beta == 1.f))
        st = run_tiles(fg::GATED_DW, bf16, false, zw, w, more, more_bytes, stream);
    return st;
}

}  // extern "C"

// ---- 4-bit weights -----------------------------------------------------------------

namespace {

fg_status check_int4(const fg_int4* w, int64_t N, int64_t K, int64_t group, int64_t scale_size,
                     int arg, const char* name) {
    if (!w) return fail(FG_ERR_INVALID_ARG, arg, "%s is NULL", name);
    const bool any = N > 0 && K > 0;
    if (any && !w->q) return fail(FG_ERR_INVALID_ARG, arg, "codes of %s are NULL", name);
    if (!aligned(w->q, 16) || w->ldq % 16 || w->ldq < cdiv(K, 2))
        return fail(FG_ERR_INVALID_ARG, arg,
                    "rows of codes of %s must start at multiples of 16 bytes, %lld at least apart", name,
                    (long long)cdiv(K, 2));
    if (w->ldq > FG_MAX_LD)
        return fail(FG_ERR_UNSUPPORTED, arg, "leading dimension of %s above FG_MAX_LD", name);
    if ((any && !w->s) || !aligned(w->s, (uintptr_t)scale_size) || w->lds < N)
        return fail(FG_ERR_INVALID_ARG, arg, "%s has no scales, misaligned ones, or lds < %lld", name,
                    (long long)N);
    if (w->z && w->ldz < N)
        return fail(FG_ERR_INVALID_ARG, arg, "zero points of %s: ldz < %lld", name, (long long)N);
    const int64_t groups = cdiv(K, group), most = 1ll << 31;
    if (groups > 0 && (w->lds >= most / scale_size / groups || (w->z && w->ldz >= most / groups)))
        return fail(FG_ERR_UNSUPPORTED, arg, "scales or zero points of %s of 2 GiB or more", name);
    return FG_OK;
}

fg_status run_int4(int64_t T, int64_t N, int64_t K, int32_t group, fg_type type, fg_type scale_type,
                   const void* x, int64_t ldx, const fg_int4* w0, const fg_int4* w1, bool gated,
                   int32_t activation, void* out, int64_t ldo, hipStream_t stream) {
    clear_error();
    if (T < 0 || T > FG_INT4_MAX_ROWS)
        return fail(FG_ERR_INVALID_ARG, 1, "T=%lld outside 0 .. %d", (long long)T, FG_INT4_MAX_ROWS);
    if (N < 0) return fail(FG_ERR_INVALID_ARG, 2, "N < 0");
    if (K < 0) return fail(FG_ERR_INVALID_ARG, 3, "K < 0");
    if (group != 32 && group != 64 && group != 128)
        return fail(FG_ERR_INVALID_ARG, 4, "group must be 32, 64 or 128");
    if (type != FG_TYPE_F32 && type != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 5, "type must be FG_TYPE_F32 or FG_TYPE_BF16");
    if (scale_type != FG_TYPE_F32 && scale_type != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 6, "scale_type must be FG_TYPE_F32 or FG_TYPE_BF16");
    const int64_t size = type_size(type), scale_size = type_size(scale_type);
    fg_status st;
    if ((st = check_matrix(x, ldx, T, K, size, 16, 7, "x")) != FG_OK) return st;
    if ((st = check_int4(w0, N, K, group, scale_size, 9, gated ? "gate" : "w")) != FG_OK) return st;
    if (gated) {
        if ((st = check_int4(w1, N, K, group, scale_size, 10, "up")) != FG_OK) return st;
        if (activation < FG_ACT_NONE || activation > FG_ACT_SILU)
            return fail(FG_ERR_INVALID_ARG, 11, "unknown activation %d", activation);
    }
    if ((st = check_matrix(out, ldo, T, N, size, size, 12, "out")) != FG_OK) return st;
    if (N > kMaxDim || K > kMaxDim)
        return fail(FG_ERR_UNSUPPORTED, 0, "N and K are limited to 2^30");
    if (T == 0 || N == 0) return FG_OK;
    if ((st = check_device()) != FG_OK) return st;
    fg::RowsParams p;
    memset(&p, 0, sizeof p);
    p.T = (int32_t)T;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.x_bf16 = type == FG_TYPE_BF16;
    p.act = activation;
    p.group = group;
    p.s_bf16 = scale_type == FG_TYPE_BF16;
    p.matrices = gated ? 2 : 1;
    p.x = x;
    p.ldx = ldx;
    for (int m = 0; m < p.matrices; ++m) {
        const fg_int4& w = m ? *w1 : *w0;
        p.w[m] = fg::RowsWeights{w.q, w.ldq, w.s, w.lds, w.z, w.ldz};
    }
    p.out = out;
    p.ldo = ldo;
    return launched(fg::launch_rows(p, stream), "4-bit product kernel");
}

}  // namespace

extern "C" {

fg_status fg_gemm_int4(int64_t T, int64_t N, int64_t K, int32_t group, fg_type type,
                       fg_type scale_type, const void* x, int64_t ldx, const fg_int4* w, void* out,
                       int64_t ldo, hipStream_t stream) {
    return run_int4(T, N, K, group, type, scale_type, x, ldx, w, nullptr, false, 0, out, ldo, stream);
}

fg_status fg_gated_int4(int64_t T, int64_t N, int64_t K, int32_t group, fg_type type,
                        fg_type scale_type, const void* x, int64_t ldx, const fg_int4* gate,
                        const fg_int4* up, int32_t activation, void* out, int64_t ldo,
                        hipStream_t stream) {
    return run_int4(T, N, K, group, type, scale_type, x, ldx, gate, up, true, activation, out, ldo,
                    stream);
}

}  // extern "C"
