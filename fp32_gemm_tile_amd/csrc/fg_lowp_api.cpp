// Host side of include/fp32gemm_fp8.h and include/fp32gemm_moe.h: argument
// validation, quick returns, the choice of kernel and launches on the
// caller's stream.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/fp32gemm_fp8.h"
#include "../../include/fp32gemm_moe.h"
#include "../../include/fp32gemm_tune.h"
#include "fg_host.h"
#include "fg_lowp_kernels.h"

using fg::cdiv;
using fg::check_device;
using fg::clear_error;
using fg::fail;

namespace {

constexpr int64_t kMaxDim = 1ll << 30;  // as fg_sgemm

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

fg_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(FG_ERR_HIP, 0, "%s: %s", what, hipGetErrorString(e));
    return FG_OK;
}

// A matrix of codes: rows of at least `cols` bytes at multiples of 16.
fg_status check_codes(const void* w, int64_t ld, int64_t cols, int arg, const char* name) {
    if (ld < std::max<int64_t>(1, cols))
        return fail(FG_ERR_INVALID_ARG, arg + 1, "leading dimension of %s: %lld < %lld", name,
                    (long long)ld, (long long)cols);
    if (ld % 16 || !aligned(w, 16))
        return fail(FG_ERR_INVALID_ARG, ld % 16 ? arg + 1 : arg,
                    "rows of %s must start at multiples of 16 bytes", name);
    if (ld > FG_MAX_LD)
        return fail(FG_ERR_UNSUPPORTED, arg + 1, "leading dimension of %s above FG_MAX_LD", name);
    return FG_OK;
}

fg_status check_scales(const float* s, int64_t ld, int64_t outer, int arg, const char* name) {
    if (!s) return fail(FG_ERR_INVALID_ARG, arg, "%s is NULL", name);
    if (!aligned(s, 4)) return fail(FG_ERR_INVALID_ARG, arg, "%s is not 4-byte aligned", name);
    if (ld < std::max<int64_t>(1, outer))
        return fail(FG_ERR_INVALID_ARG, arg + 1, "leading dimension of %s: %lld < %lld", name,
                    (long long)ld, (long long)outer);
    return FG_OK;
}

int type_size(int t) { return t == FG_TYPE_F32 ? 4 : (t == FG_TYPE_BF16 ? 2 : 1); }

// ---- block-scaled product ----------------------------------------------------

// Tile that every call runs (fg_set_fp8_tile; -1: the cheapest).
std::atomic<int> g_fp8_tile{-1};

// Shape of the tile kernel and number of slices of K.
struct Plan {
    int shape;
    int64_t splits;
};

// The cheapest by estimate: rounds of one workgroup per CU, each taking the
// blocks of K one after the other, or the stream of both operands; slices of K
// (at most 16) cost another kernel and their partial sums' way to memory and
// back. Slices pay for small results of long sums (bfloat16 C, the best tile each:
// 256 x 256 x 65536 44.0 us in one slice, 23.6 in four; 1024 x 1024 x 65536 199
// and 136 in eight, where four are chosen, 141), and cost where a sum is short
// (512 x 512 x 16384 19.3 us in one, 26.1 in two).
Plan plan_gemm(int64_t M, int64_t N, int64_t K, size_t ws_bytes) {
    constexpr double kCUs = 256, kStream = 6.5e6, kPartial = 4e6;  // bytes per us
    constexpr double kLaunch = 1.6, kFirst = 1.5, kFinish = 7, kNear = 2.5;  // us
    constexpr double kMaxTiles = 1 << 23;  // of 512 threads: a grid has fewer than 2^32
    const int64_t kb = cdiv(K, fg::kScaleBlock);
    const double stream = ((double)M * K + (double)N * K) / kStream;
    const double slice = (double)M * N * 4;
    Plan best{-1, 1};
    double best_us = 0;
    const int only = g_fp8_tile.load();
    for (int s = 0; s < fg::fp8_num_shapes(); ++s) {
        if (only >= 0 && s != only) continue;
        const fg::Fp8Shape sh = fg::fp8_shape(s);
        const double near_us = sh.block_us;
        const double tiles = (double)cdiv(M, sh.bm) * (double)cdiv(N, sh.bn);
        if (tiles >= kMaxTiles) continue;
        for (int64_t n = 1; n <= 16; n *= 2) {
            const int64_t per = cdiv(kb, n), used = cdiv(kb, per);
            if (used != n || (n > 1 && (double)n * slice > (double)ws_bytes)) break;
            const double rounds = std::ceil(tiles * (double)n / kCUs);
            const double per_block = stream > kNear && tiles * (double)n <= kCUs
                                         ? std::max(near_us, (double)sh.far_us) : near_us;
            const double share = std::min(1.0, 4 * tiles * (double)n / kCUs);
            double us = kLaunch + std::max(rounds * (sh.start_us + (double)per * per_block),
                                           kFirst + stream / share);
            if (n > 1) us += kFinish + 2 * (double)n * slice / kPartial;
            if (best.shape < 0 || us < best_us) {
                best = Plan{s, n};
                best_us = us;
            }
        }
    }
    return best;
}

}  // namespace

extern "C" {

fg_status fg_quantize_fp8(fg_type type, fg_block block, int64_t M, int64_t N, const void* X,
                          int64_t ldx, uint8_t* Q, int64_t ldq, float* S, int64_t lds,
                          uint8_t* QT, int64_t ldqt, float* ST, int64_t ldst,
                          hipStream_t stream) {
    clear_error();
    if (type != FG_TYPE_F32 && type != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 1, "type must be FG_TYPE_F32 or FG_TYPE_BF16");
    if (block != FG_BLOCK_ROW && block != FG_BLOCK_TILE)
        return fail(FG_ERR_INVALID_ARG, 2, "unknown block kind %d", (int)block);
    if (M < 0) return fail(FG_ERR_INVALID_ARG, 3, "M < 0");
    if (N < 0) return fail(FG_ERR_INVALID_ARG, 4, "N < 0");
    if (M > 0 && N > 0 && !X) return fail(FG_ERR_INVALID_ARG, 5, "X is NULL");
    if (!aligned(X, (uintptr_t)type_size(type)))
        return fail(FG_ERR_INVALID_ARG, 5, "X is not aligned to its type");
    if (ldx < std::max<int64_t>(1, N))
        return fail(FG_ERR_INVALID_ARG, 6, "ldx=%lld < N=%lld", (long long)ldx, (long long)N);
    if (!Q && !QT) return fail(FG_ERR_INVALID_ARG, 7, "neither Q nor QT given");
    const bool tile = block == FG_BLOCK_TILE;
    fg_status st;
    if (Q) {
        if ((st = check_codes(Q, ldq, N, 7, "Q")) != FG_OK) return st;
        if ((st = check_scales(S, lds, tile ? cdiv(M, 128) : M, 9, "S")) != FG_OK) return st;
    }
    if (QT) {
        if ((st = check_codes(QT, ldqt, M, 11, "QT")) != FG_OK) return st;
        if ((st = check_scales(ST, ldst, tile ? cdiv(N, 128) : N, 13, "ST")) != FG_OK) return st;
    }
    if (M > kMaxDim || N > kMaxDim)
        return fail(FG_ERR_UNSUPPORTED, 0, "M and N are limited to 2^30");
    if (M == 0 || N == 0) return FG_OK;
    if ((st = check_device()) != FG_OK) return st;

    fg::QuantParams p;
    memset(&p, 0, sizeof p);
    p.x = X;
    p.ldx = ldx;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.q = Q;
    p.ldq = ldq;
    p.s = S;
    p.lds = lds;
    p.qt = QT;
    p.ldqt = ldqt;
    p.st = ST;
    p.ldst = ldst;
    p.bf16 = type == FG_TYPE_BF16;
    p.tile = tile;
    return launched(fg::launch_quantize_fp8(p, stream), "quantisation kernel");
}

int32_t fg_fp8_num_tiles(void) { return fg::fp8_num_shapes(); }

fg_status fg_fp8_tile(int32_t tile, int32_t* rows_a, int32_t* rows_b) {
    clear_error();
    if (tile < 0 || tile >= fg::fp8_num_shapes())
        return fail(FG_ERR_INVALID_ARG, 1, "no tile %d", tile);
    if (!rows_a) return fail(FG_ERR_INVALID_ARG, 2, "rows_a is NULL");
    if (!rows_b) return fail(FG_ERR_INVALID_ARG, 3, "rows_b is NULL");
    *rows_a = fg::fp8_shape(tile).bm;
    *rows_b = fg::fp8_shape(tile).bn;
    return FG_OK;
}

fg_status fg_select_fp8(int64_t M, int64_t N, int64_t K, size_t workspace_bytes, int32_t* tile,
                        int32_t* slices) {
    clear_error();
    if (M <= 0) return fail(FG_ERR_INVALID_ARG, 1, "M < 1");
    if (N <= 0) return fail(FG_ERR_INVALID_ARG, 2, "N < 1");
    if (K <= 0) return fail(FG_ERR_INVALID_ARG, 3, "K < 1");
    if (!tile) return fail(FG_ERR_INVALID_ARG, 5, "tile is NULL");
    if (!slices) return fail(FG_ERR_INVALID_ARG, 6, "slices is NULL");
    if (M > kMaxDim || N > kMaxDim || K > FG_MAX_LD)
        return fail(FG_ERR_UNSUPPORTED, 0, "M and N are limited to 2^30, K to FG_MAX_LD");
    const Plan plan = plan_gemm(M, N, K, workspace_bytes);
    if (plan.shape < 0) return fail(FG_ERR_UNSUPPORTED, 0, "2^23 or more output tiles");
    *tile = plan.shape;
    *slices = (int32_t)plan.splits;
    return FG_OK;
}

fg_status fg_set_fp8_tile(int32_t tile) {
    clear_error();
    if (tile < -1 || tile >= fg::fp8_num_shapes())
        return fail(FG_ERR_INVALID_ARG, 1, "no tile %d", tile);
    g_fp8_tile.store(tile);
    return FG_OK;
}

size_t fg_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    const int64_t splits = plan_gemm(M, N, K, (size_t)-1 / 2).splits;
    return splits > 1 ? (size_t)(splits * M * N) * 4 : 0;
}

fg_status fg_gemm_fp8(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t* A,
                      int64_t lda, const float* SA, int64_t ldsa, const uint8_t* B, int64_t ldb,
                      const float* SB, int64_t ldsb, fg_block block_b, float beta, void* C,
                      int64_t ldc, fg_type type_c, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    clear_error();
    if (M < 0) return fail(FG_ERR_INVALID_ARG, 1, "M < 0");
    if (N < 0) return fail(FG_ERR_INVALID_ARG, 2, "N < 0");
    if (K < 0) return fail(FG_ERR_INVALID_ARG, 3, "K < 0");
    if (block_b != FG_BLOCK_ROW && block_b != FG_BLOCK_TILE)
        return fail(FG_ERR_INVALID_ARG, 13, "unknown block kind %d", (int)block_b);
    if (type_c != FG_TYPE_F32 && type_c != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 17, "type_c must be FG_TYPE_F32 or FG_TYPE_BF16");
    const bool product = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    const bool tile = block_b == FG_BLOCK_TILE;
    fg_status st;
    if (product) {
        if (!A) return fail(FG_ERR_INVALID_ARG, 5, "A is NULL");
        if ((st = check_codes(A, lda, K, 5, "A")) != FG_OK) return st;
        if ((st = check_scales(SA, ldsa, M, 7, "SA")) != FG_OK) return st;
        if (!B) return fail(FG_ERR_INVALID_ARG, 9, "B is NULL");
        if ((st = check_codes(B, ldb, K, 9, "B")) != FG_OK) return st;
        if ((st = check_scales(SB, ldsb, tile ? cdiv(N, 128) : N, 11, "SB")) != FG_OK) return st;
    }
    if (M > 0 && N > 0) {
        if (!C) return fail(FG_ERR_INVALID_ARG, 15, "C is NULL");
        if (!aligned(C, (uintptr_t)type_size(type_c)))
            return fail(FG_ERR_INVALID_ARG, 15, "C is not aligned to its type");
    }
    if (ldc < std::max<int64_t>(1, N))
        return fail(FG_ERR_INVALID_ARG, 16, "ldc=%lld < N=%lld", (long long)ldc, (long long)N);
    if (workspace && !aligned(workspace, 16))
        return fail(FG_ERR_INVALID_ARG, 18, "workspace is not 16-byte aligned");
    if (M > kMaxDim || N > kMaxDim)
        return fail(FG_ERR_UNSUPPORTED, 0, "M and N are limited to 2^30");
    if (ldc > FG_MAX_LD) return fail(FG_ERR_UNSUPPORTED, 16, "ldc above FG_MAX_LD");
    if (M == 0 || N == 0) return FG_OK;
    if (!product && beta == 1.0f) return FG_OK;

    fg::Fp8Params p;
    memset(&p, 0, sizeof p);
    p.A = A;
    p.B = B;
    p.SA = SA;
    p.SB = SB;
    p.C = C;
    p.lda = lda;
    p.ldsa = ldsa;
    p.ldb = ldb;
    p.ldsb = ldsb;
    p.ldc = ldc;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.alpha = alpha;
    p.beta = beta;
    p.c_bf16 = type_c == FG_TYPE_BF16;
    if (!product) {
        if ((st = check_device()) != FG_OK) return st;
        p.alpha = 0.f;
        return launched(fg::launch_fp8_finish(p, stream), "scaling kernel");
    }
    const Plan plan = plan_gemm(M, N, K, workspace ? workspace_bytes : 0);
    if (plan.shape < 0) return fail(FG_ERR_UNSUPPORTED, 0, "2^23 or more output tiles");
    if ((st = check_device()) != FG_OK) return st;
    p.kb = (int32_t)cdiv(K, fg::kScaleBlock);
    p.splits = (int32_t)plan.splits;
    p.kb_per_split = (int32_t)cdiv(p.kb, plan.splits);
    p.ws = static_cast<float*>(workspace);
    st = launched(fg::launch_gemm_fp8(plan.shape, tile, p, stream), "fp8 product kernel");
    if (st == FG_OK && p.splits > 1)
        st = launched(fg::launch_fp8_finish(p, stream), "fp8 reduction kernel");
    return st;
}

}  // extern "C"

// ---- mixture-of-experts layer ------------------------------------------------

namespace {

int64_t round_up(int64_t v, int64_t a) { return cdiv(v, a) * a; }

int64_t moe_h_ld(int64_t I) { return round_up(I, 16); }
int64_t moe_xs_ld(int64_t H) { return round_up(H, fg::kScaleBlock); }

// Groups of G tokens: no more than pairs, and no more than one partial group
// per expert.
int64_t most_groups(int64_t T, int64_t k, int64_t E, int64_t G) {
    return std::min(T * k, T <= G ? E : E + T * k / G);
}

// Offsets of the workspace's parts, for any types (h and x: at most three
// bfloat16 terms; groups of at least five tokens).
struct MoeSpace {
    size_t plan, logits, groups_x, groups_h, tickets, pieces, h, xs, end;
    MoeSpace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
        size_t at = 0;
        auto take = [&](int64_t bytes) {
            const size_t here = at;
            at += (size_t)round_up(bytes, 256);
            return here;
        };
        const int64_t groups = most_groups(T, k, E, 5);
        plan = take(sizeof(fg::MoePlan));
        logits = take(T * E * 8);
        groups_x = take(groups * (int64_t)sizeof(fg::MoeGroup));
        groups_h = take(groups * (int64_t)sizeof(fg::MoeGroup));
        tickets = take(cdiv(H, 16) * 4);
        int pieces_of_rows = 0;
        for (int type : {fg::TYPE_F32, fg::TYPE_BF16, fg::TYPE_E4M3})
            pieces_of_rows = std::max(
                pieces_of_rows, fg::moe_down_workgroups(type, (int)H, (int)I, (int)groups));
        pieces = take(round_up(H, 32) * 4 * T * pieces_of_rows);
        h = take(T * k * moe_h_ld(I) * 6);
        xs = take(T * moe_xs_ld(H) * 6);
        end = at;
    }
};

bool moe_sizes_ok(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    return T >= 0 && T <= FG_MOE_MAX_TOKENS && E >= 1 && E <= FG_MOE_MAX_EXPERTS && k >= 1 &&
           k <= E && k <= FG_MOE_MAX_TOP_K && H >= 1 && H <= FG_MOE_MAX_DIM && I >= 1 &&
           I <= FG_MOE_MAX_DIM;
}

fg_status check_experts(const fg_experts& m, int wtype, int64_t E, int64_t rows, int64_t cols,
                        int arg, const char* name) {
    const int64_t size = type_size(wtype);
    if (!m.w) return fail(FG_ERR_INVALID_ARG, arg, "%s is NULL", name);
    if (m.ld < cols || (E > 1 && m.stride < 0))
        return fail(FG_ERR_INVALID_ARG, arg, "%s: leading dimension %lld < %lld, or a negative stride",
                    name, (long long)m.ld, (long long)cols);
    if (!aligned(m.w, 16) || m.ld * size % 16 || (E > 1 && m.stride * size % 16))
        return fail(FG_ERR_INVALID_ARG, arg, "rows of %s must start at multiples of 16 bytes", name);
    if (m.ld > FG_MAX_LD)
        return fail(FG_ERR_UNSUPPORTED, arg, "leading dimension of %s above FG_MAX_LD", name);
    if (wtype == FG_TYPE_E4M3) {
        if (!m.scales || !aligned(m.scales, 4))
            return fail(FG_ERR_INVALID_ARG, arg, "%s has no scales, or misaligned ones", name);
        if (m.lds < cdiv(rows, 128) || (E > 1 && m.scale_stride < 0))
            return fail(FG_ERR_INVALID_ARG, arg, "scales of %s: leading dimension %lld < %lld", name,
                        (long long)m.lds, (long long)cdiv(rows, 128));
    }
    return FG_OK;
}

fg::ExpertMatrix expert_matrix(const fg_experts& m) {
    return fg::ExpertMatrix{m.w, m.ld, m.stride, m.scales, m.lds, m.scale_stride};
}

}  // namespace

extern "C" {

size_t fg_moe_workspace_size(int32_t tokens, int32_t top_k, int32_t experts, int32_t hidden,
                             int32_t inner) {
    if (!moe_sizes_ok(tokens, top_k, experts, hidden, inner)) return 0;
    return MoeSpace(tokens, top_k, experts, hidden, inner).end;
}

fg_status fg_moe(const fg_moe_layer* layer, void* workspace, size_t workspace_bytes,
                 hipStream_t stream) {
    clear_error();
    if (!layer) return fail(FG_ERR_INVALID_ARG, 1, "layer is NULL");
    const fg_moe_layer& l = *layer;
    if (l.tokens < 0 || l.tokens > FG_MOE_MAX_TOKENS)
        return fail(FG_ERR_INVALID_ARG, 1, "tokens=%d outside 0 .. %d", l.tokens, FG_MOE_MAX_TOKENS);
    if (l.experts < 1 || l.experts > FG_MOE_MAX_EXPERTS)
        return fail(FG_ERR_INVALID_ARG, 2, "experts=%d outside 1 .. %d", l.experts,
                    FG_MOE_MAX_EXPERTS);
    if (l.top_k < 1 || l.top_k > l.experts || l.top_k > FG_MOE_MAX_TOP_K)
        return fail(FG_ERR_INVALID_ARG, 3, "top_k=%d outside 1 .. min(experts, %d)", l.top_k,
                    FG_MOE_MAX_TOP_K);
    if (l.hidden < 1 || l.hidden > FG_MOE_MAX_DIM)
        return fail(FG_ERR_INVALID_ARG, 4, "hidden=%d outside 1 .. %d", l.hidden, FG_MOE_MAX_DIM);
    if (l.inner < 1 || l.inner > FG_MOE_MAX_DIM)
        return fail(FG_ERR_INVALID_ARG, 5, "inner=%d outside 1 .. %d", l.inner, FG_MOE_MAX_DIM);
    if (l.type != FG_TYPE_F32 && l.type != FG_TYPE_BF16)
        return fail(FG_ERR_INVALID_ARG, 6, "type must be FG_TYPE_F32 or FG_TYPE_BF16");
    if (l.weight_type != FG_TYPE_F32 && l.weight_type != FG_TYPE_BF16 &&
        l.weight_type != FG_TYPE_E4M3)
        return fail(FG_ERR_INVALID_ARG, 7, "unknown weight type %d", l.weight_type);
    if (l.activation < FG_ACT_NONE || l.activation > FG_ACT_SILU)
        return fail(FG_ERR_INVALID_ARG, 8, "unknown activation %d", l.activation);
    if (l.renormalize != 0 && l.renormalize != 1)
        return fail(FG_ERR_INVALID_ARG, 9, "renormalize must be 0 or 1");
    const int64_t T = l.tokens, E = l.experts, H = l.hidden, I = l.inner;
    const uintptr_t size = (uintptr_t)type_size(l.type);
    if (T > 0 && (!l.x || !aligned(l.x, size)))
        return fail(FG_ERR_INVALID_ARG, 10, "x is NULL or misaligned");
    if (l.ldx < H) return fail(FG_ERR_INVALID_ARG, 11, "ldx=%lld < hidden", (long long)l.ldx);
    fg_status st;
    if (T > 0) {
        if ((st = check_experts(l.gate, l.weight_type, E, I, H, 12, "gate")) != FG_OK) return st;
        if ((st = check_experts(l.up, l.weight_type, E, I, H, 13, "up")) != FG_OK) return st;
        if ((st = check_experts(l.down, l.weight_type, E, H, I, 14, "down")) != FG_OK) return st;
    }
    if (l.router) {
        if (l.router_type != FG_TYPE_F32 && l.router_type != FG_TYPE_BF16)
            return fail(FG_ERR_INVALID_ARG, 17, "router_type must be FG_TYPE_F32 or FG_TYPE_BF16");
        if (!aligned(l.router, (uintptr_t)type_size(l.router_type)))
            return fail(FG_ERR_INVALID_ARG, 15, "router is misaligned");
        if (l.ldr < H) return fail(FG_ERR_INVALID_ARG, 16, "ldr=%lld < hidden", (long long)l.ldr);
    }
    if (T > 0 && (!l.ids || !aligned(l.ids, 4)))
        return fail(FG_ERR_INVALID_ARG, 18, "ids is NULL or misaligned");
    if (T > 0 && (!l.weights || !aligned(l.weights, 4)))
        return fail(FG_ERR_INVALID_ARG, 19, "weights is NULL or misaligned");
    if (T > 0 && (!l.out || !aligned(l.out, size)))
        return fail(FG_ERR_INVALID_ARG, 20, "out is NULL or misaligned");
    if (l.ldo < H) return fail(FG_ERR_INVALID_ARG, 21, "ldo=%lld < hidden", (long long)l.ldo);
    if (T == 0) return FG_OK;
    if (!workspace || !aligned(workspace, 16))
        return fail(FG_ERR_INVALID_ARG, 22, "workspace is NULL or not 16-byte aligned");
    const size_t need = fg_moe_workspace_size(l.tokens, l.top_k, l.experts, l.hidden, l.inner);
    if (workspace_bytes < need)
        return fail(FG_ERR_INVALID_ARG, 23, "workspace of %zu bytes, need %zu", workspace_bytes, need);
    if ((st = check_device()) != FG_OK) return st;

    fg::MoeParams p;
    memset(&p, 0, sizeof p);
    p.T = l.tokens;
    p.E = l.experts;
    p.k = l.top_k;
    p.H = l.hidden;
    p.I = l.inner;
    p.x_bf16 = l.type == FG_TYPE_BF16;
    p.wtype = l.weight_type;
    p.act = l.activation;
    p.renorm = l.renormalize;
    p.vec_x = aligned(l.x, 16) && l.ldx * (int64_t)size % 16 == 0;
    p.x = l.x;
    p.ldx = l.ldx;
    p.gate = expert_matrix(l.gate);
    p.up = expert_matrix(l.up);
    p.down = expert_matrix(l.down);
    p.router = l.router;
    p.ldr = l.ldr;
    p.router_bf16 = l.router_type == FG_TYPE_BF16;
    p.vec_r = l.router && aligned(l.router, 16) && l.ldr * type_size(l.router_type) % 16 == 0;
    p.ids = l.ids;
    p.weights = l.weights;
    p.out = l.out;
    p.ldo = l.ldo;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    const MoeSpace space(T, l.top_k, E, H, I);
    p.plan = reinterpret_cast<fg::MoePlan*>(ws + space.plan);
    p.logits = reinterpret_cast<double*>(ws + space.logits);
    p.tickets = reinterpret_cast<int32_t*>(ws + space.tickets);
    p.pieces = reinterpret_cast<float*>(ws + space.pieces);
    p.h = reinterpret_cast<uint16_t*>(ws + space.h);
    const bool wide = p.wtype == fg::TYPE_F32;  // x and h stay binary32
    p.h_ld = (int32_t)moe_h_ld(I);
    p.h_plane = T * l.top_k * moe_h_ld(I);
    p.h_bytes = p.h_plane * (wide ? 4 : 6);
    // x is read in place where its rows are aligned and of the operands' type
    const int64_t extent = ((T - 1) * l.ldx + H) * (int64_t)size;
    if (p.vec_x && wide != (p.x_bf16 != 0) && (wide || p.x_bf16) && H % 8 == 0 &&
        extent < (1ll << 31) && l.ldx <= FG_MAX_LD) {
        p.xs = const_cast<void*>(l.x);
        p.xs_ld = (int32_t)l.ldx;
        p.xs_cols = (int32_t)H;
        p.xs_bytes = extent;
    } else {
        p.xs = ws + space.xs;
        p.xs_made = 1;
        p.xs_ld = p.xs_cols = (int32_t)moe_xs_ld(H);
        p.xs_plane = T * moe_xs_ld(H);
        p.xs_bytes = p.xs_plane * (wide ? 4 : (p.x_bf16 ? 2 : 6));
    }
    // groups: as many tokens as fill 16 columns with the terms of x and of h
    p.gx = fg::moe_group_size(wide || p.x_bf16 ? 1 : 3);
    p.gh = fg::moe_group_size(wide ? 1 : 3);
    p.most_x = (int32_t)most_groups(T, l.top_k, E, p.gx);
    p.most_h = (int32_t)most_groups(T, l.top_k, E, p.gh);
    p.groups_x = reinterpret_cast<fg::MoeGroup*>(ws + space.groups_x);
    if (T == 1) p.gh = p.gx;  // (one token to a group whatever its size)
    p.groups_h =
        p.gh == p.gx ? p.groups_x : reinterpret_cast<fg::MoeGroup*>(ws + space.groups_h);
    p.down_wgs = fg::moe_down_workgroups(p.wtype, p.H, p.I, p.most_h);
    if (l.router)
        st = launched(fg::launch_moe_route(p, stream), "router kernel");
    else
        st = launched(fg::launch_moe_plan(p, stream), "kernel that groups the tokens");
    if (st != FG_OK) return st;
    return launched(fg::launch_moe_experts(p, stream), "expert kernel");
}

}  // extern "C"
