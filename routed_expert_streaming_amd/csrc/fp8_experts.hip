// Routed experts' SwiGLU feed-forward on FP8 slabs: per token and expert
//   g = W1 x, u = W3 x, h = silu(g) * u, y = W2 h
// with x and h quantised to E4M3 in blocks of 1 x 128 and fp32 sums.
//
// g and u are sums of exact products (codes converted to bf16): what the FP8 matrix cores
// cut would move codes of h, and the outputs were then 1.3 times as far from the exact
// ones as their rounding to bf16 leaves them.  y has nothing behind it but that rounding
// and takes the FP8 cores.
#include "common.h"
#include "ffn.h"
#include "fp8_mma.h"
#include "fp8_quant.h"
#include "fp8_rows.h"

namespace {

using moe::f32x4;

constexpr int kMaxE = 1024;
constexpr int kMaxPairs = 16384;   // of a permutation
constexpr int kScanPairs = 512;    // up to here a workgroup finds its expert's pairs itself

struct ExpertArgs {
    moe::Fp8Act a;  // gate/up: x, a row a token; down: h, a row a pair, then a row a token of the shared expert
    int T, H, I, E, k;
    const int32_t *topk_idx;
    const void *const *table;
    const uint8_t *shared, *mask;
    const int32_t *count, *offset, *pair_of_row;  // or NULL: workgroups find their pairs
    float *out;  // gate/up: h [rows, I]; down: y [rows, H]
};

// The rows of one group: pair numbers, or T * k + t for the shared expert's.
struct Group {
    const uint8_t *slab;
    const int32_t *pairs;  // NULL: all tokens, in order
    int rows;
};

// Group blockIdx.y.  With a permutation: expert blockIdx.y, the shared expert last.
// Without: pair blockIdx.y stands for its expert where it is the expert's first pair, and
// the expert's other pairs are found by all waves together; list: kScanPairs numbers.
__device__ __forceinline__ Group find_group(const ExpertArgs &p, int32_t *list) {
    const int P = p.T * p.k, g = blockIdx.y, lane = threadIdx.x & 63;
    const int groups = p.count ? p.E : P;
    if (g >= groups) return {p.shared, nullptr, p.T};
    const int e = p.count ? g : p.topk_idx[g];
    if ((unsigned)e >= (unsigned)p.E || (p.mask && !p.mask[e])) return {nullptr, nullptr, 0};
    if (p.count) return {(const uint8_t *)p.table[e], p.pair_of_row + p.offset[e], p.count[e]};
    int n = 0;
    for (int b = 0; b < P; b += 64) {
        const bool mine = b + lane < P && p.topk_idx[b + lane] == e;
        const uint64_t m = __ballot(mine);
        if (n == 0 && m && b + __ffsll((long long)m) - 1 < g) return {nullptr, nullptr, 0};  // not the first
        if (mine && threadIdx.x < 64) list[n + __popcll(m & ((1ull << lane) - 1))] = b + lane;
        n += __popcll(m);
    }
    __syncthreads();
    return {(const uint8_t *)p.table[e], list, n};
}

// GATEUP: blockIdx.x is 16 columns of h, tile 0 their rows of W1 and tile 1 of W3; down:
// 16 * NT rows of W2.
template <bool GATEUP, int MT, int NT, int WK, int U>
__global__ __launch_bounds__(64 * WK) void fp8_experts_rows_kernel(ExpertArgs p) {
    static_assert(!GATEUP || NT == 2, "a tile of each matrix");
    __shared__ f32x4 part[WK][NT * MT][64];
    __shared__ int32_t list[kScanPairs];
    const Group g = find_group(p, list);
    if (g.rows == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int K = GATEUP ? p.H : p.I, N = GATEUP ? p.I : p.H, n0 = blockIdx.x * 16 * (GATEUP ? 1 : NT);
    const uint8_t *w[NT];
    const float *ws[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const moe::Fp8Slab m = moe::fp8_slab(g.slab, p.H, p.I, GATEUP ? t : 2);
        const int n = min(n0 + (GATEUP ? 0 : 16 * t), N - 1);
        w[t] = m.w + (size_t)min(n + r, N - 1) * K;
        ws[t] = m.s + (size_t)(n / 128) * m.s_row;
    }
    auto row_of = [&](int m) { return g.pairs ? g.pairs[m] : p.T * p.k + m; };
    for (int m0 = 0; m0 < g.rows; m0 += 16 * MT) {
        const uint8_t *a[MT];
        const float *as[MT];
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int m = min(m0 + 16 * u + r, g.rows - 1);
            const int row = GATEUP ? (g.pairs ? g.pairs[m] / p.k : m) : row_of(m);
            a[u] = p.a.codes + (size_t)row * p.a.stride;
            as[u] = reinterpret_cast<const float *>(p.a.scales + (size_t)row * p.a.scale_stride);
        }
        f32x4 acc[NT][MT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        moe::multiply_rows<GATEUP, MT, NT, U, WK>(wave, K, q, w, ws, a, as, acc);
        if (m0) __syncthreads();  // the last rows' sums are read
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < MT; ++u) part[wave][t * MT + u][lane] = acc[t][u];
        __syncthreads();
        constexpr int ITEMS = GATEUP ? MT : NT * MT;
#pragma unroll
        for (int i0 = 0; i0 < ITEMS; i0 += WK) {
            const int i = i0 + wave;
            if (i >= ITEMS) break;
            const int m = m0 + 16 * (i % MT) + r, n = n0 + 16 * (i / MT) + 4 * q;
            f32x4 v = moe::joined<WK, NT * MT>(part, i, lane);
            if constexpr (GATEUP) {
                const f32x4 up = moe::joined<WK, NT * MT>(part, MT + i, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = moe::silu(v[j]) * up[j];
            }
            if (m < g.rows && n < N)  // N % 32 == 0: all four columns exist
                *reinterpret_cast<float4 *>(p.out + (size_t)row_of(m) * N + n) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

struct Space {
    size_t xq, xs, h, hq, hs, count, offset, pairs, y, total;
};
Space layout(int T, int H, int I, int E, int k, bool shared) {
    Space w{};
    const size_t rows = (size_t)T * k + (shared ? (size_t)T : 0);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += moe::align_up(bytes, 256);
        return at;
    };
    w.xq = take((size_t)T * H);
    w.xs = take((size_t)T * moe::fp8_scale_row(H));
    w.h = take(rows * I * 4);
    w.hq = take(rows * I);
    w.hs = take(rows * moe::fp8_scale_row(I));
    w.count = take((size_t)E * 4);
    w.offset = take((size_t)(E + 1) * 4);
    w.pairs = take((size_t)T * k * 4);
    w.y = take(rows * H * 4);
    w.total = o;
    return w;
}

int experts(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
            const void *const *expert_table, const void *shared_slab, const uint8_t *expert_mask, float *y,
            uint8_t *ws, const Space &sp, hipStream_t s) {
    const bool shared = shared_slab != nullptr;
    const int rows = T * k + (shared ? T : 0);
    ExpertArgs a{};
    a.T = T, a.H = H, a.I = I, a.E = E, a.k = k;
    a.topk_idx = topk_idx;
    a.table = expert_table;
    a.shared = (const uint8_t *)shared_slab;
    a.mask = expert_mask;
    const bool scan = T * k <= kScanPairs;
    if (!scan) {
        int32_t *count = (int32_t *)(ws + sp.count), *offset = (int32_t *)(ws + sp.offset);
        int32_t *pairs = (int32_t *)(ws + sp.pairs);
        const int rc = moe::permute_launch(topk_idx, T, k, E, count, offset, pairs, s);
        if (rc != MOE_OK) return rc;
        a.count = count, a.offset = offset, a.pair_of_row = pairs;
    }
    const int groups = (scan ? T * k : E) + (shared ? 1 : 0);
    float *h = (float *)(ws + sp.h);
    int rc = moe::fp8_quant_rows(x, MOE_BF16, (size_t)2 * H, T, H, false, ws + sp.xq, (size_t)H,
                                 (float *)(ws + sp.xs), moe::fp8_scale_row(H), s);
    if (rc != MOE_OK) return rc;
    a.a = {ws + sp.xq, ws + sp.xs, (size_t)H, moe::fp8_scale_row(H)};
    a.out = h;
    hipLaunchKernelGGL((fp8_experts_rows_kernel<true, 1, 2, 8, 2>), dim3(I / 16, groups), dim3(512), 0, s, a);
    MOE_LAUNCH_CHECK("fp8_experts_rows_kernel<gate/up>");
    rc = moe::fp8_quant_rows(h, MOE_FP32, (size_t)4 * I, rows, I, false, ws + sp.hq, (size_t)I,
                             (float *)(ws + sp.hs), moe::fp8_scale_row(I), s);
    if (rc != MOE_OK) return rc;
    a.a = {ws + sp.hq, ws + sp.hs, (size_t)I, moe::fp8_scale_row(I)};
    a.out = y;
    hipLaunchKernelGGL((fp8_experts_rows_kernel<false, 1, 2, 8, 2>), dim3((H + 31) / 32, groups), dim3(512), 0, s, a);
    MOE_LAUNCH_CHECK("fp8_experts_rows_kernel<down>");
    return MOE_OK;
}

int check(const char *who, const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
          const void *const *expert_table, const void *shared_slab, const void *out, const void *workspace,
          size_t workspace_bytes, Space *sp) {
    if (H <= 0 || I <= 0 || H % 32 || I % 32 || H > 16384 || I > 16384)
        return moe::fail(MOE_E_SHAPE, "%s: H=%d and I=%d must be positive multiples of 32 up to 16384", who, H, I);
    if (E < 1 || E > kMaxE || k < 1 || k > E) return moe::fail(MOE_E_SHAPE, "%s: E=%d k=%d", who, E, k);
    if ((long long)T * k > kMaxPairs)
        return moe::fail(MOE_E_SHAPE, "%s: T*k=%lld above %d", who, (long long)T * k, kMaxPairs);
    if (!x || !topk_idx || !expert_table || !out || !workspace) return moe::fail(MOE_E_ARG, "%s: NULL pointer", who);
    if (((uintptr_t)x | (uintptr_t)shared_slab | (uintptr_t)out | (uintptr_t)workspace) % 16)
        return moe::fail(MOE_E_ARG, "%s: x, slabs, output and workspace must be 16-byte aligned", who);
    *sp = layout(T, H, I, E, k, shared_slab != nullptr);
    if (workspace_bytes < sp->total)
        return moe::fail(MOE_E_NOMEM, "%s: workspace %zu < %zu bytes", who, workspace_bytes, sp->total);
    return MOE_OK;
}

}  // namespace

extern "C" size_t moe_expert_bytes_fp8(int hidden, int inter) {
    if (hidden <= 0 || inter <= 0 || hidden % 32 || inter % 32) return 0;
    return moe::fp8_slab_bytes(hidden, inter);
}

extern "C" size_t moe_fp8_expert_ffn_workspace_bytes(int T, int H, int I, int E, int k, int has_shared) {
    if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
    return layout(T, H, I, E, k, has_shared != 0).total;
}

extern "C" int moe_fp8_expert_ffn(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
                                  const void *const *expert_table, const void *shared_slab,
                                  const uint8_t *expert_mask, float *y, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    if (T < 0) return moe::fail(MOE_E_ARG, "fp8_expert_ffn: T=%d < 0", T);
    if (T == 0) return MOE_OK;
    Space sp{};
    const int rc = check("fp8_expert_ffn", x, T, H, I, E, topk_idx, k, expert_table, shared_slab, y, workspace,
                         workspace_bytes, &sp);
    if (rc != MOE_OK) return rc;
    return experts(x, T, H, I, E, topk_idx, k, expert_table, shared_slab, expert_mask, y, (uint8_t *)workspace, sp,
                   (hipStream_t)stream);
}

extern "C" int moe_fp8_expert_ffn_combine(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx,
                                          const float *topk_w, int k, const void *const *expert_table,
                                          const void *shared_slab, uint16_t *out, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    if (T < 0) return moe::fail(MOE_E_ARG, "fp8_expert_ffn_combine: T=%d < 0", T);
    if (T == 0) return MOE_OK;
    if (!topk_w) return moe::fail(MOE_E_ARG, "fp8_expert_ffn_combine: NULL pointer");
    Space sp{};
    int rc = check("fp8_expert_ffn_combine", x, T, H, I, E, topk_idx, k, expert_table, shared_slab, out, workspace,
                   workspace_bytes, &sp);
    if (rc != MOE_OK) return rc;
    float *y = (float *)((uint8_t *)workspace + sp.y);
    rc = experts(x, T, H, I, E, topk_idx, k, expert_table, shared_slab, nullptr, y, (uint8_t *)workspace, sp,
                 (hipStream_t)stream);
    if (rc != MOE_OK) return rc;
    return moe_combine(y, topk_w, T, k, H, shared_slab != nullptr, out, stream);
}
