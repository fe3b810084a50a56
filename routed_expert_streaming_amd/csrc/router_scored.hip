// Router by scores: logits as the other router's (products and sums in fp64, rounded once
// to fp32), sigmoid or softmax scores, a balance bias that only the choice sees, groups
// of experts, top-k and renormalised, scaled weights.
//
// Scores and the choice are 64-bit: fp32 scores of saturated logits would tie, and a
// balance bias next to them would decide by their rounding.
//
// One wavefront a token; lane l holds experts l, l + 64, ...  A group's worth (its largest
// score or the sum of its two largest) is found by as many lanes as fit the wave, from
// the scores in LDS; the groups are then ranked by counting, and the top-k runs over
// order-preserving 64-bit codes in registers.
#include <cmath>

#include "common.h"
#include "router.h"
#include "topk.h"

namespace {

constexpr int kSmallT = 32;  // up to here the logits come from router_partials
constexpr int kMaxE = moe::kTopkMaxE;
constexpr int kMaxGroups = 64;

struct Choice {
    int E, k, score, groups, top_groups, top2, renorm;
    float scale;
};

// What this wave wrote to LDS before is what its lanes read after.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// order-preserving code of a score: 0 is absent, a NaN ranks first
__device__ __forceinline__ uint64_t score_ord(double c) {
    if (c != c) return ~0ull;
    if (c == 0.0) c = 0.0;  // -0 -> +0
    const uint64_t u = (uint64_t)__double_as_longlong(c);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// The largest of the lanes' codes, in every lane.
__device__ __forceinline__ uint64_t wave_max_code(uint64_t v) {
    const uint32_t hi = moe::topk_wave_max((uint32_t)(v >> 32));
    const uint32_t lo = moe::topk_wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The two largest of both pairs.
__device__ __forceinline__ void merge2(double &a, double &b, double c, double d) {
    const double low = fmin(a, c);
    a = fmax(a, c);
    b = fmax(low, fmax(b, d));
}

// Slots of one token from its logits (l[j]: expert lane + 64 j).  cs: this wave's E
// scores in LDS, sel: its k chosen scores.
template <int PER>
__device__ __forceinline__ void choose(const float (&l)[PER], const float *balance, const Choice &c, double *cs,
                                       double *sel, int32_t *idx_out, float *w_out) {
    const int lane = threadIdx.x & 63;
    double p[PER];
    if (c.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (lane + 64 * j < c.E) top = fmaxf(top, l[j]);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            p[j] = exp((double)l[j] - (double)top);
            if (lane + 64 * j < c.E) sum += p[j];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] /= sum;
    }
    double s[PER];
    uint64_t ord[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 64 * j;
        s[j] = p[j] + (balance && e < c.E ? (double)balance[e] : 0.0);
        ord[j] = e < c.E ? score_ord(s[j]) : 0ull;
    }
    if (c.top_groups < c.groups) {
        const int n = c.E / c.groups;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (lane + 64 * j < c.E) cs[lane + 64 * j] = s[j];
        wave_sync();
        int per = 64;  // lanes of a group
        while (per * c.groups > 64) per >>= 1;
        const int g = lane / per;
        double a = -INFINITY, b = -INFINITY;
        bool nan = false;
        if (g < c.groups)
            for (int i = lane % per; i < n; i += per) {
                const double v = cs[g * n + i];
                nan |= v != v;
                merge2(a, b, v, -INFINITY);
            }
        for (int o = 1; o < per; o <<= 1) {
            const double c1 = __shfl_xor(a, o, 64), c2 = __shfl_xor(b, o, 64);
            nan |= (bool)__shfl_xor((int)nan, o, 64);
            merge2(a, b, c1, c2);
        }
        const uint64_t worth = score_ord(nan ? NAN : c.top2 ? a + b : a);
        int rank = 0;
        for (int h = 0; h < c.groups; ++h) {
            const uint64_t other = __shfl((unsigned long long)worth, h * per, 64);
            rank += other > worth || (other == worth && h < g);
        }
        const uint64_t in = __ballot(g < c.groups && rank < c.top_groups);  // lane g * per: group g
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 64 * j;
            if (e < c.E && !(in >> (e / n * per) & 1)) ord[j] = 0ull;
        }
    }
    int slot = 0;
    for (int i = 0; i < c.k; ++i) {
        uint64_t best = 0;
        int best_j = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (ord[j] > best) best = ord[j], best_j = j;  // strict: the lower index wins a tie inside the lane
        const uint64_t top = wave_max_code(best);
        uint32_t e = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint64_t m = __ballot(best == top && best_j == j);
            if (m) {
                e = 64u * j + (uint32_t)(__ffsll((long long)m) - 1);
                break;
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((uint32_t)(lane + 64 * j) == e) {  // the owner drops the winner
                ord[j] = 0ull;
                sel[i] = p[j];
            }
        if (lane == i) slot = (int)e;
    }
    wave_sync();
    double w = lane < c.k ? sel[lane] : 0.0;
    if (c.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (lane < c.k) {
        idx_out[lane] = slot;
        w_out[lane] = (float)((double)c.scale * w);
    }
}

// Dynamic LDS: four waves' scores [E] (when groups are dropped), then their chosen ones [64].
template <int PER, bool PARTIAL>
__global__ __launch_bounds__(256) void router_choose_kernel(const void *__restrict__ from, size_t from_stride, int T,
                                                            int nslices, const float *__restrict__ bias,
                                                            const float *__restrict__ balance, Choice c,
                                                            int32_t *__restrict__ idx, float *__restrict__ w) {
    extern __shared__ double lds[];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    if (t >= T) return;
    const void *src = (const char *)from + blockIdx.y * from_stride;
    if (bias) bias += (size_t)blockIdx.y * c.E;
    if (balance) balance += (size_t)blockIdx.y * c.E;
    const size_t at = ((size_t)blockIdx.y * T + t) * c.k;
    float l[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = min(lane + 64 * j, c.E - 1);
        if constexpr (PARTIAL)
            l[j] = moe::router_logit((const double *)src + (size_t)t * c.E * moe::kMaxSlices, nslices, bias, e);
        else
            l[j] = ((const float *)src)[(size_t)t * c.E + e];
    }
    const int scores = c.top_groups < c.groups ? c.E : 0;
    choose<PER>(l, balance, c, lds + wave * scores, lds + 4 * scores + 64 * wave, idx + at, w + at);
}

template <bool PARTIAL>
int launch_choose(const void *from, size_t from_stride, int layers, int T, int H, const float *bias,
                  const float *balance, const Choice &c, int32_t *idx, float *w, hipStream_t s) {
    const dim3 grid((T + 3) / 4, layers), block(256);
    const size_t lds = ((c.top_groups < c.groups ? (size_t)4 * c.E : 0) + 256) * sizeof(double);
    const int nslices = (H + moe::kSlice - 1) / moe::kSlice;
    auto *kernel = c.E <= 64    ? router_choose_kernel<1, PARTIAL>
                   : c.E <= 128 ? router_choose_kernel<2, PARTIAL>
                   : c.E <= 256 ? router_choose_kernel<4, PARTIAL>
                   : c.E <= 512 ? router_choose_kernel<8, PARTIAL>
                                : router_choose_kernel<16, PARTIAL>;
    hipLaunchKernelGGL(kernel, grid, block, lds, s, from, from_stride, T, nslices, bias, balance, c, idx, w);
    MOE_LAUNCH_CHECK("router_choose_kernel");
    return MOE_OK;
}

// Bytes of one layer's workspace: fp64 partial logits, or fp32 logits.
size_t layer_bytes(int T, int E) {
    return T <= kSmallT ? (size_t)T * E * moe::kMaxSlices * sizeof(double)
                        : moe::align_up((size_t)T * E * sizeof(float), 256);
}

}  // namespace

extern "C" size_t moe_router_scored_workspace_bytes(int n_layers, int T, int E, int H) {
    if (n_layers <= 0 || T <= 0 || E <= 0 || E > kMaxE || H <= 0) return 0;
    return (size_t)n_layers * layer_bytes(T, E);
}

extern "C" int moe_router_scored(const uint16_t *x, int n_layers, int T, int H, const float *w_router,
                                 const float *bias, const float *balance, int E, int k, const moe_routing *routing,
                                 int32_t *topk_idx, float *topk_w, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    if (T < 0 || n_layers < 0)
        return moe::fail(MOE_E_ARG, "router_scored: T=%d, n_layers=%d must be >= 0", T, n_layers);
    if (!routing) return moe::fail(MOE_E_ARG, "router_scored: NULL routing");
    if (routing->score != MOE_SCORE_SOFTMAX && routing->score != MOE_SCORE_SIGMOID)
        return moe::fail(MOE_E_ARG, "router_scored: score=%d", routing->score);
    if (routing->group_rule != MOE_GROUP_MAX && routing->group_rule != MOE_GROUP_TOP2)
        return moe::fail(MOE_E_ARG, "router_scored: group_rule=%d", routing->group_rule);
    if (!std::isfinite(routing->scale)) return moe::fail(MOE_E_ARG, "router_scored: scale is not finite");
    if (H <= 0 || H % 32 != 0 || H > moe::kSlice * moe::kMaxSlices)
        return moe::fail(MOE_E_SHAPE, "router_scored: H=%d must be a positive multiple of 32 up to %d", H,
                         moe::kSlice * moe::kMaxSlices);
    if (E <= 0 || E > kMaxE) return moe::fail(MOE_E_SHAPE, "router_scored: E=%d outside 1..%d", E, kMaxE);
    const int groups = routing->n_groups, top = routing->top_groups;
    if (groups < 1 || groups > kMaxGroups || E % groups)
        return moe::fail(MOE_E_SHAPE, "router_scored: %d groups of %d experts (at most %d, of equal size)", groups, E,
                         kMaxGroups);
    if (top < 1 || top > groups) return moe::fail(MOE_E_SHAPE, "router_scored: top_groups=%d of %d", top, groups);
    if (top < groups && routing->group_rule == MOE_GROUP_TOP2 && E / groups < 2)
        return moe::fail(MOE_E_SHAPE, "router_scored: two scores of groups of one expert");
    if (k < 1 || k > moe::kTopkMaxK || k > E / groups * top)
        return moe::fail(MOE_E_SHAPE, "router_scored: k=%d outside 1..min(%d, experts of %d groups)", k,
                         moe::kTopkMaxK, top);
    if (T == 0 || n_layers == 0) return MOE_OK;
    if (!x || !w_router || !topk_idx || !topk_w || !workspace)
        return moe::fail(MOE_E_ARG, "router_scored: NULL pointer");
    if (n_layers > 65535) return moe::fail(MOE_E_SHAPE, "router_scored: n_layers=%d above 65535", n_layers);
    if (((uintptr_t)x | (uintptr_t)w_router) % 16 || (uintptr_t)workspace % 16)
        return moe::fail(MOE_E_ARG, "router_scored: x, w_router and workspace must be 16-byte aligned");
    const size_t per = layer_bytes(T, E), need = (size_t)n_layers * per;
    if (workspace_bytes < need)
        return moe::fail(MOE_E_NOMEM, "router_scored: workspace %zu < %zu bytes", workspace_bytes, need);
    const Choice c{E, k, routing->score, groups, top, routing->group_rule == MOE_GROUP_TOP2, routing->renormalise,
                   routing->scale};
    hipStream_t s = (hipStream_t)stream;
    if (T <= kSmallT) {
        const int rc = moe::router_partials(x, T, H, w_router, E, (double *)workspace, s, n_layers, per);
        if (rc != MOE_OK) return rc;
        return launch_choose<true>(workspace, per, n_layers, T, H, bias, balance, c, topk_idx, topk_w, s);
    }
    for (int l = 0; l < n_layers; ++l) {
        const int rc = moe::router_logits_rows(x + (size_t)l * T * H, T, H, w_router + (size_t)l * E * H,
                                               bias ? bias + (size_t)l * E : nullptr, E,
                                               (float *)((char *)workspace + (size_t)l * per), s);
        if (rc != MOE_OK) return rc;
    }
    return launch_choose<false>(workspace, per, n_layers, T, H, bias, balance, c, topk_idx, topk_w, s);
}
