// Router by scores: logits as the other router's (products and sums in fp64, rounded once
// to fp32), sigmoid or softmax scores, a balance bias that only the choice sees, groups
// of experts, top-k and renormalised, scaled weights.
//
// Scores and the choice are 64-bit: fp32 scores of saturated logits would tie, and a
// balance bias next to them would decide by their rounding.
//
// One wavefront a token; lane l holds experts l, l + 64, ...  A group's worth (its largest
// score or the sum of its two largest) is found by as many lanes as fit the wave, from
// the scores in LDS; the groups are then ranked by counting.  Where every logit is exact
// the top-k runs over order-preserving 64-bit codes in registers, a winner after the other
// (0.65 us each: two reductions of 32 bits over the wave).  Where the logits come with a
// bound on their error, nearly every token is chosen by 32-bit scores with margins, and
// only what these tell apart too little is summed and scored again in 64 bits.
//
// What bounds it: latency.  One token of 4096 x 128: 3.7 us of logits (a launch, a row of w
// a workgroup) and 5.1 of choice.  16 layers of 32 tokens of 6144 x 256: 20 of logits (5 TB/s
// of w) and 24 of choice, 9 of them sums made again; 2048 tokens: 31 and 35, 18 of them.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "router.h"
#include "router_rows.h"
#include "router_split.h"
#include "topk.h"

namespace {

constexpr int kSmallT = 32;  // up to here the logits come from router_partials
constexpr int kMaxE = moe::kTopkMaxE;
constexpr int kMaxGroups = 64;
constexpr int kMaxT = (1 << 26) - 4;  // 64 threads a token: a grid of fewer than 2^32

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

__device__ __forceinline__ double ord_score(uint64_t v) {
    return __longlong_as_double((long long)((v >> 63) ? v & 0x7FFFFFFFFFFFFFFFull : ~v));
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
__device__ __forceinline__ void merge2(float &a, float &b, float c, float d) {
    const float low = fminf(a, c);
    a = fmaxf(a, c);
    b = fmaxf(low, fmaxf(b, d));
}

// A lane's value, in every lane; lane: the same in all.
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float from_lane(float v, int lane) {
    return __uint_as_float(from_lane(__float_as_uint(v), lane));
}
__device__ __forceinline__ double from_lane(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double(
        (long long)((uint64_t)from_lane((uint32_t)(u >> 32), lane) << 32 | from_lane((uint32_t)u, lane)));
}

// Where a token's logits come from.
struct Logits {
    enum Kind { PARTIALS, ROUNDED, SPLIT } kind;  // fp64 partial sums; fp32 logits; fp32 parts with a bound on their error
    const char *ws;
    size_t stride;            // bytes between layers
    moe::RouterSplit sp;      // of SPLIT
    const uint16_t *x;        // [layers, T, H] and
    const float *w, *bias;    // [layers, E, H], for SPLIT's exact sums; [layers, E] or NULL
    int T, H;
};

// This wave's quarter of two logits as the definition has them: products and sums in fp64.
// (Three loads of each row in flight; six took the same time and twice the code.)
__device__ __forceinline__ void exact_quarters(const uint16_t *const (&x)[2], const float *const (&w)[2], int H,
                                               double (&sum)[2]) {
    constexpr int AT_ONCE = 3;
    double a[2] = {0.0, 0.0};
    for (int h0 = 4 * threadIdx.x; h0 < H; h0 += 1024 * AT_ONCE) {
        uint2 xv[2][AT_ONCE];
        float4 wv[2][AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = h0 + 1024 * i;
                xv[k][i] = h < H ? *reinterpret_cast<const uint2 *>(x[k] + h) : make_uint2(0u, 0u);
                wv[k][i] = h < H ? *reinterpret_cast<const float4 *>(w[k] + h) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                a[k] += (double)bf16_bits_to_f32(xv[k][i].x & 0xFFFFu) * (double)wv[k][i].x;
                a[k] += (double)bf16_bits_to_f32(xv[k][i].x >> 16) * (double)wv[k][i].y;
                a[k] += (double)bf16_bits_to_f32(xv[k][i].y & 0xFFFFu) * (double)wv[k][i].z;
                a[k] += (double)bf16_bits_to_f32(xv[k][i].y >> 16) * (double)wv[k][i].w;
            }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) sum[k] = wave_sum_f64(a[k]);
}

// The largest of the lanes' values, none of them negative, in every lane.
__device__ __forceinline__ float wave_max_positive(float v) {
    return __uint_as_float(moe::topk_wave_max(__float_as_uint(v)));
}

// Slots of one token (lane l: experts l + 64 j).  cs: this wave's E scores in LDS, sel: its
// k chosen scores (and its groups' bounds).
//
// SPLIT: logit j is within off[j] of the definition's.  Scores that are further apart than
// both may be off keep their order, so only where two that matter are not -- a group's
// worth next to the last group that stays, an expert next to another one among the first k
// -- the logits behind them are summed again in fp64, and the choice is made again.  A
// logit that is not finite, or whose bound is not, is summed again first.
// The four waves of the workgroup do those sums together, two at a time, a quarter of the
// columns each (asked: the experts that each asks for [4][E], asks: how many, -1 where it is
// done, quarters: two rounds' sums, summed: the logits [4][E]); there: this wave has a token.
template <int PER, bool SPLIT>
__device__ __forceinline__ void choose(float (&l)[PER], float (&off)[PER], bool there, const Choice &c,
                                       const float *balance, const uint16_t *x, const float *w, const float *bias,
                                       int H, double *cs, double *sel, uint16_t *asked, int *asks,
                                       double (*quarters)[2][4], float *summed,
                                       int32_t *idx_out, float *w_out) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool sigmoid = c.score == MOE_SCORE_SIGMOID, drop = c.top_groups < c.groups;
    const int n = c.E / c.groups;  // experts of a group
    int per = 64;                  // lanes of a group
    while (per * c.groups > 64) per >>= 1;
    int slot = 0;
    int told = SPLIT ? 0 : 3;  // what is told apart: all logits finite, then the groups, then the experts
    // one choice; whether some logits (again: bit j, logit j) are to be summed again before the next
    auto once = [&](uint32_t &again) __attribute__((always_inline)) {
        // scores
        double p[PER], key[PER];
        if (sigmoid) {
#pragma unroll
            for (int j = 0; j < PER; ++j) p[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        } else {
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 64 * j < c.E) most = max(most, moe::topk_ord(l[j]));
            const float top = moe::topk_logit(moe::topk_wave_max(most));
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
        // How far a key may be off at most: a sigmoid by a quarter of its logit; of a softmax
        // (SPLIT has none with a balance) only the ratios matter, so its sum may be any number.
        // (e^d - 1 <= d + d^2 up to 1; the margins are for these bounds' own rounding and the
        // 64-bit functions'.)
        float far32 = 0.0f, far_logit32 = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 64 * j;
            key[j] = p[j] + (balance && e < c.E ? (double)balance[e] : 0.0);
            if (SPLIT && e < c.E) {
                const float d = off[j];
                far32 = fmaxf(far32, sigmoid ? 0.25f * d : d <= 1.0f ? (float)p[j] * (d + d * d) : 1e30f);
                far_logit32 = fmaxf(far_logit32, d);
                if (told == 0 && !(fabsf(l[j]) < 1e30f && d < 1e30f)) again |= 1u << j;
            }
        }
        double far = 0.0, far_logit = 0.0;
        if (SPLIT) {
            far = 1.0001 * (double)wave_max_positive(far32) + 1e-15;
            far_logit = 1.0001 * (double)wave_max_positive(far_logit32) + 1e-15;
        }
        bool step = SPLIT && told == 0 && __any(again != 0);  // sum some logits again before going on
        uint64_t in = ~0ull;                                  // bit g * per: group g stays
        if (drop && !step) {
            wave_sync();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 64 * j < c.E) cs[lane + 64 * j] = key[j];
            wave_sync();
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
            const double value = nan ? NAN : c.top2 ? a + b : a;
            const uint64_t worth = score_ord(value);
            int rank = 0;
            for (int h = 0; h < c.groups; ++h) {
                const uint64_t other = __shfl((unsigned long long)worth, h * per, 64);
                rank += other > worth || (other == worth && h < g);
            }
            const bool stays = g < c.groups && rank < c.top_groups;
            in = __ballot(stays);
            if (SPLIT && told <= 1) {
                // groups that are not told from one on the other side of the border, and of those
                // the experts that may be among the ones that make the worth
                const double gap = c.top2 ? 4.0 * far : 2.0 * far;
                const double in_least = ord_score(~wave_max_code(stays ? ~worth : 0ull));
                const double out_most = ord_score(wave_max_code(g < c.groups && !stays ? worth : 0ull));
                const uint64_t close =
                    __ballot(g < c.groups && !(stays ? value - out_most > gap : in_least - value > gap));
                if (close) {
                    if (lane % per == 0 && g < c.groups) sel[g] = (c.top2 ? b : a) - 2.0 * far;
                    wave_sync();
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int e = lane + 64 * j, ge = e / n;
                        if (e < c.E && (close >> (ge * per) & 1) && off[j] > 0.0f && !(key[j] < sel[ge])) again |= 1u << j;
                    }
                    step = __any(again != 0);
                    if (step) told = 2;
                }
            }
        }
        if (!step) {
            uint64_t ord[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int e = lane + 64 * j;
                ord[j] = e < c.E && (!drop || (in >> (e / n * per) & 1)) ? score_ord(key[j]) : 0ull;
            }
            const bool look = SPLIT && told < 3;
            double before = 0.0;  // the last winner's key or logit
            int before_e = 0;
            for (int i = 0; i < c.k || look; ++i) {
                uint64_t best = 0;
                int best_j = 0;
                float best_l = 0.0f;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (ord[j] > best) {  // strict: the lower index wins a tie inside the lane
                        best = ord[j];
                        best_j = j;
                        best_l = l[j];
                    }
                const uint64_t top = wave_max_code(best);
                if (i >= c.k && top == 0) break;
                uint32_t e = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const uint64_t m = __ballot(best == top && best_j == j);
                    if (m) {
                        e = 64u * j + (uint32_t)(__ffsll((long long)m) - 1);
                        break;
                    }
                }
                if (look) {
                    // next to the one before it: both again (softmax: by their logits, or where the
                    // scores end)
                    const double now = sigmoid ? ord_score(top) : (double)__shfl(best_l, (int)(e & 63), 64);
                    const bool close = i > 0 && (!(before - now > 2.0 * (sigmoid ? far : far_logit)) ||
                                                 (!sigmoid && ord_score(top) < 1e-290));
                    if (i >= c.k && !close) break;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int mine = lane + 64 * j;
                        if (close && (mine == (int)e || mine == before_e) && off[j] > 0.0f) again |= 1u << j;
                    }
                    before = now;
                    before_e = (int)e;
                }
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if ((uint32_t)(lane + 64 * j) == e) {  // the owner drops the winner
                        ord[j] = 0ull;
                        if (i < c.k) sel[i] = p[j];
                    }
                if (lane == i) slot = (int)e;
            }
            told = 3;
            step = SPLIT && __any(again != 0);
        } else if (told == 0) {
            told = 1;
        }
        return step;
    };
    // SPLIT's way for nearly every token, in 32 bits: scores with their rounding added to what
    // they may be off by; the groups (those at the border once more, with the logits that make
    // their worth summed again); the winners with all that are not told from them, which are
    // then ordered by 64-bit scores of their logits, summed again where need be.  Lane i: the
    // i-th of `entries`.  Left to the above: logits or scores that are not finite, groups that
    // are not told apart in 32 bits then either, more than 64 entries, softmax's 64-bit zeros.
    // (6144 x 256, 16 layers of 32 tokens: 27 us by the above alone, 24 so; 2048 tokens 44 and 36.)
    int entries = 0, entry = 0;
    float entry_l = 0.0f, top_l = 0.0f;
    uint64_t redo = 0;  // entries whose logits are summed again
    enum { START, GROUPS, RANKED, SLOW } way = START;
    auto quick = [&](uint32_t &again) __attribute__((always_inline)) {
        float key[PER], far = 0.0f, far_logit = 0.0f, size = 1.0f;
        bool odd = false;
        if (!sigmoid) {
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 64 * j < c.E) most = max(most, moe::topk_ord(l[j]));
            top_l = moe::topk_logit(moe::topk_wave_max(most));
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 64 * j;
            const float d = off[j], v = expf(sigmoid ? -l[j] : l[j] - top_l), q = sigmoid ? 1.0f / (1.0f + v) : v;
            key[j] = q;
            if (e >= c.E) continue;
            if (balance) key[j] += balance[e];
            far = fmaxf(far, sigmoid ? 0.25f * d : d <= 1.0f ? q * (d + d * d) : 1e30f);
            far_logit = fmaxf(far_logit, d);
            odd |= !(fabsf(l[j]) < 1e30f && d < 1e30f) || !(fabsf(key[j]) < 1e30f || key[j] == -INFINITY);
            if (key[j] > -INFINITY) size = fmaxf(size, fabsf(key[j]));
        }
        if (__any(odd)) return SLOW;
        // a score is within 2^-21 of itself (the exponential, 1 +, 1 /), at most 1; and the sum's rounding
        const float rounding = 0x1p-21f * wave_max_positive(size);
        far = 1.001f * wave_max_positive(far) + rounding;
        far_logit = 1.001f * wave_max_positive(far_logit) + 0x1p-21f;
        uint64_t in = ~0ull;
        if (drop) {
            float *keys = reinterpret_cast<float *>(cs);
            wave_sync();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 64 * j < c.E) keys[lane + 64 * j] = key[j];
            wave_sync();
            const int g = lane / per;
            float a = -INFINITY, b = -INFINITY;
            if (g < c.groups)
                for (int i = lane % per; i < n; i += per) merge2(a, b, keys[g * n + i], -INFINITY);
            for (int o = 1; o < per; o <<= 1) {
                const float c1 = __shfl_xor(a, o, 64), c2 = __shfl_xor(b, o, 64);
                merge2(a, b, c1, c2);
            }
            const float value = c.top2 ? a + b : a;
            const uint32_t worth = moe::topk_ord(value);
            int rank = 0;
            for (int h = 0; h < c.groups; ++h) {
                const uint32_t other = from_lane(worth, h * per);
                rank += other > worth || (other == worth && h < g);
            }
            const bool stays = g < c.groups && rank < c.top_groups;
            in = __ballot(stays);
            const float gap = (c.top2 ? 4.01f : 2.01f) * (way == START ? far : rounding);
            const float in_least = moe::topk_logit(~moe::topk_wave_max(stays ? ~worth : 0u));
            const float out_most = moe::topk_logit(moe::topk_wave_max(g < c.groups && !stays ? worth : 0u));
            const uint64_t close =
                __ballot(g < c.groups && !(stays ? value - out_most > gap : in_least - value > gap));
            if (close) {
                if (way != START) return SLOW;
                // of those groups the experts that may be among the ones that make the worth
                if (lane % per == 0 && g < c.groups) sel[g] = (c.top2 ? b : a) - 2.01f * far;
                wave_sync();
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int e = lane + 64 * j, ge = e / n;
                    if (e < c.E && (close >> (ge * per) & 1) && off[j] > 0.0f && !(key[j] < sel[ge])) again |= 1u << j;
                }
                return GROUPS;
            }
        }
        uint32_t ord[PER];  // softmax: by the logits
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 64 * j;
            ord[j] = e < c.E && (!drop || (in >> (e / n * per) & 1)) ? moe::topk_ord(sigmoid ? key[j] : l[j]) : 0u;
        }
        const float apart = 2.01f * (sigmoid ? far : far_logit);
        float before = 0.0f;
        uint64_t sums = 0;  // entries whose logits are sums with a bound
        for (int i = 0;; ++i) {
            uint32_t best = 0;
            int best_j = 0;
            float best_l = 0.0f, best_off = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (ord[j] > best) best = ord[j], best_j = j, best_l = l[j], best_off = off[j];
            const uint32_t top = moe::topk_wave_max(best);
            if (top == 0) break;
            const float now = moe::topk_logit(top);
            const bool close = i > 0 && !(before - now > apart);
            if (i >= c.k && !close) break;
            if (i >= 64 || (!sigmoid && now - top_l < -600.0f)) return SLOW;
            const int at = __ffsll((long long)__ballot(best == top)) - 1, at_j = __builtin_amdgcn_readlane(best_j, at);
            const float at_l = from_lane(best_l, at);
            if (from_lane(best_off, at) > 0.0f) sums |= 1ull << i;
            if (close) redo |= 3ull << (i - 1);
            if (lane == i) entry = at + 64 * at_j, entry_l = at_l;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (j == at_j && lane == at) ord[j] = 0u;
            before = now;
            entries = i + 1;
        }
        redo &= sums;
        for (uint64_t m = redo; m; m &= m - 1) {
            const int e = __builtin_amdgcn_readlane(entry, __ffsll((long long)m) - 1);
            if (lane == (e & 63)) again |= 1u << (e >> 6);
        }
        return RANKED;
    };
    if constexpr (!SPLIT) {
        uint32_t again = 0;
        if (there) once(again);
    } else {
        for (bool open = there;;) {
            uint32_t again = 0;
            if (open && way == RANKED) {
                open = false;
            } else if (open) {
                if (way != SLOW) way = quick(again);
                if (way == SLOW) {
                    again = 0;
                    open = once(again);
                    if (!open) again = 0;
                } else if (way == RANKED) {
                    open = redo != 0;
                }
            }
            int mine = 0;  // this wave's experts, one after the other
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t m = __ballot(again >> j & 1);
                if (again >> j & 1) asked[wave * c.E + mine + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(lane + 64 * j);
                mine += __popcll(m);
            }
            if (lane == 0) asks[wave] = open ? mine : -1;
            __syncthreads();
            int upto[4], any = 0;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = __builtin_amdgcn_readfirstlane(asks[v]);
                any |= m >= 0;
                upto[v] = (v ? upto[v - 1] : 0) + (m > 0 ? m : 0);
            }
            if (!any) break;
            for (int at = 0, round = 0; at < upto[3]; at += 2, ++round) {
                int pair[2];  // of [4][E]; the last one again where there are no more
                const uint16_t *xs[2];
                const float *wr[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = min(at + k, upto[3] - 1), v = (i >= upto[0]) + (i >= upto[1]) + (i >= upto[2]);
                    const int first = v == 0 ? 0 : v == 1 ? upto[0] : v == 2 ? upto[1] : upto[2];
                    const int e = __builtin_amdgcn_readfirstlane(asked[v * c.E + i - first]);
                    pair[k] = v * c.E + e, xs[k] = x + (size_t)v * H, wr[k] = w + (size_t)e * H;
                }
                double v[2];
                exact_quarters(xs, wr, H, v);
                double(*q)[4] = quarters[round & 1];
                if (lane < 2) q[lane][wave] = lane ? v[1] : v[0];
                __syncthreads();
                if (threadIdx.x < 2) {
                    const int k = threadIdx.x, at_pair = k ? pair[1] : pair[0];
                    summed[at_pair] = (float)(((q[k][0] + q[k][1]) + (q[k][2] + q[k][3])) +
                                              (bias ? (double)bias[at_pair % c.E] : 0.0));
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (again >> j & 1) l[j] = summed[wave * c.E + lane + 64 * j], off[j] = 0.0f;
        }
    }
    if (!there) return;
    if (SPLIT && way == RANKED) {
        if (redo >> lane & 1) entry_l = summed[wave * c.E + entry];
        const double v = exp(sigmoid ? -(double)entry_l : (double)entry_l - (double)top_l);
        double p = sigmoid ? 1.0 / (1.0 + v) : v;
        const double key = balance && lane < entries ? p + (double)balance[entry] : p;
        int rank = 0;
        for (int i = 0; i < entries; ++i) {
            const double other = from_lane(key, i);
            rank += other > key || (other == key && __builtin_amdgcn_readlane(entry, i) < entry);
        }
        if (!sigmoid && !c.renorm) {  // the sum of all: 32-bit terms, as precise as the logits are
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 64 * j < c.E) sum += (double)expf(l[j] - top_l);
            p /= wave_sum_f64(sum);
        }
        wave_sync();
        if (lane < entries && rank < c.k) {
            sel[rank] = p;
            asked[wave * c.E + rank] = (uint16_t)entry;
        }
        wave_sync();
        slot = lane < c.k ? asked[wave * c.E + lane] : 0;
    }
    wave_sync();
    double wt = lane < c.k ? sel[lane] : 0.0;
    if (c.renorm) {
        double all = 0.0;
        for (int i = 0; i < c.k; ++i) all += sel[i];
        wt = all == 0.0 ? 0.0 : wt / all;
    }
    if (lane < c.k) {
        idx_out[lane] = slot;
        w_out[lane] = (float)((double)c.scale * wt);
    }
}

// Dynamic LDS: four waves' scores [E] (when groups are dropped), their chosen ones [64], then
// (SPLIT) what is asked for and the four tokens' exact logits [E].
template <int PER, int KIND>
__global__ __launch_bounds__(256, 2) void router_choose_kernel(Logits from, const float *__restrict__ balance, Choice c,
                                                            int32_t *__restrict__ idx, float *__restrict__ w) {
    extern __shared__ double lds[];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, T = from.T;
    const int mine = blockIdx.x * 4 + wave, t = min(mine, T - 1);
    const char *src = from.ws + blockIdx.y * from.stride;
    const float *bias = from.bias ? from.bias + (size_t)blockIdx.y * c.E : nullptr;
    if (balance) balance += (size_t)blockIdx.y * c.E;
    const size_t row = (size_t)blockIdx.y * T + t;
    float l[PER], off[PER];
    if constexpr (KIND == Logits::SPLIT) {
        // the parts' sums and norms, so many parts' loads in flight at a time
        constexpr int AT_ONCE = PER <= 4 ? 8 : PER == 8 ? 4 : 2;
        const int parts = from.sp.parts;
        const float *part = reinterpret_cast<const float *>(src + from.sp.partial) + (size_t)t * c.E;
        const float *xnorm = reinterpret_cast<const float *>(src + from.sp.xn) + t;
        const float *wnorm = reinterpret_cast<const float *>(src + from.sp.wn);
        double v[PER];
        float xn = 0.0f, wn[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = 0.0, wn[j] = 0.0f;
        for (int i0 = 0; i0 < parts; i0 += AT_ONCE) {
            float a[AT_ONCE][PER], b[AT_ONCE][PER], d[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int pi = min(i0 + i, parts - 1);
                d[i] = xnorm[(size_t)pi * T];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int e = min(lane + 64 * j, c.E - 1);
                    a[i][j] = part[(size_t)pi * T * c.E + e];
                    b[i][j] = wnorm[(size_t)pi * c.E + e];
                }
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                if (i0 + i >= parts) break;
                xn += d[i];
#pragma unroll
                for (int j = 0; j < PER; ++j) v[j] += a[i][j], wn[j] += b[i][j];
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            l[j] = (float)(v[j] + (bias ? (double)bias[min(lane + 64 * j, c.E - 1)] : 0.0));
            off[j] = moe::router_split_error(from.sp.columns, xn, wn[j], l[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = min(lane + 64 * j, c.E - 1);
            off[j] = 0.0f;
            if constexpr (KIND == Logits::PARTIALS)
                l[j] = moe::router_logit((const double *)src + (size_t)t * c.E * moe::kMaxSlices,
                                         (from.H + moe::kSlice - 1) / moe::kSlice, bias, e);
            else
                l[j] = ((const float *)src)[(size_t)t * c.E + e];
        }
    }
    const int scores = c.top_groups < c.groups ? c.E : 0;
    double *sel = lds + 4 * scores + 64 * wave;
    double(*quarters)[2][4] = reinterpret_cast<double(*)[2][4]>(lds + 4 * scores + 256);
    float *summed = reinterpret_cast<float *>(quarters + 2);
    int *asks = reinterpret_cast<int *>(summed + 4 * c.E);
    choose<PER, KIND == Logits::SPLIT>(l, off, mine < T, c, balance, from.x + ((size_t)blockIdx.y * T + 4 * blockIdx.x) * from.H,
                                       from.w + (size_t)blockIdx.y * c.E * from.H, bias, from.H, lds + wave * scores, sel,
                                       reinterpret_cast<uint16_t *>(asks + 4), asks, quarters, summed, idx + row * c.k,
                                       w + row * c.k);
}

template <int KIND>
int launch_choose(const Logits &from, int layers, const float *balance, const Choice &c, int32_t *idx, float *w,
                  hipStream_t s) {
    const dim3 grid((from.T + 3) / 4, layers), block(256);
    const size_t lds = ((c.top_groups < c.groups ? (size_t)4 * c.E : 0) + 256) * sizeof(double) +
                       (KIND == Logits::SPLIT ? 16 * sizeof(double) + (size_t)4 * c.E * 6 + 16 : 0);
    auto *kernel = c.E <= 64    ? router_choose_kernel<1, KIND>
                   : c.E <= 128 ? router_choose_kernel<2, KIND>
                   : c.E <= 256 ? router_choose_kernel<4, KIND>
                   : c.E <= 512 ? router_choose_kernel<8, KIND>
                                : router_choose_kernel<16, KIND>;
    hipLaunchKernelGGL(kernel, grid, block, lds, s, from, balance, c, idx, w);
    MOE_LAUNCH_CHECK("router_choose_kernel");
    return MOE_OK;
}

// Bytes of one layer's workspace by where its logits come from.
size_t exact_bytes(int T, int E) {
    return T <= kSmallT ? (size_t)T * E * moe::kMaxSlices * sizeof(double)
                        : moe::align_up((size_t)T * E * sizeof(float), 256);
}
// Where the logits come from the split sums.  Calls of sigmoid scores with a balance, in a
// graph, us with exact sums and split:
//   tokens                    4         8         9        12        16        17        32
//   1 layer, 4096 x 128    11  19    15  19    16  19    19  19    23  20    24  20    37  21
//   1 layer, 6144 x 256    16  24    20  25    21  25    24  26    28  26    29  27    51  29
//   1 layer, 1024 x 64     10  13    14  14    15  15    18  15    22  15    23  15    37  15
//   8 layers, 4096 x 128   16  23    23  24    25  24    30  24    36  25    37  26    61  25
//   16 layers, 6144 x 256  52  40    74  41    80  41    96  42   118  44   123  43   214  45
// So the split would pay from 9 to 13 tokens of one layer on, and from fewer of many large
// layers; the rule keeps the weights of up to 16 tokens (8 of several layers) exact.
bool split_pays(int layers, int T) { return T > (layers > 1 ? 8 : 16); }

}  // namespace

extern "C" size_t moe_router_scored_workspace_bytes(int n_layers, int T, int E, int H) {
    if (n_layers <= 0 || T <= 0 || T > kMaxT || E <= 0 || E > kMaxE || H <= 0) return 0;
    // enough for every call of fewer tokens or layers too, whichever way their logits come
    size_t exact = exact_bytes(T, E);
    if (T > kSmallT) exact = std::max(exact, exact_bytes(kSmallT, E));
    exact *= (size_t)n_layers;
    return split_pays(n_layers, T) ? std::max(exact, moe::router_split_most(n_layers, T, E, H)) : exact;
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
    if (n_layers > 65535 || T > kMaxT)
        return moe::fail(MOE_E_SHAPE, "router_scored: n_layers=%d above 65535 or T=%d above %d", n_layers, T, kMaxT);
    if (((uintptr_t)x | (uintptr_t)w_router) % 16 || (uintptr_t)workspace % 16)
        return moe::fail(MOE_E_ARG, "router_scored: x, w_router and workspace must be 16-byte aligned");
    const size_t need = moe_router_scored_workspace_bytes(n_layers, T, E, H);
    if (workspace_bytes < need)
        return moe::fail(MOE_E_NOMEM, "router_scored: workspace %zu < %zu bytes", workspace_bytes, need);
    const Choice c{E, k, routing->score, groups, top, routing->group_rule == MOE_GROUP_TOP2, routing->renormalise,
                   routing->scale};
    hipStream_t s = (hipStream_t)stream;
    Logits from{Logits::PARTIALS, (const char *)workspace, exact_bytes(T, E), {}, x, w_router, bias, T, H};
    // A softmax next to a balance takes exact sums: the split's bound is on ratios of its scores,
    // and beside a balance their sum's error counts too.  2048 x 6144 x 256: 205 us (51 without
    // the balance); 16 layers of 32 tokens: 216 (42).
    if (split_pays(n_layers, T) && !(balance && routing->score == MOE_SCORE_SOFTMAX)) {
        from.kind = Logits::SPLIT;
        from.sp = moe::router_split_layout(n_layers, T, E, H);
        from.stride = from.sp.total;
        const int rc = moe::router_split(x, n_layers, T, H, w_router, E, from.sp, workspace, s);
        if (rc != MOE_OK) return rc;
        return launch_choose<Logits::SPLIT>(from, n_layers, balance, c, topk_idx, topk_w, s);
    }
    if (T <= kSmallT) {
        const int rc = moe::router_partials(x, T, H, w_router, E, (double *)workspace, s, n_layers, from.stride);
        if (rc != MOE_OK) return rc;
        return launch_choose<Logits::PARTIALS>(from, n_layers, balance, c, topk_idx, topk_w, s);
    }
    from.kind = Logits::ROUNDED;
    for (int l = 0; l < n_layers; ++l) {
        const int rc = moe::router_logits_rows(x + (size_t)l * T * H, T, H, w_router + (size_t)l * E * H,
                                               bias ? bias + (size_t)l * E : nullptr, E,
                                               (float *)((char *)workspace + (size_t)l * from.stride), s);
        if (rc != MOE_OK) return rc;
    }
    return launch_choose<Logits::ROUNDED>(from, n_layers, balance, c, topk_idx, topk_w, s);
}
