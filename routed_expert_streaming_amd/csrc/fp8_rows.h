// Few rows of activations: W straight into registers, K split over a workgroup's waves.
//
// A workgroup owns 16 * NT rows of W and walks over its rows of A 16 * MT at a time; its
// WK waves take steps of U blocks of 128 columns in turn and their sums are joined
// through LDS, in wave order.  A step's operands are loaded while the one before is
// multiplied.  Rows past the last one repeat it (their results are not stored).
#pragma once
#include "fp8_mma.h"

namespace moe {

struct Fp8Act {
    const uint8_t *codes, *scales;
    size_t stride, scale_stride;  // bytes between rows
};

// acc[t][u] += rows of W (tile t) x rows of A (tile u) over the wave's steps.
// w[t]: this lane's row of the tile (from its piece q); ws[t]: the tile's scales, one
// per block; a[u], as[u]: this lane's row of the activations and its scales.
template <int MT, int NT, int U>
struct Fp8Step {
    Fp8Frag w[NT][U], x[MT][U];
    float ws[NT][U], as[MT][U];
};
template <int MT, int NT, int U>
__device__ __forceinline__ void load_step(Fp8Step<MT, NT, U> &s, int step, int K, int q,
                                          const uint8_t *const (&w)[NT], const float *const (&ws)[NT],
                                          const uint8_t *const (&a)[MT], const float *const (&as)[MT]) {
    const int blocks = (K + 127) / 128;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int b = min(step * U + i, blocks - 1);
        const int last = min(8, (K - 128 * b) / 16) - 1;  // last piece of the block
        const int lo = 128 * b + 16 * min(q, last), hi = 128 * b + 16 * min(q + 4, last);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s.w[t][i].lo = load_global_u4(w[t] + lo);
            s.w[t][i].hi = load_global_u4(w[t] + hi);
            s.ws[t][i] = ws[t][b];
        }
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            s.x[u][i].lo = load_global_u4(a[u] + lo);
            s.x[u][i].hi = load_global_u4(a[u] + hi);
            s.as[u][i] = as[u][b];
        }
    }
}
template <bool WIDE, int MT, int NT, int U>
__device__ __forceinline__ void multiply_step(Fp8Step<MT, NT, U> &s, int step, int K, int q, f32x4 (&acc)[NT][MT]) {
    const int blocks = (K + 127) / 128;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int b = step * U + i;
        if (b < blocks) {
            const int pieces = (K - 128 * b) / 16;
            if (pieces < 8) {
#pragma unroll
                for (int t = 0; t < NT; ++t) cut_frag(s.w[t][i], q, pieces);
#pragma unroll
                for (int u = 0; u < MT; ++u) cut_frag(s.x[u][i], q, pieces);
            }
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const auto x = operand<WIDE>(s.x[u][i]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][u] = fma4(mfma_fp8(operand<WIDE>(s.w[t][i]), x), s.ws[t][i] * s.as[u][i], acc[t][u]);
            }
        }
    }
}
template <bool WIDE, int MT, int NT, int U, int WK>
__device__ __forceinline__ void multiply_rows(int wave, int K, int q, const uint8_t *const (&w)[NT],
                                              const float *const (&ws)[NT], const uint8_t *const (&a)[MT],
                                              const float *const (&as)[MT], f32x4 (&acc)[NT][MT]) {
    const int steps = ((K + 127) / 128 + U - 1) / U;
    if (wave >= steps) return;
    Fp8Step<MT, NT, U> now, next;
    load_step(now, wave, K, q, w, ws, a, as);
    for (int s = wave; s < steps; s += WK) {
        const bool more = s + WK < steps;
        if (more) load_step(next, s + WK, K, q, w, ws, a, as);
        multiply_step<WIDE>(now, s, K, q, acc);
        if (more) now = next;
    }
}

// ---------------------------------------------------------------- a few rows, quantised here
// Up to 16 rows of unquantised activations that fit LDS whole: the workgroup quantises them
// itself, while its first weights are on their way, which saves a launch.  Row m: its codes at xs + m * few_row(K), then its scales.
constexpr int kFewRows = 4;  // tokens of the experts
__host__ __device__ inline int few_row(int K) {
    const int blocks = (K + 127) / 128;
    return blocks * 128 + (blocks + 3) / 4 * 16 + 16;  // (the last 16: other banks for the next row)
}
template <int TYPE>
__device__ __forceinline__ void quantise_few(uint8_t *xs, const uint8_t *x, size_t stride, int rows, int K, int tid,
                                             int threads) {
    const int per = (K + 127) / 128 * 16;  // lanes of a row, 16 a block
    for (int u = tid; u < rows * per; u += threads) {  // threads % 16 == 0: the lanes of a block stay together
        const int m = u / per, c = u - m * per;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (8 * c < K) load8<TYPE>(x + (size_t)m * stride + (size_t)c * (TYPE == MOE_FP32 ? 32 : 16), v);
        const float s = fp8_scale(row16_max(top_of(v)), false);
        uint8_t *row = xs + m * few_row(K);
        *reinterpret_cast<uint2 *>(row + 8 * c) = fp8_codes8<false>(v, s);  // zeros behind K
        if ((c & 15) == 0) *reinterpret_cast<float *>(row + per * 8 + (c >> 4) * 4) = s;
    }
}
// acc[t] += rows of W x the rows in LDS over the wave's steps; xs: this lane's row.
// ready(): called once, when the wave's first weights are on their way.
template <bool WIDE, int NT, int U, int WK, class Ready>
__device__ __forceinline__ void multiply_few(int wave, int K, int q, const uint8_t *const (&w)[NT],
                                             const float *const (&ws)[NT], const uint8_t *xs, f32x4 (&acc)[NT],
                                             Ready ready) {
    const int blocks = (K + 127) / 128, steps = (blocks + U - 1) / U;
    struct Weights {
        Fp8Frag w[NT][U];
        float s[NT][U];
    } now, next;
    auto load = [&](Weights &d, int step) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int b = min(step * U + i, blocks - 1), last = min(8, (K - 128 * b) / 16) - 1;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                d.w[t][i].lo = load_global_u4(w[t] + 128 * b + 16 * min(q, last));
                d.w[t][i].hi = load_global_u4(w[t] + 128 * b + 16 * min(q + 4, last));
                d.s[t][i] = ws[t][b];
            }
        }
    };
    if (wave < steps) load(now, wave);
    ready();
    for (int s = wave; s < steps; s += WK) {
        const bool more = s + WK < steps;
        if (more) load(next, s + WK);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int b = s * U + i;
            if (b >= blocks) break;
            const int pieces = (K - 128 * b) / 16;
            if (pieces < 8)
#pragma unroll
                for (int t = 0; t < NT; ++t) cut_frag(now.w[t][i], q, pieces);
            const Fp8Frag x{*reinterpret_cast<const uint4 *>(xs + 128 * b + 16 * q),
                            *reinterpret_cast<const uint4 *>(xs + 128 * b + 16 * q + 64)};
            const float xs_scale = *reinterpret_cast<const float *>(xs + blocks * 128 + 4 * b);
            const auto xo = operand<WIDE>(x);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[t] = fma4(mfma_fp8(operand<WIDE>(now.w[t][i]), xo), now.s[t][i] * xs_scale, acc[t]);
        }
        if (more) now = next;
    }
}

// The waves' sums of tile i -> this wave's registers, in wave order.
template <int WK, int TILES>
__device__ __forceinline__ f32x4 joined(const f32x4 (*part)[TILES][64], int i, int lane) {
    f32x4 v = part[0][i][lane];
#pragma unroll
    for (int k = 1; k < WK; ++k) v += part[k][i][lane];
    return v;
}

}  // namespace moe
