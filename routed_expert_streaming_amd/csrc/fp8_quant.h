// E4M3 quantisation of blocks of 128 columns, shared by the row quantiser and the
// products that take unquantised activations.
//
// A block (1 x 128 or 128 x 128 values) gets one fp32 scale s and E4M3 codes:
//   s = fp32(|x|max / 448), at least 2^-126      (the largest magnitude lands on 448)
//     or the smallest power of two >= |x|max / 448, at least 2^-126;
//     1 for a block of zeros, NaN (and codes 0) for one with an infinity or a NaN;
//   code = x / s to the nearest E4M3 value, ties to the even code.
// The code is the rounding of the true quotient: the fp32 quotient is made odd where it
// is not exact (round to odd), after which the convert's rounding to 4 bits is the only
// one.  Rounding the fp32 quotient instead would change about one code in 2^20.
#pragma once
#include "common.h"

namespace moe {

constexpr float kFp8Top = 448.0f;
constexpr int kFp8Block = 128;

// Scale of a block from the bits of its largest magnitude.
__device__ __forceinline__ float fp8_scale(uint32_t top, bool pow2) {
    if (top == 0u) return 1.0f;
    if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if (!pow2) return fmaxf(__uint_as_float(top) / kFp8Top, 0x1p-126f);
    // 448 = 1.75 * 2^8: 2^(e-8) while the significand is at most 1.75, else the next
    const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(e > 1 ? e : 1) << 23);
}

// Four values -> four codes.  inv: 1 / s rounded; s a finite scale.
// A power of two divides exactly (what the product flushes or rounds is below half of
// the smallest code).
template <bool POW2>
__device__ __forceinline__ uint32_t fp8_codes4(const float (&x)[4], float s, float inv) {
    float q[4];
    if constexpr (POW2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = x[j] * inv;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = fabsf(x[j]);
            const float q0 = a * inv;
            const float q1 = fmaf(fmaf(-q0, s, a), inv, q0);  // within an ulp of a / s
            const float rest = fmaf(-q1, s, a);               // exact: its sign is the quotient's side
            uint32_t b = __float_as_uint(q1);
            b = (b - (rest < 0.0f ? 1u : 0u)) | (rest != 0.0f ? 1u : 0u);
            q[j] = __uint_as_float(b | (__float_as_uint(x[j]) & 0x80000000u));
        }
    }
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], c, true);
}

// 4 W values of this lane -> as many codes, by the block's scale (NaN: codes 0).
template <bool POW2, int W>
__device__ __forceinline__ void fp8_codes(const float (&x)[4 * W], float s, uint32_t (&c)[W]) {
    float t = s, up = 1.0f;
    if (!POW2 && s < 0x1p-60f) {  // keep the quotient's remainder above fp32's smallest number
        up = 0x1p64f;
        t = s * up;
    }
    const float inv = 1.0f / t;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float a[4] = {x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
        if (!POW2 && up != 1.0f)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] *= up;
        c[i] = s == s ? fp8_codes4<POW2>(a, t, inv) : 0u;
    }
}
template <bool POW2>
__device__ __forceinline__ uint2 fp8_codes8(const float (&x)[8], float s) {
    uint32_t c[2];
    fp8_codes<POW2, 2>(x, s, c);
    return make_uint2(c[0], c[1]);
}

// Largest of a value over the 16 lanes of a row of lanes (16i .. 16i + 15).
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // row_mirror
    return v;
}

// Eight consecutive values of TYPE at p (16-byte aligned; 32 bytes of fp32) in fp32.
template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8]) {
    const uint4 a = load_global_u4(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (TYPE == MOE_FP32) {
        const uint4 b = load_global_u4(p + 16);
        const uint32_t z[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]), v[4 + j] = __uint_as_float(z[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = TYPE == MOE_BF16 ? bf16_bits_to_f32(w[j] & 0xFFFFu) : fp16_bits_to_f32(w[j] & 0xFFFFu);
            v[2 * j + 1] = TYPE == MOE_BF16 ? __uint_as_float(w[j] & 0xFFFF0000u) : fp16_bits_to_f32(w[j] >> 16);
        }
    }
}

template <int N>
__device__ __forceinline__ uint32_t top_of(const float (&v)[N]) {
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) t = max(t, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return t;
}

inline int fp8_blocks(int n) { return n / kFp8Block + (n % kFp8Block ? 1 : 0); }
// bytes between the scale rows of quantised activations that the library lays out
__host__ __device__ inline size_t fp8_scale_row(int K) { return ((size_t)(K / kFp8Block + (K % kFp8Block ? 1 : 0)) * 4 + 15) / 16 * 16; }

// rows of TYPE values -> codes and scales of 1 x 128 blocks (checked arguments)
int fp8_quant_rows(const void *x, int x_type, size_t x_stride, int rows, int K, bool pow2, uint8_t *codes,
                   size_t codes_stride, float *scales, size_t scales_stride, hipStream_t s);

}  // namespace moe
