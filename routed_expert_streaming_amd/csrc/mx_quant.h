// MXFP4 quantisation of one 32-column block, shared by the row quantiser and the
// block norm that writes quantised rows.
//
// A block of 32 values gets one power-of-two scale 2^(v-127) and 32 E2M1 codes
// (magnitudes 0 0.5 1 1.5 2 3 4 6):
//   e  = exponent of the block's largest magnitude, 2^e <= |x|max < 2^(e+1);
//   v  = e - 2 + 127 (floor rule: the largest magnitude lands in [4, 8) and
//        saturates at 6), one more when |x|max > 6 * 2^(e-2) (fit rule: nothing
//        saturates), at least 0;
//   q  = x / 2^(v-127) to the nearest magnitude, ties to the even code.
// All of it is exact but that last rounding: v comes from the exponent bits, and
// dividing by a power of two and the hardware's convert (round to nearest even,
// saturating) are one rounding of the true quotient.  A block that holds an
// infinity or a NaN gets v = 255, MXFP4's NaN, and codes 0; a block of zeros v = 0.
//
// Four neighbouring lanes hold a block, eight values each.
#pragma once
#include "common.h"

namespace moe {

// Largest of a value over the four lanes of a block (lanes 4i .. 4i+3).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
    return v;
}

// E8M0 byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top, bool fit) {
    const uint32_t e = top >> 23;  // biased; 0 for zero and fp32 subnormals (then v = 0)
    if (e == 255u) return 255u;
    const uint32_t v = e + ((fit && (top & 0x7FFFFFu) > 0x400000u) ? 1u : 0u);
    return v > 2u ? v - 2u : 0u;
}

// The scale operand of gfx950's scaled converts: they take its exponent field as an
// E8M0 byte (0 is 2^-127, 255 NaN).
__device__ __forceinline__ float mx_scale_operand(uint32_t v) { return __uint_as_float(v << 23); }

// Eight values of this lane -> four code bytes (byte b: value 2b in bits 0-3, 2b+1
// in bits 4-7); v is the block's E8M0 byte.  x: eight floats, or four words of bf16 or
// fp16 pairs.
__device__ __forceinline__ uint32_t mx_codes8(const float (&x)[8], uint32_t v) {
    const float scale = mx_scale_operand(v);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], scale, 3);
    return v == 255u ? 0u : c;
}
typedef _Float16 moe_f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t mx_codes8_bf16(const uint4 x, uint32_t v) {
    const float scale = mx_scale_operand(v);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(moe_bf16x2, x.x), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(moe_bf16x2, x.y), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(moe_bf16x2, x.z), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(moe_bf16x2, x.w), scale, 3);
    return v == 255u ? 0u : c;
}
__device__ __forceinline__ uint32_t mx_codes8_f16(const uint4 x, uint32_t v) {
    const float scale = mx_scale_operand(v);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(moe_f16x2, x.x), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(moe_f16x2, x.y), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(moe_f16x2, x.z), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(moe_f16x2, x.w), scale, 3);
    return v == 255u ? 0u : c;
}

// Bits of the largest magnitude of this lane's eight values (a NaN's bits are above
// every number's): fp32 values, or the 16-bit pattern of bf16 or fp16 pairs.
__device__ __forceinline__ uint32_t mx_top8(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    return top;
}
__device__ __forceinline__ uint32_t mx_top8_half(const uint4 x) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
    const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(x.x), mag(x.y)),
                                              __builtin_elementwise_max(mag(x.z), mag(x.w)));
    return max((uint32_t)m[0], (uint32_t)m[1]);
}

// Eight codes -> their values in bf16 (two significant bits: exact; infinite beyond
// bf16's range, NaN for v = 255).
__device__ __forceinline__ uint4 mx_values8(uint32_t c, uint32_t v) {
    const float scale = mx_scale_operand(v);
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3)));
}

// Scale byte of block `block` of a row whose codes start at row, by the block's
// first lane; the lane of the last block also zeroes the row's padding.
__device__ __forceinline__ void mx_store_scale(uint8_t *row, int K, int block, uint32_t v) {
    uint8_t *s = row + K / 2;
    s[block] = (uint8_t)v;
    if (block == K / 32 - 1)
        for (int p = block + 1; p < (K / 32 + 15) / 16 * 16; ++p) s[p] = 0;
}

}  // namespace moe
