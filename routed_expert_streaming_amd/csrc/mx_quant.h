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

// Eight values of this lane -> four code bytes (byte b: value 2b in bits 0-3, 2b+1
// in bits 4-7); v is the block's E8M0 byte.
__device__ __forceinline__ uint32_t mx_codes8(const float (&x)[8], uint32_t v) {
    if (v == 255u) return 0u;
    // The convert divides by the scale's exponent field.  Below 2^-63 both sides
    // are moved up by 2^64 first (exact), so that neither is a subnormal there.
    const bool low = v < 64u;
    const float up = low ? 0x1p64f : 1.0f;
    const float scale = __uint_as_float((v + (low ? 64u : 0u)) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0] * up, x[1] * up, scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2] * up, x[3] * up, scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4] * up, x[5] * up, scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6] * up, x[7] * up, scale, 3);
    return c;
}

// Bits of the largest magnitude of this lane's eight values (a NaN's bits are
// above every number's).
__device__ __forceinline__ uint32_t mx_top8(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    return top;
}

// 2^(v-127) (v = 255: NaN) and the value of an E2M1 code (bits 0-3), both exact in fp32.
__device__ __forceinline__ float mx_block_scale(uint32_t v) {
    return v == 255u ? __builtin_nanf("") : __uint_as_float(v ? v << 23 : 0x00400000u);
}
__device__ __forceinline__ float mx_e2m1(uint32_t q) {
    const uint32_t m = q & 7u;  // 2 * magnitude of codes 0..7, four bits each: 0 1 2 3 4 6 8 12
    const float a = 0.5f * (float)(0xC8643210u >> (4 * m) & 15u);
    return q & 8u ? -a : a;
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
