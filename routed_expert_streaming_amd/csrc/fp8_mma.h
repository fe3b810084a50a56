// E4M3 products on gfx950's matrix cores with fp32 scales per block of 128 columns:
// what the dense product and the experts' kernels share.
//
// v_mfma_f32_16x16x128_f8f6f4 sums 128 products, one block's: lane 16q + r holds 32 of
// the 128 columns of row r of both operands (which 32 does not matter as long as both
// agree; here the 16-byte pieces q and q + 4 of the block's eight, so that four lanes
// read 64 neighbouring bytes).  Each product starts from zero and its result enters the
// fp32 sums times its two scales, a fused multiply-add per output: the scales are not
// powers of two, which the instruction's own scaling would need.  W is the first
// operand: a lane then holds outputs n = 4q .. 4q + 3 of one m = r, so that a row's
// scale is one value a lane.
//
// What the instruction keeps (measured, every E4M3 form of it alike): of each 8 products
// (8 neighbouring bytes of a lane) only the bits down to 2^-13 of the largest one's
// exponent, the rest cut off; the sums of eights are added in fp32.  Random data comes
// out 2e-5 off, far below bf16's rounding.  Where y is fp32 the codes are therefore
// converted to bf16 (exact) and multiplied by v_mfma_f32_16x16x32_bf16, whose sums of
// such products are exact but for fp32's rounding, at half the rate.
#pragma once
#include "common.h"
#include "fp8_quant.h"
#include "lds_dma.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Frag {
    uint4 lo, hi;  // pieces q and q + 4 of a block of a row
};

__device__ __forceinline__ f32x4 mfma_fp8(const Fp8Frag &w, const Fp8Frag &a) {
    const i32x8 wv{(int)w.lo.x, (int)w.lo.y, (int)w.lo.z, (int)w.lo.w,
                   (int)w.hi.x, (int)w.hi.y, (int)w.hi.z, (int)w.hi.w};
    const i32x8 av{(int)a.lo.x, (int)a.lo.y, (int)a.lo.z, (int)a.lo.w,
                   (int)a.hi.x, (int)a.hi.y, (int)a.hi.z, (int)a.hi.w};
    // formats 0: E4M3; no scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// 8 codes -> bf16
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(
        bf16x8, make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true))));
}
struct WideFrag {
    bf16x8 v[4];
};
__device__ __forceinline__ WideFrag widen(const Fp8Frag &f) {
    return {{widen8(f.lo.x, f.lo.y), widen8(f.lo.z, f.lo.w), widen8(f.hi.x, f.hi.y), widen8(f.hi.z, f.hi.w)}};
}
__device__ __forceinline__ f32x4 mfma_fp8(const WideFrag &w, const WideFrag &a) {
    f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[s], a.v[s], c, 0, 0, 0);
    return c;
}
// The operand as the products take it.
template <bool WIDE>
__device__ __forceinline__ auto operand(const Fp8Frag &f) {
    if constexpr (WIDE)
        return widen(f);
    else
        return f;
}

__device__ __forceinline__ f32x4 fma4(const f32x4 v, float s, const f32x4 c) {
    return f32x4{fmaf(v[0], s, c[0]), fmaf(v[1], s, c[1]), fmaf(v[2], s, c[2]), fmaf(v[3], s, c[3])};
}

// Pieces past the end of a row are zeros (both operands': 0 x NaN is not 0).
__device__ __forceinline__ void cut_frag(Fp8Frag &f, int q, int pieces) {
    if (q >= pieces) f.lo = make_uint4(0u, 0u, 0u, 0u);
    if (q + 4 >= pieces) f.hi = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// FP8 expert slab: W1 [I,H], W3 [I,H], W2 [H,I] codes, then the scales of their blocks
// of 128 x 128, matrix by matrix, row by row.
struct Fp8Slab {
    const uint8_t *w;
    const float *s;
    int s_row;  // scales of a row of blocks
};
__device__ __forceinline__ Fp8Slab fp8_slab(const uint8_t *slab, int H, int I, int which) {
    const int hb = (H + 127) / 128, ib = (I + 127) / 128;
    const float *s = reinterpret_cast<const float *>(slab + (size_t)3 * H * I) + (size_t)which * ib * hb;
    return {slab + (size_t)which * H * I, s, which == 2 ? ib : hb};
}
inline size_t fp8_slab_bytes(int H, int I) {
    return align_up((size_t)3 * H * I + (size_t)12 * fp8_blocks(H) * fp8_blocks(I), 16);
}

}  // namespace moe
