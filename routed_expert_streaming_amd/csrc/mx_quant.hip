// Rows of bf16, fp16 or fp32 values -> MXFP4 rows (K/2 code bytes, K/32 scale
// bytes, zero padding to 16), the layout of the MXFP4 expert slabs: weights of a
// checkpoint into slabs, activations on their way into moe_mx_matmul.
//
// Bound by memory: 2 or 4 bytes read and 17/32 byte written per value, 2 more when
// the values the codes stand for are asked for (2048 x 6144 bf16 with values: 57 MB
// in 9.1 us, 6.2 TB/s from and to the caches).  A lane takes eight neighbouring
// values (16 or 32 bytes), so a wave reads and writes whole lines and a block's
// maximum is two quad permutes away, with no LDS; gfx950's scaled converts do the
// rounding.  With every store into the caches this took 9.6 us, rounding in plain
// arithmetic 11.5, two or four units a lane 9.6 and 9.3.
#include "common.h"
#include "mx_quant.h"
#include "dequant.h"

namespace {

constexpr int kThreads = 256;

// Whether the values are written: not, or into the caches, or past them (non-temporal
// stores; 2048 x 6144 9.1 us against 9.6, 1533 x 2080 fp32 4.6 against 5.0), from an
// XCD's L2 on.
enum { kNoValues, kValues, kStreamValues };
constexpr int64_t kStreamFrom = 4 << 20;

// One lane per eight values, numbered along the rows (units of a row: K / 8).
template <int TYPE, int VALUES>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(const uint8_t *__restrict__ x, size_t x_stride,
                                                            uint32_t units, uint32_t per, bool fit,
                                                            uint8_t *__restrict__ out, size_t out_stride,
                                                            uint16_t *__restrict__ values) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;  // K % 32 == 0: the four lanes of a block leave together
    const uint32_t row = u / per, c = u - row * per;
    const uint8_t *src = x + row * x_stride + (size_t)c * (TYPE == MOE_FP32 ? 32 : 16);
    uint32_t s, codes;
    if constexpr (TYPE == MOE_FP32) {
        const uint4 a = load_global_u4(src), b = load_global_u4(src + 16);
        const float v[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                            __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
        s = moe::mx_scale_byte(moe::quad_max(moe::mx_top8(v)), fit);
        codes = moe::mx_codes8(v, s);
    } else {
        const uint4 a = load_global_u4(src);
        const uint32_t top = moe::quad_max(moe::mx_top8_half(a));
        if constexpr (TYPE == MOE_BF16) {
            s = moe::mx_scale_byte(top << 16, fit);
            codes = moe::mx_codes8_bf16(a, s);
        } else {
            s = moe::mx_scale_byte(__float_as_uint(fp16_bits_to_f32(top)), fit);
            codes = moe::mx_codes8_f16(a, s);
        }
    }
    uint8_t *orow = out + row * out_stride;
    *reinterpret_cast<uint32_t *>(orow + 4 * (size_t)c) = codes;
    if ((c & 3) == 0) moe::mx_store_scale(orow, 8 * (int)per, (int)(c >> 2), s);
    if constexpr (VALUES != kNoValues) {
        const uint4 v = moe::mx_values8(codes, s);
        moe_u32x4 *to = reinterpret_cast<moe_u32x4 *>(values + 8 * (size_t)u);
        if constexpr (VALUES == kStreamValues)
            __builtin_nontemporal_store(moe_u32x4{v.x, v.y, v.z, v.w}, to);
        else
            *to = moe_u32x4{v.x, v.y, v.z, v.w};
    }
}

template <int TYPE>
void launch(const uint8_t *x, size_t x_stride, uint32_t units, uint32_t per, bool fit, uint8_t *out, size_t out_stride,
            uint16_t *values, hipStream_t s) {
    const dim3 grid((units + kThreads - 1) / kThreads), block(kThreads);
    auto *kernel = !values                                    ? mx_quant_kernel<TYPE, kNoValues>
                   : (int64_t)units * 16 < kStreamFrom ? mx_quant_kernel<TYPE, kValues>
                                                       : mx_quant_kernel<TYPE, kStreamValues>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, x, x_stride, units, per, fit, out, out_stride, values);
}

}  // namespace

extern "C" size_t moe_mx_row_bytes(int K) { return K > 0 && K % 32 == 0 ? moe::mx_row_bytes(K) : 0; }

extern "C" int moe_mx_quant(const void *x, int x_type, int64_t x_stride, int rows, int K, int scale_rule,
                            uint8_t *out, int64_t out_stride, uint16_t *values, void *stream) {
    if (rows < 0) return moe::fail(MOE_E_ARG, "mx_quant: rows=%d < 0", rows);
    if (x_type != MOE_BF16 && x_type != MOE_FP16 && x_type != MOE_FP32)
        return moe::fail(MOE_E_ARG, "mx_quant: x_type=%d", x_type);
    if (scale_rule != MOE_MX_SCALE_FLOOR && scale_rule != MOE_MX_SCALE_FIT)
        return moe::fail(MOE_E_ARG, "mx_quant: scale_rule=%d", scale_rule);
    if (K <= 0 || K % 32) return moe::fail(MOE_E_SHAPE, "mx_quant: K=%d must be a positive multiple of 32", K);
    if (rows == 0) return MOE_OK;
    if (!x || !out) return moe::fail(MOE_E_ARG, "mx_quant: NULL pointer");
    const int64_t size = x_type == MOE_FP32 ? 4 : 2, need = (int64_t)moe::mx_row_bytes(K);
    if (rows > 1 && (x_stride < size * K || out_stride < need))
        return moe::fail(MOE_E_SHAPE, "mx_quant: rows %lld and %lld bytes apart, %lld and %lld long",
                         (long long)x_stride, (long long)out_stride, (long long)(size * K), (long long)need);
    if (((uintptr_t)x | (uintptr_t)out | (uintptr_t)values) % 16 || (rows > 1 && (x_stride % 16 || out_stride % 16)))
        return moe::fail(MOE_E_ARG, "mx_quant: pointers and strides must be multiples of 16 bytes");
    const bool fit = scale_rule == MOE_MX_SCALE_FIT;
    // at most 2^30 lanes a launch: 32-bit unit numbers whatever the matrix
    const int per = K / 8, chunk = (1 << 30) / per;
    for (int r0 = 0; r0 < rows; r0 += chunk) {
        const int n = rows - r0 < chunk ? rows - r0 : chunk;
        const uint32_t units = (uint32_t)n * (uint32_t)per;
        const uint8_t *xp = (const uint8_t *)x + (size_t)r0 * x_stride;
        uint8_t *op = out + (size_t)r0 * out_stride;
        uint16_t *vp = values ? values + (size_t)r0 * K : nullptr;
        hipStream_t s = (hipStream_t)stream;
        if (x_type == MOE_BF16)
            launch<MOE_BF16>(xp, x_stride, units, per, fit, op, out_stride, vp, s);
        else if (x_type == MOE_FP16)
            launch<MOE_FP16>(xp, x_stride, units, per, fit, op, out_stride, vp, s);
        else
            launch<MOE_FP32>(xp, x_stride, units, per, fit, op, out_stride, vp, s);
        MOE_LAUNCH_CHECK("mx_quant_kernel");
        if (rows - r0 <= chunk) break;  // r0 + chunk may pass INT_MAX
    }
    return MOE_OK;
}
