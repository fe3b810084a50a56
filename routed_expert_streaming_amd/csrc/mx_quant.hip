// Rows of bf16, fp16 or fp32 values -> MXFP4 rows (K/2 code bytes, K/32 scale
// bytes, zero padding to 16), the layout of the MXFP4 expert slabs: weights of a
// checkpoint into slabs, activations on their way into moe_mx_matmul.
//
// Bound by memory: 2 or 4 bytes read and 17/32 byte written per value (2 more
// when the values the codes stand for are asked for), about 40 VALU instructions
// per lane of eight values.  A lane takes eight neighbouring values (16 or 32
// bytes), so a wave reads and writes whole lines and a block's maximum is two
// quad permutes away, with no LDS.
#include "common.h"
#include "mx_quant.h"
#include "dequant.h"

namespace {

constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t *p, float (&x)[8]) {
    if constexpr (TYPE == MOE_FP32) {
        const uint4 a = load_global_u4(p), b = load_global_u4(p + 16);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
    } else {
        const uint4 a = load_global_u4(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h = j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu;
            x[j] = TYPE == MOE_BF16 ? bf16_bits_to_f32(h) : fp16_bits_to_f32(h);
        }
    }
}

// One lane per eight values, numbered along the rows (units of a row: K / 8).
template <int TYPE>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(const uint8_t *__restrict__ x, size_t x_stride,
                                                            uint32_t units, int K, bool fit,
                                                            uint8_t *__restrict__ out, size_t out_stride,
                                                            uint16_t *__restrict__ values) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;  // K % 32 == 0: the four lanes of a block leave together
    const uint32_t per = (uint32_t)K / 8, row = u / per, c = u - row * per;
    float v[8];
    load8<TYPE>(x + row * x_stride + (size_t)c * (TYPE == MOE_FP32 ? 32 : 16), v);
    const uint32_t s = moe::mx_scale_byte(moe::quad_max(moe::mx_top8(v)), fit);
    const uint32_t codes = moe::mx_codes8(v, s);
    uint8_t *orow = out + row * out_stride;
    *reinterpret_cast<uint32_t *>(orow + 4 * (size_t)c) = codes;
    if ((c & 3) == 0) moe::mx_store_scale(orow, K, (int)(c >> 2), s);
    if (values) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // E2M1 * 2^(s-127): two significant bits, so bf16 holds it exactly up to
            // 6 * 2^125 (beyond: infinity)
            const uint32_t q = codes >> (8 * j);
            const float f = moe::mx_block_scale(s);
            w[j] = f32_to_bf16_bits(moe::mx_e2m1(q) * f) | f32_to_bf16_bits(moe::mx_e2m1(q >> 4) * f) << 16;
        }
        *reinterpret_cast<uint4 *>(values + (size_t)row * K + 8 * (size_t)c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
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
        const dim3 grid((units + kThreads - 1) / kThreads), block(kThreads);
        hipStream_t s = (hipStream_t)stream;
        if (x_type == MOE_BF16)
            hipLaunchKernelGGL(mx_quant_kernel<MOE_BF16>, grid, block, 0, s, xp, (size_t)x_stride, units, K, fit, op,
                               (size_t)out_stride, vp);
        else if (x_type == MOE_FP16)
            hipLaunchKernelGGL(mx_quant_kernel<MOE_FP16>, grid, block, 0, s, xp, (size_t)x_stride, units, K, fit, op,
                               (size_t)out_stride, vp);
        else
            hipLaunchKernelGGL(mx_quant_kernel<MOE_FP32>, grid, block, 0, s, xp, (size_t)x_stride, units, K, fit, op,
                               (size_t)out_stride, vp);
        MOE_LAUNCH_CHECK("mx_quant_kernel");
        if (rows - r0 <= chunk) break;  // r0 + chunk may pass INT_MAX
    }
    return MOE_OK;
}
