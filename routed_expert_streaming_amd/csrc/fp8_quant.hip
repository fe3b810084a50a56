// Rows of bf16, fp16 or fp32 values -> E4M3 codes with an fp32 scale for each block of
// 1 x 128 (activations) or 128 x 128 (weights) values.
#include "common.h"
#include "fp8_quant.h"

namespace {

constexpr int kThreads = 256;

// 1 x 128: 16 neighbouring lanes hold a block, eight values each, so that its maximum
// is four lane exchanges away.  Lanes of a last block that end behind the row have
// nothing.  units: lanes of all rows; per: of one (16 a block).  2048 x 6144 bf16: 10 us,
// 3.8 TB/s (a large copy 4.7); 6 of them are instructions: about ten for a value's exact
// rounding.  Stores past the caches took 4% less alone, but the product reads the codes next.
template <int TYPE, bool POW2>
__global__ __launch_bounds__(kThreads) void fp8_quant_rows_kernel(const uint8_t *__restrict__ x, size_t x_stride,
                                                                  uint32_t units, uint32_t per, int K,
                                                                  uint8_t *__restrict__ codes, size_t codes_stride,
                                                                  uint8_t *__restrict__ scales,
                                                                  size_t scales_stride) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;  // per % 16 == 0: the lanes of a block leave together
    const uint32_t row = u / per, c = u - row * per;
    const bool in = 8 * (int)c < K;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) moe::load8<TYPE>(x + row * x_stride + (size_t)c * (TYPE == MOE_FP32 ? 32 : 16), v);
    const float s = moe::fp8_scale(moe::row16_max(moe::top_of(v)), POW2);
    if (in) *reinterpret_cast<uint2 *>(codes + row * codes_stride + 8 * (size_t)c) = moe::fp8_codes8<POW2>(v, s);
    if ((c & 15) == 0) *reinterpret_cast<float *>(scales + row * scales_stride + 4 * (size_t)(c >> 4)) = s;
}

// 128 x 128: one workgroup a block, held in registers between the maximum and the codes;
// thread t has columns 8 * (t % 16) .. + 7 of rows t / 16, + 16, ...  1533 x 2080 fp32 (204
// blocks on 256 CUs): 5.0 us, 3.2 TB/s.
template <int TYPE, bool POW2>
__global__ __launch_bounds__(kThreads) void fp8_quant_blocks_kernel(const uint8_t *__restrict__ x, size_t x_stride,
                                                                    int rows, int K, uint8_t *__restrict__ codes,
                                                                    size_t codes_stride,
                                                                    uint8_t *__restrict__ scales,
                                                                    size_t scales_stride) {
    __shared__ uint32_t tops[kThreads / 64];
    const int r0 = blockIdx.y * 128 + threadIdx.x / 16, c = blockIdx.x * 128 + 8 * (threadIdx.x & 15);
    float v[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (r < rows && c < K)
            moe::load8<TYPE>(x + (size_t)r * x_stride + (size_t)c * (TYPE == MOE_FP32 ? 4 : 2), v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, moe::top_of(v[i]));
    top = moe::row16_max(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) top = max(top, tops[i]);
    const float s = moe::fp8_scale(top, POW2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < rows && c < K)
            *reinterpret_cast<uint2 *>(codes + (size_t)r * codes_stride + c) = moe::fp8_codes8<POW2>(v[i], s);
    }
    if (threadIdx.x == 0)
        *reinterpret_cast<float *>(scales + (size_t)blockIdx.y * scales_stride + 4 * (size_t)blockIdx.x) = s;
}

template <int TYPE, bool POW2>
int launch_rows(const uint8_t *x, size_t x_stride, int rows, int K, uint8_t *codes, size_t codes_stride,
                uint8_t *scales, size_t scales_stride, hipStream_t s) {
    // at most 2^30 lanes a launch: 32-bit unit numbers whatever the matrix
    const int per = 16 * moe::fp8_blocks(K), chunk = (1 << 30) / per;
    for (int r0 = 0; r0 < rows;) {
        const int n = rows - r0 < chunk ? rows - r0 : chunk;
        const uint32_t units = (uint32_t)n * (uint32_t)per;
        hipLaunchKernelGGL((fp8_quant_rows_kernel<TYPE, POW2>), dim3((units + kThreads - 1) / kThreads),
                           dim3(kThreads), 0, s, x + (size_t)r0 * x_stride, x_stride, units, (uint32_t)per, K,
                           codes + (size_t)r0 * codes_stride, codes_stride, scales + (size_t)r0 * scales_stride,
                           scales_stride);
        MOE_LAUNCH_CHECK("fp8_quant_rows_kernel");
        r0 += n;
    }
    return MOE_OK;
}

template <int TYPE, bool POW2>
int launch_blocks(const uint8_t *x, size_t x_stride, int rows, int K, uint8_t *codes, size_t codes_stride,
                  uint8_t *scales, size_t scales_stride, hipStream_t s) {
    // at most 2^22 workgroups a launch
    const int all = moe::fp8_blocks(rows), most = (1 << 22) / moe::fp8_blocks(K) < 32768
                                                      ? (1 << 22) / moe::fp8_blocks(K)
                                                      : 32768;
    for (int b0 = 0; b0 < all; b0 += most) {
        const int r0 = b0 * 128, n = all - b0 < most ? all - b0 : most;
        hipLaunchKernelGGL((fp8_quant_blocks_kernel<TYPE, POW2>), dim3(moe::fp8_blocks(K), n), dim3(kThreads), 0, s,
                           x + (size_t)r0 * x_stride, x_stride, rows - r0, K, codes + (size_t)r0 * codes_stride,
                           codes_stride, scales + (size_t)b0 * scales_stride, scales_stride);
        MOE_LAUNCH_CHECK("fp8_quant_blocks_kernel");
    }
    return MOE_OK;
}

template <int TYPE>
int launch(bool blocks, bool pow2, const uint8_t *x, size_t x_stride, int rows, int K, uint8_t *codes,
           size_t codes_stride, uint8_t *scales, size_t scales_stride, hipStream_t s) {
    if (blocks)
        return pow2 ? launch_blocks<TYPE, true>(x, x_stride, rows, K, codes, codes_stride, scales, scales_stride, s)
                    : launch_blocks<TYPE, false>(x, x_stride, rows, K, codes, codes_stride, scales, scales_stride, s);
    return pow2 ? launch_rows<TYPE, true>(x, x_stride, rows, K, codes, codes_stride, scales, scales_stride, s)
                : launch_rows<TYPE, false>(x, x_stride, rows, K, codes, codes_stride, scales, scales_stride, s);
}

int quant(const void *x, int x_type, size_t x_stride, int rows, int K, bool blocks, bool pow2, uint8_t *codes,
          size_t codes_stride, float *scales, size_t scales_stride, hipStream_t s) {
    const uint8_t *xp = (const uint8_t *)x;
    uint8_t *sp = (uint8_t *)scales;
    if (x_type == MOE_BF16)
        return launch<MOE_BF16>(blocks, pow2, xp, x_stride, rows, K, codes, codes_stride, sp, scales_stride, s);
    if (x_type == MOE_FP16)
        return launch<MOE_FP16>(blocks, pow2, xp, x_stride, rows, K, codes, codes_stride, sp, scales_stride, s);
    return launch<MOE_FP32>(blocks, pow2, xp, x_stride, rows, K, codes, codes_stride, sp, scales_stride, s);
}

}  // namespace

namespace moe {

int fp8_quant_rows(const void *x, int x_type, size_t x_stride, int rows, int K, bool pow2, uint8_t *codes,
                   size_t codes_stride, float *scales, size_t scales_stride, hipStream_t s) {
    return quant(x, x_type, x_stride, rows, K, false, pow2, codes, codes_stride, scales, scales_stride, s);
}

}  // namespace moe

extern "C" int moe_fp8_quant(const void *x, int x_type, int64_t x_stride, int rows, int K, int block_rows,
                             int scale_rule, uint8_t *codes, int64_t codes_stride, float *scales,
                             int64_t scales_stride, void *stream) {
    constexpr int kMaxK = 1 << 28;
    if (rows < 0) return moe::fail(MOE_E_ARG, "fp8_quant: rows=%d < 0", rows);
    if (x_type != MOE_BF16 && x_type != MOE_FP16 && x_type != MOE_FP32)
        return moe::fail(MOE_E_ARG, "fp8_quant: x_type=%d", x_type);
    if (block_rows != 1 && block_rows != 128) return moe::fail(MOE_E_ARG, "fp8_quant: block_rows=%d", block_rows);
    if (scale_rule != MOE_FP8_SCALE_AMAX && scale_rule != MOE_FP8_SCALE_POW2)
        return moe::fail(MOE_E_ARG, "fp8_quant: scale_rule=%d", scale_rule);
    if (K <= 0 || K % 16 || K > kMaxK)
        return moe::fail(MOE_E_SHAPE, "fp8_quant: K=%d must be a positive multiple of 16 up to %d", K, kMaxK);
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return moe::fail(MOE_E_ARG, "fp8_quant: NULL pointer");
    const int64_t size = x_type == MOE_FP32 ? 4 : 2;
    const bool blocks = block_rows == 128;
    const int scale_rows = blocks ? moe::fp8_blocks(rows) : rows;
    if (rows > 1 && (x_stride < size * K || codes_stride < K))
        return moe::fail(MOE_E_SHAPE, "fp8_quant: rows %lld and %lld bytes apart, %lld and %d long",
                         (long long)x_stride, (long long)codes_stride, (long long)(size * K), K);
    if (scale_rows > 1 && scales_stride < 4 * (int64_t)moe::fp8_blocks(K))
        return moe::fail(MOE_E_SHAPE, "fp8_quant: scale rows %lld bytes apart, %d long", (long long)scales_stride,
                         4 * moe::fp8_blocks(K));
    if (((uintptr_t)x | (uintptr_t)codes) % 16 || (rows > 1 && (x_stride % 16 || codes_stride % 16)))
        return moe::fail(MOE_E_ARG, "fp8_quant: pointers and strides of x and codes must be multiples of 16 bytes");
    if ((uintptr_t)scales % 4 || (scale_rows > 1 && scales_stride % 4))
        return moe::fail(MOE_E_ARG, "fp8_quant: scales or their stride is not a multiple of 4 bytes");
    return quant(x, x_type, rows > 1 ? (size_t)x_stride : 0, rows, K, blocks, scale_rule == MOE_FP8_SCALE_POW2, codes,
                 rows > 1 ? (size_t)codes_stride : 0, scales, scale_rows > 1 ? (size_t)scales_stride : 0,
                 (hipStream_t)stream);
}
