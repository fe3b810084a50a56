// y[m,n] = sum_k A[m,k] W[n,k] + bias[n] with W in MXFP4 rows and A in bf16 or in
// MXFP4 rows, on gfx950's matrix cores.
//
// A wave owns 16-row tiles of W and of A and walks K in groups of 128 columns.
// Lane l = 16q + r holds block q of the group (columns 32q .. 32q+31: 16 code
// bytes, one scale byte) of row r of a tile, as the rows lie in memory.
//  * A in MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands' codes and
//    E8M0 bytes as they are.
//  * A in bf16: the codes become bf16 (exact: an E2M1 value times a power of two)
//    and v_mfma_f32_16x16x32_bf16 runs four times per group; product s takes
//    columns 32q + 8s .. 32q + 8s + 7 from lane quarter q of both operands, so W
//    stays in the same order (a sum over k does not care which lanes hold it).
// W is the first operand: a lane then holds four consecutive n of one m, which it
// stores together.  Sums are fp32; waves that split K are joined through LDS in
// wave order.
#include "common.h"
#include "dequant.h"

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct MatArgs {
    const uint8_t *a, *w;
    size_t a_stride, w_stride;  // bytes between rows
    int M, N, K;
    const float *bias;
    uint8_t *y;
    size_t y_stride;
    bool y_f32;
};

// 8 consecutive weights (one dword of codes) -> bf16, times 2^(v-127) given as a float
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t c, float scale) {
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
    const uint32_t w2 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
    const uint32_t w3 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
    return __builtin_bit_cast(bf16x8_t, make_uint4(w0, w1, w2, w3));
}

__device__ __forceinline__ float scale_f32(uint32_t v) {
    return v == 255u ? __builtin_nanf("") : __uint_as_float(v ? v << 23 : 0x00400000u);
}

__device__ __forceinline__ f32x4_t mfma_mx(const uint4 w, const uint4 a, f32x4_t c, int ws, int as) {
    const i32x8_t wv{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8_t av{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, c, 4, 4, 0, ws, 0, as);  // 4: FP4 E2M1
}

// Four outputs n .. n+3 of row m (those below N), bias added, rounded once.
__device__ __forceinline__ void store4(const MatArgs &p, int m, int n, const f32x4_t v) {
    if (m >= p.M) return;
    uint8_t *row = p.y + (size_t)m * p.y_stride;
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = v[j] + (p.bias && n + j < p.N ? p.bias[n + j] : 0.0f);
    if (p.y_f32) {
        float *o = (float *)row + n;
        if (n + 3 < p.N && (uintptr_t)o % 16 == 0) {
            *reinterpret_cast<float4 *>(o) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) o[j] = f[j];
        }
    } else {
        uint16_t *o = (uint16_t *)row + n;
        if (n + 3 < p.N && (uintptr_t)o % 8 == 0) {
            *reinterpret_cast<uint2 *>(o) = make_uint2(f32_to_bf16_bits(f[0]) | f32_to_bf16_bits(f[1]) << 16,
                                                       f32_to_bf16_bits(f[2]) | f32_to_bf16_bits(f[3]) << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) o[j] = (uint16_t)f32_to_bf16_bits(f[j]);
        }
    }
}

// Waves WM x WN x WK; a wave owns MT tiles of A rows, NT tiles of W rows and every
// WK-th group of K.  Rows past M or N repeat the last row (their results are not
// stored); columns past K enter as zeros.
template <bool MX, int MT, int NT, int WM, int WN, int WK>
__global__ __launch_bounds__(64 * WM * WN * WK) void mx_matmul_direct_kernel(MatArgs p) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wk = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;
    const int m0 = (blockIdx.y * WM + wm) * 16 * MT, n0 = (blockIdx.x * WN + wn) * 16 * NT;
    const uint8_t *wp[NT], *ap[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) wp[t] = p.w + (size_t)min(n0 + 16 * t + r, p.N - 1) * p.w_stride;
#pragma unroll
    for (int t = 0; t < MT; ++t) ap[t] = p.a + (size_t)min(m0 + 16 * t + r, p.M - 1) * p.a_stride;
    f32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const size_t half = (size_t)p.K / 2;
    const int ng = (p.K + 127) / 128;
    for (int g = wk; g < ng; g += WK) {
        const bool in = 128 * g + 32 * q < p.K;
        const int b = in ? 4 * g + q : 0;  // block of 32 columns
        uint4 w[NT];
        uint32_t ws[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            w[t] = load_global_u4(wp[t] + 16 * (size_t)b);
            ws[t] = load_stream_u8(wp[t] + half + b);
            if (!in) w[t] = make_uint4(0u, 0u, 0u, 0u), ws[t] = 127u;
        }
        if constexpr (MX) {
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                uint4 x = load_global_u4(ap[u] + 16 * (size_t)b);
                uint32_t xs = load_stream_u8(ap[u] + half + b);
                if (!in) x = make_uint4(0u, 0u, 0u, 0u), xs = 127u;
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][u] = mfma_mx(w[t], x, acc[t][u], (int)ws[t], (int)xs);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8_t wv[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t c = s == 0 ? w[t].x : s == 1 ? w[t].y : s == 2 ? w[t].z : w[t].w;
                    wv[t] = codes_bf16(c, scale_f32(ws[t]));
                }
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    uint4 x = load_global_u4(ap[u] + 64 * (size_t)b + 16 * s);
                    if (!in) x = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv[t], __builtin_bit_cast(bf16x8_t, x), acc[t][u], 0, 0, 0);
                }
            }
        }
    }
    if constexpr (WK > 1) {
        // join: wave wk > 0 leaves its sums in LDS, wave 0 of each (wm, wn) adds them in order
        __shared__ f32x4_t part[(WK - 1) * WM * WN][NT * MT][64];
        if (wk > 0)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < MT; ++u) part[wave - WM * WN][t * MT + u][lane] = acc[t][u];
        __syncthreads();
        if (wk > 0) return;
        for (int k = 1; k < WK; ++k)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < MT; ++u) acc[t][u] += part[(k - 1) * WM * WN + wave][t * MT + u][lane];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) store4(p, m0 + 16 * u + r, n0 + 16 * t + 4 * q, acc[t][u]);
}

template <bool MX, int MT, int NT, int WM, int WN, int WK>
void launch_direct(const MatArgs &p, hipStream_t s) {
    const dim3 grid((p.N + 16 * NT * WN - 1) / (16 * NT * WN), (p.M + 16 * MT * WM - 1) / (16 * MT * WM));
    hipLaunchKernelGGL((mx_matmul_direct_kernel<MX, MT, NT, WM, WN, WK>), grid, dim3(64 * WM * WN * WK), 0, s, p);
}

template <bool MX>
void launch(const MatArgs &p, hipStream_t s) {
    if (p.M <= 16)
        launch_direct<MX, 1, 1, 1, 1, 4>(p, s);
    else
        launch_direct<MX, 4, 4, 2, 2, 1>(p, s);
}

}  // namespace

extern "C" size_t moe_mx_matmul_workspace_bytes(int M, int N, int K, int a_type) {
    (void)M, (void)N, (void)K, (void)a_type;
    return 0;
}

extern "C" int moe_mx_matmul(const void *a, int a_type, int64_t a_stride, const uint8_t *w, int64_t w_stride, int M,
                             int N, int K, const float *bias, void *y, int y_type, int64_t y_stride, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0) return moe::fail(MOE_E_ARG, "mx_matmul: M=%d, N=%d", M, N);
    if (a_type != MOE_BF16 && a_type != MOE_MXFP4) return moe::fail(MOE_E_ARG, "mx_matmul: a_type=%d", a_type);
    if (y_type != MOE_BF16 && y_type != MOE_FP32) return moe::fail(MOE_E_ARG, "mx_matmul: y_type=%d", y_type);
    if (K <= 0 || K % 32) return moe::fail(MOE_E_SHAPE, "mx_matmul: K=%d must be a positive multiple of 32", K);
    if (M == 0 || N == 0) return MOE_OK;
    if (!a || !w || !y) return moe::fail(MOE_E_ARG, "mx_matmul: NULL pointer");
    const int64_t row = (int64_t)moe::mx_row_bytes(K), size = y_type == MOE_FP32 ? 4 : 2;
    const int64_t a_row = a_type == MOE_MXFP4 ? row : 2 * (int64_t)K;
    if ((M > 1 && (a_stride < a_row || y_stride < size * N)) || (N > 1 && w_stride < row))
        return moe::fail(MOE_E_SHAPE, "mx_matmul: a row stride (%lld, %lld, %lld) is below the row's bytes",
                         (long long)a_stride, (long long)w_stride, (long long)y_stride);
    if (((uintptr_t)a | (uintptr_t)w) % 16 || (M > 1 && a_stride % 16) || (N > 1 && w_stride % 16))
        return moe::fail(MOE_E_ARG, "mx_matmul: operands' pointers and strides must be multiples of 16 bytes");
    if ((uintptr_t)y % size || (M > 1 && y_stride % size) || (uintptr_t)bias % 4)
        return moe::fail(MOE_E_ARG, "mx_matmul: y, its stride or bias is not aligned to its type");
    const size_t need = moe_mx_matmul_workspace_bytes(M, N, K, a_type);
    if (workspace_bytes < need || (need && !workspace))
        return moe::fail(MOE_E_NOMEM, "mx_matmul: workspace %zu < %zu bytes", workspace_bytes, need);
    const MatArgs p{(const uint8_t *)a, w, (size_t)a_stride, (size_t)w_stride, M, N, K, bias, (uint8_t *)y,
                    (size_t)y_stride, y_type == MOE_FP32};
    if (a_type == MOE_MXFP4)
        launch<true>(p, (hipStream_t)stream);
    else
        launch<false>(p, (hipStream_t)stream);
    MOE_LAUNCH_CHECK("mx_matmul_kernel");
    return MOE_OK;
}
