// y[m,n] = sum over blocks b of 128 columns of a_scale[m,b] w_scale[n/128,b] sum_k A[m,k] W[n,k],
// plus bias[n]: E4M3 rows of activations (or bf16 ones, quantised first) times E4M3
// weights in blocks of 128 x 128.  Sums over k are fp32.
//
// A call, kernels alone: 1 x 4096 x 4096 6 us (one launch, 2.8 TB/s); 32 x 6144 x 6144 3 for
// the activations and 11 (3.4 TB/s of weights); 2048 x 6144 x 6144 10 and 75 to 85 with the
// clock (1.8 to 2.1 PFLOP/s).
#include "common.h"
#include "fp8_mma.h"
#include "fp8_quant.h"
#include "fp8_rows.h"
#include "fp8_tile.h"

namespace {

using moe::f32x4;

constexpr int kMaxRows = 1 << 26;        // M and N
constexpr int kMaxK = 1 << 27;
constexpr int64_t kMaxStride = 1 << 28;
// bytes of a bf16 y from which a tile kernel writes past the caches (2048 x 6144 x 6144: 3.5
// us less, which the caches took to write back at the kernel's end)
constexpr int64_t kStreamFrom = 4 << 20;

struct MatArgs {
    moe::Fp8Act a;
    const uint8_t *w;
    size_t w_stride;
    const uint8_t *ws;
    size_t ws_stride;  // bytes between rows of blocks' scales
    int M, N, K;
    const float *bias;
    uint8_t *y;
    size_t y_stride;
    bool ends;  // the caller's rows of scales, which may end inside 16 bytes
    __device__ __forceinline__ uint8_t *row(int m) const { return y + (size_t)m * y_stride; }
};

// Four outputs n .. n+3 of row m (those below N), bias added, rounded once.  F32: y's type.
template <bool F32>
__device__ __forceinline__ void store4(const MatArgs &p, int m, int n, const f32x4 v) {
    if (m >= p.M) return;
    uint8_t *row = p.y + (size_t)m * p.y_stride;
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = v[j] + (p.bias && n + j < p.N ? p.bias[n + j] : 0.0f);
    if constexpr (F32) {
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
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) o[j] = (uint16_t)pack_bf16(f[j], 0.0f);
        }
    }
}

template <bool WIDE, int MT, int NT, int WK, int U>
__global__ __launch_bounds__(64 * WK) void fp8_matmul_rows_kernel(MatArgs p) {
    __shared__ f32x4 part[WK][NT * MT][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int m0 = blockIdx.y * 16 * MT, n0 = blockIdx.x * 16 * NT;
    const uint8_t *w[NT], *a[MT];
    const float *ws[NT], *as[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = min(n0 + 16 * t, p.N - 1);
        w[t] = p.w + (size_t)min(n + r, p.N - 1) * p.w_stride;
        ws[t] = reinterpret_cast<const float *>(p.ws + (size_t)(n / 128) * p.ws_stride);
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int m = min(m0 + 16 * u + r, p.M - 1);
        a[u] = p.a.codes + (size_t)m * p.a.stride;
        as[u] = reinterpret_cast<const float *>(p.a.scales + (size_t)m * p.a.scale_stride);
    }
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe::multiply_rows<WIDE, MT, NT, U, WK>(wave, p.K, q, w, ws, a, as, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) part[wave][t * MT + u][lane] = acc[t][u];
    __syncthreads();
#pragma unroll
    for (int i0 = 0; i0 < NT * MT; i0 += WK) {
        const int i = i0 + wave;
        if (i >= NT * MT) break;
        store4<WIDE>(p, m0 + 16 * (i % MT) + r, n0 + 16 * (i / MT) + 4 * q,
                     moe::joined<WK, NT * MT>(part, i, lane));
    }
}

template <bool WIDE, int MT, int NT, int WK, int U>
void launch_rows(MatArgs p, hipStream_t s) {
    const int most = 32768 * 16 * MT, all = p.M;  // rows of A a grid holds
    for (int m = 0;; m += most) {
        p.M = min(all - m, most);
        const dim3 grid((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT));
        hipLaunchKernelGGL((fp8_matmul_rows_kernel<WIDE, MT, NT, WK, U>), grid, dim3(64 * WK), 0, s, p);
        if (all - m <= most) return;
        p.a.codes += (size_t)most * p.a.stride;
        p.a.scales += (size_t)most * p.a.scale_stride;
        p.y += (size_t)most * p.y_stride;
    }
}

// ENDS as fp8_tile's.  Kernels of their own: with both ways in one, 32 x 6144 x 6144 took 13.3 us
// instead of 12.5 although only the first was taken.
template <bool WIDE, class T, bool STREAM, bool ENDS>
__global__ __launch_bounds__(64 * T::WAVES) void fp8_matmul_tile_kernel(MatArgs p, int m_tiles, int n_tiles) {
    __shared__ uint4 smem4[T::LDS / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    constexpr int MT = T::MT, NT = T::NT;
    constexpr int SN = 128 % (16 * NT) == 0 ? 1 : NT;  // a wave's columns lie in one block of W's rows, or each tile's do
    // consecutive workgroups go to the 8 XCDs in turn: each XCD takes a run of
    // neighbouring tiles, m fastest, so that its L2 holds the W rows they share
    const int tiles = m_tiles * n_tiles, per = (tiles + 7) / 8;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= tiles) return;
    const int m0 = tile % m_tiles * T::BM, n0 = tile / m_tiles * T::BN;
    const int m_last = min(T::BM, p.M - m0) - 1, n_last = min(T::BN, p.N - n0) - 1;
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = all % T::GROUP;
    const int wm = wave / T::WN, wn = wave % T::WN;
    const float *ws[SN];
#pragma unroll
    for (int i = 0; i < SN; ++i)
        ws[i] = reinterpret_cast<const float *>(
            p.ws + (size_t)(min(n0 + (wn * NT + i) * 16, p.N - 1) / 128) * p.ws_stride);
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe::fp8_tile<T, WIDE, SN, ENDS>(
        smem, p.w + (size_t)n0 * p.w_stride, p.a.codes + (size_t)m0 * p.a.stride,
        p.a.scales + (size_t)m0 * p.a.scale_stride, ws, p.K,
        [&](int row) { return (uint32_t)min(row, n_last) * (uint32_t)p.w_stride; },
        [&](int row) { return (uint32_t)min(row, m_last) * (uint32_t)p.a.stride; },
        [&](int row) { return (uint32_t)min(row, m_last) * (uint32_t)p.a.scale_stride; }, acc);
    if (p.bias)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float c = p.bias[min(n0 + (wn * NT + t) * 16 + 4 * q + j, p.N - 1)];
#pragma unroll
                for (int u = 0; u < MT; ++u) acc[t][u][j] += c;
            }
    if constexpr (WIDE)
        moe::store_tile<T, MT, NT, float>(p, smem, m0, n0, wm, wn, lane, acc, all < T::GROUP);
    else
        moe::store_tile<T, MT, NT, uint16_t, STREAM>(p, smem, m0, n0, wm, wn, lane, acc, all < T::GROUP);
}

template <bool WIDE, class T>
void launch_tile(const MatArgs &p, hipStream_t s) {
    const int m_tiles = (p.M + T::BM - 1) / T::BM, n_tiles = (p.N + T::BN - 1) / T::BN;
    const unsigned grid = (unsigned)(((int64_t)m_tiles * n_tiles + 7) / 8 * 8);
    auto *kernel = p.ends ? fp8_matmul_tile_kernel<WIDE, T, false, true> : fp8_matmul_tile_kernel<WIDE, T, false, false>;
    if constexpr (!WIDE)
        if ((int64_t)p.M * p.N * 2 >= kStreamFrom)
            kernel = p.ends ? fp8_matmul_tile_kernel<WIDE, T, true, true> : fp8_matmul_tile_kernel<WIDE, T, true, false>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * T::WAVES), 0, s, p, m_tiles, n_tiles);
}

// Up to 16 rows of bf16 activations, quantised by each workgroup (16 rows of W) for itself.
template <bool WIDE, int WK, int U>
__global__ __launch_bounds__(64 * WK) void fp8_matmul_few_kernel(MatArgs p) {
    extern __shared__ uint4 few_smem[];
    __shared__ f32x4 part[WK][1][64];
    uint8_t *xs = reinterpret_cast<uint8_t *>(few_smem);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const uint8_t *const w[1] = {p.w + (size_t)min(n0 + r, p.N - 1) * p.w_stride};
    const float *const ws[1] = {reinterpret_cast<const float *>(p.ws + (size_t)(n0 / 128) * p.ws_stride)};
    f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    moe::multiply_few<WIDE, 1, U, WK>(wave, p.K, q, w, ws, xs + min(r, p.M - 1) * moe::few_row(p.K), acc, [&]() {
        moe::quantise_few<MOE_BF16>(xs, p.a.codes, p.a.stride, p.M, p.K, threadIdx.x, 64 * WK);
        __syncthreads();
    });
    part[wave][0][lane] = acc[0];
    __syncthreads();
    if (wave == 0) store4<WIDE>(p, r, n0 + 4 * q, moe::joined<WK, 1>(part, 0, lane));
}

// Which kernel a product takes: the least estimated time, in us.  A round of as many
// workgroups as the CUs hold takes a + b per turn, a turn being KW blocks of 128 columns
// (of the rows kernels, 16 blocks); b grows from `few` workgroups to a full round (they
// share L2 and power).  Measured at K = 1536 .. 6144, kernels alone:
//                      y bf16: a, b few .. full       y fp32
//   rows, 16 x 16      1.6  2.0 (+ 0.04 a row)          the same
//   rows, 16 x 32      2.6  2.4 (+ 0.04 a row)          the same
//   16 x 32,   KW 4    2.5  0.56                        2.5  0.62
//   32 x 32,   KW 4    2.6  0.68                        2.9  0.82
//   32 x 64,   KW 4    3.8  0.85                        3.2  1.20 (two stages)
//   64 x 64,   KW 2    3.7  0.64                        5.0  0.84
//   128 x 64,  KW 2    2.7  1.15                        3.0  1.36
//   128 x 128, KW 1    4.9  0.60 .. 0.63                --  (two groups: 4.0  1.76)
//   128 x 128, 4 waves 4.6  0.87 .. 1.20, two a CU      --
//   256 x 192          7.0  1.27 .. 1.41                --
//   256 x 256          8.0  1.36 .. 1.70                --
// So 32 x 6144 x 6144 takes 10.9 us in 32 x 32 tiles (16.7 where each wave streams W and A
// for itself), 2048 rows 75 us in 256 x 192 ones and 101 in 128 x 128.
enum Kind { FEW, ROWS1, ROWS2, T16, T32, T32W, T64, T128N, T128, T128P, T256N, T256 };

Kind plan(bool wide, int M, int N, int K, bool near) {
    const int nb = moe::fp8_blocks(K);
    auto over = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const struct {
        Kind kind;
        int bm, bn, kw, slots;
        float a, few, full;
    } tiles[2][12] = {{{ROWS1, 16, 16, 16, 2, 1.6f, 2.0f + 0.04f * (float)M, 3.0f + 0.10f * (float)M},
                       {ROWS2, 16, 32, 16, 1, 2.6f, 2.4f + 0.04f * (float)M, 2.4f + 0.04f * (float)M},
                       {T16, 16, 32, 4, 1, 2.5f, 0.56f, 0.60f},
                       {T32, 32, 32, 4, 1, 2.6f, 0.68f, 0.68f},
                       {T32W, 32, 64, 4, 1, 3.8f, 0.85f, 0.87f},
                       {T64, 64, 64, 2, 1, 3.7f, 0.64f, 0.68f},
                       {T128N, 128, 64, 2, 1, 2.7f, 1.10f, 1.18f},
                       {T128, 128, 128, 1, 1, 4.9f, 0.60f, 0.63f},
                       {T128P, 128, 128, 1, 2, 4.6f, 0.80f, 1.20f},
                       {T256N, 256, 192, 1, 1, 7.0f, 1.25f, 1.41f},
                       {T256, 256, 256, 1, 1, 8.0f, 1.30f, 1.70f}},
                      {{ROWS1, 16, 16, 16, 2, 1.6f, 2.0f + 0.04f * (float)M, 3.0f + 0.10f * (float)M},
                       {ROWS2, 16, 32, 16, 1, 2.6f, 2.4f + 0.04f * (float)M, 2.4f + 0.04f * (float)M},
                       {T16, 16, 32, 4, 1, 2.5f, 0.62f, 0.65f},
                       {T32, 32, 32, 4, 1, 2.9f, 0.82f, 0.82f},
                       {T32W, 32, 64, 4, 1, 3.2f, 1.20f, 1.25f},
                       {T64, 64, 64, 2, 1, 5.0f, 0.84f, 0.86f},
                       {T128N, 128, 64, 2, 1, 3.0f, 1.36f, 1.50f},
                       {T128, 128, 128, 2, 1, 4.0f, 1.70f, 2.10f}}};
    Kind best = ROWS1;
    if (!near) return M <= 16 ? ROWS1 : ROWS2;
    float least = 1e30f;
    for (const auto &t : tiles[wide]) {
        if (t.bm == 0 || ((t.kind == ROWS1 || t.kind == ROWS2) && M > 16)) continue;
        const int64_t wgs = over(M, t.bm) * over(N, t.bn), round = 256 * t.slots, rest = wgs % round;
        if (wgs > 4000000) continue;  // below 2^32 threads
        const float turns = (float)over(nb, t.kw), whole = t.a + t.full * turns;
        const float part = rest ? t.a + (t.few + (t.full - t.few) * (float)rest / (float)round) * turns : 0.0f;
        const float us = (float)(wgs / round) * whole + part;
        if (us < least) least = us, best = t.kind;
    }
    return best;
}

// Rows (of A, of its scales, of W) further apart than this take the rows kernels: a tile's
// lane offsets are 32 bits.
constexpr int64_t kTileStride = 8 << 20;

// Which activations the kernel quantises itself: one tile of rows that leave LDS room for two
// workgroups a CU, where every workgroup doing so takes less than a launch for all of them.
// Kernels alone, two launches and one, us: 1 x 4096 x 4096 8.1 and 6.8; 1 x 12288 x 12288 45
// and 36; 8 x 4096 x 1024 6.3 and 4.6; 16 x 4096 x 1024 6.4 and 6.2, x 12288 9.0 and 11.9;
// 4 x 4096 x 4096 9.2 and 9.3, x 12288 14 and 18; 3 x 12288 x 6144 17 and 19.
constexpr int kFewBytes = 52 << 10, kFewWgs = 1024;
constexpr int64_t kFewValues = 11 << 10, kFewValuesNarrow = 18 << 10;  // of A; for a round of workgroups
bool few(bool quantise, int M, int N, int K) {
    const int64_t values = (int64_t)M * K;
    return quantise && M <= 16 && (int64_t)M * moe::few_row(K) <= kFewBytes && N <= 16 * kFewWgs &&
           (M == 1 || values <= (N <= 4096 ? kFewValuesNarrow : kFewValues));
}

// WIDE: fp32 outputs, from products of codes converted to bf16.
template <bool WIDE>
int run(const MatArgs &p, Kind kind, hipStream_t s) {
    switch (kind) {
        case FEW:
            hipLaunchKernelGGL((fp8_matmul_few_kernel<WIDE, 8, 2>), dim3((p.N + 15) / 16), dim3(512),
                               (size_t)p.M * moe::few_row(p.K), s, p);
            break;
        case ROWS1: launch_rows<WIDE, 1, 1, 8, 2>(p, s); break;
        case ROWS2: launch_rows<WIDE, 1, 2, 8, 2>(p, s); break;
        case T16: launch_tile<WIDE, moe::Fp8Tile<1, 2, 1, 1, 4, 4, 4>>(p, s); break;
        case T32: launch_tile<WIDE, moe::Fp8Tile<1, 2, 2, 1, 3, 3, 4>>(p, s); break;
        case T32W: launch_tile<WIDE, moe::Fp8Tile<1, 4, 2, 1, WIDE ? 2 : 3, WIDE ? 2 : 3, 4>>(p, s); break;
        case T64: launch_tile<WIDE, moe::Fp8Tile<2, 2, 2, 2, 3, 3, 2>>(p, s); break;
        case T128N: launch_tile<WIDE, moe::Fp8Tile<2, 2, 4, 2, 2, 2, 2>>(p, s); break;
        case T128:
            if constexpr (WIDE)
                launch_tile<WIDE, moe::Fp8Tile<2, 2, 4, 4, 2, 2, 2>>(p, s);
            else
                launch_tile<WIDE, moe::Fp8Tile<2, 4, 4, 2, 3, 3>>(p, s);
            break;
        default:
            if constexpr (!WIDE) {
                if (kind == T128P)
                    launch_tile<WIDE, moe::Fp8Tile<2, 2, 4, 4, 2, 2>>(p, s);
                else if (kind == T256N)
                    launch_tile<WIDE, moe::Fp8Tile<2, 4, 8, 3, 2, 3>>(p, s);
                else
                    launch_tile<WIDE, moe::Fp8Tile<2, 4, 8, 4, 2, 2>>(p, s);
            }
    }
    MOE_LAUNCH_CHECK("fp8_matmul_kernel");
    return MOE_OK;
}

// Quantised activations in the workspace: codes, then scales.
struct Space {
    size_t codes, scales, total;
};
Space layout(int M, int N, int K, bool quantise) {
    Space w{};
    if (!quantise || few(quantise, M, N, K)) return w;
    w.scales = moe::align_up((size_t)M * K, 256);
    w.total = w.scales + moe::align_up((size_t)M * moe::fp8_scale_row(K), 256);
    return w;
}

}  // namespace

extern "C" size_t moe_fp8_matmul_workspace_bytes(int M, int N, int K, int a_type) {
    if (M <= 0 || N <= 0 || K <= 0 || K % 16 || M > kMaxRows || N > kMaxRows || K > kMaxK) return 0;
    if (a_type != MOE_BF16 && a_type != MOE_FP8) return 0;
    return layout(M, N, K, a_type == MOE_BF16).total;
}

extern "C" int moe_fp8_matmul(const void *a, int a_type, int64_t a_stride, const float *a_scales,
                              int64_t a_scales_stride, const uint8_t *w, int64_t w_stride, const float *w_scales,
                              int64_t w_scales_stride, int M, int N, int K, const float *bias, void *y, int y_type,
                              int64_t y_stride, void *workspace, size_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0) return moe::fail(MOE_E_ARG, "fp8_matmul: M=%d, N=%d", M, N);
    if (a_type != MOE_BF16 && a_type != MOE_FP8) return moe::fail(MOE_E_ARG, "fp8_matmul: a_type=%d", a_type);
    if (y_type != MOE_BF16 && y_type != MOE_FP32) return moe::fail(MOE_E_ARG, "fp8_matmul: y_type=%d", y_type);
    if (K <= 0 || K % 16) return moe::fail(MOE_E_SHAPE, "fp8_matmul: K=%d must be a positive multiple of 16", K);
    if (M > kMaxRows || N > kMaxRows || K > kMaxK)
        return moe::fail(MOE_E_SHAPE, "fp8_matmul: M=%d, N=%d above %d or K=%d above %d", M, N, kMaxRows, K, kMaxK);
    if (M == 0 || N == 0) return MOE_OK;
    const bool quantise = a_type == MOE_BF16;
    if (!a || !w || !w_scales || !y || (!quantise && !a_scales))
        return moe::fail(MOE_E_ARG, "fp8_matmul: NULL pointer");
    const int64_t size = y_type == MOE_FP32 ? 4 : 2, a_row = quantise ? 2 * (int64_t)K : K;
    const int64_t srow = 4 * (int64_t)moe::fp8_blocks(K);
    if ((M > 1 && (a_stride < a_row || y_stride < size * N || (!quantise && a_scales_stride < srow))) ||
        (N > 1 && w_stride < K) || (N > 128 && w_scales_stride < srow))
        return moe::fail(MOE_E_SHAPE, "fp8_matmul: a row stride (%lld, %lld, %lld, %lld, %lld) is below the row's bytes",
                         (long long)a_stride, (long long)a_scales_stride, (long long)w_stride,
                         (long long)w_scales_stride, (long long)y_stride);
    if (((uintptr_t)a | (uintptr_t)w) % 16 || (M > 1 && a_stride % 16) || (N > 1 && w_stride % 16))
        return moe::fail(MOE_E_ARG, "fp8_matmul: operands' pointers and strides must be multiples of 16 bytes");
    if (!quantise && ((uintptr_t)a_scales % 16 || (M > 1 && a_scales_stride % 16)))
        return moe::fail(MOE_E_ARG, "fp8_matmul: a_scales and its stride must be multiples of 16 bytes");
    if ((uintptr_t)w_scales % 4 || (N > 128 && w_scales_stride % 4))
        return moe::fail(MOE_E_ARG, "fp8_matmul: w_scales or its stride is not a multiple of 4 bytes");
    if ((uintptr_t)y % size || (M > 1 && y_stride % size) || (uintptr_t)bias % 4)
        return moe::fail(MOE_E_ARG, "fp8_matmul: y, its stride or bias is not aligned to its type");
    if ((M > 1 && (a_stride > kMaxStride || (!quantise && a_scales_stride > kMaxStride))) ||
        (N > 1 && w_stride > kMaxStride))
        return moe::fail(MOE_E_SHAPE, "fp8_matmul: operands' rows more than %lld bytes apart", (long long)kMaxStride);
    const Space sp = layout(M, N, K, quantise);
    if (workspace_bytes < sp.total || (sp.total && !workspace))
        return moe::fail(MOE_E_NOMEM, "fp8_matmul: workspace %zu < %zu bytes", workspace_bytes, sp.total);
    if (sp.total && (uintptr_t)workspace % 16)
        return moe::fail(MOE_E_ARG, "fp8_matmul: workspace is not 16-byte aligned");
    hipStream_t s = (hipStream_t)stream;
    MatArgs p{};
    p.a = {(const uint8_t *)a, (const uint8_t *)a_scales, M > 1 ? (size_t)a_stride : 0,
           M > 1 ? (size_t)a_scales_stride : 0};
    p.w = w;
    p.w_stride = N > 1 ? (size_t)w_stride : 0;
    p.ws = (const uint8_t *)w_scales;
    p.ws_stride = N > 128 ? (size_t)w_scales_stride : 0;
    p.M = M, p.N = N, p.K = K;
    p.bias = bias;
    p.y = (uint8_t *)y;
    p.y_stride = M > 1 ? (size_t)y_stride : 0;
    p.ends = !quantise && moe::fp8_blocks(K) % 4 != 0;
    const bool here = few(quantise, M, N, K);
    if (quantise && !here) {
        uint8_t *codes = (uint8_t *)workspace + sp.codes;
        float *scales = (float *)((uint8_t *)workspace + sp.scales);
        const int rc = moe::fp8_quant_rows(a, MOE_BF16, p.a.stride, M, K, false, codes, (size_t)K, scales,
                                           moe::fp8_scale_row(K), s);
        if (rc != MOE_OK) return rc;
        p.a = {codes, (const uint8_t *)scales, (size_t)K, moe::fp8_scale_row(K)};
    }
    const size_t far = (size_t)kTileStride;
    const bool near = (M == 1 || (p.a.stride < far && p.a.scale_stride < far)) && (N == 1 || p.w_stride < far);
    const bool wide = y_type == MOE_FP32;
    const Kind kind = here ? FEW : plan(wide, M, N, K, near);
    return wide ? run<true>(p, kind, s) : run<false>(p, kind, s);
}
