// Router logits of many tokens, x [T,H] bf16 times w [E,H] fp32, on the bf16 matrix cores.
//
// An fp32 weight is the exact sum of three bf16 numbers (8 significant bits each, cut off
// the top), and products of bf16 numbers are exact in fp32, so three products of bf16
// matrices give the fp32 product but for the additions' rounding.  That is kept small and
// bounded: 64 columns at a time are summed from zero, the two small planes first, and
// joined in fp32; the parts of H are joined in fp64 by the reader, who also gets the norms
// of the rows of x and w and with them a bound on each logit's error.
//
// A workgroup owns 16 MT tokens x 128 experts (16 a wave) and one part of H, and walks it
// in stages of 64 columns through a ring of three (four of 32 tokens) LDS stages filled by
// direct loads; weights come in as fp32 and are split in registers, each by one wave (11
// instructions for two weights, beside six products of 16 cycles for every eight a lane).
// 2048 x 6144 x 256: 30 us, 0.64 PFLOP/s of bf16 products; the fp64 matrix cores took 209.
// 16 layers of 32 tokens: 20 us, 5 TB/s of weights.
#include <algorithm>

#include "common.h"
#include "lds_dma.h"
#include "router_split.h"
#include "tile.h"

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCols = 64;   // of a stage
constexpr int kBN = 128;    // experts of a workgroup
constexpr int kWaves = 8;

template <int MT>
struct Tile {
    static constexpr int BM = 16 * MT, X_BYTES = BM * 128, W_BYTES = kBN * 256, STAGE = X_BYTES + W_BYTES;
    static constexpr int STAGES = 160 * 1024 / STAGE < 4 ? 160 * 1024 / STAGE : 4;
    static constexpr int X_LOADS = X_BYTES / 1024, X_EACH = (X_LOADS + kWaves - 1) / kWaves, W_EACH = kBN / 4 / kWaves;
    static constexpr int EACH = X_EACH + W_EACH;
};

struct Planes {
    bf16x8_t p[3];  // of 8 weights: large, middle, small
};
__device__ __forceinline__ Planes split8(const float (&w)[8]) {
    uint32_t d[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = w[2 * j], b = w[2 * j + 1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
            d[i][j] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);  // the upper halves
            a -= __uint_as_float(ua & 0xFFFF0000u);
            b -= __uint_as_float(ub & 0xFFFF0000u);
        }
    }
    Planes s;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        s.p[i] = __builtin_bit_cast(bf16x8_t, make_uint4(d[i][0], d[i][1], d[i][2], d[i][3]));
    return s;
}

template <int MT>
__global__ __launch_bounds__(64 * kWaves) void router_split_kernel(const uint16_t *__restrict__ x, int T, int H,
                                                                   const float *__restrict__ w, int E, int m_tiles,
                                                                   moe::RouterSplit sp, uint8_t *__restrict__ ws) {
    using L = Tile<MT>;
    constexpr int S = L::STAGES;
    __shared__ uint4 smem4[S * L::STAGE / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = blockIdx.x % m_tiles * L::BM, e0 = blockIdx.x / m_tiles * kBN, part = blockIdx.y;
    const int h0 = part * sp.columns, cols = min(sp.columns, H - h0), ns = (cols + kCols - 1) / kCols;
    const int halves = (cols - (ns - 1) * kCols) / 32;  // of the last stage: 1 or 2 (H % 32 == 0)
    const uint16_t *xb = x + (size_t)blockIdx.z * T * H + (size_t)m0 * H + h0;
    const float *wb = w + (size_t)blockIdx.z * E * H + (size_t)e0 * H + h0;
    ws += blockIdx.z * sp.total;
    const uint32_t lds0 = lds_addr(smem);

    // x: 8 rows x 128 bytes a load, w: 4 rows x 256; a row's 16-byte pieces change places by
    // a key of the row
    const int px = (lane & 7) ^ moe::bank_key<8>((8 * wave + (lane >> 3)) & 15);
    const int pw = (lane & 15) ^ moe::bank_key<16>((4 * wave + (lane >> 4)) & 15);
    const uint32_t cut_x = 16 * (px - min(px, 4 * halves - 1)), cut_w = 16 * (pw - min(pw, 8 * halves - 1));
    uint32_t x_at[L::X_EACH], w_at[L::W_EACH];
    auto x_load = [&](int j) __attribute__((always_inline)) { return (j * kWaves + wave) % L::X_LOADS; };
#pragma unroll
    for (int j = 0; j < L::X_EACH; ++j)
        x_at[j] = (uint32_t)min(8 * x_load(j) + (lane >> 3), T - 1 - m0) * (uint32_t)(2 * H) + 16 * px;
#pragma unroll
    for (int j = 0; j < L::W_EACH; ++j)
        w_at[j] = (uint32_t)min(4 * (j * kWaves + wave) + (lane >> 4), E - 1 - e0) * (uint32_t)(4 * H) + 16 * pw;
    auto issue = [&](int i) __attribute__((always_inline)) {
        const uint32_t at = lds0 + (uint32_t)(i % S) * L::STAGE;
#pragma unroll
        for (int j = 0; j < L::X_EACH; ++j)
            dma16(xb + (size_t)i * kCols, x_at[j] - (i == ns - 1 ? cut_x : 0u), at + 1024u * x_load(j));
#pragma unroll
        for (int j = 0; j < L::W_EACH; ++j)
            dma16(wb + (size_t)i * kCols, w_at[j] - (i == ns - 1 ? cut_w : 0u),
                  at + L::X_BYTES + 1024u * (j * kWaves + wave));
    };

    f32x4_t sum[MT];
    float xn[(MT + kWaves - 1) / kWaves] = {}, wn = 0.0f;  // squares of this wave's share of the rows of x, and of its w
#pragma unroll
    for (int u = 0; u < MT; ++u) sum[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < S - 1 && i < ns; ++i) issue(i);
    for (int g = 0; g < ns; ++g) {
        // stage g has landed once only the S - 2 after it are in flight; every wave is done
        // with stage g - 1, whose place the next load takes
        if (g + S - 1 <= ns)
            wait_vm<(S - 2) * L::EACH>();
        else
            wait_vm<0>();
        ring_barrier();
        if (g + S - 1 < ns) issue(g + S - 1);
        const uint8_t *st = smem + (uint32_t)(g % S) * L::STAGE;
        const uint8_t *xs = st + r * 128, *wr = st + L::X_BYTES + (wave * 16 + r) * 256;
        f32x4_t acc[MT];
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        Planes wp[2];
        bf16x8_t xv[2][MT];
        const bool both = g + 1 < ns || halves == 2;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s == 1 && !both) break;
            float f[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 v = *reinterpret_cast<const float4 *>(wr + 16 * ((8 * s + 2 * q + h) ^ moe::bank_key<16>(r)));
                f[4 * h] = v.x, f[4 * h + 1] = v.y, f[4 * h + 2] = v.z, f[4 * h + 3] = v.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) wn = fmaf(f[j], f[j], wn);
            wp[s] = split8(f);
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const uint4 v = *reinterpret_cast<const uint4 *>(xs + u * 2048 + 16 * ((4 * s + q) ^ moe::bank_key<8>(r)));
                xv[s][u] = __builtin_bit_cast(bf16x8_t, v);
                if (u % kWaves == wave) {
                    float &n = xn[u / kWaves];
                    n = dot2_bf16(v.x, v.x, n);
                    n = dot2_bf16(v.y, v.y, n);
                    n = dot2_bf16(v.z, v.z, n);
                    n = dot2_bf16(v.w, v.w, n);
                }
            }
        }
        // the small planes of all 64 columns first, while the sums are small
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s == 1 && !both) break;
#pragma unroll
                for (int u = 0; u < MT; ++u)
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wp[s].p[p], xv[s][u], acc[u], 0, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < MT; ++u) sum[u] += acc[u];
    }
    wait_vm<0>();

    float *partial = reinterpret_cast<float *>(ws + sp.partial) + (size_t)part * T * E;
    const int e = e0 + wave * 16 + 4 * q;
    if (e < E)
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int t = m0 + 16 * u + r;
            if (t >= T) continue;
            float *o = partial + (size_t)t * E + e;
            if (E % 4 == 0) {
                *reinterpret_cast<float4 *>(o) = make_float4(sum[u][0], sum[u][1], sum[u][2], sum[u][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < E) o[j] = sum[u][j];
            }
        }
    wn += __shfl_xor(wn, 16, 64);
    wn += __shfl_xor(wn, 32, 64);
    if (blockIdx.x % m_tiles == 0 && q == 0 && e0 + wave * 16 + r < E)
        reinterpret_cast<float *>(ws + sp.wn)[(size_t)part * E + e0 + wave * 16 + r] = wn;
#pragma unroll
    for (int i = 0; i < (MT + kWaves - 1) / kWaves; ++i) {
        float n = xn[i];
        n += __shfl_xor(n, 16, 64);
        n += __shfl_xor(n, 32, 64);
        const int u = i * kWaves + wave, t = m0 + 16 * u + r;
        if (e0 == 0 && q == 0 && u < MT && t < T) reinterpret_cast<float *>(ws + sp.xn)[(size_t)part * T + t] = n;
    }
}

}  // namespace

namespace moe {

static constexpr int64_t kCUs = 256;
static int most_parts(int H) { return std::max(1, std::min((H + kCols - 1) / kCols / 4, 16)); }

RouterSplit router_split_layout(int layers, int T, int E, int H) {
    RouterSplit sp{};
    // as many parts as make one workgroup a CU, of at least four stages, at most 16
    const int64_t tiles = (int64_t)layers * ((E + kBN - 1) / kBN) * (T <= 32 ? 1 : (T + 127) / 128);
    const int stages = (H + kCols - 1) / kCols;
    const int parts = std::max(1, std::min((int)(kCUs / std::min(tiles, kCUs)), most_parts(H)));
    sp.columns = (stages + parts - 1) / parts * kCols;
    sp.parts = (H + sp.columns - 1) / sp.columns;
    size_t o = 0;
    sp.partial = o;
    o += align_up((size_t)sp.parts * T * E * 4, 256);
    sp.xn = o;
    o += align_up((size_t)sp.parts * T * 4, 256);
    sp.wn = o;
    o += align_up((size_t)sp.parts * E * 4, 256);
    sp.total = o;
    return sp;
}

// Fewer tokens or layers may be summed in more parts.  Two or more parts are chosen where
// parts * layers * tiles of experts * tiles of at most 128 tokens are at most kCUs.
size_t router_split_most(int layers, int T, int E, int H) {
    const int64_t cap = most_parts(H), all = (int64_t)layers * T, room = kCUs / ((E + kBN - 1) / kBN);
    const int64_t rows = std::max(all, std::min(cap * all, 128 * room));  // parts x layers x tokens
    const int64_t parts = std::max((int64_t)layers, std::min(cap * layers, room));
    return 4 * ((size_t)rows * (E + 1) + (size_t)parts * E) + (size_t)layers * 3 * 256;  // (rounded up by arrays)
}

int router_split(const uint16_t *x, int layers, int T, int H, const float *w_router, int E, const RouterSplit &sp,
                 void *workspace, hipStream_t s) {
    const int n_tiles = (E + kBN - 1) / kBN, m_tiles = T <= 32 ? 1 : (T + 127) / 128;
    const dim3 grid(m_tiles * n_tiles, sp.parts, layers), block(64 * kWaves);
    auto *kernel = T <= 32 ? router_split_kernel<2> : router_split_kernel<8>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, x, T, H, w_router, E, m_tiles, sp, (uint8_t *)workspace);
    MOE_LAUNCH_CHECK("router_split_kernel");
    return MOE_OK;
}

}  // namespace moe
