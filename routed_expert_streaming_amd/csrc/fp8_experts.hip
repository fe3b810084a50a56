// Routed experts' SwiGLU feed-forward on FP8 slabs: per token and expert
//   g = W1 x, u = W3 x, h = silu(g) * u, y = W2 h
// with x and h quantised to E4M3 in blocks of 1 x 128 and fp32 sums.
//
// g and u are sums of exact products (codes converted to bf16): what the FP8 matrix cores
// cut would move codes of h, and the outputs were then 1.3 times as far from the exact
// ones as their rounding to bf16 leaves them.  y has nothing behind it but that rounding
// and takes the FP8 cores.
#include <algorithm>

#include "common.h"
#include "fp8_mma.h"
#include "fp8_quant.h"
#include "fp8_rows.h"
#include "fp8_tall.h"
#include "fp8_tile.h"

namespace {

using moe::f32x4;

constexpr int kMaxE = 1024;
constexpr int kMaxPairs = 16384;   // of a permutation
// Up to here, and up to kFewRows tokens, a workgroup finds its expert's pairs itself: no
// permutation, no launch for a quantisation.  Top 8 of 128 experts of 4096 x 1536 and a
// shared one, this way and by tiles: 1 token 48 and 80 us, 2 tokens 75 and 89, 3 tokens 102
// and 109, 4 tokens 127 and 125.
constexpr int kScanPairs = 32;
constexpr int kFewBytes = 44 * 1024;  // of LDS for their rows, beside up to 16 KB for the sums

struct ExpertArgs {
    moe::Fp8Act a;      // tile kernels.  gate/up: x, a row a token; down: h
    const uint8_t *in;  // few tokens.  gate/up: x in bf16; down: h in fp32
    int T, H, I, E, k;
    const int32_t *topk_idx;
    const void *const *table;
    const uint8_t *shared, *mask;
    uint8_t *out;         // few tokens: fp32 h [rows, I] or y [rows, H]; tile kernels: codes of h, or y
    uint8_t *out_scales;  // tile kernel, gate/up: h's
    const int32_t *offset, *pair_of_row, *tiles;  // tile kernels
};

// ---------------------------------------------------------------- few tokens
// Group blockIdx.y: pair blockIdx.y stands for its expert where it is the expert's first
// pair, and all waves together find the expert's other pairs (no launch for a
// permutation); the shared expert, all tokens in order, comes last.  Rows of h and y: pair
// numbers, then T * k + t.  list: kScanPairs numbers.
struct Group {
    const uint8_t *slab;
    const int32_t *pairs;  // NULL: all tokens, in order
    int rows;
};
__device__ __forceinline__ Group find_group(const ExpertArgs &p, int32_t *list) {
    static_assert(kScanPairs <= 64, "a ballot");
    const int P = p.T * p.k, g = blockIdx.y, lane = threadIdx.x & 63;
    if (g >= P) return {p.shared, nullptr, p.T};
    const int e = p.topk_idx[g];
    if ((unsigned)e >= (unsigned)p.E || (p.mask && !p.mask[e])) return {nullptr, nullptr, 0};
    const bool mine = lane < P && p.topk_idx[lane] == e;
    const uint64_t m = __ballot(mine);
    if (__ffsll((long long)m) - 1 < g) return {nullptr, nullptr, 0};  // not the first
    if (mine && threadIdx.x < 64) list[__popcll(m & ((1ull << lane) - 1))] = lane;
    __syncthreads();
    return {(const uint8_t *)p.table[e], list, (int)__popcll(m)};
}

// GATEUP: blockIdx.x is 16 columns of h, tile 0 their rows of W1 and tile 1 of W3; down:
// 16 * NT rows of W2.  A workgroup quantises its rows (x in bf16, h in fp32) itself while
// its first weights are on their way; at_once rows fit the LDS.  Weights bound it: 113 MB of
// W1 and W3 in 27 us, 57 MB of W2 in 16.  Steps of one block (U) and few waves on a short K
// leave more workgroups a CU: with two blocks a step 59 us a token, so 48.
template <bool GATEUP, int NT, int WK, int U>
__global__ __launch_bounds__(64 * WK) void fp8_experts_few_kernel(ExpertArgs p, int at_once) {
    static_assert(!GATEUP || NT == 2, "a tile of each matrix");
    extern __shared__ uint4 few_smem[];
    __shared__ f32x4 part[WK][NT][64];
    __shared__ int32_t list[kScanPairs];
    uint8_t *const xs = reinterpret_cast<uint8_t *>(few_smem);
    const Group g = find_group(p, list);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int K = GATEUP ? p.H : p.I, N = GATEUP ? p.I : p.H, n0 = blockIdx.x * 16 * (GATEUP ? 1 : NT);
    if (g.rows == 0) return;
    const uint8_t *w[NT];
    const float *ws[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const moe::Fp8Slab m = moe::fp8_slab(g.slab, p.H, p.I, GATEUP ? t : 2);
        const int n = min(n0 + (GATEUP ? 0 : 16 * t), N - 1);
        w[t] = m.w + (size_t)min(n + r, N - 1) * K;
        ws[t] = m.s + (size_t)(n / 128) * m.s_row;
    }
    auto row_of = [&](int m) { return g.pairs ? g.pairs[m] : p.T * p.k + m; };
    for (int m0 = 0; m0 < g.rows; m0 += at_once) {
        const int rows = min(at_once, g.rows - m0);
        f32x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (m0) __syncthreads();  // the last rows and their sums are read
        moe::multiply_few<GATEUP, NT, U, WK>(
            wave, K, q, w, ws, xs + min(r, rows - 1) * moe::few_row(K), acc, [&]() {
                for (int m = 0; m < rows; ++m) {
                    const int row = GATEUP ? (g.pairs ? g.pairs[m0 + m] / p.k : m0 + m) : row_of(m0 + m);
                    moe::quantise_few<GATEUP ? MOE_BF16 : MOE_FP32>(
                        xs + m * moe::few_row(K), p.in + (size_t)row * K * (GATEUP ? 2 : 4), 0, 1, K, threadIdx.x,
                        64 * WK);
                }
                __syncthreads();
            });
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][t][lane] = acc[t];
        __syncthreads();
        constexpr int ITEMS = GATEUP ? 1 : NT;
        for (int i = wave; i < ITEMS; i += WK) {
            const int n = n0 + 16 * i + 4 * q;
            f32x4 v = moe::joined<WK, NT>(part, i, lane);
            if constexpr (GATEUP) {
                const f32x4 up = moe::joined<WK, NT>(part, 1, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = moe::silu(v[j]) * up[j];
            }
            if (r < rows && n < N)  // N % 32 == 0: all four columns exist
                reinterpret_cast<float4 *>(p.out)[((size_t)row_of(m0 + r) * N + n) / 4] =
                    make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

// ---------------------------------------------------------------- many tokens
// The (token, expert) pairs in expert order; a workgroup owns BM rows of one expert and 128
// columns of h or 256 of y.  Rows of h: the pairs' places in that order, then T * k + t; so
// the down projection reads neighbouring rows.
constexpr int kGroupBits = 11;  // of a tile's number: its expert (E: the shared one); above: which of its BM rows
constexpr int kPrepare = 1024;  // threads of the kernel that comes first

// One launch before the products.  Workgroup 0 sorts the pairs by expert, stable, and lists
// the tiles of BM rows: offset [E + 1], pair_of_row, tiles[0] how many, tiles[1 ..] each
// one's expert and place.  Its 16 waves take neighbouring runs of pairs; lanes with the
// same expert find each other by ballots over the number's bits, so that a pair's place
// (its expert's offset, plus that expert's pairs of the waves before, plus its rank in its
// own) needs neither atomics nor a second sort.  Pairs of masked experts have their places
// but no tiles; pairs with a number outside 0 .. E-1 have none.  The other workgroups
// quantise x: codes, or (WIDE) the codes' values in bf16, and scales.  2048 tokens of 4096,
// top 8: 24 us, 3% of the call, most of it the sort; 32 tokens 7.
struct PrepareArgs {
    const uint16_t *x;
    uint8_t *xq;
    float *xs;
    int T, H, E, k, BM;
    const int32_t *topk_idx;
    const uint8_t *mask;
    bool shared;
    int32_t *offset, *pairs, *tiles;
};

__device__ __forceinline__ int wave_scan(int v) {  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, 64);
        if ((int)(threadIdx.x & 63) >= o) v += u;
    }
    return v;
}

__device__ __forceinline__ void sort_pairs(const PrepareArgs &p, uint16_t *count) {  // count: [16][E]
    __shared__ int sums[2][16];
    constexpr int kPer = kMaxPairs / 1024;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = p.T * p.k;
    const int run = (n + 1023) / 1024 * 64;  // pairs of a wave
    int ex[kPer], rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = wave * run + 64 * i + lane;
        ex[i] = 64 * i < run && at < n ? p.topk_idx[at] : -1;
        if ((unsigned)ex[i] >= (unsigned)p.E) ex[i] = -1;
    }
    for (int i = tid; i < 16 * p.E; i += 1024) count[i] = 0;
    __syncthreads();
    uint16_t *mine = count + wave * p.E;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (64 * i < run) {
            uint64_t same = __ballot(ex[i] >= 0);
#pragma unroll
            for (int b = 0; b < 10; ++b) {
                if ((p.E - 1) >> b == 0) break;
                const uint64_t ones = __ballot(ex[i] >> b & 1);
                same &= (ex[i] >> b & 1) ? ones : ~ones;
            }
            const int below = __popcll(same & ((1ull << lane) - 1));
            if (ex[i] >= 0) {
                const int before = mine[ex[i]];  // read by all lanes of the expert before the first of them writes
                rank[i] = before + below;
                if (below == 0) mine[ex[i]] = (uint16_t)(before + __popcll(same));
            }
        }
    __syncthreads();
    // one expert a thread: its pairs, its tiles
    int pairs = 0;
    if (tid < p.E)
        for (int w = 0; w < 16; ++w) {
            const int c = count[w * p.E + tid];
            count[w * p.E + tid] = (uint16_t)pairs;
            pairs += c;
        }
    const int tiles = tid < p.E && (!p.mask || p.mask[tid]) ? (pairs + p.BM - 1) / p.BM : 0;
    const int pair_sum = wave_scan(pairs), tile_sum = wave_scan(tiles);
    if (lane == 63) sums[0][wave] = pair_sum, sums[1][wave] = tile_sum;
    __syncthreads();
    int first = pair_sum - pairs, tile0 = tile_sum - tiles, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if (w < wave) first += sums[0][w], tile0 += sums[1][w];
        all += sums[1][w];
    }
    if (tid < p.E) p.offset[tid] = first;
    if (tid == p.E - 1) p.offset[p.E] = first + pairs;
    for (int i = 0; i < tiles; ++i) p.tiles[1 + tile0 + i] = tid | i << kGroupBits;
    const int more = p.shared ? (p.T + p.BM - 1) / p.BM : 0;
    for (int i = tid; i < more; i += 1024) p.tiles[1 + all + i] = p.E | i << kGroupBits;
    if (tid == 0) p.tiles[0] = all + more;
    if (tid < p.E) reinterpret_cast<int *>(count + 16 * p.E)[tid] = first;
    __syncthreads();
    const int *offset = reinterpret_cast<const int *>(count + 16 * p.E);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (64 * i < run && ex[i] >= 0) p.pairs[offset[ex[i]] + mine[ex[i]] + rank[i]] = wave * run + 64 * i + lane;
}

template <bool WIDE>
__global__ __launch_bounds__(kPrepare) void fp8_experts_prepare_kernel(PrepareArgs p) {
    extern __shared__ uint16_t counts[];
    if (blockIdx.x == 0) {
        sort_pairs(p, counts);
        return;
    }
    const int per = 16 * ((p.H + 127) / 128), u = (blockIdx.x - 1) * kPrepare + threadIdx.x;
    if (u >= p.T * per) return;  // T * per: a multiple of 16
    const int row = u / per, c = u - row * per;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (8 * c < p.H) moe::load8<MOE_BF16>(reinterpret_cast<const uint8_t *>(p.x + (size_t)row * p.H + 8 * c), v);
    const float s = moe::fp8_scale(moe::row16_max(moe::top_of(v)), false);
    const uint2 codes = moe::fp8_codes8<false>(v, s);
    if (8 * c < p.H) {
        if constexpr (WIDE)
            *reinterpret_cast<uint4 *>(p.xq + ((size_t)row * p.H + 8 * c) * 2) =
                __builtin_bit_cast(uint4, moe::widen8(codes.x, codes.y));
        else
            *reinterpret_cast<uint2 *>(p.xq + (size_t)row * p.H + 8 * c) = codes;
    }
    if ((c & 15) == 0) p.xs[(size_t)row * (moe::fp8_scale_row(p.H) / 4) + (c >> 4)] = s;
}

// Rows of y, for store_tile.
struct YRows {
    int M, N;
    uint8_t *y;
    size_t y_stride;
    const int32_t *pairs;
    __device__ __forceinline__ uint8_t *row(int m) const { return y + (size_t)(pairs ? pairs[m] : m) * y_stride; }
};

// One tile: rows rows of an expert from its m0-th on x columns n0 and up.
struct TileOf {
    const uint8_t *slab;
    const int32_t *pairs;  // of these rows; NULL: tokens m0 and up
    int first, m0, n0, rows;
    bool shared;
};
template <bool GATEUP, class T>
__device__ __forceinline__ void experts_tile(const ExpertArgs &p, const TileOf &at, uint8_t *smem) {
    constexpr int BN = GATEUP ? T::BN / 2 : T::BN, MT = T::MT, NT = T::NT;  // columns of h or y
    const int H = p.H, I = p.I, P = p.T * p.k, K = GATEUP ? H : I;
    const int first = at.first, m0 = at.m0, n0 = at.n0, rows = at.rows;
    const uint8_t *const slab = at.slab;
    const int32_t *const pairs = at.pairs;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / T::WN, wn = wave % T::WN;

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto row_of = [&](int row) { return min(row, rows - 1); };
    if constexpr (GATEUP) {
        // a wave's first NT / 2 tiles are rows of W1, the others the same rows of W3
        const moe::Fp8Slab w1 = moe::fp8_slab(slab, H, I, 0), w3 = moe::fp8_slab(slab, H, I, 1);
        const float *const ws[2] = {w1.s + (size_t)(n0 / 128) * w1.s_row, w3.s + (size_t)(n0 / 128) * w3.s_row};
        auto token = [&](int row) { return (uint32_t)(pairs ? pairs[row_of(row)] / p.k : m0 + row_of(row)); };
        auto w_off = [&](int row) {
            const int w = row / (16 * NT), t = row / 16 % NT, c = n0 + (w * (NT / 2) + t % (NT / 2)) * 16 + row % 16;
            return (uint32_t)((t >= NT / 2 ? I : 0) + min(c, I - 1)) * (uint32_t)H;
        };
        auto a_off = [&](int row) { return token(row) * (uint32_t)p.a.stride; };
        auto s_off = [&](int row) { return token(row) * (uint32_t)p.a.scale_stride; };
        if constexpr (T::TALL)
            moe::fp8_tall<T, 2>(smem, w1.w, p.a.codes, p.a.scales, ws, K, w_off, a_off, s_off, acc);
        else
            moe::fp8_tile<T, true, 2>(smem, w1.w, p.a.codes, p.a.scales, ws, K, w_off, a_off, s_off, acc);
        // h, its largest magnitude per row over the block's columns, its codes
        uint32_t(*tops)[T::WN] = reinterpret_cast<uint32_t(*)[T::WN]>(smem);
        uint8_t *codes = smem + T::BM * T::WN * 4;
        constexpr int PITCH = BN + 16, HT = NT / 2;  // a wave's tiles of h
        static_assert(BN == 128 && NT % 2 == 0, "a workgroup holds whole blocks of h");
        float h[MT][4 * HT];
#pragma unroll
        for (int u = 0; u < MT; ++u) {
#pragma unroll
            for (int j = 0; j < 4 * HT; ++j) {
                const int c = n0 + (wn * HT + j / 4) * 16 + 4 * q + j % 4;
                h[u][j] = c < I ? moe::silu(acc[j / 4][u][j % 4]) * acc[HT + j / 4][u][j % 4] : 0.0f;
            }
            uint32_t top = moe::top_of(h[u]);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
            if (q == 0) tops[(wm * MT + u) * 16 + r][wn] = top;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int m = (wm * MT + u) * 16 + r;
            uint32_t top = 0, c[HT];
#pragma unroll
            for (int w = 0; w < T::WN; ++w) top = max(top, tops[m][w]);
            const float s = moe::fp8_scale(top, false);
            moe::fp8_codes<false, HT>(h[u], s, c);
#pragma unroll
            for (int t = 0; t < HT; ++t)
                *reinterpret_cast<uint32_t *>(codes + m * PITCH + (wn * HT + t) * 16 + 4 * q) = c[t];
            if (wn == 0 && q == 0 && m < rows)
                *reinterpret_cast<float *>(p.out_scales + (size_t)(first + m0 + m) * moe::fp8_scale_row(I) +
                                           4 * (size_t)(n0 / 128)) = s;
        }
        __syncthreads();
        for (int v = threadIdx.x; v < T::BM * (BN / 16); v += 64 * T::WAVES) {
            const int m = v / (BN / 16), c = v % (BN / 16) * 16;
            if (m < rows && n0 + c < I)
                *reinterpret_cast<uint4 *>(p.out + (size_t)(first + m0 + m) * I + n0 + c) =
                    *reinterpret_cast<const uint4 *>(codes + m * PITCH + c);
        }
    } else {
        const moe::Fp8Slab w2 = moe::fp8_slab(slab, H, I, 2);
        const float *const ws[1] = {w2.s + (size_t)(min(n0 + wn * NT * 16, H - 1) / 128) * w2.s_row};
        const uint8_t *w = w2.w + (size_t)n0 * I, *h = p.a.codes + (size_t)(first + m0) * p.a.stride,
                      *hs = p.a.scales + (size_t)(first + m0) * p.a.scale_stride;
        auto w_off = [&](int row) { return (uint32_t)min(row, H - 1 - n0) * (uint32_t)I; };
        auto a_off = [&](int row) { return (uint32_t)row_of(row) * (uint32_t)p.a.stride; };
        auto s_off = [&](int row) { return (uint32_t)row_of(row) * (uint32_t)p.a.scale_stride; };
        if constexpr (T::TALL)
            moe::fp8_tall<T, 1>(smem, w, h, hs, ws, K, w_off, a_off, s_off, acc);
        else
            moe::fp8_tile<T, false, 1>(smem, w, h, hs, ws, K, w_off, a_off, s_off, acc);
        const YRows y{rows, H, p.out + (at.shared ? (size_t)(P + m0) * H * 4 : 0), (size_t)H * 4, pairs};
        moe::store_tile<T, MT, NT, float, true>(y, smem, 0, n0, wm, wn, lane, acc);
    }
}

// T: the tile, the tallest one of the heights where several are listed.
// 2048 tokens, top 8 of 128 of 4096 x 1536 and a shared one: gate/up 0.71 PFLOP/s on the
// bf16 matrix cores (busy 48% of the time, the clock down to 1.9 GHz), down 0.83 on the FP8
// ones with 2 TB/s of W2 and y.  A wave waits a third of its time at turns.
template <bool GATEUP, class T>
__global__ __launch_bounds__(64 * T::WAVES, T::TALL ? 2 : 1) void fp8_experts_tile_kernel(ExpertArgs p) {
    constexpr int BN = GATEUP ? T::BN / 2 : T::BN;
    __shared__ uint4 smem4[T::LDS / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    // Each XCD takes a run of neighbouring tiles, an expert's rows fastest: the tiles that
    // share rows of W start together and read them from its L2.  (With the columns fastest
    // they drifted apart: 2.9 GB came from memory for 1.6 GB of W1 and W3.)
    const int N = GATEUP ? p.I : p.H;
    const int n_tiles = (N + BN - 1) / BN, tiles = p.tiles[0] * n_tiles, per = (tiles + 7) / 8;
    const int i = blockIdx.x >> 3, tile = (blockIdx.x & 7) * per + i;
    if (i >= per || tile >= tiles) return;
    const int number = p.tiles[1 + tile / n_tiles], e = number & ((1 << kGroupBits) - 1);
    TileOf at;
    at.shared = e == p.E;
    at.first = at.shared ? p.T * p.k : p.offset[e];
    const int all = at.shared ? p.T : p.offset[e + 1] - at.first;  // rows
    const int m_tiles = (all + T::BM - 1) / T::BM;
    const int height = 16 * (((all + 15) / 16 + m_tiles - 1) / m_tiles);  // alike; with none left empty
    const int local = tile - (tile / n_tiles - (number >> kGroupBits)) * n_tiles;  // of the expert's tiles
    at.m0 = local % m_tiles * height, at.n0 = local / m_tiles * BN, at.rows = min(height, all - at.m0);
    at.pairs = at.shared ? nullptr : p.pair_of_row + at.first + at.m0;
    at.slab = at.shared ? p.shared : (const uint8_t *)p.table[e];
    if constexpr (T::TALL) {
        if (T::MT > 8 && at.rows > 128)
            experts_tile<GATEUP, moe::Fp8Tall<T::WN, (T::MT > 8 ? 10 : 4), T::EXACT>>(p, at, smem);
        else if (T::MT > 6 && at.rows > 96)
            experts_tile<GATEUP, moe::Fp8Tall<T::WN, (T::MT > 6 ? 8 : 4), T::EXACT>>(p, at, smem);
        else if (T::MT > 4 && at.rows > 64)
            experts_tile<GATEUP, moe::Fp8Tall<T::WN, (T::MT > 4 ? 6 : 4), T::EXACT>>(p, at, smem);
        else
            experts_tile<GATEUP, moe::Fp8Tall<T::WN, 4, T::EXACT>>(p, at, smem);
    } else {
        experts_tile<GATEUP, T>(p, at, smem);
    }
}

struct Space {
    size_t xq, xs, h, hq, hs, offset, pairs, tiles, y, total;
};
bool few(int T, int k) { return T <= moe::kFewRows && (int64_t)T * k <= kScanPairs; }

// Rows of a tile, by the rows an expert has on average.  Tiles of 16 rows leave two
// workgroups a CU and keep up with memory (32 tokens, top 8 of 128 experts of 4096 x 1536:
// 2.1 GB of weights in 380 us); tall ones read and convert each row of W once for all of an
// expert's rows.  Those experts, a call in a graph, us in tiles of 16, 64 and up to 160 rows:
//   rows an expert    8    16    24    32    48    64    96   128
//   16              447   497   575   680   865  1056  1436  1833
//   64              494   503   503   515   559   680   848  1005
//   160             493   493   507   517   542   603   702   833
int tile_rows(int T, int E, int k) {
    const int64_t pairs = (int64_t)T * k;
    return pairs >= (int64_t)64 * E ? 160 : pairs >= (int64_t)24 * E ? 64 : 16;
}

Space layout(int T, int H, int I, int E, int k, bool shared) {
    Space w{};
    const size_t rows = (size_t)T * k + (shared ? (size_t)T : 0);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += moe::align_up(bytes, 256);
        return at;
    };
    if (few(T, k)) {
        w.h = take(rows * I * 4);
    } else {
        const int BM = tile_rows(T, E, k);
        w.xq = take((size_t)T * H * (BM > 16 ? 2 : 1));
        w.xs = take((size_t)T * moe::fp8_scale_row(H));
        w.hq = take(rows * I);
        w.hs = take(rows * moe::fp8_scale_row(I));
        w.offset = take((size_t)(E + 1) * 4);
        w.pairs = take((size_t)T * k * 4);
        w.tiles = take(4 * (1 + rows / 16 + (size_t)E + 1));  // (16: the size grows with T)
    }
    w.y = take(rows * H * 4);
    w.total = o;
    return w;
}

// Enough for every call of fewer tokens too: a few rows' h is in fp32.
size_t workspace_of(int T, int H, int I, int E, int k, bool shared) {
    const int some = std::min(std::min(T, moe::kFewRows), kScanPairs / k);  // the most tokens that `few` takes
    return std::max(layout(T, H, I, E, k, shared).total, some ? layout(some, H, I, E, k, shared).total : 0);
}

template <bool GATEUP, class T>
int launch_tiles(const ExpertArgs &a, int rows, hipStream_t s) {
    // at most so many tiles of rows: every expert's last one may be short
    const int experts = a.E < a.T * a.k ? a.E : a.T * a.k, most = rows / T::BM + experts + 1;
    const int columns = GATEUP ? (a.I + T::BN / 2 - 1) / (T::BN / 2) : (a.H + T::BN - 1) / T::BN;
    hipLaunchKernelGGL((fp8_experts_tile_kernel<GATEUP, T>), dim3((unsigned)((most * columns + 7) / 8 * 8)),
                       dim3(64 * T::WAVES), 0, s, a);
    MOE_LAUNCH_CHECK("fp8_experts_tile_kernel");
    return MOE_OK;
}

template <bool GATEUP, int NT, int WK, int U>
int launch_few(const ExpertArgs &a, bool shared, hipStream_t s) {
    const int row = moe::few_row(GATEUP ? a.H : a.I), N = GATEUP ? a.I : a.H, columns = GATEUP ? 16 : 16 * NT;
    const int at_once = std::min(a.T, kFewBytes / row);  // at least 2: 16384 columns take 17 KB
    hipLaunchKernelGGL((fp8_experts_few_kernel<GATEUP, NT, WK, U>),
                       dim3((N + columns - 1) / columns, a.T * a.k + (shared ? 1 : 0)), dim3(64 * WK),
                       (size_t)at_once * row, s, a, at_once);
    MOE_LAUNCH_CHECK("fp8_experts_few_kernel");
    return MOE_OK;
}

int experts(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
            const void *const *expert_table, const void *shared_slab, const uint8_t *expert_mask, float *y,
            uint8_t *ws, const Space &sp, hipStream_t s) {
    const bool shared = shared_slab != nullptr;
    const int rows = T * k + (shared ? T : 0);
    ExpertArgs a{};
    a.T = T, a.H = H, a.I = I, a.E = E, a.k = k;
    a.topk_idx = topk_idx;
    a.table = expert_table;
    a.shared = (const uint8_t *)shared_slab;
    a.mask = expert_mask;
    if (few(T, k)) {
        a.in = (const uint8_t *)x;
        a.out = ws + sp.h;
        int rc = launch_few<true, 2, 8, 1>(a, shared, s);
        if (rc != MOE_OK) return rc;
        a.in = ws + sp.h;
        a.out = (uint8_t *)y;
        return launch_few<false, 2, 4, 1>(a, shared, s);
    }
    float *xs = (float *)(ws + sp.xs);
    const moe::Fp8Act ha{ws + sp.hq, ws + sp.hs, (size_t)I, moe::fp8_scale_row(I)};
    a.a = {ws + sp.xq, ws + sp.xs, (size_t)H, moe::fp8_scale_row(H)};
    const int BM = tile_rows(T, E, k);
    PrepareArgs pa{x, ws + sp.xq, xs, T, H, E, k, BM, topk_idx, expert_mask, shared, (int32_t *)(ws + sp.offset),
                   (int32_t *)(ws + sp.pairs), (int32_t *)(ws + sp.tiles)};
    const unsigned blocks = 1 + (unsigned)(((size_t)T * 16 * moe::fp8_blocks(H) + kPrepare - 1) / kPrepare);
    const size_t lds = (size_t)E * (16 * sizeof(uint16_t) + sizeof(int));
    auto *prepare = BM > 16 ? fp8_experts_prepare_kernel<true> : fp8_experts_prepare_kernel<false>;
    hipLaunchKernelGGL(prepare, dim3(blocks), dim3(kPrepare), lds, s, pa);
    MOE_LAUNCH_CHECK("fp8_experts_prepare_kernel");
    a.offset = pa.offset, a.pair_of_row = pa.pairs, a.tiles = pa.tiles;
    a.out = ws + sp.hq;
    a.out_scales = ws + sp.hs;
    if (BM > 16) a.a.stride = (size_t)2 * H;  // bf16
    int rc = BM == 160  ? launch_tiles<true, moe::Fp8Tall<8, 10, true>>(a, rows, s)
             : BM == 64 ? launch_tiles<true, moe::Fp8Tall<8, 4, true>>(a, rows, s)
                        : launch_tiles<true, moe::Fp8Tile<1, 8, 1, 2, 2, 2>>(a, rows, s);
    if (rc != MOE_OK) return rc;
    a.a = ha;
    a.out = (uint8_t *)y;
    return BM == 160  ? launch_tiles<false, moe::Fp8Tall<4, 10, false>>(a, rows, s)
           : BM == 64 ? launch_tiles<false, moe::Fp8Tall<4, 4, false>>(a, rows, s)
                      : launch_tiles<false, moe::Fp8Tile<1, 8, 1, 2, 2, 2>>(a, rows, s);
}

int check(const char *who, const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
          const void *const *expert_table, const void *shared_slab, const void *out, const void *workspace,
          size_t workspace_bytes, Space *sp) {
    if (H <= 0 || I <= 0 || H % 32 || I % 32 || H > 16384 || I > 16384)
        return moe::fail(MOE_E_SHAPE, "%s: H=%d and I=%d must be positive multiples of 32 up to 16384", who, H, I);
    if (E < 1 || E > kMaxE || k < 1 || k > E) return moe::fail(MOE_E_SHAPE, "%s: E=%d k=%d", who, E, k);
    if ((long long)T * k > kMaxPairs)
        return moe::fail(MOE_E_SHAPE, "%s: T*k=%lld above %d", who, (long long)T * k, kMaxPairs);
    if (!x || !topk_idx || !expert_table || !out || !workspace) return moe::fail(MOE_E_ARG, "%s: NULL pointer", who);
    if (((uintptr_t)x | (uintptr_t)shared_slab | (uintptr_t)out | (uintptr_t)workspace) % 16)
        return moe::fail(MOE_E_ARG, "%s: x, slabs, output and workspace must be 16-byte aligned", who);
    const size_t need = workspace_of(T, H, I, E, k, shared_slab != nullptr);
    if (workspace_bytes < need)
        return moe::fail(MOE_E_NOMEM, "%s: workspace %zu < %zu bytes", who, workspace_bytes, need);
    *sp = layout(T, H, I, E, k, shared_slab != nullptr);
    return MOE_OK;
}

}  // namespace

extern "C" size_t moe_expert_bytes_fp8(int hidden, int inter) {
    if (hidden <= 0 || inter <= 0 || hidden % 32 || inter % 32) return 0;
    return moe::fp8_slab_bytes(hidden, inter);
}

extern "C" size_t moe_fp8_expert_ffn_workspace_bytes(int T, int H, int I, int E, int k, int has_shared) {
    if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
    return workspace_of(T, H, I, E, k, has_shared != 0);
}

extern "C" int moe_fp8_expert_ffn(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx, int k,
                                  const void *const *expert_table, const void *shared_slab,
                                  const uint8_t *expert_mask, float *y, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    if (T < 0) return moe::fail(MOE_E_ARG, "fp8_expert_ffn: T=%d < 0", T);
    if (T == 0) return MOE_OK;
    Space sp{};
    const int rc = check("fp8_expert_ffn", x, T, H, I, E, topk_idx, k, expert_table, shared_slab, y, workspace,
                         workspace_bytes, &sp);
    if (rc != MOE_OK) return rc;
    return experts(x, T, H, I, E, topk_idx, k, expert_table, shared_slab, expert_mask, y, (uint8_t *)workspace, sp,
                   (hipStream_t)stream);
}

extern "C" int moe_fp8_expert_ffn_combine(const uint16_t *x, int T, int H, int I, int E, const int32_t *topk_idx,
                                          const float *topk_w, int k, const void *const *expert_table,
                                          const void *shared_slab, uint16_t *out, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    if (T < 0) return moe::fail(MOE_E_ARG, "fp8_expert_ffn_combine: T=%d < 0", T);
    if (T == 0) return MOE_OK;
    if (!topk_w) return moe::fail(MOE_E_ARG, "fp8_expert_ffn_combine: NULL pointer");
    Space sp{};
    int rc = check("fp8_expert_ffn_combine", x, T, H, I, E, topk_idx, k, expert_table, shared_slab, out, workspace,
                   workspace_bytes, &sp);
    if (rc != MOE_OK) return rc;
    float *y = (float *)((uint8_t *)workspace + sp.y);
    rc = experts(x, T, H, I, E, topk_idx, k, expert_table, shared_slab, nullptr, y, (uint8_t *)workspace, sp,
                 (hipStream_t)stream);
    if (rc != MOE_OK) return rc;
    return moe_combine(y, topk_w, T, k, H, shared_slab != nullptr, out, stream);
}
