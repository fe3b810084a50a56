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

#ifndef MOE_TCFG
#define MOE_TCFG 2, 4, 8, 3
#endif
#ifndef MOE_BCFG
#define MOE_BCFG 2, 4, 4, 4
#endif
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

// One product of 16 x 16 x 128; byte B of ws / as is the lane's block's scale.
template <int B>
__device__ __forceinline__ f32x4_t mfma_mx(const uint4 w, const uint4 a, f32x4_t c, int ws, int as) {
    const i32x8_t wv{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const i32x8_t av{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, c, 4, 4, B, ws, B, as);  // 4: FP4 E2M1
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
                for (int t = 0; t < NT; ++t) acc[t][u] = mfma_mx<0>(w[t], x, acc[t][u], (int)ws[t], (int)xs);
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

// ---------------------------------------------------------------- many rows: tiles through LDS
// A workgroup owns BM x BN outputs (WM x WN waves of MT x NT tiles of 16 x 16) and
// walks K in groups of 128 columns through a ring of STAGES LDS stages, filled by
// direct global -> LDS loads STAGES - 1 groups ahead.
//  * MXFP4 rows next to MXFP4 rows: a stage is two groups, one load instruction 8
//    rows x 128 code bytes; next to bf16 rows a stage is one group, 16 rows x 64
//    bytes.  Eight neighbouring lanes on one 128-byte run take 37 cycles an
//    instruction, four on 64 bytes 50 (measured with the products left out), and
//    these loads are what bounds the kernel.
//  * bf16 rows: one instruction brings 4 rows x 256 bytes.
//  In all a row's 16-byte pieces change places by a key of the row (bank_key).
//  * scales: every fourth group, the 16 scale bytes of each row for the next four
//    groups come in raw (4 bytes per group, one per quarter) and one thread per
//    row turns them into one dword per quarter whose byte b belongs to group b:
//    the products select it by its number (MXFP4) or shift it out (bf16).
// The last group may end inside (K % 128 != 0): lanes past K load the last block
// again, their operands become zeros and their scales 1.
constexpr int kG = 128;          // columns of a group

typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ uint32_t lds_addr(const void *lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_u8 *)lds);
}
// Direct global -> LDS load of 16 bytes per lane: base (uniform) + off (this lane's
// byte offset) -> LDS byte lds + 16 * lane.  Inline asm, because the compiler would
// make every LDS read wait for all of these; the waits below count them instead
// (a wave's loads complete in order).  s_nop 4: the wait states a vector memory
// instruction needs after a VALU write of an SGPR it reads and after the M0 write.
__device__ __forceinline__ void dma16(const void *base, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
// Waits until at most N of the wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Workgroup barrier that leaves vector memory in flight; this wave's LDS accesses
// are done when it arrives.
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int N>
struct IntC {
    static constexpr int value = N;
};
template <int B, int E, class F>
__device__ __forceinline__ void static_for(F &&f) {
    if constexpr (B < E) {
        f(IntC<B>{});
        static_for<B + 1, E>(f);
    }
}

__device__ __forceinline__ uint4 zero_unless(bool keep, uint4 v) {
    return make_uint4(keep ? v.x : 0u, keep ? v.y : 0u, keep ? v.z : 0u, keep ? v.w : 0u);
}

// What the 16-byte pieces of row r of 16 are moved by (xor), for rows of 4, 8 or 16
// pieces: a wave's 16-byte LDS reads are served in sets of 16 lanes that take rows
// 0-3 and 12-15 from one quarter and rows 4-11 from the next (or the other way
// round); with these keys every such set, and 16 consecutive lanes too, falls into
// different banks (row-wise order measured 44% of the LDS cycles as conflicts).
template <int PIECES>
__device__ __forceinline__ int bank_key(int r) {
    const int k = 0x78 >> 2 * (r >> 2 & 3) & 3;  // 0 2 3 1 for rows 0-3, 4-7, 8-11, 12-15
    return PIECES == 4 ? k : PIECES == 8 ? k | (r >> 1 & 1) << 2 : k << 2 | (r & 3);
}

template <bool MX, int WM, int WN, int MT, int NT>
struct Tile {
    static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = WM * WN;
    static constexpr int KS = MX ? 2 : 1;                 // 128-column groups of a stage
    static constexpr int CODES = 64 * KS;                 // code bytes of a row of a stage
    static constexpr int A_ROW = MX ? CODES : 256 * KS;   // bytes of a row of A
    static constexpr int W_BYTES = BN * CODES, A_BYTES = BM * A_ROW, STAGE = W_BYTES + A_BYTES;
    static constexpr int SCALE_ROWS = BN + (MX ? BM : 0);  // rows of W, then rows of A
    static constexpr int RAW_LOADS = SCALE_ROWS / 16;      // load instructions of 16 groups' scales
    static constexpr int RAW_BYTES = SCALE_ROWS * 64, PACKED_BYTES = SCALE_ROWS * 16;
    static constexpr int W_LOADS = W_BYTES / 1024, LOADS = STAGE / 1024;  // load instructions of a stage
    static constexpr int PER_WAVE = (LOADS + WAVES - 1) / WAVES;          // by each wave (some twice, see issue)
    static constexpr int RAW_PER_WAVE = (RAW_LOADS + WAVES - 1) / WAVES;
    static constexpr int FIT = (160 * 1024 - RAW_BYTES - PACKED_BYTES) / STAGE, STAGES = FIT < 3 ? FIT : 3;
    static constexpr int RING = STAGES * STAGE, LDS = RING + RAW_BYTES + PACKED_BYTES;
    static_assert(STAGES >= 2 && LOADS >= WAVES && RAW_LOADS >= WAVES, "tile does not fit its workgroup");
};

// The sums of a workgroup's tile -> y, through the (now free) ring so that the
// stores are whole rows: the direct order, four n of 16 different m, took 10 us of a
// 2048 x 6144 output where whole rows take 4.  In as many parts of m as the ring's
// size asks for.
template <class T, int WN, int MT, int NT, typename OUT>
__device__ __forceinline__ void store_tile(const MatArgs &p, uint8_t *smem, int m0, int n0, int wm, int wn, int lane,
                                           const f32x4_t (&acc)[NT][MT]) {
    constexpr int PITCH = T::BN * (int)sizeof(OUT) + 16;
    constexpr int FULL = T::BM * PITCH, PARTS = FULL <= T::LDS ? 1 : FULL <= 2 * T::LDS ? 2 : 4;
    static_assert(MT % PARTS == 0 && FULL <= PARTS * T::LDS, "a part of the tile fits the LDS");
    constexpr int PM = MT / PARTS, ROWS = T::BM / PARTS;  // row tiles per wave, rows of a part
    constexpr int PER16 = 16 / (int)sizeof(OUT), UNITS = T::BN / PER16;
    const int r = lane & 15, q = lane >> 4;
    const bool wide = ((uintptr_t)p.y | p.y_stride) % 16 == 0;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        if (part) __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int nl = (wn * NT + t) * 16 + 4 * q;
            float b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = p.bias && n0 + nl + j < p.N ? p.bias[n0 + nl + j] : 0.0f;
#pragma unroll
            for (int u = 0; u < PM; ++u) {
                const f32x4_t v = acc[t][part * PM + u];
                uint8_t *o = smem + ((wm * PM + u) * 16 + r) * PITCH + nl * (int)sizeof(OUT);
                if constexpr (sizeof(OUT) == 4)
                    *reinterpret_cast<float4 *>(o) = make_float4(v[0] + b[0], v[1] + b[1], v[2] + b[2], v[3] + b[3]);
                else
                    *reinterpret_cast<uint2 *>(o) =
                        make_uint2(f32_to_bf16_bits(v[0] + b[0]) | f32_to_bf16_bits(v[1] + b[1]) << 16,
                                   f32_to_bf16_bits(v[2] + b[2]) | f32_to_bf16_bits(v[3] + b[3]) << 16);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < ROWS * UNITS; i += 64 * T::WAVES) {
            const int lr = i / UNITS, c = i - lr * UNITS;
            // row lr of the part: wave row lr / (16 * PM), its tile part * PM + ...
            const int m = m0 + lr / (16 * PM) * (16 * MT) + part * 16 * PM + lr % (16 * PM), n = n0 + c * PER16;
            if (m >= p.M || n >= p.N) continue;
            const uint4 v = *reinterpret_cast<const uint4 *>(smem + lr * PITCH + 16 * c);
            OUT *o = reinterpret_cast<OUT *>(p.y + (size_t)m * p.y_stride) + n;
            if (wide && n + PER16 <= p.N) {
                *reinterpret_cast<uint4 *>(o) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < PER16; ++j)
                    if (n + j < p.N) {
                        if constexpr (sizeof(OUT) == 4)
                            o[j] = __uint_as_float(w[j]);
                        else
                            o[j] = (OUT)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
                    }
            }
        }
    }
}

template <bool MX, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void
mx_matmul_tile_kernel(MatArgs p, int m_tiles, int n_tiles) {
    using T = Tile<MX, WM, WN, MT, NT>;
    constexpr int S = T::STAGES;
    __shared__ uint4 smem4[T::LDS / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    uint8_t *raw = smem + T::RING;            // 64 scale bytes per row: of 16 groups
    uint8_t *packed = raw + T::RAW_BYTES;     // four dwords per row, one per quarter: of 4 groups
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    // consecutive workgroups go to the 8 XCDs in turn: each XCD takes a run of
    // neighbouring tiles, m fastest, so that its L2 holds the W rows they share
    const int tiles = m_tiles * n_tiles, per = (tiles + 7) / 8;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= tiles) return;
    const int m0 = tile % m_tiles * T::BM, n0 = tile / m_tiles * T::BN;
    const int ng = (p.K + kG - 1) / kG, ns = (ng + T::KS - 1) / T::KS;  // groups, stages
    const int nq = (p.K - (ng - 1) * kG) / 32;              // blocks of the last group
    const int nb = nq + 4 * (ng - 1 - (ns - 1) * T::KS);    // blocks of the last stage
    const int m_last = min(T::BM, p.M - m0) - 1, n_last = min(T::BN, p.N - n0) - 1;
    const uint8_t *wbase = p.w + (size_t)n0 * p.w_stride, *abase = p.a + (size_t)m0 * p.a_stride;
    const uint32_t lds0 = lds_addr(smem), raw0 = lds_addr(raw);

    // the wave's load instructions of a stage: number c < LOADS fills KB c of the
    // stage (W rows first); past the end the wave repeats its previous one
    // (a wave's instructions take rows that are equal modulo 16, so its lanes keep
    // their pieces)
    static_assert(T::WAVES % 4 == 0, "rows of a wave's load instructions modulo 16");
    constexpr int PIECES = T::CODES / 16, ROWS = 64 / PIECES;  // of a row of codes; rows of an instruction
    const int piece = (lane % PIECES) ^ bank_key<PIECES>(wave * ROWS + lane / PIECES);
    const int piece_a = MX ? piece : r ^ bank_key<16>(4 * (wave - T::W_LOADS) + q);
    // what the last stage's lanes step back by, past K
    const uint32_t cut = 16 * (piece - min(piece, nb - 1)), cut_a = MX ? cut : 16 * (piece_a - min(piece_a, 4 * nb - 1));
    uint32_t off[T::PER_WAVE];
#pragma unroll
    for (int j = 0; j < T::PER_WAVE; ++j) {
        const int c0 = j * T::WAVES + wave, c = c0 < T::LOADS ? c0 : c0 - T::WAVES;
        if (c < T::W_LOADS)
            off[j] = (uint32_t)min(c * ROWS + lane / PIECES, n_last) * (uint32_t)p.w_stride + 16 * piece;
        else
            off[j] = (uint32_t)min(MX ? (c - T::W_LOADS) * ROWS + lane / PIECES : 4 * (c - T::W_LOADS) + q, m_last) *
                         (uint32_t)p.a_stride +
                     16 * piece_a;
    }
    // the wave's instruction j of stage i, into the place of stage `as`
    auto issue_one = [&](int i, int as, int j) {
        const int c0 = j * T::WAVES + wave, c = c0 < T::LOADS ? c0 : c0 - T::WAVES;
        const uint8_t *base = c < T::W_LOADS ? wbase + T::CODES * (size_t)i : abase + T::A_ROW * (size_t)i;
        dma16(base, off[j] - (i == ns - 1 ? c < T::W_LOADS ? cut : cut_a : 0u), lds0 + (uint32_t)(as % S) * T::STAGE + 1024u * c);
    };
    // scales: an instruction brings 64 bytes of each of 16 rows (places past the row's
    // last 16 bytes repeat those)
    const int nr = (ng + 3) / 4;                      // runs of four groups
    const int last16 = ((p.K / 32 + 15) / 16 - 1);    // last 16 scale bytes of a row
    auto issue_scales = [&](int h) __attribute__((always_inline)) {  // of runs h .. h + 3 (h % 4 == 0)
#pragma unroll
        for (int j = 0; j < T::RAW_PER_WAVE; ++j) {
            const int c0 = j * T::WAVES + wave, c = c0 < T::RAW_LOADS ? c0 : c0 - T::WAVES;
            const bool isw = 16 * c < T::BN;
            const int row = 16 * c + (lane >> 2) - (isw ? 0 : T::BN);
            const uint32_t at = (uint32_t)min(row, isw ? n_last : m_last) * (uint32_t)(isw ? p.w_stride : p.a_stride);
            const uint8_t *base = (isw ? wbase : abase) + (size_t)p.K / 2 + 16 * (size_t)h;
            dma16(base, at + 16 * min(lane & 3, last16 - h), raw0 + 1024u * c);
        }
    };
    auto pack_scales = [&](int h) __attribute__((always_inline)) {
        const int in = p.K / 32 - 16 * h;  // blocks that exist (none past the last run)
#pragma unroll
        for (int row0 = 0; row0 < T::SCALE_ROWS; row0 += 64 * T::WAVES) {
            const int row = min(row0 + tid, T::SCALE_ROWS - 1);  // several threads write the last row alike
            const uint4 v = reinterpret_cast<const uint4 *>(raw)[4 * row + (h & 3)];
            uint32_t d[4] = {v.x, v.y, v.z, v.w};  // d[b] byte k: group 4h + b, quarter k
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int n = min(max(in - 4 * b, 0), 4);
                const uint32_t keep = n == 4 ? ~0u : (1u << 8 * n) - 1u;
                d[b] = (d[b] & keep) | (0x7F7F7F7Fu & ~keep);
            }
            // 4 x 4 byte transposition
            const uint32_t a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u);
            const uint32_t a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
            const uint32_t b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
            const uint32_t b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
            reinterpret_cast<uint4 *>(packed)[row] =
                make_uint4(__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                           __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u));
        }
    };

    f32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // Operands in registers.  A's are read again for the next group (MXFP4) or the
    // next product of the group (bf16: a quarter of it) right after the products that
    // used them, tile by tile between the products of the other tiles; W's alternate.
    uint4 w[2][NT], x[MT];
    uint32_t sw[NT], sa[MT], sw_next[NT];
    const uint8_t *w_at = smem + (wn * NT * 16 + r) * T::CODES;
    const uint8_t *x_at = smem + T::W_BYTES + (wm * MT * 16 + r) * T::A_ROW;
    const uint32_t *scale_at = reinterpret_cast<const uint32_t *>(packed) + 4 * r + q;
    auto stage_of = [&](int g) { return (uint32_t)(g / T::KS % S) * T::STAGE; };
    auto read_w = [&](int g, int t) {
        return *reinterpret_cast<const uint4 *>(w_at + stage_of(g) + t * 16 * T::CODES +
                                                16 * ((4 * (g % T::KS) + q) ^ bank_key<PIECES>(r)));
    };
    auto read_x = [&](int g, int s, int u) {
        const int piece = MX ? (4 * (g % T::KS) + q) ^ bank_key<PIECES>(r) : (4 * q + s) ^ bank_key<16>(r);
        return *reinterpret_cast<const uint4 *>(x_at + stage_of(g) + u * 16 * T::A_ROW + 16 * piece);
    };
    auto read_sw = [&](int t) { return scale_at[(wn * NT + t) * 64]; };
    auto read_sa = [&](int u) { return scale_at[4 * T::BN + (wm * MT + u) * 64]; };
    // the last group's quarters past K become zeros: W's (A's MXFP4 codes are finite
    // whatever was read) and bf16 A's
    auto cut_w = [&](uint4 (&d)[NT]) {
        if (nq < 4)
#pragma unroll
            for (int t = 0; t < NT; ++t) d[t] = zero_unless(q < nq, d[t]);
    };
    auto cut_x = [&]() {
        if (!MX && nq < 4)
#pragma unroll
            for (int u = 0; u < MT; ++u) x[u] = zero_unless(q < nq, x[u]);
    };

    // Issue order, which the waits count on: scales of runs 0 .. 3, stages 0 .. S-1,
    // then at the turn from stage i to i + 1: [four runs' scales], stage i + S.  Past
    // the last stage the last one is loaded again, into the places no one reads any
    // more, so that the loop needs no branch.
    issue_scales(0);
    wait_vm<0>();
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < T::PER_WAVE; ++j) issue_one(min(i, ns - 1), i, j);
    ring_barrier();
    pack_scales(0);
    wait_vm<(S - 1) * T::PER_WAVE>();
    ring_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t) w[0][t] = read_w(0, t), sw[t] = sw_next[t] = read_sw(t);
#pragma unroll
    for (int u = 0; u < MT; ++u) x[u] = read_x(0, 0, u), sa[u] = MX ? read_sa(u) : 0u;

    // The turn to the next stage: it has landed once only the loads issued after it
    // are in flight.  Every wave's operands of this stage are in registers when it
    // arrives (its LDS reads are done), so stage i + S may overwrite it.
    auto turn = [&](int g) {
        wait_vm<(S - 2) * T::PER_WAVE>();
        ring_barrier();
        // the scales of runs 4j .. 4j+3 have all been packed two stages ago
        if (g % 16 == 11 && g / 4 + 2 < nr) issue_scales(g / 4 + 2);
    };
    // keeps the products of tile column u ahead of the LDS reads that follow in the
    // source (and their sums in place): left to itself the compiler gathers reads
    // and products of two groups and spills
    auto pin = [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(acc[t][u])::"memory");
    };
    // group g, with the operands of group g + 1 read on the way (garbage past the
    // last one: the reads stay inside the ring); last: g is the last group
    auto group = [&](int g, auto b_const, bool last) __attribute__((always_inline)) {
        constexpr int b = decltype(b_const)::value, cur = b & 1, nxt = cur ^ 1;  // b = g % 4
        constexpr bool turns = (b + 1) % T::KS == 0;
        const int i = g / T::KS;
        if constexpr (MX) {
#pragma unroll
            for (int u = 0; u < MT; ++u) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][u] = mfma_mx<b>(w[cur][t], x[u], acc[t][u], (int)sw[t], (int)sa[u]);
                pin(u);
                if (turns && u == 0) turn(g);
                if (u < NT) {
                    w[nxt][u] = read_w(g + 1, u);
                    if (b == 3) sw_next[u] = read_sw(u);
                }
                x[u] = read_x(g + 1, 0, u);
                if (b == 3) sa[u] = read_sa(u);
                if (turns)
#pragma unroll
                    for (int j = 0; j < T::PER_WAVE; ++j)
                        if (j % MT == u) issue_one(min(i + S, ns - 1), i + S, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            bf16x8_t wv[2][NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) wv[0][t] = codes_bf16(w[cur][t].x, scale_f32(sw[t] >> 8 * b & 255u));
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int u = 0; u < MT; ++u) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv[s & 1][t], __builtin_bit_cast(bf16x8_t, x[u]), acc[t][u], 0, 0, 0);
                    pin(u);
                    if (s == 3 && u == 0) turn(g);
                    if (s == 3)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (t % MT == u) {
                                w[nxt][t] = read_w(g + 1, t);
                                if (b == 3) sw_next[t] = read_sw(t);
                            }
                    x[u] = s < 3 ? read_x(g, s + 1, u) : read_x(g + 1, 0, u);
                    if (s < 3)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (t % MT == u)
                                wv[(s + 1) & 1][t] = codes_bf16(s == 0 ? w[cur][t].y : s == 1 ? w[cur][t].z : w[cur][t].w,
                                                                scale_f32(sw[t] >> 8 * b & 255u));
                    if (s == 3)
#pragma unroll
                        for (int j = 0; j < T::PER_WAVE; ++j)
                            if (j % MT == u) issue_one(min(i + S, ns - 1), i + S, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (last && s < 3) cut_x();
            }
        }
        // the next run's scales: in since the wait above; shown to all by the barrier
        // at this run's end
        if (b == 3 - T::KS) pack_scales(g / 4 + 1);
        if (b == 3)
#pragma unroll
            for (int t = 0; t < NT; ++t) sw[t] = sw_next[t];
    };
    int g = 0;
    for (; g + 4 < ng; g += 4) static_for<0, 4>([&](auto b) { group(g + decltype(b)::value, b, false); });
    // the last 1 to 4 groups
    static_for<0, 4>([&](auto b_const) {
        constexpr int b = decltype(b_const)::value;
        if (g + b < ng) {
            const bool last = g + b == ng - 1;
            if (last) cut_w(w[b & 1]), cut_x();
            group(g + b, b_const, last);
        }
    });
    wait_vm<0>();     // no load may still write the ring
    __syncthreads();  // the ring becomes the output's staging
    if (p.y_f32)
        store_tile<T, WN, MT, NT, float>(p, smem, m0, n0, wm, wn, lane, acc);
    else
        store_tile<T, WN, MT, NT, uint16_t>(p, smem, m0, n0, wm, wn, lane, acc);
}

template <bool MX, int MT, int NT, int WM, int WN, int WK>
void launch_direct(const MatArgs &p, hipStream_t s) {
    const dim3 grid((p.N + 16 * NT * WN - 1) / (16 * NT * WN), (p.M + 16 * MT * WM - 1) / (16 * MT * WM));
    hipLaunchKernelGGL((mx_matmul_direct_kernel<MX, MT, NT, WM, WN, WK>), grid, dim3(64 * WM * WN * WK), 0, s, p);
}

template <bool MX, int WM, int WN, int MT, int NT>
void launch_tile(const MatArgs &p, hipStream_t s) {
    using T = Tile<MX, WM, WN, MT, NT>;
    const int m_tiles = (p.M + T::BM - 1) / T::BM, n_tiles = (p.N + T::BN - 1) / T::BN;
    const unsigned grid = (unsigned)(((int64_t)m_tiles * n_tiles + 7) / 8 * 8);
    hipLaunchKernelGGL((mx_matmul_tile_kernel<MX, WM, WN, MT, NT>), dim3(grid), dim3(64 * T::WAVES), 0, s, p,
                       m_tiles, n_tiles);
}

template <bool MX>
void launch(const MatArgs &p, hipStream_t s) {
    // a tile's lane offsets are 32 bits: rows further apart take the direct kernel
    const bool near = p.w_stride < (8u << 20) && p.a_stride < (8u << 20);
    if (p.M <= 16)
        launch_direct<MX, 1, 1, 1, 1, 4>(p, s);
    else if (p.M <= 64 || !near)
        launch_direct<MX, 4, 4, 2, 2, 1>(p, s);
    else if constexpr (MX)
        launch_tile<MX, MOE_TCFG>(p, s);
    else
        launch_tile<MX, MOE_BCFG>(p, s);
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
