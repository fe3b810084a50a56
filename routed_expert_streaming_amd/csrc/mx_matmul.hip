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
//  * MXFP4 rows: one load instruction brings a tile's 16 rows x 64 code bytes in
//    lane order (lane 16q + r: block q of row r), which is the order the products
//    read them in: 16 consecutive bytes per lane, no bank conflicts.
//  * bf16 rows: one instruction brings 4 rows x 256 bytes; the 16-byte piece p of
//    row m lies at place p ^ (m % 16), so that the 16 rows a product reads at one
//    piece number lie in different banks.
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

template <bool MX, int WM, int WN, int MT, int NT>
struct Tile {
    static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = WM * WN;
    static constexpr int W_BYTES = BN * 64, A_BYTES = BM * (MX ? 64 : 256), STAGE = W_BYTES + A_BYTES;
    static constexpr int SCALE_ROWS = BN + (MX ? BM : 0);  // rows of W, then rows of A
    static constexpr int SCALE_LOADS = (SCALE_ROWS + 63) / 64;
    static constexpr int SCALE_BYTES = SCALE_LOADS * 64 * 16;
    static constexpr int LOADS = STAGE / 1024;                    // load instructions of a group
    static constexpr int PER_WAVE = (LOADS + WAVES - 1) / WAVES;  // by each wave (some twice, see issue)
    static constexpr int SCALES_PER_WAVE = (SCALE_LOADS + WAVES - 1) / WAVES;
    static constexpr int STAGES = (160 * 1024 - 2 * SCALE_BYTES) / STAGE < 4 ? (160 * 1024 - 2 * SCALE_BYTES) / STAGE : 4;
    static constexpr int LDS = STAGES * STAGE + 2 * SCALE_BYTES;
    static_assert(STAGES >= 3 && LOADS >= WAVES && SCALE_ROWS <= 64 * WAVES, "tile does not fit its workgroup");
};

template <bool MX, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(64 * WM * WN) void mx_matmul_tile_kernel(MatArgs p, int m_tiles, int n_tiles) {
    using T = Tile<MX, WM, WN, MT, NT>;
    constexpr int AHEAD = T::STAGES - 1;
    __shared__ uint4 smem4[T::LDS / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    uint8_t *raw = smem + T::STAGES * T::STAGE;              // 16 scale bytes per row
    uint8_t *packed = raw + T::SCALE_BYTES;                  // four dwords per row, one per quarter
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    // consecutive workgroups go to the 8 XCDs in turn: each XCD takes a run of
    // neighbouring tiles, m fastest, so that its L2 holds the W rows they share
    const int tiles = m_tiles * n_tiles, per = (tiles + 7) / 8;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || tile >= tiles) return;
    const int m0 = tile % m_tiles * T::BM, n0 = tile / m_tiles * T::BN;
    const int ng = (p.K + kG - 1) / kG;
    const int nq = (p.K - (ng - 1) * kG) / 32;  // blocks of the last group
    const int m_last = min(T::BM, p.M - m0) - 1, n_last = min(T::BN, p.N - n0) - 1;
    const uint8_t *wbase = p.w + (size_t)n0 * p.w_stride, *abase = p.a + (size_t)m0 * p.a_stride;
    const uint32_t lds0 = lds_addr(smem), raw0 = lds_addr(raw);

    // the wave's load instructions of a group: number c < LOADS fills KB c of the
    // stage (W tiles first); past the end the wave repeats its previous one
    uint32_t off[T::PER_WAVE], cut[T::PER_WAVE];  // lane offsets; what the last group's lanes step back by
#pragma unroll
    for (int j = 0; j < T::PER_WAVE; ++j) {
        const int c0 = j * T::WAVES + wave, c = c0 < T::LOADS ? c0 : c0 - T::WAVES;
        if (c < T::W_BYTES / 1024) {
            off[j] = (uint32_t)min(16 * c + r, n_last) * (uint32_t)p.w_stride + 16 * q;
            cut[j] = 16 * (q - min(q, nq - 1));
        } else if (MX) {
            off[j] = (uint32_t)min(16 * (c - T::W_BYTES / 1024) + r, m_last) * (uint32_t)p.a_stride + 16 * q;
            cut[j] = 16 * (q - min(q, nq - 1));
        } else {
            const int m = 4 * (c - T::W_BYTES / 1024) + q, piece = r ^ (m & 15);
            off[j] = (uint32_t)min(m, m_last) * (uint32_t)p.a_stride + 16 * piece;
            cut[j] = 16 * (piece - min(piece, 4 * nq - 1));
        }
    }
    auto issue = [&](int g) {
        const uint32_t st = lds0 + (uint32_t)(g % T::STAGES) * T::STAGE;
        const bool last = g == ng - 1;
#pragma unroll
        for (int j = 0; j < T::PER_WAVE; ++j) {
            const int c0 = j * T::WAVES + wave, c = c0 < T::LOADS ? c0 : c0 - T::WAVES;
            const bool w = c < T::W_BYTES / 1024;
            const uint8_t *base = w ? wbase + 64 * (size_t)g : abase + (MX ? 64 : 256) * (size_t)g;
            dma16(base, last ? off[j] - cut[j] : off[j], st + 1024u * c);
        }
    };
    uint32_t soff[T::SCALES_PER_WAVE];
#pragma unroll
    for (int j = 0; j < T::SCALES_PER_WAVE; ++j) {
        const int c0 = j * T::WAVES + wave, c = c0 < T::SCALE_LOADS ? c0 : c0 % T::SCALE_LOADS;
        const int row = min(64 * c + lane, T::SCALE_ROWS - 1);
        soff[j] = row < T::BN ? (uint32_t)min(row, n_last) * (uint32_t)p.w_stride
                              : (uint32_t)min(row - T::BN, m_last) * (uint32_t)p.a_stride;
    }
    auto issue_scales = [&](int h) {  // of groups 4h .. 4h+3
#pragma unroll
        for (int j = 0; j < T::SCALES_PER_WAVE; ++j) {
            const int c0 = j * T::WAVES + wave, c = c0 < T::SCALE_LOADS ? c0 : c0 % T::SCALE_LOADS;
            const uint8_t *base = (64 * c < T::BN ? wbase : abase) + (size_t)p.K / 2 + 16 * (size_t)h;
            dma16(base, soff[j], raw0 + 1024u * c);
        }
    };
    static_assert(!MX || T::BN % 64 == 0, "a scale load is all W rows or all A rows");
    auto pack_scales = [&](int h) {
        if (tid >= T::SCALE_ROWS) return;
        const uint4 v = reinterpret_cast<const uint4 *>(raw)[tid];
        uint32_t d[4] = {v.x, v.y, v.z, v.w};  // d[b] byte q: group 4h + b, quarter q
        const int in = p.K / 32 - 16 * h;      // blocks that exist
        if (in < 16)
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (4 * b + k >= in) d[b] = (d[b] & ~(255u << 8 * k)) | 127u << 8 * k;
        // 4 x 4 byte transposition
        const uint32_t a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
        const uint32_t b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
        reinterpret_cast<uint4 *>(packed)[tid] =
            make_uint4(__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                       __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u));
    };

    f32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint32_t sw[NT], sa[MT];

    // issue order: scales 0, groups 0 .. AHEAD-1; then in group g: [scales of the
    // next four when g % 4 == 0], group g + AHEAD
    issue_scales(0);
    wait_vm<0>();
    for (int g = 0; g < AHEAD && g < ng; ++g) issue(g);
    ring_barrier();
    pack_scales(0);

    auto group = [&](int g, auto b_const) {
        constexpr int b = decltype(b_const)::value;  // g % 4
        // group g has landed once only the loads issued after it are in flight
        if (g + AHEAD - 1 < ng)
            wait_vm<(AHEAD - 1) * T::PER_WAVE>();
        else
            wait_vm<0>();
        ring_barrier();  // every wave's part of group g is there, and group g - 1 has been read
        if (b == 0 && g + 4 < ng) issue_scales(g / 4 + 1);
        if (g + AHEAD < ng) issue(g + AHEAD);
        if (b == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sw[t] = reinterpret_cast<const uint32_t *>(packed)[(wn * NT + t) * 64 + 4 * r + q];
            if (MX)
#pragma unroll
                for (int u = 0; u < MT; ++u)
                    sa[u] = reinterpret_cast<const uint32_t *>(packed)[4 * T::BN + (wm * MT + u) * 64 + 4 * r + q];
        }
        // the next four groups' scales: issued in this run's first group, so landed
        // with this one's loads (with AHEAD <= 3 they were issued before those)
        if (b == 3 && g + 1 < ng) pack_scales(g / 4 + 1);
        const uint8_t *st = smem + (size_t)(g % T::STAGES) * T::STAGE;
        const bool keep = g < ng - 1 || q < nq;
        uint4 w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            w[t] = zero_unless(keep, reinterpret_cast<const uint4 *>(st)[(wn * NT + t) * 64 + lane]);
        if constexpr (MX) {
            const uint4 *as = reinterpret_cast<const uint4 *>(st + T::W_BYTES) + wm * MT * 64 + lane;
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const uint4 x = as[u * 64];  // past K: finite codes times W's zeros
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][u] = mfma_mx<b>(w[t], x, acc[t][u], (int)sw[t], (int)sa[u]);
            }
        } else {
            const uint8_t *as = st + T::W_BYTES + (wm * MT * 16 + r) * 256;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8_t wv[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t c = s == 0 ? w[t].x : s == 1 ? w[t].y : s == 2 ? w[t].z : w[t].w;
                    wv[t] = codes_bf16(c, scale_f32(sw[t] >> 8 * b & 255u));
                }
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    const uint4 x = zero_unless(
                        keep, *reinterpret_cast<const uint4 *>(as + u * 16 * 256 + 16 * ((4 * q + s) ^ r)));
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv[t], __builtin_bit_cast(bf16x8_t, x), acc[t][u], 0, 0, 0);
                }
            }
        }
    };
    for (int g0 = 0; g0 < ng; g0 += 4)
        static_for<0, 4>([&](auto b) {
            if (g0 + decltype(b)::value < ng) group(g0 + decltype(b)::value, b);
        });
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            store4(p, m0 + (wm * MT + u) * 16 + r, n0 + (wn * NT + t) * 16 + 4 * q, acc[t][u]);
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
        launch_tile<MX, 2, 4, 8, 3>(p, s);
    else
        launch_tile<MX, 2, 4, 4, 4>(p, s);
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
