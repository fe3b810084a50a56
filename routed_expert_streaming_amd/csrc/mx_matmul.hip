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
// stores together.  Sums are fp32; waves and parts that split K are joined in a fixed
// order.
//
// Three families, chosen by plan(): up to 16 rows of A (bound by W's bytes), up to
// about 64 (W's bytes and A's re-reads), more (LDS tiles, bound by the loads into LDS,
// then by the matrix cores).
#include "common.h"
#include "dequant.h"
#include "lds_dma.h"
#include "mx_quant.h"

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int64_t kMaxStride = 1 << 28;  // 16 rows' offsets stay in 32 bits
constexpr int kMaxRows = 1 << 26;        // M and N: a rows kernel's grid stays below 2^32 threads
constexpr int kMaxK = 1 << 27;

struct MatArgs {
    const uint8_t *a, *w;
    size_t a_stride, w_stride;  // bytes between rows
    int M, N, K;
    const float *bias;
    uint8_t *y;
    size_t y_stride;
    bool y_f32;
};

// 8 consecutive weights (one dword of codes) -> bf16, times 2^(v-127) as the converts take it
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t c, float scale) {
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
    const uint32_t w2 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
    const uint32_t w3 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
    return __builtin_bit_cast(bf16x8_t, make_uint4(w0, w1, w2, w3));
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
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) o[j] = (uint16_t)pack_bf16(f[j], 0.0f);
        }
    }
}

__device__ __forceinline__ uint4 zero_unless(bool keep, uint4 v) {
    return make_uint4(keep ? v.x : 0u, keep ? v.y : 0u, keep ? v.z : 0u, keep ? v.w : 0u);
}

// This lane's part of 512 columns (run h) of an MXFP4 row: blocks 16h + 4q .. + 3.
struct Run {
    uint4 c[4];
    uint32_t s;  // byte j: block j's scale
};
// Rows row0 .. row0 + 15 of an operand (those past the last repeat it): a uniform base
// and this lane's offset, row r's codes from column 128q on.
struct Rows {
    const uint8_t *base;
    uint32_t off;
};
__device__ __forceinline__ Rows rows_at(const uint8_t *m, size_t stride, int row0, int rows, int r, int q) {
    const int first = min(row0, rows - 1);
    return {m + (size_t)first * stride, (uint32_t)min(r, rows - 1 - first) * (uint32_t)stride + 64u * q};
}
// (blocks past K repeat the row's last one; the scale dword lies inside the row, whose
// scales are padded to 16 bytes)
__device__ __forceinline__ Run load_run(const MatArgs &p, const Rows &m, int h, int q) {
    Run v;
    const int n = p.K / 32 - 16 * h;  // blocks of the run
    const uint8_t *c = m.base + 256 * (size_t)h;
    if (n >= 16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v.c[j] = load_global_u4(c + m.off + 16 * j);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v.c[j] = load_global_u4(c + m.off - 64u * q + 16u * min(4 * q + j, n - 1));
    }
    v.s = load_stream_u32(m.base + (size_t)p.K / 2 + 16 * (size_t)h + (m.off - 60u * q));
    return v;
}
// blocks past K: zeros, scale 1
__device__ __forceinline__ void cut_run(const MatArgs &p, Run &v, int h, int q) {
    const int n = p.K / 32 - (16 * h + 4 * q);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j >= n) {
            v.c[j] = make_uint4(0u, 0u, 0u, 0u);
            v.s = (v.s & ~(255u << 8 * j)) | 127u << 8 * j;
        }
}
// The compiler waits for these loads here (and not later, behind loads issued since).
__device__ __forceinline__ void wait_run(Run &v) {
    asm volatile("" : "+v"(v.c[0].x), "+v"(v.c[1].x), "+v"(v.c[2].x), "+v"(v.c[3].x), "+v"(v.s));
}
// acc += a run of W times the same run of bf16 A, whose rows lie kXRow bytes apart in
// LDS: 16 more than a run, so that 16 rows' 16-byte pieces lie in different banks.
// xs: this lane's row and quarter.
constexpr int kXRow = 1040;
template <int MT, int NT>
__device__ __forceinline__ void multiply_run(const Run (&w)[NT], const uint8_t *(&xs)[MT], f32x4_t (&acc)[NT][MT]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float sc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[t] = moe::mx_scale_operand(w[t].s >> 8 * j & 255u);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf16x8_t wv[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 c = w[t].c[j];
                wv[t] = codes_bf16(s == 0 ? c.x : s == 1 ? c.y : s == 2 ? c.z : c.w, sc[t]);
            }
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xs[u] + 64 * j + 16 * s);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[t], __builtin_bit_cast(bf16x8_t, x),
                                                                        acc[t][u], 0, 0, 0);
            }
        }
    }
}
// Run h of a row of bf16 A into LDS (lane l: its 16-byte piece l; past K the last one).
__device__ __forceinline__ void dma_run(const MatArgs &p, int m, int h, int lane, uint32_t lds) {
    const int pieces = p.K / 8 - 64 * h;
    dma16(p.a + (size_t)m * p.a_stride + 1024 * (size_t)h, 16 * min(lane, pieces - 1), lds);
}
// Zeros past K in the last run of `rows` rows at xs, once it is there.
__device__ __forceinline__ void zero_past_k(const MatArgs &p, uint8_t *xs, int rows, int h, int lane) {
    if (8 * lane >= p.K - 512 * h)
        for (int m = 0; m < rows; ++m)
            *reinterpret_cast<uint4 *>(xs + m * kXRow + 16 * lane) = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------- few rows: W straight into registers
// One workgroup owns 16 * MT rows of A and 16 * NT rows of W; its WK waves split K
// in runs of 512 columns (wave k takes runs k, k + WK, ...) and their sums are
// joined through LDS, in wave order.  In a run lane 16q + r holds blocks 4q .. 4q+3
// of row r: 64 code bytes and one dword of scales, so a row's 256 bytes are read as
// whole lines, and product j takes block 4q + j from every quarter.  W is read once
// from memory, the next run's while this one is multiplied; A comes from the caches.
// 1 x 65536 x 4096 in MXFP4 takes 30 us (142 MB, 4.7 TB/s; a large copy reaches 4.9),
// 32 x 6144 x 6144 8.3 us (2.5 TB/s: 192 workgroups, whose 8 waves have 12 runs between
// them, and A's run is loaded only where it is used).  K split over the waves of a workgroup, not whole rows to
// each, because 16 whole rows at a time keep the memory's pages open: with the same
// loads alone a workgroup over 16 rows read 5.8 TB/s, one over 64 rows 4.0.
// Rows past M or N repeat the last row (their results are not stored); blocks past K
// repeat the row's last block, as zeros.
//
// bf16 A: a run of a row is 1 KB, one direct global -> LDS load into the wave's own
// rows (XR of them, two runs in turn).  32 rows of two waves fill a CU's LDS, and two of
// its SIMDs have no wave: 32 x 6144 x 6144 14.9 us, bound by six turns one after the other.
template <bool MX, int MT, int NT, int WK, int XR>
__global__ __launch_bounds__(64 * WK) void mx_matmul_rows_kernel(MatArgs p) {
    static_assert(MX || XR <= 16 * MT, "rows of A in LDS");
    constexpr int XBUF = MX ? 0 : WK * 2 * XR * kXRow, JOIN = WK * NT * MT * 1024;
    __shared__ uint4 smem4[(XBUF > JOIN ? XBUF : JOIN) / 16];
    uint8_t *smem = reinterpret_cast<uint8_t *>(smem4);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int m0 = blockIdx.y * 16 * MT, n0 = blockIdx.x * 16 * NT;
    const int blocks = p.K / 32, runs = (blocks + 15) / 16, xrows = min(XR, p.M - m0);
    Rows wr[NT], ar[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) wr[t] = rows_at(p.w, p.w_stride, n0 + 16 * t, p.N, r, q);
#pragma unroll
    for (int u = 0; u < MT; ++u) ar[u] = rows_at(p.a, p.a_stride, m0 + 16 * u, p.M, r, q);
    f32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    uint8_t *xw = smem + wave * (2 * XR * kXRow);
    const uint32_t xbuf = lds_addr(smem) + (uint32_t)wave * (2 * XR * kXRow);
    auto load_x = [&](int h, int i) __attribute__((always_inline)) {  // run h of A into buffer i of the wave
        for (int m = 0; m < xrows; ++m) dma_run(p, m0 + m, h, lane, xbuf + (uint32_t)(i * XR + m) * kXRow);
    };
    // With one tile the waves themselves are enough in flight (72 registers, three
    // workgroups a CU: 1 x 65536 x 4096 29.5 us; with the next run too, 85 registers
    // and two, 35 us).
    constexpr bool AHEAD = !MX || NT * MT > 1;
    Run w[NT];
    if (AHEAD && wave < runs) {
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t] = load_run(p, wr[t], wave, q);
        if (!MX) load_x(wave, 0);
    }
    int buf = 0;
    for (int h = wave; h < runs; h += WK, buf ^= 1) {
        const bool last = h == runs - 1 && blocks % 16 != 0;
        if (!MX) {
            wait_vm<0>();
            if (last) zero_past_k(p, xw + buf * XR * kXRow, xrows, h, lane);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (AHEAD)
                wait_run(w[t]);
            else
                w[t] = load_run(p, wr[t], h, q);
        Run next[NT];
        if (AHEAD && h + WK < runs) {
#pragma unroll
            for (int t = 0; t < NT; ++t) next[t] = load_run(p, wr[t], h + WK, q);
            if (!MX) load_x(h + WK, buf ^ 1);
        }
        if (last)
#pragma unroll
            for (int t = 0; t < NT; ++t) cut_run(p, w[t], h, q);
        if constexpr (MX) {
            Run x[MT];
#pragma unroll
            for (int u = 0; u < MT; ++u) x[u] = load_run(p, ar[u], h, q);
            if (last)
#pragma unroll
                for (int u = 0; u < MT; ++u) cut_run(p, x[u], h, q);
            static_for<0, 4>([&](auto j_const) __attribute__((always_inline)) {
                constexpr int j = decltype(j_const)::value;
#pragma unroll
                for (int u = 0; u < MT; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[t][u] = mfma_mx<j>(w[t].c[j], x[u].c[j], acc[t][u], (int)w[t].s, (int)x[u].s);
            });
        } else {
            const uint8_t *xs[MT];
#pragma unroll
            for (int u = 0; u < MT; ++u) xs[u] = xw + (buf * XR + min(16 * u + r, xrows - 1)) * kXRow + 256 * q;
            multiply_run<MT, NT>(w, xs, acc);
        }
        if (AHEAD)
#pragma unroll
            for (int t = 0; t < NT; ++t) w[t] = next[t];
    }
    // join: tile i is summed by wave i % WK
    if (!MX) __syncthreads();  // the rows of A are read
    f32x4_t(*part)[NT * MT][64] = reinterpret_cast<f32x4_t(*)[NT * MT][64]>(smem);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) part[wave][t * MT + u][lane] = acc[t][u];
    __syncthreads();
#pragma unroll
    for (int i0 = 0; i0 < NT * MT; i0 += WK) {
        const int i = i0 + wave;
        if (i >= NT * MT) break;
        f32x4_t v = part[0][i][lane];
#pragma unroll
        for (int k = 1; k < WK; ++k) v += part[k][i][lane];
        store4(p, m0 + 16 * (i % MT) + r, n0 + 16 * (i / MT) + 4 * q, v);
    }
}

// bf16 A of at most 16 rows that fit LDS (KB of it) whole: the workgroup brings them in
// once and goes over tiles of 16 rows of W, blockIdx.x, + gridDim.x, ..., its waves
// sharing each tile's runs as above, the next tile's W in flight while this one is
// joined.  4 x 65536 x 4096 (fp32 y): 32 us, 4.5 TB/s over W; from global memory, 16
// scattered loads a run, 42 us, and with A brought in for each tile 40 us.  Four waves
// and three workgroups a CU: eight waves each took 35 us, four workgroups 42 (the last
// of 16 tiles a CU then runs alone).  1 x 4096 x 4096, one tile a CU, takes 4.2 us: A, then
// two runs a wave one after the other, then the join, each a latency.
template <int WK, int KB>
__global__ __launch_bounds__(64 * WK) void mx_matmul_few_kernel(MatArgs p, int tiles) {
    __shared__ uint4 xs4[KB * 64];
    __shared__ f32x4_t part[2][WK][64];
    uint8_t *xs = reinterpret_cast<uint8_t *>(xs4);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int blocks = p.K / 32, runs = (blocks + 15) / 16;
    Rows wr = rows_at(p.w, p.w_stride, 16 * blockIdx.x, p.N, r, q);
    Run w[1];
    if (wave < runs) w[0] = load_run(p, wr, wave, q);
    const uint32_t lds0 = lds_addr(xs);
    for (int h = wave; h < runs; h += WK)
        for (int m = 0; m < p.M; ++m) dma_run(p, m, h, lane, lds0 + (uint32_t)(h * p.M + m) * kXRow);
    wait_vm<0>();  // a wave reads only what it loaded itself
    if (blocks % 16 != 0 && (runs - 1) % WK == wave)
        zero_past_k(p, xs + (size_t)(runs - 1) * p.M * kXRow, p.M, runs - 1, lane);
    const uint8_t *xrow = xs + min(r, p.M - 1) * kXRow + 256 * q;
    int i = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++i) {
        f32x4_t acc[1][1] = {{f32x4_t{0.f, 0.f, 0.f, 0.f}}};
        const Rows here = wr;
        wr = rows_at(p.w, p.w_stride, 16 * min(tile + (int)gridDim.x, tiles - 1), p.N, r, q);
        for (int h = wave; h < runs; h += WK) {
            wait_run(w[0]);
            Run now[1] = {w[0]};
            const bool more = h + WK < runs;
            w[0] = load_run(p, more ? here : wr, more ? h + WK : wave, q);  // the next run, or tile
            const bool last = h == runs - 1 && blocks % 16 != 0;
            if (last) cut_run(p, now[0], h, q);
            const uint8_t *x[1] = {xrow + (size_t)h * p.M * kXRow};
            multiply_run<1, 1>(now, x, acc);
        }
        // join, in two buffers in turn, so that one barrier a tile is enough; another
        // wave each time
        part[i & 1][wave][lane] = acc[0][0];
        ring_barrier();
        if (wave == i % WK) {
            f32x4_t v = part[i & 1][0][lane];
#pragma unroll
            for (int k = 1; k < WK; ++k) v += part[i & 1][k][lane];
            store4(p, r, tile * 16 + 4 * q, v);
        }
    }
}

// ---------------------------------------------------------------- many rows: tiles through LDS
// A workgroup owns BM x BN outputs (WM x WN waves of MT x NT tiles of 16 x 16) and
// walks K in groups of 128 columns through a ring of STAGES LDS stages, filled by
// direct global -> LDS loads.
//  * MXFP4 rows next to MXFP4 rows: a stage is two groups, one load instruction 8
//    rows x 128 code bytes; next to bf16 rows a stage is one group, 16 rows x 64
//    bytes.  Eight neighbouring lanes on one 128-byte run take 37 cycles an
//    instruction, four on 64 bytes 50 (measured with the products left out).
//  * bf16 rows: one instruction brings 4 rows x 256 bytes.
//  In all a row's 16-byte pieces change places by a key of the row (bank_key).
//  * scales: every 16 groups, 64 scale bytes of each row come in raw (16 bytes a row and
//    load, as every four groups, cost a tenth of the time), and every four groups one
//    thread per row turns 16 of them into one dword per quarter whose byte b belongs to
//    group b: the products select it by its number (MXFP4) or shift it out (bf16).
// Measured, 2048 x 6144 x 6144 in MXFP4, 256 x 192 tiles, one a CU: 44 us, 3.5
// PFLOP/s.  A 128-column group takes 0.63 us; its products alone 0.45, of which the
// matrix cores are busy 0.35 (a scaled FP4 product takes 16 cycles of them: in
// registers two waves a SIMD issue one every 16.7, 8.0 PFLOP/s at the 2.04 GHz that
// the card then runs at, one wave every 17.5); its loads alone 0.35, and the 88 KB of
// LDS reads and 28 KB of LDS writes 0.39 at 128 bytes a cycle: the three share issue
// and LDS.  Prologue and epilogue take about 10 us of it.  2048 x 4096 x 6144 with
// bf16 A, 128 x 256 tiles: 80 us, 1.29 PFLOP/s (bf16 products reach 2.1 in registers; a
// library product of bf16 matrices of these sizes took 102 us).
// The last group may end inside (K % 128 != 0): lanes past K load the last block
// again, their operands become zeros and their scales 1.
constexpr int kG = 128;          // columns of a group

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
    static_assert(STAGES >= 2 && LOADS >= WAVES, "tile does not fit its workgroup");
};

// The sums of a workgroup's tile -> y, through the (now free) ring so that the
// stores are whole rows: in the registers' order, four n of 16 different m, a 2048 x
// 6144 output took 10 us, as whole rows 4.  In as many parts of m as the ring's size
// asks for.  Kept short: it runs once, from a cold instruction cache.
template <class T, int MT, int NT, typename OUT>
__device__ __forceinline__ void store_tile(const MatArgs &p, uint8_t *smem, int m0, int n0, int wm, int wn, int lane,
                                           const f32x4_t (&acc)[NT][MT]) {
    constexpr int PITCH = T::BN * (int)sizeof(OUT) + 16;
    constexpr int FULL = T::BM * PITCH, PARTS = FULL <= T::LDS ? 1 : FULL <= 2 * T::LDS ? 2 : 4;
    static_assert(MT % PARTS == 0 && FULL <= PARTS * T::LDS, "a part of the tile fits the LDS");
    constexpr int PM = MT / PARTS, ROWS = T::BM / PARTS;  // row tiles per wave, rows of a part
    constexpr int PER16 = 16 / (int)sizeof(OUT), UNITS = T::BN / PER16, THREADS = 64 * T::WAVES;
    constexpr int AT_ONCE = ROWS * UNITS % (4 * THREADS) == 0 ? 4 : ROWS * UNITS % (2 * THREADS) == 0 ? 2 : 1;
    static_assert(ROWS * UNITS % (AT_ONCE * THREADS) == 0, "whole rounds of stores");
    const int r = lane & 15, q = lane >> 4;
    // 16 bytes at a time where every row begins and ends on such a piece
    const bool wide = ((uintptr_t)p.y | p.y_stride) % 16 == 0 && p.N % PER16 == 0;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        if (part) __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < PM; ++u) {
                const f32x4_t v = acc[t][part * PM + u];
                uint8_t *o = smem + ((wm * PM + u) * 16 + r) * PITCH + ((wn * NT + t) * 16 + 4 * q) * (int)sizeof(OUT);
                if constexpr (sizeof(OUT) == 4)
                    *reinterpret_cast<f32x4_t *>(o) = v;
                else
                    *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
        __syncthreads();
        // row lr of the part: wave row lr / (16 * PM), its tiles part * PM and up
        auto row_of = [&](int lr) { return m0 + lr / (16 * PM) * (16 * MT) + part * 16 * PM + lr % (16 * PM); };
        if (wide) {
#pragma unroll 1
            for (int i0 = threadIdx.x; i0 < ROWS * UNITS; i0 += AT_ONCE * THREADS) {
                uint4 v[AT_ONCE];
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) {
                    const int i = i0 + e * THREADS;
                    v[e] = *reinterpret_cast<const uint4 *>(smem + i / UNITS * PITCH + 16 * (i % UNITS));
                }
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) {
                    const int i = i0 + e * THREADS, m = row_of(i / UNITS), n = n0 + i % UNITS * PER16;
                    if (m < p.M && n < p.N)
                        *reinterpret_cast<uint4 *>(p.y + (size_t)m * p.y_stride + (size_t)n * sizeof(OUT)) = v[e];
                }
            }
        } else {  // value by value, a wave on neighbouring ones
            const int cols = min(T::BN, p.N - n0);
            for (int lr = threadIdx.x / 64; lr < ROWS; lr += T::WAVES) {
                const int m = row_of(lr);
                if (m >= p.M) continue;
                OUT *o = reinterpret_cast<OUT *>(p.y + (size_t)m * p.y_stride) + n0;
                const OUT *v = reinterpret_cast<const OUT *>(smem + lr * PITCH);
                for (int n = lane; n < cols; n += 64) o[n] = v[n];
            }
        }
    }
}

template <bool MX, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4))) void
mx_matmul_tile_kernel(MatArgs p, int m_tiles, int n_tiles, int k_part) {
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
    const int m_last = min(T::BM, p.M - m0) - 1, n_last = min(T::BN, p.N - n0) - 1;
    // this workgroup's columns k0 .. k0 + K - 1 (k_part a multiple of 512: whole runs of scales)
    const int k0 = blockIdx.y * k_part, K = min(k_part, p.K - k0);
    const uint8_t *wbase = p.w + (size_t)n0 * p.w_stride + k0 / 2;
    const uint8_t *abase = p.a + (size_t)m0 * p.a_stride + (MX ? (size_t)k0 / 2 : 2 * (size_t)k0);
    const size_t scales = (size_t)p.K / 2 - k0 / 2 + k0 / 32;  // from there
    const uint32_t lds0 = lds_addr(smem), raw0 = lds_addr(raw);
    const int ng = (K + kG - 1) / kG, ns = (ng + T::KS - 1) / T::KS;  // groups, stages
    const int nq = (K - (ng - 1) * kG) / 32;              // blocks of the last group
    const int nb = nq + 4 * (ng - 1 - (ns - 1) * T::KS);    // blocks of the last stage

    // the wave's load instructions of a stage: number c < LOADS fills KB c of the
    // stage (W rows first); past the end the wave repeats its previous one
    // (a wave's instructions take rows that are equal modulo 16, so its lanes keep
    // their pieces)
    static_assert(T::WAVES % 4 == 0, "rows of a wave's load instructions modulo 16");
    constexpr int PIECES = T::CODES / 16, ROWS = 64 / PIECES;  // of a row of codes; rows of an instruction
    const int piece = (lane % PIECES) ^ bank_key<PIECES>(wave * ROWS + lane / PIECES);
    const int piece_a = MX ? piece : r ^ bank_key<16>(4 * (wave - T::W_LOADS) + q);
    // what the last stage's lanes step back by, past K
    const uint32_t cut = 16 * (piece - min(piece, nb - 1));
    const uint32_t cut_a = MX ? cut : 16 * (piece_a - min(piece_a, 4 * nb - 1));
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
        dma16(base, off[j] - (i == ns - 1 ? c < T::W_LOADS ? cut : cut_a : 0u),
              lds0 + (uint32_t)(as % S) * T::STAGE + 1024u * c);
    };
    // scales: an instruction brings 64 bytes of each of 16 rows (places past the row's
    // last 16 bytes repeat those)
    const int nr = (ng + 3) / 4;                      // runs of four groups
    const int last16 = nr - 1;                        // last 16 scale bytes of these columns
    auto issue_scales = [&](int h) __attribute__((always_inline)) {  // of runs h .. h + 3 (h % 4 == 0)
#pragma unroll
        for (int j = 0; j < T::RAW_PER_WAVE; ++j) {
            const int c0 = j * T::WAVES + wave, c = c0 < T::RAW_LOADS ? c0 : c0 % T::RAW_LOADS;
            const bool isw = 16 * c < T::BN;
            const int row = 16 * c + (lane >> 2) - (isw ? 0 : T::BN);
            const uint32_t at = (uint32_t)min(row, isw ? n_last : m_last) * (uint32_t)(isw ? p.w_stride : p.a_stride);
            const uint8_t *base = (isw ? wbase : abase) + scales + 16 * (size_t)h;
            dma16(base, at + 16 * min(lane & 3, last16 - h), raw0 + 1024u * c);
        }
    };
    auto pack_scales = [&](int h) __attribute__((always_inline)) {
        const int in = K / 32 - 16 * h;  // blocks that exist (none past the last run)
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
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < T::PER_WAVE; ++j) issue_one(min(i, ns - 1), i, j);
    wait_vm<S * T::PER_WAVE>();
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
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t % MT == u) {
                        w[nxt][t] = read_w(g + 1, t);
                        if (b == 3) sw_next[t] = read_sw(t);
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
            for (int t = 0; t < NT; ++t)
                wv[0][t] = codes_bf16(w[cur][t].x, moe::mx_scale_operand(sw[t] >> 8 * b & 255u));
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
                                wv[(s + 1) & 1][t] =
                                    codes_bf16(s == 0 ? w[cur][t].y : s == 1 ? w[cur][t].z : w[cur][t].w,
                                               moe::mx_scale_operand(sw[t] >> 8 * b & 255u));
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
    p.y += (size_t)blockIdx.y * p.M * p.y_stride;  // (parts of K: their sums one after the other)
    if (p.bias)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float c = p.bias[min(n0 + (wn * NT + t) * 16 + 4 * q + j, p.N - 1)];
#pragma unroll
                for (int u = 0; u < MT; ++u) acc[t][u][j] += c;
            }
    if (p.y_f32)
        store_tile<T, MT, NT, float>(p, smem, m0, n0, wm, wn, lane, acc);
    else
        store_tile<T, MT, NT, uint16_t>(p, smem, m0, n0, wm, wn, lane, acc);
}

template <bool MX, int MT, int NT, int WK, int XR>
void launch_rows(MatArgs p, hipStream_t s) {
    const int most = 65535 * 16 * MT, all = p.M;  // rows of A a grid holds
    for (int m = 0;; m += most) {
        p.M = min(all - m, most);
        const dim3 grid((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT));
        hipLaunchKernelGGL((mx_matmul_rows_kernel<MX, MT, NT, WK, XR>), grid, dim3(64 * WK), 0, s, p);
        if (all - m <= most) return;
        p.a += (size_t)most * p.a_stride;
        p.y += (size_t)most * p.y_stride;
    }
}

template <int WK, int KB>
void launch_few(const MatArgs &p, int per_cu, hipStream_t s) {
    const int tiles = (p.N + 15) / 16;
    hipLaunchKernelGGL((mx_matmul_few_kernel<WK, KB>), dim3(min(tiles, 256 * per_cu)), dim3(64 * WK), 0, s, p, tiles);
}

template <bool MX, int WM, int WN, int MT, int NT>
void launch_tile(const MatArgs &p, int k_part, hipStream_t s) {
    using T = Tile<MX, WM, WN, MT, NT>;
    const int m_tiles = (p.M + T::BM - 1) / T::BM, n_tiles = (p.N + T::BN - 1) / T::BN;
    const dim3 grid((unsigned)(((int64_t)m_tiles * n_tiles + 7) / 8 * 8), (unsigned)((p.K + k_part - 1) / k_part));
    hipLaunchKernelGGL((mx_matmul_tile_kernel<MX, WM, WN, MT, NT>), grid, dim3(64 * T::WAVES), 0, s, p, m_tiles,
                       n_tiles, k_part);
}

// The parts' sums [parts][M][N] added in order, bias, rounding once.
__global__ __launch_bounds__(256) void mx_matmul_join_kernel(const float *__restrict__ sums, int parts, MatArgs p) {
    const size_t all = (size_t)p.M * p.N, step = (size_t)gridDim.x * 256;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
        float v = sums[i];
        for (int k = 1; k < parts; ++k) v += sums[k * all + i];
        const size_t m = i / (uint32_t)p.N, n = i - m * p.N;
        if (p.bias) v += p.bias[n];
        uint8_t *row = p.y + m * p.y_stride;
        if (p.y_f32)
            reinterpret_cast<float *>(row)[n] = v;
        else
            reinterpret_cast<uint16_t *>(row)[n] = (uint16_t)pack_bf16(v, 0.0f);
    }
}

// Which kernel a product takes: the least estimated time, in us, over the tile sizes
// and parts of K.  A round of one workgroup per CU takes a + b per 128 columns; b grows
// from `few` workgroups to a full round (they share L2 and the power budget).  Measured
// at K = 2048 and 6144:
//   MXFP4 A   256 x 192  7 + 0.52 .. 0.78   128 x 128  3 + 0.31 .. 0.41     64 x 64  3 + 0.17 .. 0.18
//   bf16 A    128 x 256  6 + 1.23 .. 1.60   128 x 128  2.8 + 0.81 .. 1.06   64 x 64  2.5 + 0.47
// (of 64 x 64 tiles a CU holds two workgroups: rounds after the first take 0.65 of it)
// and the rows kernel 2 (bf16 2.2) + 2.1 per turn of its waves' runs, which is low for
// MXFP4 A and wide outputs: 32 x 6144 x 6144 takes 8.3 us where it says 6.2, 128 x 4096 x
// 4096 12.0 where it says 8.2 and takes the rows kernel before 64 x 64 tiles at 8.6.
// So 128 x 6144 x 6144 in MXFP4 takes 31 us in 256 x 192 tiles and 12 us in 64 x 64
// ones, 2048 rows 44 us and 129 us.  Parts cost a second kernel, about 3 us, and their
// sums written and read: 64 x 6144 x 6144 with bf16 A 25 us in one part, 18 us in two.
struct Plan {
    enum Kind { FEW, ROWS1, ROWS2, TILE_L, TILE_M, TILE_S } kind;
    int k_part, parts;
};
constexpr int kCUs = 256;
constexpr int64_t kMostWgs = (1LL << 32) / 512 - 8;  // of a tile kernel's 512 threads: below 2^32 in all

int64_t few_bytes(int M, int K) { return (int64_t)((K + 511) / 512) * M * kXRow; }  // bf16 A in LDS
constexpr int64_t kFewMost = 136 << 10;

// One W tile of 16 rows a workgroup while that is one round, two beyond: 32 x 2048 x 6144
// in MXFP4 5.4 us against 6.6 with two, 32 x 6144 x 6144 11.2 against 8.3; bf16 A, 32 x
// 4096 x 2048, 5.3 against 6.4.
bool one_w_tile(int M, int N) { return (int64_t)((M + 31) / 32) * ((N + 15) / 16) <= kCUs; }

Plan plan(bool mx, int M, int N, int K, bool near) {
    Plan best{Plan::ROWS1, K, 1};
    if (M <= 16) {
        if (!mx && near && few_bytes(M, K) <= kFewMost) best.kind = Plan::FEW;
        return best;
    }
    auto rounds = [](int64_t wgs) { return (double)((wgs + kCUs - 1) / kCUs); };
    auto over = [](int a, int b) { return (int64_t)((a + b - 1) / b); };
    best.kind = Plan::ROWS2;
    if (!near) return best;
    const int turns = (int)over((int)over(K, 512), mx ? 8 : 2);
    double least = rounds(over(M, 32) * over(N, 32)) * (mx ? 2.0 + 2.1 * turns : 2.2 + 2.1 * turns);
    if (one_w_tile(M, N)) least *= 0.85;
    const struct {
        Plan::Kind kind;
        int bm, bn;
        double a, few, full, more;
    } tiles[2][3] = {{{Plan::TILE_L, 128, 256, 6.0, 1.23, 1.60, 1.0},
                      {Plan::TILE_M, 128, 128, 2.8, 0.81, 1.06, 1.0},
                      {Plan::TILE_S, 64, 64, 2.5, 0.47, 0.47, 0.65}},
                     {{Plan::TILE_L, 256, 192, 7.0, 0.52, 0.78, 1.0},
                      {Plan::TILE_M, 128, 128, 3.0, 0.31, 0.41, 1.0},
                      {Plan::TILE_S, 64, 64, 3.0, 0.17, 0.18, 0.65}}};
    for (const auto &t : tiles[mx])
        for (int parts = 1; parts <= 8; parts *= 2) {
            const int64_t part = over((int)over(K, 512), parts) * 512;
            if (parts > 1 && part * (parts - 1) >= K) break;  // a part would be empty
            const int64_t wgs = over(M, t.bm) * over(N, t.bn) * parts, rest = wgs % kCUs;
            if (wgs > kMostWgs) break;
            const double groups = (double)(part < K ? part : K) / 128;
            const double join = parts > 1 ? 3.0 + (double)M * N * 8.0 * parts / 4e6 : 0.0;
            const double whole = t.a + t.full * groups;
            const double part_round = rest ? t.a + (t.few + (t.full - t.few) * (double)rest / kCUs) * groups : 0.0;
            const double tile_us =
                wgs < kCUs ? part_round : whole + t.more * ((double)(wgs / kCUs - 1) * whole + part_round);
            const double us = tile_us + join;
            if (us < least) {
                least = us;
                best = Plan{t.kind, part < K ? (int)part : K, parts};
            }
        }
    return best;
}

template <bool MX>
int run(const MatArgs &p, const Plan &how, float *sums, hipStream_t s) {
    MatArgs t = p;  // what the tile kernels write: y, or the parts' sums
    if (how.parts > 1) {
        t.y = (uint8_t *)sums;
        t.y_stride = (size_t)p.N * 4;
        t.y_f32 = true;
        t.bias = nullptr;
    }
    switch (how.kind) {
        case Plan::FEW: {
            const int64_t bytes = few_bytes(p.M, p.K);  // workgroups a CU: what LDS and registers hold
            if (bytes <= 16 << 10)
                launch_few<4, 16>(p, 3, s);
            else if (bytes <= 36 << 10)
                launch_few<4, 36>(p, 3, s);
            else if (bytes <= 64 << 10)
                launch_few<4, 64>(p, 2, s);
            else
                launch_few<8, 136>(p, 1, s);
            break;
        }
        case Plan::ROWS1:
            // A of many rows, or of bf16 rows too long for LDS, is as many bytes as a tile of
            // W: with more tiles than CUs, two tiles a workgroup read it half as often (MXFP4
            // 16 x 6144 x 6144 6.9 us against 8.3, 16 x 65536 x 4096 43 against 50, but 4 x
            // 65536 x 4096 38 against 35; bf16 16 x 6144 x 6144 10.3 against 13.6)
            if ((!MX || p.M > 8) && p.N > 16 * kCUs)
                launch_rows<MX, 1, 2, MX ? 8 : 4, 16>(p, s);
            else
                launch_rows<MX, 1, 1, MX ? 8 : 4, 16>(p, s);
            break;
        case Plan::ROWS2:
            if (one_w_tile(p.M, p.N))
                launch_rows<MX, 2, 1, MX ? 8 : 2, 32>(p, s);
            else
                launch_rows<MX, 2, 2, MX ? 8 : 2, 32>(p, s);
            break;
        case Plan::TILE_L:
            if constexpr (MX)
                launch_tile<MX, 2, 4, 8, 3>(t, how.k_part, s);
            else
                launch_tile<MX, 2, 4, 4, 4>(t, how.k_part, s);
            break;
        case Plan::TILE_M: launch_tile<MX, 2, 4, 4, 2>(t, how.k_part, s); break;
        case Plan::TILE_S: launch_tile<MX, 2, 4, 2, 1>(t, how.k_part, s); break;
    }
    MOE_LAUNCH_CHECK("mx_matmul_kernel");
    if (how.parts > 1) {
        const size_t blocks = ((size_t)p.M * p.N + 255) / 256;
        hipLaunchKernelGGL(mx_matmul_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s,
                           sums, how.parts, p);
        MOE_LAUNCH_CHECK("mx_matmul_join_kernel");
    }
    return MOE_OK;
}

// Rows further apart than this take the rows kernels: a tile's lane offsets are 32 bits.
constexpr int64_t kTileStride = 8 << 20;

size_t sums_bytes(const Plan &how, int M, int N) { return how.parts > 1 ? (size_t)how.parts * M * N * 4 : 0; }

}  // namespace

extern "C" size_t moe_mx_matmul_workspace_bytes(int M, int N, int K, int a_type) {
    if (M <= 0 || N <= 0 || K <= 0 || K % 32 || M > kMaxRows || N > kMaxRows || K > kMaxK) return 0;
    if (a_type != MOE_BF16 && a_type != MOE_MXFP4) return 0;
    return sums_bytes(plan(a_type == MOE_MXFP4, M, N, K, true), M, N);
}

extern "C" int moe_mx_matmul(const void *a, int a_type, int64_t a_stride, const uint8_t *w, int64_t w_stride, int M,
                             int N, int K, const float *bias, void *y, int y_type, int64_t y_stride, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0) return moe::fail(MOE_E_ARG, "mx_matmul: M=%d, N=%d", M, N);
    if (a_type != MOE_BF16 && a_type != MOE_MXFP4) return moe::fail(MOE_E_ARG, "mx_matmul: a_type=%d", a_type);
    if (y_type != MOE_BF16 && y_type != MOE_FP32) return moe::fail(MOE_E_ARG, "mx_matmul: y_type=%d", y_type);
    if (K <= 0 || K % 32) return moe::fail(MOE_E_SHAPE, "mx_matmul: K=%d must be a positive multiple of 32", K);
    if (M > kMaxRows || N > kMaxRows || K > kMaxK)
        return moe::fail(MOE_E_SHAPE, "mx_matmul: M=%d, N=%d above %d or K=%d above %d", M, N, kMaxRows, K, kMaxK);
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
    if ((M > 1 && a_stride > kMaxStride) || (N > 1 && w_stride > kMaxStride))
        return moe::fail(MOE_E_SHAPE, "mx_matmul: operands' rows more than %lld bytes apart", (long long)kMaxStride);
    const bool mx = a_type == MOE_MXFP4;
    const Plan how = plan(mx, M, N, K, (M == 1 || a_stride < kTileStride) && (N == 1 || w_stride < kTileStride));
    const size_t need = sums_bytes(how, M, N);
    if (workspace_bytes < need || (need && !workspace))
        return moe::fail(MOE_E_NOMEM, "mx_matmul: workspace %zu < %zu bytes", workspace_bytes, need);
    if (need && (uintptr_t)workspace % 16) return moe::fail(MOE_E_ARG, "mx_matmul: workspace is not 16-byte aligned");
    const MatArgs p{(const uint8_t *)a, w, M > 1 ? (size_t)a_stride : 0, N > 1 ? (size_t)w_stride : 0, M, N, K, bias,
                    (uint8_t *)y, M > 1 ? (size_t)y_stride : 0, y_type == MOE_FP32};
    return mx ? run<true>(p, how, (float *)workspace, (hipStream_t)stream)
              : run<false>(p, how, (float *)workspace, (hipStream_t)stream);
}
