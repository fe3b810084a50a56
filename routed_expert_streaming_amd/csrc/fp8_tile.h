// Many rows of activations: tiles through LDS.
//
// A workgroup owns BM x BN outputs (WM x WN waves of MT x NT tiles of 16 x 16) and walks
// K in blocks of 128 columns through two rings of LDS stages, one block of W's rows or of
// A's each, filled by direct global -> LDS loads of 8 rows x 128 bytes.  A row's eight
// 16-byte pieces change places by a key of the row, so that the operand reads fall into
// different banks.  The activations' scales come in by four blocks (16 bytes a row), two
// such chunks in turn; W's scales, one or a few a block for a wave's columns, lie in
// registers across the lanes, 64 blocks at a time.
//
// KW groups of waves may share the outputs and take every KW-th block each, with rings of
// their own (and an A scale chunk in every stage); their sums are joined through LDS, in
// order, at the end.  A turn from one block to the next is a chain of latencies, about 0.4
// us whatever the tile's size, which small tiles cannot fill otherwise.
#pragma once
#include "fp8_mma.h"
#include "tile.h"

namespace moe {

template <int WM_, int WN_, int MT_, int NT_, int SW_, int SA_, int KW_ = 1>
struct Fp8Tile {
    static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
    static constexpr bool TALL = false;
    static constexpr int SW = SW_, SA = SA_;  // stages of W's rows and of A's
    static constexpr int KW = KW_, GROUP = WM * WN;  // groups of waves along K, waves of one
    static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = GROUP * KW;
    static constexpr int W_BYTES = BN * 128, A_BYTES = BM * 128;
    static constexpr int W_LOADS = BN / 8, A_LOADS = BM / 8;  // load instructions of a stage, 1 KB each
    static constexpr int W_EACH = (W_LOADS + GROUP - 1) / GROUP, A_EACH = (A_LOADS + GROUP - 1) / GROUP;  // by a wave
    static constexpr int SCALE_ROWS = BM < 64 ? 64 : BM, CHUNK = SCALE_ROWS * 16;
    static constexpr int SCALE_LOADS = SCALE_ROWS / 64;
    static constexpr int CHUNKS = KW == 1 ? 2 : SA;
    static constexpr int A_RING = SW * W_BYTES, S_RING = A_RING + SA * A_BYTES, RINGS = S_RING + CHUNKS * CHUNK;
    static constexpr int JOIN = (KW - 1) * GROUP * MT * NT * 1024;  // the sums of the groups but the first
    static constexpr int LDS = KW * RINGS > JOIN ? KW * RINGS : JOIN;
    static_assert(SW >= 2 && SW <= SA && SA <= 4 && SCALE_LOADS <= GROUP && GROUP % 2 == 0 && WAVES <= 16 &&
                      LDS <= 160 * 1024,
                  "tile does not fit its workgroup");
    static_assert(SA * A_EACH + SW * W_EACH < 64, "vmcnt range");
    // loads of a wave after each column of tiles, so that all are issued within half a block
    static constexpr int EACH = W_EACH + A_EACH + (KW > 1 ? 1 : 0), SPREAD = (EACH + (MT + 1) / 2 - 1) / ((MT + 1) / 2);
    static constexpr int LAG = MT * NT % 4 == 0 ? 4 : MT * NT % 3 == 0 ? 3 : MT * NT % 2 == 0 ? 2 : 1;
};

// acc[t][u] += rows of W (tile t of this wave) x rows of A (tile u); with KW > 1 only the
// first group's waves have the sums in the end.  w, a, as: uniform
// bases at column 0; w_off(row), a_off(row), as_off(row): 32-bit byte offsets of the
// tile's rows (valid for every row of the tile); ws[i]: the scales of the wave's i-th
// NT / SN tiles, one per block.  ENDS: A's rows of scales end where their values do, so
// nothing behind them is read (else they are readable up to a multiple of 16 bytes).
// On return no load is in flight and all waves are done with the LDS.
template <class T, bool WIDE, int SN, bool ENDS = false, class WOff, class AOff, class SOff>
__device__ __forceinline__ void fp8_tile(uint8_t *smem, const uint8_t *w, const uint8_t *a, const uint8_t *as,
                                         const float *const (&ws)[SN], int K, WOff w_off, AOff a_off, SOff as_off,
                                         f32x4 (&acc)[T::NT][T::MT]) {
    constexpr int SW = T::SW, SA = T::SA, MT = T::MT, NT = T::NT;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    constexpr int KW = T::KW;
    const int kg = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / T::GROUP;  // this wave's group
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) - kg * T::GROUP, wm = wave / T::WN, wn = wave % T::WN;
    const int blocks = (K + 127) / 128, pieces = (K - 128 * (blocks - 1)) / 16;  // pieces of the last block
    const int nb = KW == 1 ? blocks : (blocks + KW - 1) / KW;                     // this group's (the last may be none)
    auto block_of = [&](int g) __attribute__((always_inline)) { return KW == 1 ? g : min(g * KW + kg, blocks - 1); };
    uint8_t *const ring = smem + kg * T::RINGS;
    const uint32_t lds0 = lds_addr(smem) + kg * T::RINGS;

    // load instruction c fills KB c of a stage, rows 8c .. 8c + 7; a wave's take rows that
    // are equal modulo 16, so its lanes keep their pieces (where there are fewer loads
    // than waves, or not a multiple, some are made twice)
    const int piece = (lane & 7) ^ bank_key<8>((8 * wave + (lane >> 3)) & 15);
    const uint32_t cut = 16 * (piece - min(piece, pieces - 1));  // what the last block's lanes step back by
    auto load_number = [&](int j, int loads) __attribute__((always_inline)) {
        const int c = j * T::GROUP + wave;
        return c < loads ? c : loads >= T::GROUP ? c - T::GROUP : c % loads;
    };
    uint32_t w_at[T::W_EACH], a_at[T::A_EACH];
#pragma unroll
    for (int j = 0; j < T::W_EACH; ++j) w_at[j] = w_off(8 * load_number(j, T::W_LOADS) + (lane >> 3)) + 16 * piece;
#pragma unroll
    for (int j = 0; j < T::A_EACH; ++j) a_at[j] = a_off(8 * load_number(j, T::A_LOADS) + (lane >> 3)) + 16 * piece;
    auto issue_w = [&](int i, int j) __attribute__((always_inline)) {
        const int b = block_of(i);
        dma16(w + 128 * (size_t)b, w_at[j] - (b == blocks - 1 ? cut : 0u),
              lds0 + (uint32_t)(i % SW) * T::W_BYTES + 1024u * load_number(j, T::W_LOADS));
    };
    auto issue_a = [&](int i, int j) __attribute__((always_inline)) {
        const int b = block_of(i);
        dma16(a + 128 * (size_t)b, a_at[j] - (b == blocks - 1 ? cut : 0u),
              lds0 + T::A_RING + (uint32_t)(i % SA) * T::A_BYTES + 1024u * load_number(j, T::A_LOADS));
    };
    const int se = wave % T::SCALE_LOADS;  // (several waves bring the same rows)
    const uint32_t s_off = as_off(min(64 * se + lane, T::BM - 1));
    // ENDS: the row's last scales where they are fewer than four, kept from the start (a load of them
    // in their turn would be waited for behind the rings': 0.3 us of a short product).  They take a
    // load's place, so the waits do not count on the scales' loads.
    constexpr int NO_SCALES = ENDS && KW > 1 ? 1 : 0;
    float last[3] = {0.f, 0.f, 0.f};
    auto issue_scales = [&](int i) __attribute__((always_inline)) {  // of stage i's block and its neighbours
        const int place = KW == 1 ? i >> 2 & 1 : i % SA, first = block_of(i) & ~3;
        const uint32_t at = T::S_RING + (uint32_t)place * T::CHUNK + 1024u * se;
        if (ENDS && first + 4 > blocks) {
            *reinterpret_cast<f32x4 *>(ring + at + 16 * lane) = f32x4{last[0], last[1], last[2], 0.f};
        } else {
            dma16(as + 4 * (size_t)first, s_off, lds0 + at);
        }
    };
    float wsv[SN];  // lane l: the scale of block 64 * (b / 64) + l
    auto load_ws = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            wsv[i] = ws[i][min(b0 + lane, blocks - 1)];
            asm volatile("" : "+v"(wsv[i]));  // waited for here, not in every block behind the rings' loads
        }
    };
    const uint8_t *w_lds = ring + (wn * NT * 16 + r) * 128, *x_lds = ring + T::A_RING + (wm * MT * 16 + r) * 128;
    const uint8_t *s_lds = ring + T::S_RING + (wm * MT * 16 + r) * 16;
    const int lo = 16 * (q ^ bank_key<8>(r)), hi = 16 * ((q + 4) ^ bank_key<8>(r));
    auto read = [&](const uint8_t *p) __attribute__((always_inline)) {
        return Fp8Frag{*reinterpret_cast<const uint4 *>(p + lo), *reinterpret_cast<const uint4 *>(p + hi)};
    };
    auto read_w = [&](int g, int t) __attribute__((always_inline)) {
        return read(w_lds + (uint32_t)(g % SW) * T::W_BYTES + t * 2048);
    };
    auto read_x = [&](int g, int u) __attribute__((always_inline)) {
        return read(x_lds + (uint32_t)(g % SA) * T::A_BYTES + u * 2048);
    };
    auto read_s = [&](int g, int u) __attribute__((always_inline)) {
        const int place = KW == 1 ? g >> 2 & 1 : g % SA;
        return *reinterpret_cast<const float *>(s_lds + place * T::CHUNK + u * 256 + 4 * (block_of(g) & 3));
    };

    // Issue order, which the waits count on: the first scales, W's stages 0 .. SW-1 and A's
    // 0 .. SA-1 by turns, then after the turn from block g to g + 1 W's stage g + SW and A's
    // g + SA (and scales before them).
    if (ENDS) {
        const float *from = reinterpret_cast<const float *>(as + s_off) + (blocks & ~3);
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if ((blocks & ~3) + j < blocks) last[j] = from[j];
    }
    load_ws(0);
    if (ENDS)
#pragma unroll
        for (int j = 0; j < 3; ++j) asm volatile("" : "+v"(last[j]));
    if (KW == 1) issue_scales(0);
#pragma unroll
    for (int i = 0; i < SA; ++i) {
        if (KW > 1 && i < nb) issue_scales(i);
        if (i < SW && i < nb)
#pragma unroll
            for (int j = 0; j < T::W_EACH; ++j) issue_w(i, j);
        if (i < nb)
#pragma unroll
            for (int j = 0; j < T::A_EACH; ++j) issue_a(i, j);
    }
    if (nb >= SA)
        wait_vm<(SW - 1) * T::W_EACH + (SA - 1) * (T::EACH - T::W_EACH - NO_SCALES)>();
    else
        wait_vm<0>();
    ring_barrier();
    // A's operands are read AHEAD columns of tiles before their products: with one, the
    // eight waves' reads in turn took longer than a column's products.
    constexpr int AHEAD = MT >= 4 ? 2 : 1;
    static_assert(MT % AHEAD == 0, "an operand's place");
    Fp8Frag wf[NT], xf[AHEAD];
    float sf[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) xf[u] = read_x(0, u), sf[u] = read_s(0, u);
#pragma unroll
    for (int t = 0; t < NT; ++t) wf[t] = read_w(0, t);

    // The turn from block g to g + 1: every wave's operands of block g are in registers
    // when it arrives, so the stages that follow may overwrite it.  Block g + 1 has landed
    // once only the loads issued after its own are in flight: after W's stage g + 1 came A's
    // g + 1 - SW + SA (itself needed where SA = SW) and what SW - 2 turns issued.
    auto turn = [&](int g) __attribute__((always_inline)) {
        if (g + SA <= nb)
            wait_vm<(SW - 2) * (T::EACH - NO_SCALES) + (SA > SW ? T::A_EACH : 0)>();  // (scales come first)
        else
            wait_vm<0>();
        ring_barrier();
    };
    // A product's result enters the sums when LAG more products have been issued, so that
    // no addition waits for its own product.  (The pin keeps that order: left to itself
    // the compiler gathers the products and spills.  256 x 256 tiles still spill 8 of their 256
    // registers, 20 bytes a lane.)
    constexpr int LAG = T::LAG;
    static_assert(NT * MT % LAG == 0, "a product's place");
    f32x4 done[LAG];
    float done_s[LAG];
#pragma unroll
    for (int i = 0; i < LAG; ++i) done[i] = f32x4{0.f, 0.f, 0.f, 0.f}, done_s[i] = 0.f;
    auto add = [&](auto i_const) __attribute__((always_inline)) {  // product i of this block's, or of the last one's
        constexpr int i = decltype(i_const)::value, n = (i + NT * MT) % (NT * MT), t = n % NT, u = n / NT;
        acc[t][u] = fma4(done[n % LAG], done_s[n % LAG], acc[t][u]);
        asm volatile("" : "+v"(acc[t][u])::"memory");
    };
    auto block = [&](int g, auto cut_const) __attribute__((always_inline)) {
        constexpr bool CUT = decltype(cut_const)::value != 0;
        const int b = block_of(g);
        if ((b & 63) < KW && g) load_ws(b & ~63);
        const bool none = KW > 1 && g * KW + kg >= blocks;  // no such block: the last one again, times 0
        float sw[SN];
#pragma unroll
        for (int i = 0; i < SN; ++i)
            sw[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[i]), b & 63));
        const int kept = CUT && b == blocks - 1 ? pieces : 8;
        if (CUT) {
#pragma unroll
            for (int t = 0; t < NT; ++t) cut_frag(wf[t], q, kept);
        }
        decltype(operand<WIDE>(wf[0])) wo[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) wo[t] = operand<WIDE>(wf[t]);
        static_for<0, MT>([&](auto u_const) __attribute__((always_inline)) {
            constexpr int u = decltype(u_const)::value;
            if (CUT) cut_frag(xf[u % AHEAD], q, kept);
            const auto x = operand<WIDE>(xf[u % AHEAD]);
            float su[SN];
#pragma unroll
            for (int i = 0; i < SN; ++i) su[i] = none ? 0.0f : sf[u % AHEAD] * sw[i];
            // the next operands (past the last block whatever the rings hold)
            constexpr int next = u + AHEAD;
            if (next == MT) turn(g);
            xf[u % AHEAD] = next < MT ? read_x(g, next) : read_x(g + 1, next - MT);
            sf[u % AHEAD] = next < MT ? read_s(g, next) : read_s(g + 1, next - MT);
            static_for<0, NT>([&](auto t_const) __attribute__((always_inline)) {
                constexpr int t = decltype(t_const)::value, i = u * NT + t;
                const f32x4 v = mfma_fp8(wo[t], x);
                asm volatile("" ::: "memory");
                add(IntC<i - LAG>{});
                done[i % LAG] = v;
                done_s[i % LAG] = su[t / (NT / SN)];
                if (u + 1 == MT) wf[t] = read_w(g + 1, t);
            });
            // the loads that the last turn made room for: from there on, spread over the products,
            // because a wave whose load the memory pipeline does not take yet issues nothing else
            constexpr int step = (u + AHEAD) % MT, turned = u + AHEAD < MT ? 1 : 0;
            if constexpr (step * T::SPREAD < T::EACH) {
                const int from = g - turned;  // the turn's block
                if (KW == 1 && step == 0 && from >= 0 && ((from + SA) & 3) == 0 && from + SA < nb) issue_scales(from + SA);
#pragma unroll
                for (int j0 = step * T::SPREAD; j0 < (step + 1) * T::SPREAD && j0 < T::EACH; ++j0) {
                    const int j = KW > 1 ? j0 - 1 : j0;  // KW > 1: the scales first
                    if (j < 0) {
                        if (from >= 0 && from + SA < nb) issue_scales(from + SA);
                    } else if (j < T::W_EACH) {
                        if (from >= 0 && from + SW < nb) issue_w(from + SW, j);
                    } else {
                        if (from >= 0 && from + SA < nb) issue_a(from + SA, j - T::W_EACH);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    const int whole = pieces < 8 ? nb - 1 : nb;
    for (int g = 0; g < whole; ++g) block(g, IntC<0>{});
    if (pieces < 8) block(nb - 1, IntC<1>{});
    static_for<NT * MT - LAG, NT * MT>(add);
    wait_vm<0>();
    __syncthreads();
    if constexpr (KW > 1) {
        f32x4(*part)[64] = reinterpret_cast<f32x4(*)[64]>(smem);
        if (kg)
#pragma unroll
            for (int i = 0; i < NT * MT; ++i)
                part[((kg - 1) * T::GROUP + wave) * NT * MT + i][lane] = acc[i / MT][i % MT];
        __syncthreads();
        if (!kg)
#pragma unroll
            for (int i = 0; i < NT * MT; ++i)
#pragma unroll
                for (int k = 1; k < KW; ++k) acc[i / MT][i % MT] += part[((k - 1) * T::GROUP + wave) * NT * MT + i][lane];
        __syncthreads();
    }
}

}  // namespace moe
