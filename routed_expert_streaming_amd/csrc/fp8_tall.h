// Tiles of 16 MT rows of A x 32 columns a wave, where W is what costs: an expert's rows, as
// many of them at once as there are.
//
// Every wave owns 32 rows of W and walks K in blocks of 128 columns against all of the
// tile's rows of A.  So W is read, and for exact
// products (EXACT: both operands as bf16) converted, once for all of those rows: a block
// of 64 rows took twice the instructions of its products, and 1.5 us, whatever their order.
//
// A comes in through two LDS stages of two parts each, W through two stages that only
// their wave reads.  A turn (wait, barrier) stands in the middle of a block, where the
// second part is needed and the first one's place becomes free, and one at its end, the
// other way round; a load has a block and a half of time.  Past a row's end A's lanes read
// its last piece again, against zeros for W's: what is not a number there is in the row.  Between two products stand an
// addition of the tile before and, in a block's first tiles, the conversion of the next
// block's W: a wave issues in order.
#pragma once
#include "fp8_mma.h"
#include "tile.h"

namespace moe {

template <int WN_, int MT_, bool EXACT_>
struct Fp8Tall {
    static constexpr int WM = 1, WN = WN_, MT = MT_, NT = 2, WAVES = WN, BM = 16 * MT, BN = 32 * WN;
    static constexpr int FIRST = (MT + 2) / 4 * 2;  // tiles of A's first part
    static constexpr bool TALL = true, EXACT = EXACT_;
    static constexpr int A_ROW = EXACT ? 256 : 128, TILE = 16 * A_ROW;
    static constexpr int W_BYTES = BN * 128, A_BYTES = MT * TILE;
    static constexpr int W_EACH = 4, A0_EACH = FIRST * TILE / 1024 / WN, A1_EACH = (MT - FIRST) * TILE / 1024 / WN;
    static constexpr int A_EACH = A0_EACH + A1_EACH, EACH = W_EACH + A_EACH;  // loads of a wave a block, 1 KB each
    static constexpr int SCALE_LOADS = (BM + 63) / 64, CHUNK = 1024 * SCALE_LOADS;
    static constexpr int A_RING = 2 * W_BYTES, S_RING = A_RING + 2 * A_BYTES, LDS = S_RING + 2 * CHUNK;
    static constexpr int CONVERT = MT < 6 ? MT - 2 : 4;  // tiles that convert
    static_assert(A0_EACH * WN * 1024 == FIRST * TILE && A1_EACH * WN * 1024 == (MT - FIRST) * TILE, "equal shares");
    static_assert(WN % 4 == 0 && MT % 2 == 0 && FIRST >= 2 && FIRST < MT && SCALE_LOADS <= WN && 4 * NT % CONVERT == 0 &&
                      LDS <= 160 * 1024,
                  "the shape below");
};

// acc[t][u] += rows of W (tile t of this wave) x rows of A (tile u).  The arguments as
// fp8_tile's; with EXACT a holds the codes' values in bf16, 256 bytes a block, and W is
// converted.  On return no load is in flight and all waves are done with the LDS.
template <class T, int SN, class WOff, class AOff, class SOff>
__device__ __forceinline__ void fp8_tall(uint8_t *smem, const uint8_t *w, const uint8_t *a, const uint8_t *as,
                                         const float *const (&ws)[SN], int K, WOff w_off, AOff a_off, SOff as_off,
                                         f32x4 (&acc)[T::NT][T::MT]) {
    constexpr int MT = T::MT, NT = T::NT, PARTS = T::EXACT ? 4 : 1;  // products a block of a tile
    constexpr bool EXACT = T::EXACT;
    using Frag = std::conditional_t<EXACT, WideFrag, Fp8Frag>;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = (K + 127) / 128, pieces = (K - 128 * (nb - 1)) / 16;  // blocks; pieces of the last (of codes)
    const uint32_t lds0 = lds_addr(smem);

    // A load fills 1 KB of a stage: 8 rows of codes, 4 of bf16.  The last block's lanes
    // step back to its last piece.
    constexpr int PA = T::A_ROW / 16;
    const int row_w = lane >> 3, row_a = lane / PA;
    uint32_t w_at[T::W_EACH], a_at[T::A_EACH];
    const int piece_w[2] = {(lane & 7) ^ bank_key<8>(row_w), (lane & 7) ^ bank_key<8>(8 + row_w)};
    const int piece_a = lane % PA ^ bank_key<PA>((64 / PA * wave + row_a) & 15);
#pragma unroll
    for (int j = 0; j < T::W_EACH; ++j) w_at[j] = w_off(32 * wave + 8 * j + row_w) + 16 * piece_w[j & 1];
#pragma unroll
    for (int j = 0; j < T::A_EACH; ++j) a_at[j] = a_off(64 / PA * (j * T::WN + wave) + row_a) + 16 * piece_a;
    auto issue_w = [&](int i) __attribute__((always_inline)) {
        if (i == nb - 1 && pieces < 8)
#pragma unroll
            for (int j = 0; j < T::W_EACH; ++j) w_at[j] -= 16 * (piece_w[j & 1] - min(piece_w[j & 1], pieces - 1));
#pragma unroll
        for (int j = 0; j < T::W_EACH; ++j)
            dma16(w + 128 * (size_t)i, w_at[j], lds0 + (i & 1) * T::W_BYTES + 4096u * wave + 1024u * j);
    };
    auto issue_a = [&](int i, auto part_const) __attribute__((always_inline)) {
        constexpr int J0 = decltype(part_const)::value ? T::A0_EACH : 0, J1 = J0 ? T::A_EACH : T::A0_EACH;
        if (i == nb - 1 && pieces < 8)
#pragma unroll
            for (int j = J0; j < J1; ++j) a_at[j] -= 16 * (piece_a - min(piece_a, PA / 8 * pieces - 1));
#pragma unroll
        for (int j = J0; j < J1; ++j)
            dma16(a + T::A_ROW * (size_t)i, a_at[j],
                  lds0 + T::A_RING + (i & 1) * T::A_BYTES + 1024u * (j * T::WN + wave));
    };
    const int se = wave % T::SCALE_LOADS;
    const uint32_t s_off = as_off(min(64 * se + lane, T::BM - 1));
    auto issue_scales = [&](int i) __attribute__((always_inline)) {  // of blocks i .. i + 3
        dma16(as + 16 * (size_t)(i >> 2), s_off, lds0 + T::S_RING + (uint32_t)(i >> 2 & 1) * T::CHUNK + 1024u * se);
    };
    float wsv[SN];  // lane l: the scale of block 64 * (b / 64) + l
    auto load_ws = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SN; ++i) {
            wsv[i] = ws[i][min(b0 + lane, nb - 1)];
            asm volatile("" : "+v"(wsv[i]));
        }
    };

    const uint8_t *w_lds = smem + 4096 * wave + 128 * r, *s_lds = smem + T::S_RING + 16 * r;
    const int lo = 16 * (q ^ bank_key<8>(r)), hi = 16 * ((q + 4) ^ bank_key<8>(r));
    const uint8_t *x_lds[2][EXACT ? 4 : 2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint8_t *row = smem + T::A_RING + p * T::A_BYTES + T::A_ROW * r;
        if constexpr (EXACT) {  // the columns of codes' pieces q and q + 4: pieces 2q, 2q + 1 and 8 further
#pragma unroll
            for (int s = 0; s < 4; ++s) x_lds[p][s] = row + 16 * ((2 * q + (s & 1) + 8 * (s >> 1)) ^ bank_key<16>(r));
        } else {
            x_lds[p][0] = row + lo, x_lds[p][1] = row + hi;
        }
    }
    auto read_w = [&](int stage, int t) __attribute__((always_inline)) {
        const uint8_t *p = w_lds + stage * T::W_BYTES + t * 2048;
        return Fp8Frag{*reinterpret_cast<const uint4 *>(p + lo), *reinterpret_cast<const uint4 *>(p + hi)};
    };
    auto read_x = [&](int stage, int u) __attribute__((always_inline)) {
        if constexpr (EXACT) {
            WideFrag f;
#pragma unroll
            for (int s = 0; s < 4; ++s) f.v[s] = *reinterpret_cast<const bf16x8 *>(x_lds[stage][s] + u * T::TILE);
            return f;
        } else {
            return Fp8Frag{*reinterpret_cast<const uint4 *>(x_lds[stage][0] + u * T::TILE),
                           *reinterpret_cast<const uint4 *>(x_lds[stage][1] + u * T::TILE)};
        }
    };
    auto scales_of = [&](int g) __attribute__((always_inline)) { return s_lds + (g >> 2 & 1) * T::CHUNK + 4 * (g & 3); };
    auto read_s = [&](const uint8_t *p, int u) __attribute__((always_inline)) {
        return *reinterpret_cast<const float *>(p + u * 256);
    };
    auto widen_part = [&](const Fp8Frag &f, int s) __attribute__((always_inline)) {  // s: which 8 of a lane's 32 codes
        return s == 0   ? widen8(f.lo.x, f.lo.y)
               : s == 1 ? widen8(f.lo.z, f.lo.w)
               : s == 2 ? widen8(f.hi.x, f.hi.y)
                        : widen8(f.hi.z, f.hi.w);
    };

    constexpr IntC<0> PART0{};
    constexpr IntC<1> PART1{};
    Frag wf[2][NT];   // block g's W in [g & 1]
    Fp8Frag raw[NT];  // EXACT: the codes of the next block's
    load_ws(0);
    issue_scales(0);
    issue_w(0);
    issue_a(0, PART0);
    if (nb > 1) issue_w(1);
    issue_a(0, PART1);
    if (nb > 1)
        wait_vm<T::EACH>();
    else
        wait_vm<T::A_EACH>();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        raw[t] = read_w(0, t);
        if (nb == 1) cut_frag(raw[t], q, pieces);
        if constexpr (EXACT) {
            wf[0][t] = widen(raw[t]);
        } else {
            wf[0][t] = raw[t];
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // W's stage 0 is read
    if (nb > 1) issue_a(1, PART0);
    if (nb > 2) issue_w(2);
    if (nb > 1) issue_a(1, PART1);
    if (nb > 2)
        wait_vm<T::EACH + T::A1_EACH>();
    else
        wait_vm<0>();
    ring_barrier();
    if constexpr (EXACT)
#pragma unroll
        for (int t = 0; t < NT; ++t) raw[t] = read_w(1, t);
    Frag xf[2] = {read_x(0, 0), read_x(0, 1)};
    float sf[2] = {read_s(scales_of(0), 0), read_s(scales_of(0), 1)};

    f32x4 v[2][NT];  // tile u's products in [u & 1], added while the next one's are made
    float vs[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) v[1][t] = f32x4{0.f, 0.f, 0.f, 0.f}, vs[1][t] = 0.0f;
    auto convert = [&](auto p_const, auto n_const) __attribute__((always_inline)) {  // the next block's W, part n
        constexpr int P = decltype(p_const)::value, n = decltype(n_const)::value;
        if constexpr (EXACT) wf[P ^ 1][n % NT].v[n / NT] = widen_part(raw[n % NT], n / NT);
        if constexpr (EXACT) asm volatile("" : "+v"(wf[P ^ 1][n % NT].v[n / NT]));
    };
    auto block = [&](int g, auto p_const) __attribute__((always_inline)) {
        constexpr int P = decltype(p_const)::value;
        if ((g & 63) == 0 && g) load_ws(g);
        float sw[SN];
#pragma unroll
        for (int i = 0; i < SN; ++i)
            sw[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[i]), g & 63));
        const uint8_t *const s_now = scales_of(g), *const s_next = scales_of(g + 1);
        if (EXACT && pieces < 8 && g + 1 == nb - 1)
#pragma unroll
            for (int t = 0; t < NT; ++t) cut_frag(raw[t], q, pieces);
        static_for<0, MT>([&](auto u_const) __attribute__((always_inline)) {
            constexpr int u = decltype(u_const)::value, CV = 4 * NT / T::CONVERT;  // W's parts a tile converts
            if constexpr (u == T::FIRST - 2) {
                if (g + 2 < nb)
                    wait_vm<T::EACH>();
                else if (g + 1 < nb)
                    wait_vm<T::A_EACH>();
                else
                    wait_vm<0>();
                ring_barrier();
                if (g + 2 < nb) {
                    if (((g + 2) & 3) == 0) issue_scales(g + 2);
                    issue_a(g + 2, PART0);
                }
                if constexpr (EXACT) {
                    if (g + 3 < nb) issue_w(g + 3);
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        wf[P ^ 1][t] = read_w(P ^ 1, t);
                        if (pieces < 8 && g + 1 == nb - 1) cut_frag(wf[P ^ 1][t], q, pieces);
                    }
                }
            }
            if constexpr (u == MT - 2) {
                if (g + (EXACT ? 3 : 2) < nb)
                    wait_vm<T::EACH>();
                else if (g + 2 < nb)
                    wait_vm<T::A_EACH>();
                else if (g + 1 < nb)
                    wait_vm<T::A1_EACH>();
                ring_barrier();
                if constexpr (!EXACT)
                    if (g + 3 < nb) issue_w(g + 3);
                if (g + 2 < nb) issue_a(g + 2, PART1);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) vs[u & 1][t] = sf[u & 1] * sw[t % SN];
            static_for<0, PARTS * NT>([&](auto i_const) __attribute__((always_inline)) {
                constexpr int i = decltype(i_const)::value, t = i % NT, s = i / NT, ADDS = 4 / PARTS;
                f32x4 &c = v[u & 1][t];
                if constexpr (EXACT)
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[P][t].v[s], xf[u & 1].v[s],
                                                                s ? c : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                else
                    c = mfma_fp8(wf[P][t], xf[u & 1]);
#pragma unroll
                for (int j = ADDS * s; j < ADDS * (s + 1); ++j) {
                    f32x4 &sum = acc[t][(u + MT - 1) % MT];
                    sum[j] = fmaf(v[(u + 1) & 1][t][j], vs[(u + 1) & 1][t], sum[j]);
                }
                if constexpr (EXACT && u < T::CONVERT)
                    if constexpr (i * CV % (4 * NT) < CV) convert(IntC<P>{}, IntC<CV * u + i * CV / (4 * NT)>{});
                // left to itself the compiler adds, and converts, at the block's end
                if constexpr (s == PARTS - 1) asm volatile("" : "+v"(acc[t][(u + MT - 1) % MT]));
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (u < MT - 2) {
                xf[u & 1] = read_x(P, u + 2);
                sf[u & 1] = read_s(s_now, u + 2);
            }
            if constexpr (u >= MT - 2) {  // past the last block whatever the rings hold
                xf[u & 1] = read_x(P ^ 1, u + 2 - MT);
                sf[u & 1] = read_s(s_next, u + 2 - MT);
            }
            if constexpr (EXACT && u == MT - 2)  // W's stage is free: its loads come after the next turn
#pragma unroll
                for (int t = 0; t < NT; ++t) raw[t] = read_w(P, t);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    int g = 0;
    for (; g + 1 < nb; g += 2) {
        block(g, IntC<0>{});
        block(g + 1, IntC<1>{});
    }
    if (g < nb) block(g, IntC<0>{});
#pragma unroll
    for (int t = 0; t < NT; ++t)
        acc[t][MT - 1] = fma4(v[(MT - 1) & 1][t], vs[(MT - 1) & 1][t], acc[t][MT - 1]);
    wait_vm<0>();
    __syncthreads();
}

}  // namespace moe
