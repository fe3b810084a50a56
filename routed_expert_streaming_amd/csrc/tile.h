// Tiles of 16 x 16 outputs through LDS, shared by the dense products: where a row's
// pieces lie, and a workgroup's sums on their way to y.
#pragma once
#include "common.h"
#include "lds_dma.h"

namespace moe {

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

// The sums of a workgroup's tile -> y, through the (now free) ring so that the
// stores are whole rows: in the registers' order, four n of 16 different m, a 2048 x
// 6144 output took 10 us, as whole rows 4.  In as many parts of m as the ring's size
// asks for.  Kept short: it runs once, from a cold instruction cache.  p: M, N, y and
// y_stride (their alignment decides the width of the stores) and row(m), where row m lies.
// mine: this wave holds sums (else it only helps to store).  STREAM: stores past the caches, for outputs that these do not hold.
template <class T, int MT, int NT, typename OUT, bool STREAM = false, class ARGS, typename F32X4>
__device__ __forceinline__ void store_tile(const ARGS &p, uint8_t *smem, int m0, int n0, int wm, int wn, int lane,
                                           const F32X4 (&acc)[NT][MT], bool mine = true) {
    constexpr int PITCH = T::BN * (int)sizeof(OUT) + 16;
    constexpr int FULL = T::BM * PITCH, PARTS = FULL <= T::LDS ? 1 : FULL <= 2 * T::LDS ? 2 : 4;
    static_assert(MT % PARTS == 0 && FULL <= PARTS * T::LDS, "a part of the tile fits the LDS");
    constexpr int PM = MT / PARTS, ROWS = T::BM / PARTS;  // row tiles per wave, rows of a part
    constexpr int PER16 = 16 / (int)sizeof(OUT), UNITS = T::BN / PER16, THREADS = 64 * T::WAVES;
    constexpr int AT_ONCE = ROWS * UNITS % (4 * THREADS) == 0 ? 4 : ROWS * UNITS % (2 * THREADS) == 0 ? 2 : 1;
    static_assert(AT_ONCE == 1 || ROWS * UNITS % (AT_ONCE * THREADS) == 0, "whole rounds of stores");
    const int r = lane & 15, q = lane >> 4;
    // 16 bytes at a time where every row begins and ends on such a piece
    const bool wide = ((uintptr_t)p.y | p.y_stride) % 16 == 0 && p.N % PER16 == 0;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        if (part) __syncthreads();
        if (mine) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < PM; ++u) {
                    const F32X4 v = acc[t][part * PM + u];
                    uint8_t *o = smem + ((wm * PM + u) * 16 + r) * PITCH + ((wn * NT + t) * 16 + 4 * q) * (int)sizeof(OUT);
                    if constexpr (sizeof(OUT) == 4)
                        *reinterpret_cast<F32X4 *>(o) = v;
                    else
                        *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                }
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
                    if (m < p.M && n < p.N) {
                        moe_u32x4 *to = reinterpret_cast<moe_u32x4 *>(p.row(m) + (size_t)n * sizeof(OUT));
                        const moe_u32x4 d{v[e].x, v[e].y, v[e].z, v[e].w};
                        if constexpr (STREAM)
                            __builtin_nontemporal_store(d, to);
                        else
                            *to = d;
                    }
                }
            }
        } else {  // value by value, a wave on neighbouring ones
            const int cols = min(T::BN, p.N - n0);
            for (int lr = threadIdx.x / 64; lr < ROWS; lr += T::WAVES) {
                const int m = row_of(lr);
                if (m >= p.M) continue;
                OUT *o = reinterpret_cast<OUT *>(p.row(m)) + n0;
                const OUT *v = reinterpret_cast<const OUT *>(smem + lr * PITCH);
                for (int n = lane; n < cols; n += 64) o[n] = v[n];
            }
        }
    }
}


}  // namespace moe
