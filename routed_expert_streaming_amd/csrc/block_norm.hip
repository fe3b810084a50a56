// The step between two blocks of a residual network, per token row t, in one pass:
//   d = add[t,:]                                            the block's output
//   d = d / sqrt(mean(d^2) + eps) * w_post                  (post-norm, optional)
//   d = gate * d                                            (optional)
//   r = resid[t,:] + scale * d                              kept as resid's type
//   x = bf16( r / sqrt(mean(r^2) + eps) * w_pre )           the next block's input
// and, from the same registers, x as an MXFP4 row for a product that takes one.
//
// Bound by memory: one read of add, resid (and an element gate), one write of
// resid and x.  One workgroup owns a row and holds it in registers between the
// two sums of squares, so nothing is read twice (2048 x 6144, fp32 residual: 151
// MB in 27.0 us, 5.6 TB/s, with x's MXFP4 rows in x's place 25.5; bf16 residual
// 21.6; one token of 4096: 3.8 us, the latency of a load, two sums and a store).
// That holds for rows of up to 32768 columns in 16-byte accesses.  Where H is not a
// multiple of 8, or a pointer not one of 16 bytes, a lane takes one value at a time
// and 4096 columns fit; longer rows are read again for each step.  Such rows are
// bound by the number of their 2- and 4-byte accesses: 2048 x 4001 41.9 us, 2048 x
// 6143 85.3.  The sums are fp32 in a fixed order (a lane's values in index order, a
// butterfly per wave, the waves in order), so results are reproducible.
#include "common.h"
#include "dequant.h"
#include "mx_quant.h"

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kReread = 8;            // items of a row that the registers do not hold
// Residual streams of this many bytes (an XCD's L2) and more, and their x, are written
// with non-temporal stores: 256 x 6144 by itself 6.7 us against 7.6, 2048 x 6144 27 us
// against 39; in a chain with the products between, 2048 rows took the same either way.
constexpr int64_t kStreamFrom = 4 << 20;
constexpr int kMaxH = 1 << 28;       // column numbers plus a step stay in 31 bits
constexpr int kMaxRows = 1 << 20;    // rows of one launch (its threads stay below 2^32)

struct NormArgs {
    const uint16_t *add;
    const float *w_post;
    const void *gate;
    const void *resid;
    void *resid_out;
    const float *w_pre;
    uint16_t *x_next;
    uint8_t *x_rows;
    int H, gate_kind;
    bool post;
    float scale, eps;
};

// V consecutive values at element i of a bf16 / fp32 array (V = 8: 16-byte aligned)
template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t *p, size_t i, float (&x)[V]) {
    if constexpr (V == 8) {
        const uint4 a = load_global_u4(p + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = bf16_bits_to_f32(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu);
    } else {
        x[0] = bf16_bits_to_f32(p[i]);
    }
}
template <int V>
__device__ __forceinline__ void load_f32(const float *p, size_t i, float (&x)[V]) {
    if constexpr (V == 8) {
        const uint4 a = load_global_u4(p + i), b = load_global_u4(p + i + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
    } else {
        x[0] = p[i];
    }
}
// 16 bytes to 16-byte aligned p; STREAM: non-temporal
template <bool STREAM>
__device__ __forceinline__ void store16(void *p, uint4 v) {
    const moe_u32x4 w{v.x, v.y, v.z, v.w};
    if constexpr (STREAM)
        __builtin_nontemporal_store(w, (moe_u32x4 *)p);
    else
        *(moe_u32x4 *)p = w;
}
template <int V, bool STREAM>
__device__ __forceinline__ void store_bf16(uint16_t *p, size_t i, const uint32_t (&h)[V]) {
    if constexpr (V == 8) {
        store16<STREAM>(p + i, make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16));
    } else {
        p[i] = (uint16_t)h[0];
    }
}

// Sum over the workgroup (every thread gets it).  part: one float per wave.
__device__ __forceinline__ float block_sum(float v, float *part) {
    v = group_sum<64>(v);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[0];
    for (int w = 1; w < waves; ++w) s += part[w];
    return s;
}

// The gated and scaled update of V values: resid + scale * gate * norm(add).
template <int V, bool RF32>
__device__ __forceinline__ void update(const NormArgs &a, size_t row, int i, float inv_post, float gate_row,
                                       const float (&d0)[V], float (&r)[V]) {
    float d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = d0[j];
    if (a.post) {
        float w[V];
        if (a.w_post) load_f32<V>(a.w_post, (size_t)i, w);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = a.w_post ? d[j] * inv_post * w[j] : d[j] * inv_post;
    }
    if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
        float g[V];
        if (a.gate_kind == MOE_GATE_CHANNEL)
            load_f32<V>((const float *)a.gate, (size_t)i, g);
        else
            load_bf16<V>((const uint16_t *)a.gate, row + i, g);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] *= g[j];
    } else if (a.gate_kind == MOE_GATE_ROW) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] *= gate_row;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = fmaf(a.scale, d[j], r[j]);
}

template <int V, bool RF32>
__device__ __forceinline__ void load_resid(const void *p, size_t i, float (&r)[V]) {
    if constexpr (RF32)
        load_f32<V>((const float *)p, i, r);
    else
        load_bf16<V>((const uint16_t *)p, i, r);
}

// Stores r as the residual stream's type; r becomes the value kept.
template <int V, bool RF32, bool STREAM>
__device__ __forceinline__ void store_resid(void *p, size_t i, float (&r)[V]) {
    if constexpr (RF32) {
        if constexpr (V == 8) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                store16<STREAM>((float *)p + i + j, make_uint4(__float_as_uint(r[j]), __float_as_uint(r[j + 1]),
                                                               __float_as_uint(r[j + 2]), __float_as_uint(r[j + 3])));
        } else {
            ((float *)p)[i] = r[0];
        }
    } else {
        uint32_t h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            h[j] = f32_to_bf16_bits(r[j]);
            r[j] = bf16_bits_to_f32(h[j]);
        }
        store_bf16<V, STREAM>((uint16_t *)p, i, h);
    }
}

// x of V values from the kept residual, stored as bf16 and / or as MXFP4 codes of
// those bf16 values (V = 8: four neighbouring lanes hold a block).
template <int V, bool STREAM>
__device__ __forceinline__ void store_next(const NormArgs &a, size_t row, int i, float inv, const float (&r)[V]) {
    uint32_t h[V];
    float w[V];
    if (a.w_pre) load_f32<V>(a.w_pre, (size_t)i, w);
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = f32_to_bf16_bits(a.w_pre ? r[j] * inv * w[j] : r[j] * inv);
    if (a.x_next) store_bf16<V, STREAM>(a.x_next, row + i, h);
    if constexpr (V == 8) {
        if (a.x_rows) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = bf16_bits_to_f32(h[j]);
            const uint32_t s = moe::mx_scale_byte(moe::quad_max(moe::mx_top8(x)), false);
            uint8_t *orow = a.x_rows + blockIdx.x * moe::mx_row_bytes(a.H);
            *reinterpret_cast<uint32_t *>(orow + i / 2) = moe::mx_codes8(x, s);
            if (((i >> 3) & 3) == 0) moe::mx_store_scale(orow, a.H, i >> 5, s);
        }
    }
}

// ITEMS > 0: thread t holds values V*(t + j*threads) .. + V-1 for j < ITEMS in
// registers (H <= V * threads * ITEMS).  ITEMS = 0: any H, the row re-read from
// memory for each of the three steps (the kept residual from resid_out).
template <int V, int ITEMS, bool RF32, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(NormArgs a) {
    __shared__ float part[2][kMaxThreads / 64];
    const size_t row = (size_t)blockIdx.x * a.H;
    const int tid = threadIdx.x, step = V * blockDim.x;
    const float gate_row = a.gate_kind == MOE_GATE_ROW ? ((const float *)a.gate)[blockIdx.x] : 1.0f;
    if constexpr (ITEMS > 0) {
        float d[ITEMS][V], r[ITEMS][V];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = V * tid + k * step;
#pragma unroll
            for (int j = 0; j < V; ++j) d[k][j] = r[k][j] = 0.0f;
            if (i < a.H) {
                if (a.add) load_bf16<V>(a.add, row + i, d[k]);
                load_resid<V, RF32>(a.resid, row + i, r[k]);
            }
        }
        if (a.add) {
            float inv_post = 1.0f;
            if (a.post) {
                float ss = 0.0f;
#pragma unroll
                for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) ss = fmaf(d[k][j], d[k][j], ss);
                inv_post = 1.0f / sqrtf(block_sum(ss, part[0]) / (float)a.H + a.eps);
            }
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = V * tid + k * step;
                if (i < a.H) {
                    update<V, RF32>(a, row, i, inv_post, gate_row, d[k], r[k]);
                    store_resid<V, RF32, STREAM>(a.resid_out, row + i, r[k]);
                }
            }
        }
        if (!a.x_next && !a.x_rows) return;
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(r[k][j], r[k][j], ss);
        const float inv = 1.0f / sqrtf(block_sum(ss, part[1]) / (float)a.H + a.eps);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = V * tid + k * step;
            if (i < a.H) store_next<V, STREAM>(a, row, i, inv, r[k]);
        }
    } else {
        const void *kept = a.resid;
        float ss = 0.0f;
        if (a.add) {
            float inv_post = 1.0f;
            if (a.post) {
                float sp = 0.0f;
                for (int i = V * tid; i < a.H; i += step) {
                    float d[V];
                    load_bf16<V>(a.add, row + i, d);
#pragma unroll
                    for (int j = 0; j < V; ++j) sp = fmaf(d[j], d[j], sp);
                }
                inv_post = 1.0f / sqrtf(block_sum(sp, part[0]) / (float)a.H + a.eps);
            }
            for (int i = V * tid; i < a.H; i += step) {
                float d[V], r[V];
                load_bf16<V>(a.add, row + i, d);
                load_resid<V, RF32>(a.resid, row + i, r);
                update<V, RF32>(a, row, i, inv_post, gate_row, d, r);
                store_resid<V, RF32, STREAM>(a.resid_out, row + i, r);
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(r[j], r[j], ss);
            }
            kept = a.resid_out;  // a lane reads back only what it wrote itself
        } else {
            for (int i = V * tid; i < a.H; i += step) {
                float r[V];
                load_resid<V, RF32>(a.resid, row + i, r);
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(r[j], r[j], ss);
            }
        }
        if (!a.x_next && !a.x_rows) return;
        const float inv = 1.0f / sqrtf(block_sum(ss, part[1]) / (float)a.H + a.eps);
        for (int i = V * tid; i < a.H; i += step) {
            float r[V];
            load_resid<V, RF32>(kept, row + i, r);
            store_next<V, STREAM>(a, row, i, inv, r);
        }
    }
}

template <int V, bool RF32, bool STREAM>
void launch(const NormArgs &a, int T, int threads, int items, hipStream_t s) {
    const dim3 grid(T), block(threads);
    // One item holds eight values of each of 1024 threads, and is taken below 256 rows: a
    // bf16 stream of that is never large enough to be written past the caches.
    static_assert(255 * 8 * kMaxThreads * 2 < kStreamFrom, "one item, bf16, past the caches");
    if constexpr (RF32 || !STREAM)
        if (items == 1) {
            hipLaunchKernelGGL((block_norm_kernel<V, 1, RF32, STREAM>), grid, block, 0, s, a);
            return;
        }
    if (items <= 2)
        hipLaunchKernelGGL((block_norm_kernel<V, 2, RF32, STREAM>), grid, block, 0, s, a);
    else if (items <= 4)
        hipLaunchKernelGGL((block_norm_kernel<V, 4, RF32, STREAM>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((block_norm_kernel<V, 0, RF32, STREAM>), grid, block, 0, s, a);
}

}  // namespace

extern "C" int moe_block_norm(const uint16_t *add, int post_norm, const float *w_post, const void *gate, int gate_kind,
                              float scale, const void *resid, void *resid_out, int resid_type, const float *w_pre,
                              int T, int H, float eps, uint16_t *x_next, uint8_t *x_rows, void *stream) {
    if (T < 0 || H <= 0) return moe::fail(MOE_E_ARG, "block_norm: T=%d, H=%d", T, H);
    if (!(eps >= 0.0f) || eps > 1.0f) return moe::fail(MOE_E_ARG, "block_norm: eps=%g outside [0, 1]", (double)eps);
    if (resid_type != MOE_FP32 && resid_type != MOE_BF16)
        return moe::fail(MOE_E_ARG, "block_norm: resid_type=%d", resid_type);
    if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT)
        return moe::fail(MOE_E_ARG, "block_norm: gate_kind=%d", gate_kind);
    if (x_rows && H % 32) return moe::fail(MOE_E_SHAPE, "block_norm: MXFP4 rows need H %% 32 == 0, H=%d", H);
    if (H > kMaxH) return moe::fail(MOE_E_SHAPE, "block_norm: H=%d above %d", H, kMaxH);
    if (w_post && !post_norm) return moe::fail(MOE_E_ARG, "block_norm: w_post without post_norm");
    if (T == 0) return MOE_OK;
    if (!resid || (add && !resid_out) || (!add && !x_next && !x_rows))
        return moe::fail(MOE_E_ARG, "block_norm: NULL pointer");
    if (add && gate_kind != MOE_GATE_NONE && !gate) return moe::fail(MOE_E_ARG, "block_norm: NULL gate");
    const bool f32 = resid_type == MOE_FP32;
    const uintptr_t size = f32 ? 4 : 2;
    if ((((uintptr_t)add | (uintptr_t)x_next) % 2) || (((uintptr_t)resid | (uintptr_t)resid_out) % size) ||
        (((uintptr_t)w_post | (uintptr_t)w_pre) % 4) ||
        (add && gate_kind != MOE_GATE_NONE && (uintptr_t)gate % (gate_kind == MOE_GATE_ELEMENT ? 2 : 4)))
        return moe::fail(MOE_E_ARG, "block_norm: a pointer is not aligned to its type");
    const uintptr_t all = (uintptr_t)add | (uintptr_t)resid | (uintptr_t)resid_out | (uintptr_t)w_post |
                          (uintptr_t)w_pre | (uintptr_t)x_next |
                          (gate_kind == MOE_GATE_CHANNEL || gate_kind == MOE_GATE_ELEMENT ? (uintptr_t)gate : 0);
    const bool wide = H % 8 == 0 && all % 16 == 0;  // 16-byte loads of eight values
    if (x_rows && (!wide || (uintptr_t)x_rows % 16))
        return moe::fail(MOE_E_ARG, "block_norm: MXFP4 rows need every pointer 16-byte aligned");
    const int V = wide ? 8 : 1;
    const int units = (H + V - 1) / V;
    const bool stream_out = (int64_t)T * H * (int64_t)size >= kStreamFrom;
    // Few rows: one item per thread, the most lanes on a row.  A row per CU and more: two
    // (2048 x 6144: 27.0 us, with one item 28.5, with three 28.0; 301 x 1001: 4.8, 5.4, 5.2).
    int items = T < 256 ? 1 : 2;
    while (items < 4 && units > items * kMaxThreads) items *= 2;
    int threads = ((units + items - 1) / items + 63) / 64 * 64;
    if (threads > kMaxThreads) threads = kMaxThreads, items = kReread;
    hipStream_t s = (hipStream_t)stream;
    for (int t0 = 0; t0 < T; t0 += kMaxRows) {
        const int n = T - t0 < kMaxRows ? T - t0 : kMaxRows;
        const size_t e = (size_t)t0 * H;  // elements before this launch's first row
        const int kind = add ? gate_kind : MOE_GATE_NONE;
        NormArgs a{add ? add + e : nullptr,
                   w_post,
                   kind == MOE_GATE_ROW       ? (const void *)((const float *)gate + t0)
                   : kind == MOE_GATE_ELEMENT ? (const void *)((const uint16_t *)gate + e)
                                              : gate,
                   (const char *)resid + e * size,
                   add ? (char *)resid_out + e * size : nullptr,
                   w_pre,
                   x_next ? x_next + e : nullptr,
                   x_rows ? x_rows + t0 * moe::mx_row_bytes(H) : nullptr,
                   H,
                   kind,
                   post_norm != 0,
                   scale,
                   eps};
        if (!wide)
            f32 ? launch<1, true, false>(a, n, threads, items, s) : launch<1, false, false>(a, n, threads, items, s);
        else if (stream_out)
            f32 ? launch<8, true, true>(a, n, threads, items, s) : launch<8, false, true>(a, n, threads, items, s);
        else
            f32 ? launch<8, true, false>(a, n, threads, items, s) : launch<8, false, false>(a, n, threads, items, s);
        MOE_LAUNCH_CHECK("block_norm_kernel");
        if (T - t0 <= kMaxRows) break;
    }
    return MOE_OK;
}
