// Device side of the expert relayouts: token rows moved to expert-major rows
// and back (include/vf_relayout.h, "Expert relayouts").
//
// plan   row_of[i] = offsets[e_i] + #{j < i : e_j = e_i}: a stable counting
//        sort of the slots i by expert.
// pack   packed[row_of[t,k]] = x[t]
// merge  out[t] = sum_k w[t,k] * packed[row_of[t,k]]
// merge backward
//        dpacked[row_of[t,k]] = w[t,k] * dout[t]
//        dw[t,k] = sum_m dout[t,m] * packed[row_of[t,k],m]
//
// All of the row kernels are bound by HBM: they move whole rows and do a few
// operations per element.  They walk the token side, so a token row is read
// (or written) once, whatever K is, and every packed row is read (or written)
// once as a whole; the row index is one 4-byte load per slot.
//
// Work split: a warp takes one span, kSpan consecutive columns of one token.
// A lane holds 8 columns of it as 8 / VW units of VW elements; unit u of lane
// l starts at column u * 32 * VW + l * VW, so each access of a warp covers
// 32 * VW consecutive elements whatever VW is.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "quant_kernel.cuh"

namespace vf {

constexpr int kSpan = 256;               // columns of a warp's span
constexpr int kExpertThreads = 256;      // threads per block of the row kernels
constexpr int kExpertWarps = kExpertThreads / 32;
constexpr int kPlanThreads = 1024;
constexpr int kGapBlocks = 4;            // blocks that zero one expert's gap rows
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Element types: storage S, exact widening to float32, one rounding back.
struct Bf16 {
    using S = uint16_t;
    static __device__ __forceinline__ float widen(S v) { return bf16_bits_to_float(v); }
    static __device__ __forceinline__ S round(float f) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
};
struct F16 {
    using S = uint16_t;
    static __device__ __forceinline__ float widen(S v) {
        return __half2float(__ushort_as_half(v));
    }
    static __device__ __forceinline__ S round(float f) {
        return __half_as_ushort(__float2half_rn(f));
    }
};
struct F32 {
    using S = uint32_t;
    static __device__ __forceinline__ float widen(S v) { return __uint_as_float(v); }
    static __device__ __forceinline__ S round(float f) { return __float_as_uint(f); }
};

template <int BYTES> struct UnitBits;
template <> struct UnitBits<16> { using T = uint4; };
template <> struct UnitBits<8> { using T = uint2; };
template <> struct UnitBits<4> { using T = uint32_t; };
template <> struct UnitBits<2> { using T = uint16_t; };
template <> struct UnitBits<1> { using T = uint8_t; };

template <class S, int VW>
__device__ __forceinline__ void load_unit(const S *p, S *v) {
    using B = typename UnitBits<int(sizeof(S)) * VW>::T;
    const B b = *reinterpret_cast<const B *>(p);
    memcpy(v, &b, sizeof(b));
}

template <class S, int VW>
__device__ __forceinline__ void store_unit(S *p, const S *v) {
    using B = typename UnitBits<int(sizeof(S)) * VW>::T;
    B b;
    memcpy(&b, v, sizeof(b));
    *reinterpret_cast<B *>(p) = b;
}

// Arguments of the row kernels.
struct ExpertArgs {
    const int32_t *row_of;        // [T][K]
    const int32_t *counts, *offsets;
    void *tokens;                 // [T][M] view
    int64_t token_stride, col_stride;    // col_stride is 1 on every path with VW > 1
    void *packed;                 // [rows][M]
    const float *weights;         // [T][K] view, or null
    int64_t weight_stride, weight_col_stride;
    uint8_t *codes;
    float *scales;
    void *grad_packed;
    float *grad_weights;
    int64_t T, M;
    int32_t K, rows, E, group;
    int32_t spans;                // ceil(M / kSpan)
    int32_t groups;               // ceil(M / group)
    uint32_t row_blocks;          // blocks of the row part; the rest zero the gap rows
};

// First column of unit u in a span.
template <int VW>
__device__ __forceinline__ int unit_col(int u, int lane) { return u * 32 * VW + lane * VW; }

// The span's units of a row; units past the row's end are zeros.
template <class S, int VW>
__device__ __forceinline__ void load_span(const S *row, int64_t stride, int64_t col0, int64_t M,
                                          int lane, S (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8 / VW; ++u) {
        const int64_t c = col0 + unit_col<VW>(u, lane);
#pragma unroll
        for (int i = 0; i < VW; ++i) v[u * VW + i] = S(0);
        if (c < M) load_unit<S, VW>(row + c * stride, v + u * VW);
    }
}

template <class S, int VW>
__device__ __forceinline__ void store_span(S *row, int64_t stride, int64_t col0, int64_t M,
                                           int lane, const S (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8 / VW; ++u) {
        const int64_t c = col0 + unit_col<VW>(u, lane);
        if (c < M) store_unit<S, VW>(row + c * stride, v + u * VW);
    }
}

// Slot k's row of token t, or -1 (dropped, or a row that does not exist).
__device__ __forceinline__ int slot_row(const ExpertArgs &a, int64_t t, int k) {
    const int r = a.row_of[t * a.K + k];
    return r >= 0 && r < a.rows ? r : -1;
}

// Zeros for the gap rows of every expert: block `b` of kGapBlocks * E.
template <class S, int VW>
__device__ __forceinline__ void zero_gaps(const ExpertArgs &a, void *packed, uint32_t b) {
    const int e = int(b / kGapBlocks);
    const int64_t first = int64_t(a.offsets[e]) + a.counts[e] + b % kGapBlocks;
    const int64_t end = min(int64_t(a.offsets[e + 1]), int64_t(a.rows));
    S zero[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) zero[i] = S(0);
    for (int64_t r = max(first, int64_t(0)); r < end; r += kGapBlocks) {
        S *row = static_cast<S *>(packed) + r * a.M;
        for (int64_t c = int64_t(threadIdx.x) * VW; c < a.M; c += kExpertThreads * VW)
            store_unit<S, VW>(row + c, zero);
    }
}

// ---- 8-bit checkpoints of a span ----------------------------------------------

// Quantises one span of a row (bfloat16 patterns v; zeros past the row's end)
// group by group and stores its codes and scales.  All 32 lanes are here.  A
// group lies within one span (group divides kSpan): within one unit of
// consecutive lanes, or over consecutive units of all lanes.
template <int VW, int FMT>
__device__ __forceinline__ void checkpoint_span(const ExpertArgs &a, int64_t row, int64_t col0,
                                                int lane, const uint16_t (&v)[8]) {
    constexpr int U = 8 / VW;
    const int lanes = min(32, a.group / VW);               // of a unit that share a group
    const int units = max(1, a.group / (32 * VW));         // that share a group
    uint32_t m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        m[u] = 0;
#pragma unroll
        for (int i = 0; i < VW; ++i) m[u] = max(m[u], uint32_t(v[u * VW + i]) & 0x7FFFu);
        for (int o = lanes >> 1; o > 0; o >>= 1) m[u] = max(m[u], __shfl_xor_sync(kAll, m[u], o));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = col0 + unit_col<VW>(u, lane);
        uint32_t top_mag = 0;
#pragma unroll
        for (int w = 0; w < U; ++w)
            if (w / units == u / units) top_mag = max(top_mag, m[w]);
        const float amax = bf16_bits_to_float(top_mag), top = top_code<FMT>();
        const bool lost = non_finite_magnitude(top_mag);
        const bool live = !lost && amax >= 0x1p-96f;
        const float inv = live ? __fdiv_rn(top, amax) : 0.0f;
        if (c >= a.M) continue;
        if (lane % lanes == 0 && u % units == 0)
            a.scales[row * a.groups + c / a.group] =
                lost ? __uint_as_float(kLostScaleBits) : live ? __fdiv_rn(amax, top) : 0.0f;
        uint16_t h[VW];
        uint8_t code[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) h[i] = v[u * VW + i];
        encode<VW, FMT>(h, inv, live, code);
        store_unit<uint8_t, VW>(a.codes + row * a.M + c, code);
    }
}

// The float32 values that a span of a checkpointed row stands for: code times
// scale, NaN where the scale is not finite.
template <int VW, int FMT>
__device__ __forceinline__ void restore_span(const ExpertArgs &a, int64_t row, int64_t col0,
                                             int lane, float (&f)[8]) {
#pragma unroll
    for (int u = 0; u < 8 / VW; ++u) {
        const int64_t c = col0 + unit_col<VW>(u, lane);
#pragma unroll
        for (int i = 0; i < VW; ++i) f[u * VW + i] = 0.0f;
        if (c >= a.M) continue;
        uint8_t code[VW];
        load_unit<uint8_t, VW>(a.codes + row * a.M + c, code);
        const float s = a.scales[row * a.groups + c / a.group];
#pragma unroll
        for (int i = 0; i < VW; ++i)
            f[u * VW + i] = lost_scale(s) ? __uint_as_float(kLostScaleBits)
                                          : __fmul_rn(code_value<FMT>(code[i]), s);
    }
}

// ---- row kernels ---------------------------------------------------------------

// Pack; FMT != 0 also keeps the tokens' checkpoint.  Walks (token, span).
template <class S, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads)
expert_pack_rows(const __grid_constant__ ExpertArgs a) {
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<S, VW>(a, a.packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    const int64_t items = a.T * a.spans;
    for (int64_t it = int64_t(blockIdx.x) * kExpertWarps + (threadIdx.x >> 5); it < items;
         it += int64_t(a.row_blocks) * kExpertWarps) {
        const int64_t t = it / a.spans, col0 = (it - t * a.spans) * kSpan;
        S v[8];
        load_span<S, VW>(static_cast<const S *>(a.tokens) + t * a.token_stride, a.col_stride,
                         col0, a.M, lane, v);
        for (int k = 0; k < a.K; ++k) {
            const int r = slot_row(a, t, k);
            if (r >= 0)
                store_span<S, VW>(static_cast<S *>(a.packed) + int64_t(r) * a.M, 1, col0, a.M,
                                  lane, v);
        }
        if constexpr (FMT != 0) checkpoint_span<VW, FMT>(a, t, col0, lane, v);
    }
}

// The pack of a checkpoint of the tokens: dequantised bfloat16 rows.
template <int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads)
expert_restore_rows(const __grid_constant__ ExpertArgs a) {
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<uint16_t, VW>(a, a.packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    const int64_t items = a.T * a.spans;
    for (int64_t it = int64_t(blockIdx.x) * kExpertWarps + (threadIdx.x >> 5); it < items;
         it += int64_t(a.row_blocks) * kExpertWarps) {
        const int64_t t = it / a.spans, col0 = (it - t * a.spans) * kSpan;
        float f[8];
        restore_span<VW, FMT>(a, t, col0, lane, f);
        uint16_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = isnan(f[i]) ? uint16_t(kLostValue2 & 0xFFFFu) : Bf16::round(f[i]);
        for (int k = 0; k < a.K; ++k) {
            const int r = slot_row(a, t, k);
            if (r >= 0)
                store_span<uint16_t, VW>(static_cast<uint16_t *>(a.packed) + int64_t(r) * a.M, 1,
                                         col0, a.M, lane, v);
        }
    }
}

// Merge; FMT != 0 also keeps the packed rows' checkpoint (a row belongs to one
// slot, so it is read once).  Walks (token, span).
template <class E, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads)
expert_merge_rows(const __grid_constant__ ExpertArgs a) {
    using S = typename E::S;
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31);
    const int64_t items = a.T * a.spans;
    for (int64_t it = int64_t(blockIdx.x) * kExpertWarps + (threadIdx.x >> 5); it < items;
         it += int64_t(a.row_blocks) * kExpertWarps) {
        const int64_t t = it / a.spans, col0 = (it - t * a.spans) * kSpan;
        float acc[8] = {};
        for (int k = 0; k < a.K; ++k) {
            const int r = slot_row(a, t, k);
            if (r < 0) continue;
            S v[8];
            load_span<S, VW>(static_cast<const S *>(a.packed) + int64_t(r) * a.M, 1, col0, a.M,
                             lane, v);
            const float w = a.weights == nullptr
                                ? 1.0f
                                : a.weights[t * a.weight_stride + k * a.weight_col_stride];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(w, E::widen(v[i]), acc[i]);
            if constexpr (FMT != 0) checkpoint_span<VW, FMT>(a, r, col0, lane, v);
        }
        S out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = E::round(acc[i]);
        store_span<S, VW>(static_cast<S *>(a.tokens) + t * a.token_stride, a.col_stride, col0,
                          a.M, lane, out);
    }
}

// Gradients of the merge; FMT != 0: the packed rows come from a checkpoint.  A
// warp walks the spans of a token, so each weight's gradient is one sum.
template <class E, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads)
expert_merge_backward_rows(const __grid_constant__ ExpertArgs a) {
    using S = typename E::S;
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<S, VW>(a, a.grad_packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    for (int64_t t = int64_t(blockIdx.x) * kExpertWarps + (threadIdx.x >> 5); t < a.T;
         t += int64_t(a.row_blocks) * kExpertWarps) {
        for (int k = 0; k < a.K; ++k) {
            const int r = slot_row(a, t, k);
            float dot = 0.0f;
            if (r >= 0) {
                const float w = a.weights[t * a.weight_stride + k * a.weight_col_stride];
                for (int64_t col0 = 0; col0 < a.M; col0 += kSpan) {
                    S g[8], d[8];
                    float y[8];
                    load_span<S, VW>(static_cast<const S *>(a.tokens) + t * a.token_stride,
                                     a.col_stride, col0, a.M, lane, g);
                    if constexpr (FMT != 0) {
                        restore_span<VW, FMT>(a, r, col0, lane, y);
                    } else {
                        S v[8];
                        load_span<S, VW>(static_cast<const S *>(a.packed) + int64_t(r) * a.M, 1,
                                         col0, a.M, lane, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = E::widen(v[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot = __fmaf_rn(E::widen(g[i]), y[i], dot);
                        d[i] = E::round(w * E::widen(g[i]));
                    }
                    store_span<S, VW>(static_cast<S *>(a.grad_packed) + int64_t(r) * a.M, 1,
                                      col0, a.M, lane, d);
                }
            }
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
            if (lane == 0) a.grad_weights[t * a.K + k] = dot;
        }
    }
}

// ---- the plan ------------------------------------------------------------------

struct PlanArgs {
    const void *experts;          // [T][K] view
    int64_t token_stride, slot_stride;
    int32_t *row_of, *slot_of, *counts, *offsets;
    int32_t *block_counts;        // [blocks][E], or null when there is one block
    int32_t K, E, align, slots, rows;
    int32_t tile;                 // slots of a block, a multiple of 32 * warps
    int32_t warps;                // warps that sort; each keeps E counters
};

// Expert of slot i, or -1 when the slot is dropped (or i is past the end).
template <class I>
__device__ __forceinline__ int slot_expert(const PlanArgs &a, int i, int end) {
    if (i >= end) return -1;
    const int t = i / a.K;
    const I e = static_cast<const I *>(a.experts)[t * a.token_stride +
                                                  int64_t(i - t * a.K) * a.slot_stride];
    return e >= 0 && e < I(a.E) ? int(e) : -1;
}

// Counts of each expert in the block's tile.
template <class I>
__global__ void __launch_bounds__(kPlanThreads)
expert_plan_counts(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t cnt[];                       // [E]
    wait_for_previous_grid();
    for (int e = int(threadIdx.x); e < a.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    const int first = int(blockIdx.x) * a.tile;
    const int end = min(a.slots, first + a.tile);
    for (int i = first + int(threadIdx.x); i < end; i += kPlanThreads) {
        const int e = slot_expert<I>(a, i, end);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = int(threadIdx.x); e < a.E; e += kPlanThreads)
        a.block_counts[int64_t(blockIdx.x) * a.E + e] = cnt[e];
}

// Inclusive prefix sum over the block's threads; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += up;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kAll, s, o);
            if (lane >= o) s += up;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    *total = warp_sums[31];
    __syncthreads();
    return v;
}

// Rows of the slots of the block's tile.  Each of a.warps warps owns a
// contiguous part of the tile: it counts its experts, the counts of the warps
// and blocks before it and the experts' offsets give its first row of every
// expert, and a second walk in slot order hands the rows out.
template <class I>
__global__ void __launch_bounds__(kPlanThreads)
expert_plan_rows(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t smem[];
    int32_t *cnt = smem;                                   // [warps][E]
    int32_t *base = smem + a.warps * a.E;                  // [E]
    __shared__ int32_t warp_sums[32];
    __shared__ int32_t end_row;
    wait_for_previous_grid();
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < a.warps * a.E; i += kPlanThreads) cnt[i] = 0;
    __syncthreads();
    const int part = a.tile / a.warps;                     // a multiple of 32
    const int first = int(blockIdx.x) * a.tile + warp * part;
    const int end = warp < a.warps ? min(a.slots, first + part) : first;
    int32_t *mine = cnt + warp * a.E;
    for (int i = first + lane; i < end; i += 32) {
        const int e = slot_expert<I>(a, i, end);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // offsets of the experts, and each warp's first row of every expert
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int before = 0, all = 0;
        if (e < a.E) {
            int own = 0;
            for (int w = 0; w < a.warps; ++w) {
                const int c = cnt[w * a.E + e];
                cnt[w * a.E + e] = own;
                own += c;
            }
            all = own;
            if (a.block_counts != nullptr) {
                all = 0;
                for (int b = 0; b < int(gridDim.x); ++b) {
                    if (b == int(blockIdx.x)) before = all;
                    all += a.block_counts[int64_t(b) * a.E + e];
                }
            }
        }
        // (in 64 bits: a count next to 2^31 rounded up would not fit)
        const int padded = int((int64_t(all) + a.align - 1) / a.align * a.align);
        int total;
        const int incl = block_scan(padded, warp_sums, &total);
        const int off = carry + incl - padded;
        carry += total;
        if (e < a.E) {
            base[e] = off + before;
            if (blockIdx.x == 0) {
                a.counts[e] = all;
                a.offsets[e] = off;
                if (e == a.E - 1) a.offsets[a.E] = off + padded;
            }
            // the gap rows behind expert e belong to no slot
            if (e % int(gridDim.x) == int(blockIdx.x))
                for (int r = off + all; r < off + padded; ++r) a.slot_of[r] = -1;
        }
    }
    if (tid == 0) end_row = carry;
    __syncthreads();
    for (int64_t r = int64_t(end_row) + int64_t(blockIdx.x) * kPlanThreads + tid; r < a.rows;
         r += int64_t(gridDim.x) * kPlanThreads)
        a.slot_of[r] = -1;
    for (int i0 = first; i0 < end; i0 += 32) {             // warp-uniform
        const int i = i0 + lane;
        const int e = slot_expert<I>(a, i, end);
        const uint32_t same = __match_any_sync(kAll, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int at = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] = at + __popc(same);
        __syncwarp();
        const int row = e >= 0 ? base[e] + at + rank : -1;
        if (i < end) a.row_of[i] = row;
        if (row >= 0) a.slot_of[row] = i;
    }
}

}  // namespace vf
