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
// once as a whole; the row index is one 4-byte load per slot.  (The merge's
// backward pass loads its token row once for every 2 or 4 slots; from the second
// time on it comes from the caches.)  Measured on GB300 (bf16, device time, bytes
// that cannot be avoided over it):
//   pack            T = 55,414, K = 8, M = 3,584   510 us   6.79 TB/s
//   merge           the same                       498 us   6.96 TB/s
//   merge backward  T = 4,096, K = 8, M = 4,096     85 us   6.53 TB/s
//   plan            1.6 M slots, 256 experts        23 us   bound by latency: two
//                   grids, each a walk of some 300 slots per warp in slot order,
//                   with one block of 1,024 threads to an SM (54 registers)
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
constexpr int kMergeResident = 4;        // blocks of the merge that fit an SM
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Element types: storage S; exact widening to float32 and one rounding back,
// for the two elements of a 32-bit word (one for F32).
struct Bf16 {
    using S = uint16_t;
    static __device__ __forceinline__ void widen(uint32_t w, float *f) {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint32_t round(const float *f) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
};
struct F16 {
    using S = uint16_t;
    static __device__ __forceinline__ void widen(uint32_t w, float *f) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        f[0] = v.x;
        f[1] = v.y;
    }
    static __device__ __forceinline__ uint32_t round(const float *f) {
        const __half2 h = __floats2half2_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
struct F32 {
    using S = uint32_t;
    static __device__ __forceinline__ void widen(uint32_t w, float *f) {
        f[0] = __uint_as_float(w);
    }
    static __device__ __forceinline__ uint32_t round(const float *f) {
        return __float_as_uint(f[0]);
    }
};

// Marks a loaded value as used, without an instruction: the compiler starts
// computing with no row before it has issued the loads of all rows that are
// marked.  Left alone it may start on the first row as soon as that is there, and
// issue the last row's loads behind it (the backward pass from INT8 codes at
// T = 55,414, K = 4, M = 3,584 took 478 us, 414 so; the merge that quantises was
// faster without).
__device__ __forceinline__ void loaded(uint32_t &x) { asm volatile("" : "+r"(x)); }
__device__ __forceinline__ void loaded(float &x) { asm volatile("" : "+f"(x)); }
__device__ __forceinline__ void loaded(uint2 &x) {
    loaded(x.x);
    loaded(x.y);
}
__device__ __forceinline__ void loaded(uint4 &x) {
    loaded(x.x);
    loaded(x.y);
    loaded(x.z);
    loaded(x.w);
}

// A lane's 8 columns of a span, as 32-bit words: unit u's elements at
// [u * VW, u * VW + VW).
template <class S> constexpr int kWords = 8 * int(sizeof(S)) / 4;
template <class S> struct Lane8 {
    uint32_t w[kWords<S>];
};

template <int BYTES> struct UnitBits;
template <> struct UnitBits<16> { using T = uint4; };
template <> struct UnitBits<8> { using T = uint2; };
template <> struct UnitBits<4> { using T = uint32_t; };
template <> struct UnitBits<2> { using T = uint16_t; };
template <> struct UnitBits<1> { using T = uint8_t; };

template <class S, int VW>
__device__ __forceinline__ void store_unit(S *p, const S *v) {
    using B = typename UnitBits<int(sizeof(S)) * VW>::T;
    B b;
    memcpy(&b, v, sizeof(b));
    *reinterpret_cast<B *>(p) = b;
}

// Packed rows whose loads a lane has in flight in the merge and its backward
// pass: 64 bytes.
template <class S> constexpr int kRowsInFlight = sizeof(S) == 2 ? 4 : 2;

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
    int64_t T;
    int32_t M, K, rows, E;
    int32_t group_log2;           // elements of a checkpoint's group
    int32_t spans;                // ceil(M / kSpan)
    int32_t groups;               // ceil(M / group)
    int32_t step_tokens, step_spans;     // row_blocks * kExpertWarps items, as Walk counts
    int32_t token_warps;          // merge backward: warps that share a token
    uint32_t row_blocks;          // blocks of the row part; the rest zero the gap rows,
    int32_t gap_blocks;           // so many of them to an expert
};

// The (token, span) items of the row blocks, one per warp at a time, spans
// fastest: the block's warps share a token's routing and cover consecutive
// columns.  The division is done once; a step adds to both numbers.
struct Walk {
    int64_t t;
    int s;

    __device__ __forceinline__ explicit Walk(const ExpertArgs &a) {
        // row_blocks * kExpertWarps fits 32 bits
        const uint32_t it = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
        t = it / uint32_t(a.spans);
        s = int(it - uint32_t(t) * uint32_t(a.spans));
    }
    __device__ __forceinline__ void step(const ExpertArgs &a) {
        t += a.step_tokens;
        s += a.step_spans;
        if (s >= a.spans) {
            s -= a.spans;
            ++t;
        }
    }
};

// First column of unit u in a span.
template <int VW>
__device__ __forceinline__ int unit_col(int u, int lane) { return u * 32 * VW + lane * VW; }

// The lane's units of a row's span; units past the row's end, and all of them
// where `there` is false, are zeros.  Small units are loaded from a
// column clamped into the row (and from row 0 where there is none: the caller
// sees to it that a row exists) and zeroed afterwards: with a condition each, the
// loads of a span waited for one another (the merge of 20,000 tokens, K = 4,
// M = 2,049 took 662 us, 186 so, and 154 with the loads marked as well).
// kClampBelow: the unit size from which on the loads are predicated instead.
template <class S, int VW, int kClampBelow = 16>
__device__ __forceinline__ Lane8<S> load_span(const void *base, int64_t offset, int64_t stride,
                                              int col0, int M, int lane,
                                              bool there = true) {
    using B = typename UnitBits<int(sizeof(S)) * VW>::T;
    constexpr int U = 8 / VW;
    B b[U] = {};
    if constexpr (sizeof(B) >= kClampBelow) {
        const S *row = static_cast<const S *>(base) + offset;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = col0 + unit_col<VW>(u, lane);
            if (there && c < M) b[u] = *reinterpret_cast<const B *>(row + int64_t(c) * stride);
        }
    } else {
        const S *row = static_cast<const S *>(base) + (there ? offset : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = min(col0 + unit_col<VW>(u, lane), M - VW);
            b[u] = *reinterpret_cast<const B *>(row + int64_t(c) * stride);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (!there || col0 + unit_col<VW>(u, lane) >= M) b[u] = B{};
    }
    Lane8<S> v;
    if constexpr (sizeof(B) >= 4) {
        memcpy(v.w, b, sizeof(v.w));
    } else {
#pragma unroll
        for (int i = 0; i < kWords<S>; ++i) v.w[i] = uint32_t(b[2 * i]) | uint32_t(b[2 * i + 1]) << 16;
    }
    return v;
}

template <class S, int VW>
__device__ __forceinline__ void store_span(void *base, int64_t offset, int64_t stride,
                                           int col0, int M, int lane,
                                           const Lane8<S> &v) {
    S *row = static_cast<S *>(base) + offset;
#pragma unroll
    for (int u = 0; u < 8 / VW; ++u) {
        const int c = col0 + unit_col<VW>(u, lane);
        if (c < M)
            store_unit<S, VW>(row + int64_t(c) * stride, reinterpret_cast<const S *>(v.w) + u * VW);
    }
}

// Two float32 fused multiply-adds, a * b + c, in one instruction (sm_100 and
// later), each rounded once.
__device__ __forceinline__ float2 fma2_rn(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%6, %7};\n\t"
        "fma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

template <class E>
__device__ __forceinline__ void widen_span(const Lane8<typename E::S> &v, float (&f)[8]) {
    constexpr int N = 4 / int(sizeof(typename E::S));
#pragma unroll
    for (int i = 0; i < kWords<typename E::S>; ++i) E::widen(v.w[i], f + N * i);
}

template <class E>
__device__ __forceinline__ Lane8<typename E::S> round_span(const float (&f)[8]) {
    constexpr int N = 4 / int(sizeof(typename E::S));
    Lane8<typename E::S> v;
#pragma unroll
    for (int i = 0; i < kWords<typename E::S>; ++i) v.w[i] = E::round(f + N * i);
    return v;
}

// The routing of up to 32 slots of token t, k0 onward: lane j holds slot k0 + j's
// row, -1 when it is dropped, past K or the token past T, or when it names a row
// that does not exist, and its weight, 0 where the row is -1 (whatever is
// stored).  Both loads are issued at once.
struct Slots {
    int row;
    float weight;

    __device__ __forceinline__ Slots(const ExpertArgs &a, int64_t t, int k0, int lane,
                                     bool weighted) {
        const bool there = t < a.T && k0 + lane < a.K;
        row = there ? a.row_of[t * a.K + k0 + lane] : -1;
        weight = 1.0f;
        if (weighted && there)
            weight = a.weights[t * a.weight_stride + (k0 + lane) * a.weight_col_stride];
        if (row < 0 || row >= a.rows) {
            row = -1;
            weight = 0.0f;
        }
    }
};

// Zeros for the gap rows of every expert: block `b` of a.gap_blocks * E.
template <class S, int VW>
__device__ __forceinline__ void zero_gaps(const ExpertArgs &a, void *packed, uint32_t b) {
    const uint32_t shares = uint32_t(a.gap_blocks);
    const int e = int(b / shares);
    const int64_t first = int64_t(a.offsets[e]) + a.counts[e] + b % shares;
    const int64_t end = min(int64_t(a.offsets[e + 1]), int64_t(a.rows));
    const S zero[VW] = {};
    for (int64_t r = max(first, int64_t(0)); r < end; r += shares) {
        S *row = static_cast<S *>(packed) + r * a.M;
        for (int64_t c = int64_t(threadIdx.x) * VW; c < a.M; c += int64_t(blockDim.x) * VW)
            store_unit<S, VW>(row + c, zero);
    }
}

// ---- 8-bit checkpoints of a span ----------------------------------------------

// fl(top / M) and fl(M / top) of the 128 bfloat16 mantissas M, as bits, in
// shared memory: quant_kernel.cuh derives a row's inverse and scale from them
// without a division.  The exponent's bias is folded in, so that adding or
// subtracting the group's exponent field gives the result.
struct ScaleTable {
    uint32_t inv[kMantissas], scale[kMantissas];
};

constexpr uint32_t kBias = 127u << 23;

template <int FMT>
__device__ __forceinline__ void fill_table(ScaleTable &tab) {
    const float top = top_code<FMT>();
    for (int i = int(threadIdx.x); i < kMantissas; i += int(blockDim.x)) {
        const float M = 1.0f + float(i) * (1.0f / 128.0f);      // exact
        tab.inv[i] = __float_as_uint(__fdiv_rn(top, M)) + kBias;
        tab.scale[i] = __float_as_uint(__fdiv_rn(M, top)) - kBias;
    }
    __syncthreads();
}

// 1 / scale of a group whose largest magnitude is the bfloat16 pattern m; 0
// where the group is not live (amax < 2^-96, or not finite).
__device__ __forceinline__ bool live_group(uint32_t m) { return m - 0x0F80u < 0x7F80u - 0x0F80u; }

__device__ __forceinline__ float group_inverse(const ScaleTable &tab, uint32_t m) {
    const uint32_t bits = tab.inv[m & 0x7Fu] - ((m << 16) & 0x7F800000u);
    return live_group(m) ? __uint_as_float(bits) : 0.0f;
}

__device__ __forceinline__ float group_scale(const ScaleTable &tab, uint32_t m) {
    if (non_finite_magnitude(m)) return __uint_as_float(kLostScaleBits);
    const uint32_t bits = tab.scale[m & 0x7Fu] + ((m << 16) & 0x7F800000u);
    return live_group(m) ? __uint_as_float(bits) : 0.0f;
}

// Quantises one span of a row (zeros past the row's end) group by group and
// stores its codes and scales.  All 32 lanes are here.  A group lies within one
// span (its size divides kSpan): within one unit, over consecutive lanes, or
// over consecutive units of all lanes.
template <int VW, int FMT>
__device__ __forceinline__ void checkpoint_span(const ExpertArgs &a, const ScaleTable &tab,
                                                int64_t row, int col0, int lane,
                                                const Lane8<uint16_t> &v) {
    static_assert(VW < 8, "expert_q_kernel.cuh has the form for 16-byte accesses");
    constexpr int U = 8 / VW;
    const int lanes = min(32, (1 << a.group_log2) / VW);        // of a unit that share a group
    const int units = max(1, (1 << a.group_log2) / (32 * VW));  // that share a group
    const uint16_t *h = reinterpret_cast<const uint16_t *>(v.w);
    uint32_t m[U];
    float inv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        m[u] = 0;
#pragma unroll
        for (int i = 0; i < VW; ++i) m[u] = max(m[u], uint32_t(h[u * VW + i]) & 0x7FFFu);
    }
    // over the units that share a group, then over the lanes, once per group
#pragma unroll
    for (int o = 1; o < U; o <<= 1)
        if (o < units) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (!(u & o)) m[u] = m[u | o] = max(m[u], m[u | o]);
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if ((u & (units - 1)) == 0) {
            for (int o = lanes >> 1; o > 0; o >>= 1)
                m[u] = max(m[u], __shfl_xor_sync(kAll, m[u], o));
            inv[u] = group_inverse(tab, m[u]);
        } else {                                                // as its group's first unit
            m[u] = m[u & (u - 1)];
            inv[u] = inv[u & (u - 1)];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = col0 + unit_col<VW>(u, lane);
        if (c >= a.M) continue;
        if ((c & ((1 << a.group_log2) - 1)) == 0)
            a.scales[row * a.groups + (c >> a.group_log2)] = group_scale(tab, m[u]);
        uint16_t x[VW];
        uint8_t code[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) x[i] = h[u * VW + i];
        encode<VW, FMT>(x, inv[u], live_group(m[u]), code);
        store_unit<uint8_t, VW>(a.codes + row * a.M + c, code);
    }
}

// The lane's codes of a span of a checkpointed row and the scales of its units;
// zeros where there are none (loads as in load_span).
template <int VW> struct KeptLane {
    typename UnitBits<VW>::T code[8 / VW];
    float scale[8 / VW];

    __device__ __forceinline__ uint2 words() const {
        uint2 w = make_uint2(0, 0);
#pragma unroll
        for (int u = 0; u < 8 / VW; ++u) {
            const uint32_t x = uint32_t(code[u]) << (8 * (u * VW % 4));
            (u * VW < 4 ? w.x : w.y) |= x;
        }
        return w;
    }
};

template <int VW>
__device__ __forceinline__ KeptLane<VW> load_kept(const ExpertArgs &a, int64_t row, int col0,
                                                  int lane, bool there = true) {
    using B = typename UnitBits<VW>::T;
    constexpr int U = 8 / VW;
    KeptLane<VW> q;
    if (!there) row = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = min(col0 + unit_col<VW>(u, lane), a.M - VW);
        q.code[u] = *reinterpret_cast<const B *>(a.codes + row * a.M + c);
        q.scale[u] = a.scales[row * a.groups + (c >> a.group_log2)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (!there || col0 + unit_col<VW>(u, lane) >= a.M) {
            q.code[u] = B(0);
            q.scale[u] = 0.0f;
        }
    return q;
}

// Code values of the lane's columns, as float32 (exact).
template <int FMT>
__device__ __forceinline__ void code_values(uint2 code, float (&f)[8]) {
    const uint32_t w[2] = {code.x, code.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == kFmtInt8) {
            const uint32_t u = w[h] ^ 0x80808080u;               // code + 128, per byte
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[4 * h + i] = __fsub_rn(
                    __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | i)), 8388736.0f);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                    __nv_fp8x2_storage_t((w[h] >> (16 * i)) & 0xFFFFu), __NV_E4M3);
                const float2 p = __half22float2(__half2(hr));    // exact: E4M3 fits in half
                f[4 * h + 2 * i] = p.x;
                f[4 * h + 2 * i + 1] = p.y;
            }
        }
    }
}

__device__ __forceinline__ float finite_or_nan(float s) {
    return lost_scale(s) ? __uint_as_float(kLostScaleBits) : s;
}

// ---- row kernels ---------------------------------------------------------------

// Pack; FMT != 0 also keeps the tokens' checkpoint.  Walks (token, span).
template <class S, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads)
expert_pack_rows(const __grid_constant__ ExpertArgs a) {
    __shared__ ScaleTable tab;
    if constexpr (FMT != 0) fill_table<FMT>(tab);
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<S, VW>(a, a.packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int col0 = at.s * kSpan;
        Slots slots(a, at.t, 0, lane, false);
        const Lane8<S> v = load_span<S, VW>(a.tokens, at.t * a.token_stride, a.col_stride, col0,
                                            a.M, lane);
        for (int k0 = 0; k0 < a.K; k0 += 32) {
            if (k0 > 0) slots = Slots(a, at.t, k0, lane, false);
            for (int j = 0; j < min(32, a.K - k0); ++j) {
                const int r = __shfl_sync(kAll, slots.row, j);
                if (r >= 0) store_span<S, VW>(a.packed, int64_t(r) * a.M, 1, col0, a.M, lane, v);
            }
        }
        if constexpr (FMT != 0) checkpoint_span<VW, FMT>(a, tab, at.t, col0, lane, v);
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
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int col0 = at.s * kSpan;
        Slots slots(a, at.t, 0, lane, false);
        const KeptLane<VW> q = load_kept<VW>(a, at.t, col0, lane);
        float f[8];
        code_values<FMT>(q.words(), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], q.scale[i / VW]);
        Lane8<uint16_t> v = round_span<Bf16>(f);
        // a lost group arrives as one NaN pattern
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lost_scale(q.scale[i / VW]))
                reinterpret_cast<uint16_t *>(v.w)[i] = uint16_t(kLostValue2 & 0xFFFFu);
        for (int k0 = 0; k0 < a.K; k0 += 32) {
            if (k0 > 0) slots = Slots(a, at.t, k0, lane, false);
            for (int j = 0; j < min(32, a.K - k0); ++j) {
                const int r = __shfl_sync(kAll, slots.row, j);
                if (r >= 0)
                    store_span<uint16_t, VW>(a.packed, int64_t(r) * a.M, 1, col0, a.M, lane, v);
            }
        }
    }
}

// Merge; FMT != 0 also keeps the packed rows' checkpoint (a row belongs to one
// slot, so it is read once).  Walks (token, span).  Four resident blocks with
// four rows in flight (64 registers) were faster than three with eight (499 and
// 539 us at T = 55,414, K = 8, M = 3,584); loading the next item's routing ahead
// made the warps drift apart and cost more than it hid (750 us and up).
template <class E, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads,
                                  VW * sizeof(typename E::S) < 16 ? 2 : kMergeResident)
expert_merge_rows(const __grid_constant__ ExpertArgs a) {
    using S = typename E::S;
    constexpr int KU = kRowsInFlight<S>;
    __shared__ ScaleTable tab;
    if constexpr (FMT != 0) fill_table<FMT>(tab);
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31);
    const bool weighted = a.weights != nullptr;
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int col0 = at.s * kSpan;
        Slots slots(a, at.t, 0, lane, weighted);
        float acc[8] = {};
        for (int k0 = 0; k0 < a.K; k0 += KU) {
            if (k0 > 0 && k0 % 32 == 0) slots = Slots(a, at.t, k0, lane, weighted);
            Lane8<S> v[KU];
            int r[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                r[j] = __shfl_sync(kAll, slots.row, k0 % 32 + j);
                // (8-byte units at M = 2,052: 75 us predicated, 109 clamped; with a
                // checkpoint 325 and 295)
                v[j] = load_span<S, VW, FMT ? 16 : 8>(a.packed, int64_t(r[j]) * a.M, 1, col0,
                                                      a.M, lane, r[j] >= 0);
            }
            if constexpr (FMT == 0) {
#pragma unroll
                for (int j = 0; j < KU; ++j)
#pragma unroll
                    for (int i = 0; i < kWords<S>; ++i) loaded(v[j].w[i]);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const float w = __shfl_sync(kAll, slots.weight, k0 % 32 + j);
                float f[8];
                widen_span<E>(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 sum = fma2_rn(make_float2(w, w), make_float2(f[i], f[i + 1]),
                                               make_float2(acc[i], acc[i + 1]));
                    acc[i] = sum.x;
                    acc[i + 1] = sum.y;
                }
            }
            if constexpr (FMT != 0) {
#pragma unroll
                for (int j = 0; j < KU; ++j)
                    if (r[j] >= 0) checkpoint_span<VW, FMT>(a, tab, r[j], col0, lane, v[j]);
            }
        }
        store_span<S, VW>(a.tokens, at.t * a.token_stride, a.col_stride, col0, a.M, lane,
                          round_span<E>(acc));
    }
}

// The sums of N values over the warp's lanes (N a power of two, at most 32):
// lane l gets the sum of value l % N.  Each step halves the values a lane
// holds, so it takes N - 1 + log2(32 / N) shuffles, not 5 N.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o < N) {
            n >>= 1;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float give = up ? v[2 * i] : v[2 * i + 1];
                    const float keep = up ? v[2 * i + 1] : v[2 * i];
                    v[i] = keep + __shfl_xor_sync(kAll, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(kAll, v[0], o);
        }
    }
    return v[0];
}

// Gradients of the merge; FMT != 0: the packed rows come from a checkpoint.
// a.token_warps warps share a token's spans and add their parts of each
// weight's gradient up in shared memory, in warp order.  KU rows' loads are in
// flight at a time: four, in four resident blocks, 85 us at T = 4,096, K = 8,
// M = 4,096; eight in three 89, eight in two 129.
template <class E, int VW, int FMT>
__global__ void __launch_bounds__(kExpertThreads, VW * sizeof(typename E::S) < 16 ? 2 : 4)
expert_merge_backward_rows(const __grid_constant__ ExpertArgs a) {
    using S = typename E::S;
    constexpr int KU = kRowsInFlight<S>;
    __shared__ float parts[kExpertWarps][KU];
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<S, VW>(a, a.grad_packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int tokens = int(blockDim.x >> 5) / a.token_warps;     // of a block at a time
    const int part = warp % a.token_warps;
    for (int64_t t0 = int64_t(blockIdx.x) * tokens; t0 < a.T;    // block-uniform
         t0 += int64_t(a.row_blocks) * tokens) {
        const int64_t t = t0 + warp / a.token_warps;
        for (int k0 = 0; k0 < a.K; k0 += KU) {
            const Slots slots(a, t, k0, lane, true);
            float2 dots[KU] = {};                                // of even and odd columns
            // (with no packed rows at all, every slot is dropped)
            for (int s = t < a.T && a.rows > 0 ? part : a.spans; s < a.spans;
                 s += a.token_warps) {
                const int col0 = s * kSpan;
                const Lane8<S> gv = load_span<S, VW>(a.tokens, t * a.token_stride, a.col_stride,
                                                     col0, a.M, lane);
                Lane8<S> v[KU];
                KeptLane<VW> q[KU];
                int r[KU];
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    r[j] = __shfl_sync(kAll, slots.row, j);
                    if constexpr (FMT != 0)
                        q[j] = load_kept<VW>(a, r[j], col0, lane, r[j] >= 0);
                    else
                        v[j] = load_span<S, VW>(a.packed, int64_t(r[j]) * a.M, 1, col0, a.M,
                                                lane, r[j] >= 0);
                }
                if constexpr (FMT == 0) {
#pragma unroll
                    for (int j = 0; j < KU; ++j)
#pragma unroll
                        for (int i = 0; i < kWords<S>; ++i) loaded(v[j].w[i]);
                }
                float g[8];
                widen_span<E>(gv, g);
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    const float w = __shfl_sync(kAll, slots.weight, j);
                    float y[8], d[8];
                    if constexpr (FMT != 0) {
                        code_values<FMT>(q[j].words(), y);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = __fmul_rn(y[i], finite_or_nan(q[j].scale[i / VW]));
                    } else {
                        widen_span<E>(v[j], y);
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        dots[j] = fma2_rn(make_float2(g[i], g[i + 1]),
                                          make_float2(y[i], y[i + 1]), dots[j]);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 p = mul2_rn(make_float2(w, w), make_float2(g[i], g[i + 1]));
                        d[i] = p.x;
                        d[i + 1] = p.y;
                    }
                    if (r[j] >= 0)
                        store_span<S, VW>(a.grad_packed, int64_t(r[j]) * a.M, 1, col0, a.M, lane,
                                          round_span<E>(d));
                }
            }
            float dot[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j)
                // a dropped slot's gradient is 0; what was summed for it are products
                // of g and 0, NaN where g is not finite (skipping them took 344 us for
                // 262 at T = 20,000, K = 4, M = 2,049 from E4M3 codes, one select after
                // the warp's sum 93 for 85 at T = 4,096, K = 8, M = 4,096)
                dot[j] = __shfl_sync(kAll, slots.row, j) >= 0 ? dots[j].x + dots[j].y : 0.0f;
            const float sum = warp_sums<KU>(dot, lane);
            __syncthreads();                                     // parts is free again
            if (lane < KU) parts[warp][lane] = sum;
            __syncthreads();
            if (part == 0 && t < a.T && lane < KU && k0 + lane < a.K) {
                float all = 0.0f;
                for (int p = 0; p < a.token_warps; ++p) all += parts[warp + p][lane];
                a.grad_weights[t * a.K + k0 + lane] = all;
            }
        }
    }
}

// ---- the plan ------------------------------------------------------------------

struct PlanArgs {
    const void *experts;          // [T][K] view
    int64_t token_stride, slot_stride;
    int32_t *row_of, *slot_of, *counts, *offsets;
    int32_t *block_counts;        // [blocks][counts_stride(E)], with more than one block
    int32_t *warp_first;          // [blocks][warps][E], the same
    int32_t K, E, align, slots, rows;
    int32_t tile;                 // slots of a block, a multiple of 32 * warps
    int32_t warps;                // warps that sort; each keeps E counters
    int32_t flat;                 // the view is contiguous: no division per slot
};

// Experts of N slots i, i + 32, ...: their loads are issued together.  -1 for a
// dropped slot and past the end.
template <class I, int N>
__device__ __forceinline__ void slot_experts(const PlanArgs &a, int i, int end, int (&e)[N]) {
    I v[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int j = i + u * 32;
        v[u] = I(-1);
        if (j >= end) continue;
        const int t = a.flat ? 0 : j / a.K;
        v[u] = static_cast<const I *>(
            a.experts)[t * a.token_stride + int64_t(j - t * a.K) * a.slot_stride];
    }
#pragma unroll
    for (int u = 0; u < N; ++u) e[u] = v[u] >= 0 && v[u] < I(a.E) ? int(v[u]) : -1;
}

// What a warp keeps of each expert while it ranks: how many slots it has seen,
// and in which lanes of the current 32 slots it occurs.
struct Seen {
    uint32_t lanes;
    int32_t count;
};

// The block's part of the slots that a warp sorts.
struct PlanPart {
    int first, end;

    __device__ __forceinline__ explicit PlanPart(const PlanArgs &a) {
        const int warp = int(threadIdx.x >> 5);
        const int part = a.tile / a.warps;                 // a multiple of 32
        first = int(blockIdx.x) * a.tile + warp * part;
        end = warp < a.warps ? min(a.slots, first + part) : first;
    }
};

// Each slot's rank among the slots of its expert in the warp's part, to row_of
// (-1 for a dropped slot); seen[e].count ends as the part's number of e's slots.
// Which lanes share an expert is found in shared memory: every lane sets its bit
// (a match instruction, and ballots of each bit of the expert, were slower).
template <class I, int N>
__device__ __forceinline__ void rank_slots(const PlanArgs &a, const PlanPart &p, Seen *seen) {
    const int lane = int(threadIdx.x & 31);
    for (int i0 = p.first; i0 < p.end; i0 += 32 * N) {  // warp-uniform
        int e[N];
        slot_experts<I, N>(a, i0 + lane, p.end, e);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (i0 + u * 32 >= p.end) break;                     // warp-uniform
            const int i = i0 + u * 32 + lane;
            if (e[u] >= 0) atomicOr(&seen[e[u]].lanes, 1u << lane);
            __syncwarp();
            const Seen s = e[u] >= 0 ? seen[e[u]] : Seen{0u, 0};
            const int rank = __popc(s.lanes & ((1u << lane) - 1));
            __syncwarp();
            if (e[u] >= 0 && rank == 0) seen[e[u]] = Seen{0u, s.count + __popc(s.lanes)};
            __syncwarp();
            if (i < p.end) a.row_of[i] = e[u] >= 0 ? s.count + rank : -1;
        }
    }
}

// Ranks to rows: base[e] is the first row of the part's slots of e.  The experts
// are read a second time and row_of is the caller's memory, so what another writer
// does to either meanwhile may give a row that does not exist: such a slot is
// dropped, and nothing is stored outside slot_of.
template <class I, int N>
__device__ __forceinline__ void place_slots(const PlanArgs &a, const PlanPart &p,
                                            const int32_t *base) {
    const int lane = int(threadIdx.x & 31);
    for (int i0 = p.first + lane; i0 < p.end; i0 += 32 * N) {
        int e[N], row[N];
#pragma unroll
        for (int u = 0; u < N; ++u)
            row[u] = i0 + u * 32 < p.end ? a.row_of[i0 + u * 32] : -1;
        slot_experts<I, N>(a, i0, p.end, e);
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (e[u] >= 0) {
                const uint32_t r = uint32_t(row[u]) + uint32_t(base[e[u]]);
                const bool there = r < uint32_t(a.rows);
                a.row_of[i0 + u * 32] = there ? int(r) : -1;
                if (there) a.slot_of[r] = i0 + u * 32;
            }
    }
}

// Inclusive prefix sum over the block's threads (whole warps); `total` gets the
// sum.
__device__ __forceinline__ int block_scan(int v, int *warp_totals, int *total) {
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int warps = int(blockDim.x >> 5);
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += up;
    }
    if (lane == 31) warp_totals[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int s = lane < warps ? warp_totals[lane] : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kAll, s, o);
            if (lane >= o) s += up;
        }
        if (lane < warps) warp_totals[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_totals[warp - 1];
    *total = warp_totals[warps - 1];
    __syncthreads();
    return v;
}

// From the warps' counts of expert e to each warp's first rank; the sum.
__device__ __forceinline__ int warp_firsts(const PlanArgs &a, Seen *seen, int e) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < a.warps; ++w) {
        const int c = seen[w * a.E + e].count;
        seen[w * a.E + e].count = sum;
        sum += c;
    }
    return sum;
}

// Stride of block_counts: whole 16-byte vectors.
__host__ __device__ __forceinline__ int64_t counts_stride(int64_t E) { return (E + 3) / 4 * 4; }

// Adds up every expert's counts of all blocks, and of those before this one, in
// shared memory (both zero before).  A thread takes four experts of every
// shares-th block.
__device__ __forceinline__ void sum_blocks(const PlanArgs &a, int32_t *all, int32_t *before) {
    constexpr int N = 8;                                   // loads at a time
    const int quads = int(counts_stride(a.E) / 4), blocks = int(gridDim.x);
    const int shares = max(1, int(blockDim.x) / quads);
    const int4 *counts = reinterpret_cast<const int4 *>(a.block_counts);
    for (int i = int(threadIdx.x); i < quads * shares; i += int(blockDim.x)) {
        const int share = i / quads, q = i - share * quads;
        int sum[4] = {}, some[4] = {};
        for (int b0 = share; b0 < blocks; b0 += N * shares) {
            int4 c[N];
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int b = b0 + u * shares;
                c[u] = b < blocks ? counts[int64_t(b) * quads + q] : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int v[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[j] += v[j];
                    if (b0 + u * shares < int(blockIdx.x)) some[j] += v[j];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * q + j < a.E) {                          // the padding is not read
                atomicAdd(&all[4 * q + j], sum[j]);
                atomicAdd(&before[4 * q + j], some[j]);
            }
    }
}

// Offsets of the experts from their counts (both in shared memory; block 0 also
// writes them out), then -1 for the rows that belong to no slot.
__device__ __forceinline__ void offsets_and_gaps(const PlanArgs &a, const int32_t *all,
                                                 int32_t *offset) {
    __shared__ int32_t warp_totals[32];
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += threads) {
        const int e = e0 + tid;
        const int count = e < a.E ? all[e] : 0;
        // (in 64 bits: a count next to 2^31 rounded up would not fit)
        const int padded = int((int64_t(count) + a.align - 1) / a.align * a.align);
        int total;
        const int off = carry + block_scan(padded, warp_totals, &total) - padded;
        carry += total;
        if (e < a.E) {
            offset[e] = off;
            if (blockIdx.x == 0) {
                a.counts[e] = count;
                a.offsets[e] = off;
                if (e == a.E - 1) a.offsets[a.E] = off + padded;
            }
        }
    }
    __syncthreads();
    if (a.align > 1)
        for (int e = int(blockIdx.x); e < a.E; e += int(gridDim.x)) {
            const int stop = e + 1 < a.E ? offset[e + 1] : carry;
            for (int64_t r = int64_t(offset[e]) + all[e] + tid; r < stop; r += threads)
                a.slot_of[r] = -1;
        }
    for (int64_t r = int64_t(carry) + int64_t(blockIdx.x) * threads + tid; r < a.rows;
         r += int64_t(gridDim.x) * threads)
        a.slot_of[r] = -1;
}

// Fills `n` counters of a warp's experts with zeros.
__device__ __forceinline__ void zero_seen(Seen *seen, int n) {
    for (int i = int(threadIdx.x); i < n; i += int(blockDim.x)) seen[i] = Seen{0u, 0};
}

// The plan by one block.  Each of a.warps warps ranks a contiguous part of the
// slots; a prefix sum over the warps and over the experts makes rows of ranks.
template <class I>
__global__ void __launch_bounds__(kPlanThreads)
expert_plan_one(const __grid_constant__ PlanArgs a) {
    extern __shared__ int2 smem[];
    Seen *seen = reinterpret_cast<Seen *>(smem);           // [warps][E]
    int32_t *base = reinterpret_cast<int32_t *>(smem);     // the same, first rows
    int32_t *all = base + 2 * a.warps * a.E;               // [E]
    int32_t *offset = all + a.E;                           // [E]
    const int threads = int(blockDim.x), lane = int(threadIdx.x & 31);
    const int warp = int(threadIdx.x >> 5);
    zero_seen(seen, a.warps * a.E);
    __syncthreads();
    wait_for_previous_grid();
    const PlanPart p(a);
    rank_slots<I, 4>(a, p, seen + warp * a.E);
    __syncthreads();
    for (int e = int(threadIdx.x); e < a.E; e += threads) all[e] = warp_firsts(a, seen, e);
    __syncthreads();
    offsets_and_gaps(a, all, offset);
    if (warp < a.warps) {
        // a warp's own first ranks become first rows, over the first half of its
        // counters
        Seen *mine = seen + warp * a.E;
        int32_t *rows = reinterpret_cast<int32_t *>(mine);
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int row = e < a.E ? mine[e].count + offset[e] : 0;
            __syncwarp();
            if (e < a.E) rows[e] = row;
            __syncwarp();
        }
        place_slots<I, 4>(a, p, rows);
    }
}

// Slots of a lane whose loads are in flight with many blocks: 22.9 us at 1.6 M
// slots of 256 experts, 26.6 with 4.
constexpr int kPlanLoads = 8;

// The plan by many blocks, in two grids.  The first ranks the slots within each
// warp's part of its block's tile ...
template <class I>
__global__ void __launch_bounds__(kPlanThreads)
expert_plan_rank(const __grid_constant__ PlanArgs a) {
    extern __shared__ int2 smem[];
    Seen *seen = reinterpret_cast<Seen *>(smem);           // [warps][E]
    const int threads = int(blockDim.x), tid = int(threadIdx.x);
    zero_seen(seen, a.warps * a.E);
    __syncthreads();
    wait_for_previous_grid();
    const PlanPart p(a);
    rank_slots<I, kPlanLoads>(a, p, seen + (tid >> 5) * a.E);
    __syncthreads();
    int32_t *counts = a.block_counts + int64_t(blockIdx.x) * counts_stride(a.E);
    for (int e = tid; e < a.E; e += threads) counts[e] = warp_firsts(a, seen, e);
    __syncthreads();
    int32_t *out = a.warp_first + int64_t(blockIdx.x) * a.warps * a.E;
    for (int i = tid; i < a.warps * a.E; i += threads) out[i] = seen[i].count;
}

// ... and the second adds what lies before: each block sums the counts of all
// blocks by itself (152 x E numbers from L2, which is cheaper than a third grid).
template <class I>
__global__ void __launch_bounds__(kPlanThreads)
expert_plan_place(const __grid_constant__ PlanArgs a) {
    extern __shared__ int2 smem[];
    int32_t *base = reinterpret_cast<int32_t *>(smem);     // [warps][E]
    int32_t *all = base + a.warps * a.E;                   // [E] counts of all blocks
    int32_t *offset = all + a.E;                           // [E]
    int32_t *before = offset + a.E;                        // [E] of the blocks before
    const int threads = int(blockDim.x), lane = int(threadIdx.x & 31);
    const int warp = int(threadIdx.x >> 5);
    for (int e = int(threadIdx.x); e < a.E; e += threads) all[e] = before[e] = 0;
    __syncthreads();
    wait_for_previous_grid();
    sum_blocks(a, all, before);
    __syncthreads();
    offsets_and_gaps(a, all, offset);
    if (warp < a.warps) {
        int32_t *rows = base + warp * a.E;
        const int32_t *firsts = a.warp_first + (int64_t(blockIdx.x) * a.warps + warp) * a.E;
        for (int e = lane; e < a.E; e += 32) rows[e] = firsts[e] + offset[e] + before[e];
        __syncwarp();
        place_slots<I, kPlanLoads>(a, PlanPart(a), rows);
    }
}

}  // namespace vf
