// Device side of a layer's row-wise operators (include/vf_relayout.h, "Gated
// activation" and "Root-mean-square norm").
//
// glu            out = s(g) g u                  s(g) = 1 / (1 + exp(-g))
// glu backward   dg = s (1 + g (1 - s)) d u,  du = g s d
// norm           h = x + residual, r = 1 / sqrt(mean(h^2) + eps), y = h r w
// norm backward  dx = r (w g - h r^2 mean(w g h)) + dtotal,  dw = sum_t g h r
//
// All are bound by HBM: each element is read and written once, with some twenty
// operations in float32 between.  Measured on GB300 (device time; bytes that cannot be
// avoided over it):
//   glu            110,828 rows, F = 2,048, bf16                 196 us   7.0 TB/s
//   glu backward   the same                                      317 us   6.9 TB/s
//   norm           T = 55,414, M = 3,584, bf16, with a residual  227 us   7.0 TB/s
//   norm to E4M3   the same                                      227 us   6.1 TB/s
//   norm backward  T = 55,413, M = 2,048, fp32, with grad_total  268 us   6.8 TB/s
//                  T = 55,414, M = 3,584, bf16, with grad_total  288 us   5.5 TB/s
#pragma once

#include <cstdint>

#include "expert_kernel.cuh"
#include "shift.cuh"

namespace vf {

// VW consecutive elements (stride 1 where VW > 1) and their float32 values.
template <class S, int VW>
struct Unit {
    using B = typename UnitBits<int(sizeof(S)) * VW>::T;
    B b;

    __device__ __forceinline__ void load(const S *p) { b = *reinterpret_cast<const B *>(p); }
    __device__ __forceinline__ void store(S *p) const { *reinterpret_cast<B *>(p) = b; }
};

template <class E, int VW>
__device__ __forceinline__ void widen_unit(const Unit<typename E::S, VW> &u, float (&f)[VW]) {
    constexpr int N = 4 / int(sizeof(typename E::S));
    if constexpr (VW < N) {
        float pair[2];
        E::widen(uint32_t(u.b), pair);
        f[0] = pair[0];
    } else {
        uint32_t w[VW / N];
        memcpy(w, &u.b, sizeof(w));
#pragma unroll
        for (int i = 0; i < VW / N; ++i) E::widen(w[i], f + N * i);
    }
}

template <class E, int VW>
__device__ __forceinline__ Unit<typename E::S, VW> round_unit(const float (&f)[VW]) {
    constexpr int N = 4 / int(sizeof(typename E::S));
    Unit<typename E::S, VW> u;
    if constexpr (VW < N) {
        const float pair[2] = {f[0], 0.0f};
        u.b = typename Unit<typename E::S, VW>::B(E::round(pair));
    } else {
        uint32_t w[VW / N];
#pragma unroll
        for (int i = 0; i < VW / N; ++i) w[i] = E::round(f + N * i);
        memcpy(&u.b, w, sizeof(w));
    }
    return u;
}

// A [n][m] view.
struct View {
    void *p;
    int64_t row, col;

    template <class S>
    __device__ __forceinline__ S *at(int64_t r, int64_t c) const {
        return static_cast<S *>(p) + r * row + c * col;
    }

    // The same where units of VW > 1 elements are taken: their column stride is 1.
    template <class S, int VW>
    __device__ __forceinline__ S *unit(int64_t r, int u) const {
        if constexpr (VW > 1) return static_cast<S *>(p) + r * row + int64_t(u) * VW;
        return at<S>(r, u);
    }
};

// ---- rows at any address -----------------------------------------------------------
//
// Rows of odd lengths start at any multiple of their elements' size.  They are read in the
// 16-byte pieces that they lie in.  Where a row's first or last piece reaches out of the view
// (in its first and last row at most, but for views that repeat a row) elements are
// read one by one.  There are two ways to take them:
// * A lane's unit is a piece, with head = the elements in front of the row in its first
//   one: unit u has columns u VW - head and on.  All views of a call have to lie alike; the
//   weight is shifted to them.  (The order of a row's sums is by its address then.)
// * A lane's unit is columns u VW and on (the codes' groups are columns, and the halves of
//   the activation's rows do not lie alike): it shifts together the two pieces that its unit
//   lies in, the second of which is the next lane's first, and stores the piece that its
//   unit and the one of the lane before it fill.

// Bytes from .. to - 1 (both even) at p, zeros for the others of the 16.
__device__ __noinline__ uint4 load_some(uint64_t p, int from, int to) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (2 * j >= from && 2 * j < to)
            w[j / 2] |= uint32_t(*reinterpret_cast<const uint16_t *>(p + 2 * j)) << (j % 2 * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row in its pieces: piece u is at start + 16 u, its bytes of the row end at span.
struct PieceRow {
    uint64_t start;
    int head, span;               // bytes in front of the row; behind its end, from the start on
    bool inside;                  // all pieces lie in the view

    __device__ __forceinline__ PieceRow() {}
    template <class S>
    __device__ __forceinline__ PieceRow(const View &v, int64_t r, int64_t rows, int m, S) {
        const uint64_t at = reinterpret_cast<uint64_t>(v.at<S>(r, 0));
        head = int(at & 15);
        start = at - uint64_t(head);
        span = head + m * int(sizeof(S));
        inside = start >= reinterpret_cast<uint64_t>(v.p) &&
                 start + uint64_t((span + 15) & ~15) <=
                     reinterpret_cast<uint64_t>(v.at<S>(rows - 1, 0)) + uint64_t(span - head);
    }

    // The row's bytes of piece u are from .. to - 1; whether those of the 32 pieces from u on
    // are whole.
    __device__ __forceinline__ int from(int u) const { return u == 0 ? head : 0; }
    __device__ __forceinline__ int to(int u) const { return min(max(span - 16 * u, 0), 16); }
    __device__ __forceinline__ bool whole(int u) const {
        return (u > 0 || head == 0) && 16 * (u + 32) <= span;
    }
    // Piece u; of a piece outside the row zeros.
    __device__ __forceinline__ uint4 load(int u) const {
        if (!inside) return load_slow(u);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (16 * u < span) v = *reinterpret_cast<const uint4 *>(start + int64_t(16 * u));
        return v;
    }
    __device__ __forceinline__ uint4 load_slow(int u) const {
        return load_some(start + int64_t(16 * u), from(u), to(u));
    }
};

// The two pieces of a unit of columns.
struct Pieces {
    uint4 lo, hi;

    __device__ __forceinline__ void load(const PieceRow &r, int unit) {
        lo = r.load(unit);
        hi = r.load(unit + 1);
    }
};

// Bytes from .. to - 1 (both even) of v, zeros for the others.
__device__ __forceinline__ uint4 some_bytes(const uint4 &v, int from, int to) {
    const auto word = [&](uint32_t w, int i) {
        const uint32_t lo = 4 * i >= from && 4 * i < to ? 0xFFFFu : 0u;
        const uint32_t hi = 4 * i + 2 >= from && 4 * i + 2 < to ? 0xFFFF0000u : 0u;
        return w & (lo | hi);
    };
    return make_uint4(word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3));
}

// The unit; zeros behind the row's end.
__device__ __forceinline__ uint4 join_pieces(const PieceRow &r, int unit, const uint4 &lo,
                                             const uint4 &hi) {
    const uint4 v = shifted(lo, hi, r.head);
    const int left = r.span - r.head - 16 * unit;
    return left >= 16 ? v : some_bytes(v, 0, max(left, 0));
}

// Bytes from .. to - 1 of v (even) to p + from and on.
__device__ __forceinline__ void store_some(uint64_t p, const uint4 &v, int from, int to) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (2 * j >= from && 2 * j < to)
            *reinterpret_cast<uint16_t *>(p + 2 * j) = uint16_t(w[j / 2] >> (j % 2 * 16));
}
__device__ __forceinline__ void store_some(uint64_t p, uint64_t v, int from, int to) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= from && j < to) *reinterpret_cast<uint8_t *>(p + j) = uint8_t(v >> (8 * j));
}

// Stores a row's first or last piece (from and to even): what is next to a multiple of 16
// bytes leaves in 8, 4 and 2 bytes.
__device__ __noinline__ void store_part(uint64_t p, uint4 v, int from, int to) {
    const bool back = from > 0;
    const int n = to - from;
    if (back && to < 16) {
        store_some(p, v, from, to);
        return;
    }
    if (n == 16) {
        *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const auto word = [&](int i) { return i & 2 ? (i & 1 ? v.w : v.z) : i & 1 ? v.y : v.x; };
    const int at4 = back ? 12 - (n & 8) : n & 8, at2 = back ? 14 - (n & 12) : n & 12;
    if (n & 8)
        *reinterpret_cast<uint2 *>(p + (back ? 8 : 0)) =
            back ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y);
    if (n & 4) *reinterpret_cast<uint32_t *>(p + at4) = word(at4 / 4);
    if (n & 2)
        *reinterpret_cast<uint16_t *>(p + at2) = uint16_t(word(at2 / 4) >> (at2 & 2 ? 16 : 0));
}

// The 8 bytes from byte `shift` (1 to 7) of lo and hi on.
__device__ __forceinline__ uint64_t shifted(uint64_t lo, uint64_t hi, int shift) {
    return lo >> (8 * shift) | hi << (64 - 8 * shift);
}
// The value of the lane before.
__device__ __forceinline__ uint4 from_before(const uint4 &v) {
    return make_uint4(__shfl_up_sync(kAll, v.x, 1), __shfl_up_sync(kAll, v.y, 1),
                      __shfl_up_sync(kAll, v.z, 1), __shfl_up_sync(kAll, v.w, 1));
}
__device__ __forceinline__ uint64_t from_before(uint64_t v) {
    return __shfl_up_sync(kAll, static_cast<unsigned long long>(v), 1);
}

// Stores a warp's units of a row of `bytes`, unit + 1 in the next lane; by all lanes of the
// warp, those with units behind the row's end too.  P: uint4 (16 bytes) or uint64_t.
template <class P>
__device__ __forceinline__ void store_shifted(void *row, int unit, int64_t bytes, const P &v,
                                              int lane) {
    constexpr int N = int(sizeof(P));
    const uint64_t p = reinterpret_cast<uint64_t>(row) + uint64_t(unit) * N;
    const int64_t left = bytes - int64_t(unit) * N;
    const int n = int(min(max(left, int64_t(0)), int64_t(N)));
    const int next = lane < 31 ? int(min(max(left - N, int64_t(0)), int64_t(N))) : 0;
    const int shift = int(p & (N - 1));                    // the same in all lanes
    if (shift == 0) {
        if (n == N) *reinterpret_cast<P *>(p) = v;
        else store_some(p, v, 0, n);
        return;
    }
    const P before = from_before(v);
    const bool whole = lane > 0 && n + shift >= N, after = next + shift >= N;
    if (whole) *reinterpret_cast<P *>(p - shift) = shifted(before, v, N - shift);
    if (!whole || !after) store_some(p, v, whole ? N - shift : 0, after ? N - shift : n);
}

// ---- arithmetic --------------------------------------------------------------------

// VW float32 operations, two to an instruction where there are two: a * b, and
// a * b + c rounded once.  b may be one value for all.
template <int VW>
__device__ __forceinline__ void mul_n(const float (&a)[VW], const float (&b)[VW],
                                      float (&o)[VW]) {
    if constexpr (VW == 1) {
        o[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < VW; i += 2) {
            const float2 p = mul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            o[i] = p.x, o[i + 1] = p.y;
        }
    }
}
template <int VW>
__device__ __forceinline__ void mul_n(const float (&a)[VW], float b, float (&o)[VW]) {
    float all[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) all[i] = b;
    mul_n<VW>(a, all, o);
}
template <int VW>
__device__ __forceinline__ void fma_n(const float (&a)[VW], const float (&b)[VW],
                                      const float (&c)[VW], float (&o)[VW]) {
    if constexpr (VW == 1) {
        o[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VW; i += 2) {
            const float2 p = fma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]),
                                     make_float2(c[i], c[i + 1]));
            o[i] = p.x, o[i + 1] = p.y;
        }
    }
}
template <int VW>
__device__ __forceinline__ void fma_n(const float (&a)[VW], float b, const float (&c)[VW],
                                      float (&o)[VW]) {
    float all[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) all[i] = b;
    fma_n<VW>(a, all, c, o);
}
// The sum of a * b added to two running sums.
template <int VW>
__device__ __forceinline__ void dot_n(const float (&a)[VW], const float (&b)[VW], float2 &sum) {
    if constexpr (VW == 1) {
        sum.x = fmaf(a[0], b[0], sum.x);
    } else {
#pragma unroll
        for (int i = 0; i < VW; i += 2)
            sum = fma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), sum);
    }
}

// ---- gated activation ------------------------------------------------------------

struct GluArgs {
    const int32_t *slot_of, *offsets;
    View gate, up, grad;          // read
    View out, out_up;             // glu: out; backward: the gradients of gate and up
    int32_t rows, E;
    int32_t F, units;             // units: of VW elements in a row
    int32_t col_blocks;
};

// s(g) = 1 / (1 + e), times e where g is negative, with e = exp(-|g|): exp(-g) overflows from
// g = -88.7 on, where s has not left float32 and the other factors may bring it far above
// its smallest values.  For 16-bit elements the fast exponential and reciprocal (of 1 to 2:
// off by one unit) do: off by some 2^-20 at |g| = 10, where a rounding to the type is 2^-9
// or 2^-12 (with the full ones the activation of 110,828 rows, F = 2,048, took 238 us at
// 201 of HBM's).
template <class S>
__device__ __forceinline__ float sigmoid(float g) {
    float e, s;
    if constexpr (sizeof(S) == 4) {
        e = expf(-fabsf(g));
        s = __frcp_rn(1.0f + e);
    } else {
        e = __expf(-fabsf(g));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    }
    if (g < 0.0f) s *= e;
    return s;
}

// A thread takes one unit of columns of U rows at a time; blockDim is (columns, rows).
// ANY: rows at any address, in columns.
template <class E, int VW, bool BACKWARD, bool ANY>
__global__ void __launch_bounds__(256)
expert_glu_rows(const __grid_constant__ GluArgs a) {
    using S = typename E::S;
    static_assert(!ANY || (sizeof(S) == 2 && VW == 8), "units of 16 bytes");
    constexpr int U = ANY ? 1 : 2;
    wait_for_previous_grid();
    const int used = min(max(a.offsets[a.E], 0), a.rows);
    const int unit = int(blockIdx.x % uint32_t(a.col_blocks) * blockDim.x + threadIdx.x);
    const int lane = int(threadIdx.x & 31);
    if (unit - (ANY ? lane : 0) >= a.units) return;
    const auto store = [&](const View &view, int64_t r, const Unit<S, VW> &u) {
        if constexpr (ANY)
            store_shifted(view.at<S>(r, 0), unit, int64_t(a.F) * sizeof(S), u.b, lane);
        else
            u.store(view.unit<S, VW>(r, unit));
    };
    const int64_t step = int64_t(gridDim.x / uint32_t(a.col_blocks)) * blockDim.y * U;
    for (int64_t r0 = (int64_t(blockIdx.x / uint32_t(a.col_blocks)) * blockDim.y + threadIdx.y) * U;
         r0 < used; r0 += step) {
        bool there[U];
        Unit<S, VW> gate[U], up[U], grad[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            there[i] = r0 + i < used && a.slot_of[r0 + i] >= 0;
            gate[i].b = up[i].b = grad[i].b = {};
        }
        if constexpr (ANY) {
            if (there[0]) {
                const View *const views[3] = {&a.gate, &a.up, &a.grad};
                Unit<S, VW> *const units[3] = {gate, up, grad};
                constexpr int N = BACKWARD ? 3 : 2;
                PieceRow rows[N];
                Pieces pieces[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    rows[k] = PieceRow(*views[k], r0, a.rows, a.F, S());
                    pieces[k].load(rows[k], unit);
                }
#pragma unroll
                for (int k = 0; k < N; ++k)
                    units[k][0].b = join_pieces(rows[k], unit, pieces[k].lo, pieces[k].hi);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (!ANY && there[i]) {
                gate[i].load(a.gate.unit<const S, VW>(r0 + i, unit));
                up[i].load(a.up.unit<const S, VW>(r0 + i, unit));
                if constexpr (BACKWARD) grad[i].load(a.grad.unit<const S, VW>(r0 + i, unit));
            }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float g[VW], u[VW], d[VW], y[VW];
            widen_unit<E, VW>(gate[i], g);
            widen_unit<E, VW>(up[i], u);
            if constexpr (BACKWARD) widen_unit<E, VW>(grad[i], d);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float s = sigmoid<S>(g[j]);
                if constexpr (BACKWARD) {
                    // what is small first: no product leaves float32 where the
                    // result does not
                    y[j] = s * (1.0f + g[j] * (1.0f - s)) * d[j] * u[j];
                    u[j] = g[j] * s * d[j];
                } else {
                    y[j] = g[j] * s * u[j];
                }
                if (!there[i]) y[j] = u[j] = 0.0f;         // a gap row
            }
            if (r0 + i >= used) continue;
            store(a.out, r0 + i, round_unit<E, VW>(y));
            if constexpr (BACKWARD) store(a.out_up, r0 + i, round_unit<E, VW>(u));
        }
    }
}

// ---- root-mean-square norm -------------------------------------------------------

struct NormArgs {
    View x, residual, total, out; // residual.p null: none; backward: x is the total
    View grad, grad_total, grad_x;
    const void *weight;
    uint8_t *codes;
    float *scales;
    float *partial;               // backward: [blocks][M]
    float *grad_weight;
    int64_t T;
    int32_t M, units;             // units: of VW elements in a row
    int32_t weight32;             // the weight is float32
    int32_t warps;                // warps of a row
    int32_t group, groups;        // columns to a scale, scales of a row
    float eps, inv_m;             // 1 / M
    int32_t blocks;
};

template <class E, int VW>
__device__ __forceinline__ void load_weight(const NormArgs &a, int64_t c, float (&w)[VW]) {
    if (a.weight32) {
        const float *p = static_cast<const float *>(a.weight) + c;
        if constexpr (VW >= 4) {
#pragma unroll
            for (int i = 0; i < VW; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p + i);
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VW; ++i) w[i] = p[i];
        }
    } else {
        Unit<typename E::S, VW> u;
        u.load(static_cast<const typename E::S *>(a.weight) + c);
        widen_unit<E, VW>(u, w);
    }
}

// The weight from any column c on, zeros outside it, where it starts at a multiple of 16 bytes.
// All lanes of a warp are here.
template <class E, int VW>
__device__ __forceinline__ void load_weight_at(const NormArgs &a, int c, float (&w)[VW]) {
    using S = typename E::S;
    const int each = a.weight32 ? 4 : 16 / int(sizeof(S));
    const int c0 = c & -each, o = c & (each - 1);
    const uint4 *const p = static_cast<const uint4 *>(a.weight) + (a.weight32 ? c0 >> 2 : c0 / VW);
    if (a.weight32) {
        constexpr int N = VW / 4 + 1;
        float f[4 * N];
        if (__all_sync(kAll, c >= 0 && c0 + 4 * N <= a.M)) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint4 v = p[i];
                memcpy(f + 4 * i, &v, 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
                f[i] = 0.0f;
                if (c0 + i >= 0 && c0 + i < a.M)
                    f[i] = static_cast<const float *>(a.weight)[c0 + i];
            }
        }
#pragma unroll
        for (int i = 0; i < VW + 2; ++i) f[i] = o & 2 ? f[i + 2] : f[i];
#pragma unroll
        for (int i = 0; i < VW; ++i) w[i] = o & 1 ? f[i + 1] : f[i];
    } else {
        Unit<S, VW> u;
        if (__all_sync(kAll, c >= 0 && c0 + 2 * VW <= a.M)) {
            u.b = shifted(p[0], p[1], o * int(sizeof(S)));
        } else {
            uint32_t h[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                h[i] = 0;
                if (c + i >= 0 && c + i < a.M) h[i] = static_cast<const S *>(a.weight)[c + i];
            }
            if constexpr (VW == 8)
                u.b = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                 h[6] | h[7] << 16);
        }
        widen_unit<E, VW>(u, w);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// The sum over a row's warps, to all of them; `parts` has a float for every warp of
// the block.  Every thread of the block is here.
__device__ __forceinline__ float row_sum(float v, float *parts, int warps) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int warp = int(threadIdx.x >> 5);
    __syncthreads();                                       // parts is free again
    if ((threadIdx.x & 31) == 0) parts[warp] = v;
    __syncthreads();
    const int first = warp - warp % warps;
    float all = 0.0f;
    for (int i = 0; i < warps; ++i) all += parts[first + i];
    return all;
}

__device__ __forceinline__ float inverse_rms(const NormArgs &a, float squares) {
    return __frcp_rn(__fsqrt_rn(squares * a.inv_m + a.eps));
}

// A group's scale and inverse from its largest magnitude (as float32 bits, so that
// infinities and NaN are above all others): the lossy transport's format.
__device__ __forceinline__ bool group_scale32(uint32_t m, float top, float &inv, float &scale) {
    inv = scale = 0.0f;
    if (m >= 0x7F800000u) scale = __uint_as_float(kLostScaleBits);
    if (m - 0x0F800000u >= 0x7F800000u - 0x0F800000u) return false;    // below 2^-96, or lost
    const float amax = __uint_as_float(m);
    inv = __fdiv_rn(top, amax);
    scale = __fdiv_rn(amax, top);
    return true;
}

template <int FMT>
__device__ __forceinline__ uint8_t encode32(float y, float inv) {
    const float q = __fmul_rn(y, inv);
    if constexpr (FMT == kFmtInt8)
        return uint8_t(int8_t(min(127, max(-127, __float2int_rn(q)))));
    else
        return uint8_t(__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3));
}

// Four values to four codes, with the steps of encode8 (|y| is at most the group's
// amax, so that no INT8 clamp would act).
template <int FMT>
__device__ __forceinline__ uint32_t encode32x4(const float *y, float inv) {
    uint32_t lo, hi;
    if constexpr (FMT == kFmtInt8) {
        lo = __byte_perm(rint_bits(__fmul_rn(y[0], inv)), rint_bits(__fmul_rn(y[1], inv)), 0x0040);
        hi = __byte_perm(rint_bits(__fmul_rn(y[2], inv)), rint_bits(__fmul_rn(y[3], inv)), 0x0040);
    } else {
        const float2 inv2 = make_float2(inv, inv);
        lo = __nv_cvt_float2_to_fp8x2(mul2_rn(make_float2(y[0], y[1]), inv2), __NV_SATFINITE,
                                      __NV_E4M3);
        hi = __nv_cvt_float2_to_fp8x2(mul2_rn(make_float2(y[2], y[3]), inv2), __NV_SATFINITE,
                                      __NV_E4M3);
    }
    return __byte_perm(lo, hi, 0x5410);
}

// The larger magnitude of two floats in one instruction, the sign as it falls; NaN
// where one is NaN.
__device__ __forceinline__ float max_magnitude32(float a, float b) {
    float d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The norm with a row held in the registers of a.warps warps, NV units of VW
// elements to a lane.  FMT: 0 writes out, else codes (VW = 8 or 4, a group is 4 to 32
// lanes).  ANY: rows at any address, taken in pieces for out and in columns for codes.
template <class E, int VW, int NV, int FMT, bool ANY>
__global__ void __launch_bounds__(1024)
norm_rows(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    constexpr bool kPieces = ANY && FMT == 0, kColumns = ANY && FMT != 0;
    __shared__ float parts[32];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int part = warp % a.warps;
    const int64_t t = int64_t(blockIdx.x) * int(blockDim.x / 32 / a.warps) + warp / a.warps;
    const auto unit_of = [&](int j) { return (j * a.warps + part) * 32 + lane; };
    PieceRow row, other_row;
    if constexpr (ANY) {
        row = PieceRow(a.x, t, a.T, a.M, S());
        other_row = a.residual.p ? PieceRow(a.residual, t, a.T, a.M, S()) : row;
    }
    const int head = kPieces ? row.head / int(sizeof(S)) : 0;
    const auto store = [&](const View &view, int j, bool there, const Unit<S, VW> &u) {
        if constexpr (kPieces) {
            const uint64_t p = reinterpret_cast<uint64_t>(view.at<S>(t, 0)) - uint64_t(row.head) +
                               int64_t(16 * unit_of(j));
            if (t < a.T && row.whole(unit_of(j) - lane)) *reinterpret_cast<uint4 *>(p) = u.b;
            else if (there) store_part(p, u.b, row.from(unit_of(j)), row.to(unit_of(j)));
        } else if constexpr (kColumns) {
            if (t < a.T)
                store_shifted(view.at<S>(t, 0), unit_of(j), int64_t(a.M) * sizeof(S), u.b, lane);
        } else if (there) {
            u.store(view.unit<S, VW>(t, unit_of(j)));
        }
    };
    Unit<S, VW> x[NV], other[NV];
    bool there[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        there[j] = t < a.T && (kPieces ? 16 * unit_of(j) < row.span : unit_of(j) < a.units);
        x[j].b = other[j].b = {};
    }
    if constexpr (kPieces) {
        if (t < a.T) {
#pragma unroll
            for (int j = 0; j < NV; ++j) x[j].b = row.load(unit_of(j));
            if (a.residual.p)
#pragma unroll
                for (int j = 0; j < NV; ++j) other[j].b = other_row.load(unit_of(j));
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!row.whole(unit_of(j) - lane)) {
                    const int from = row.from(unit_of(j)), to = row.to(unit_of(j));
                    x[j].b = some_bytes(x[j].b, from, to);
                    other[j].b = some_bytes(other[j].b, from, to);
                }
        }
    } else if constexpr (kColumns) {
        if (t < a.T) {
            Pieces px[NV], pother[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) px[j].load(row, unit_of(j));
            if (a.residual.p)
#pragma unroll
                for (int j = 0; j < NV; ++j) pother[j].load(other_row, unit_of(j));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                x[j].b = join_pieces(row, unit_of(j), px[j].lo, px[j].hi);
                if (a.residual.p)
                    other[j].b = join_pieces(other_row, unit_of(j), pother[j].lo, pother[j].hi);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (there[j]) x[j].load(a.x.unit<const S, VW>(t, unit_of(j)));
        if (a.residual.p)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (there[j]) other[j].load(a.residual.unit<const S, VW>(t, unit_of(j)));
    }
    float y[NV][VW];
    if (a.residual.p) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[VW];
            widen_unit<E, VW>(x[j], y[j]);
            widen_unit<E, VW>(other[j], f);
            fma_n<VW>(y[j], 1.0f, f, f);                   // the sum, rounded once
            x[j] = round_unit<E, VW>(f);
            store(a.total, j, there[j], x[j]);
        }
    }
    float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        widen_unit<E, VW>(x[j], y[j]);
        dot_n<VW>(y[j], y[j], squares);
    }
    const float r = inverse_rms(a, row_sum(squares.x + squares.y, parts, a.warps));
    // A group's scale takes two divisions and is the same in all of its lanes: lane j of
    // a group (it has four at least) divides for unit j, and the others get it from
    // there (at T = 55,414, M = 3,584, E4M3: 296 us with all of them in every lane).
    static_assert(FMT == 0 || NV <= 4, "a lane of the group for every unit");
    uint32_t largest[NV] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = int64_t(unit_of(j)) * VW;
        float w[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) w[i] = 0.0f;
        if constexpr (ANY) load_weight_at<E, VW>(a, int(c) - head, w);
        else if (there[j]) load_weight<E, VW>(a, c, w);
        mul_n<VW>(y[j], r, y[j]);
        mul_n<VW>(y[j], w, y[j]);
        if constexpr (FMT == 0) {
            store(a.out, j, there[j], round_unit<E, VW>(y[j]));
        } else {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < VW; ++i)
                m = max_magnitude32(m, kColumns && c + i >= a.M ? 0.0f : y[j][i]);
            // (a zero times a NaN or an infinite root is a NaN: not in the row's columns)
            largest[j] = there[j] ? __float_as_uint(m) & 0x7FFFFFFFu : 0u;
        }
    }
    if constexpr (FMT != 0) {
        const int lanes = a.group / VW;
        for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                largest[j] = max(largest[j], __shfl_xor_sync(kAll, largest[j], o));
        const int mine = lane % lanes, first = lane - mine;
        uint32_t m = largest[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) m = mine == j ? largest[j] : m;
        float inv, scale;
        const bool live = group_scale32(m, top_code<FMT>(), inv, scale);
        if (!live) inv = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = unit_of(j);
            const float q = __shfl_sync(kAll, inv, first + j);
            uint32_t code[VW / 4];
#pragma unroll
            for (int i = 0; i < VW / 4; ++i)               // not live: NaN and infinities too
                code[i] = q == 0.0f ? 0u : encode32x4<FMT>(y[j] + 4 * i, q);
            if constexpr (kColumns) {
                static_assert(VW == 8, "units of 8 codes");
                if (t < a.T)
                    store_shifted(a.codes + t * a.M, unit, a.M,
                                  uint64_t(code[1]) << 32 | code[0], lane);
            } else if (there[j]) {
                store_unit<uint32_t, VW / 4>(
                    reinterpret_cast<uint32_t *>(a.codes + t * a.M + int64_t(unit) * VW), code);
            }
            // (lane j of a row's last group may lie behind the row's end)
            if (mine == j && t < a.T && unit - mine < a.units)
                a.scales[t * a.groups + unit / lanes] = scale;
        }
    }
}

// The norm of rows of any length and strides: a block to a row, which is read
// again (or its total, by the thread that wrote it) once the sum is there.
template <class E, int FMT>
__global__ void __launch_bounds__(256)
norm_any(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    __shared__ float parts[32];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int warps = int(blockDim.x >> 5);
    const bool sum = a.residual.p != nullptr;
    const View &h = sum ? a.total : a.x;
    const int span = FMT == 0 ? 256 : a.group;             // columns of a warp at a time
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float squares = 0.0f;
        for (int64_t c0 = int64_t(warp) * span; c0 < a.M; c0 += int64_t(warps) * span)
            for (int64_t c = c0 + lane; c < min(c0 + span, int64_t(a.M)); c += 32) {
                Unit<S, 1> u;
                float f[1];
                u.load(a.x.at<const S>(t, c));
                widen_unit<E, 1>(u, f);
                if (sum) {
                    float g[1];
                    u.load(a.residual.at<const S>(t, c));
                    widen_unit<E, 1>(u, g);
                    f[0] += g[0];
                    u = round_unit<E, 1>(f);
                    u.store(a.total.at<S>(t, c));
                    widen_unit<E, 1>(u, f);
                }
                squares = fmaf(f[0], f[0], squares);
            }
        const float r = inverse_rms(a, row_sum(squares, parts, warps));
        for (int64_t c0 = int64_t(warp) * span; c0 < a.M; c0 += int64_t(warps) * span) {
            float y[8];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t c = c0 + i * 32 + lane;
                y[i] = 0.0f;
                if (i * 32 >= span || c >= a.M) continue;
                Unit<S, 1> u;
                float f[1], w[1];
                u.load(h.at<const S>(t, c));
                widen_unit<E, 1>(u, f);
                load_weight<E, 1>(a, c, w);
                y[i] = f[0] * r * w[0];
                m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                if constexpr (FMT == 0) {
                    f[0] = y[i];
                    round_unit<E, 1>(f).store(a.out.at<S>(t, c));
                }
            }
            if constexpr (FMT != 0) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
                float inv, scale;
                const bool live = group_scale32(m, top_code<FMT>(), inv, scale);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t c = c0 + i * 32 + lane;
                    if (i * 32 < span && c < a.M)
                        a.codes[t * a.M + c] = live ? encode32<FMT>(y[i], inv) : uint8_t(0);
                }
                if (lane == 0) a.scales[t * a.groups + c0 / a.group] = scale;
            }
        }
    }
}

// Two sums over a row's warps by one barrier; `turn` alternates from call to call.
__device__ __forceinline__ float2 row_sums(float u, float v, float2 (*parts)[32], int turn,
                                           int warps) {
    float2 s = make_float2(warp_sum(u), warp_sum(v));
    if (warps == 1) return s;
    const int warp = int(threadIdx.x >> 5);
    if ((threadIdx.x & 31) == 0) parts[turn][warp] = s;
    __syncthreads();
    const int first = warp - warp % warps;
    s = make_float2(0.0f, 0.0f);
    for (int i = 0; i < warps; ++i) {
        s.x += parts[turn][first + i].x;
        s.y += parts[turn][first + i].y;
    }
    return s;
}

// Rows of a group of warps in shared memory, one of them worked on.  (With three, fewer
// blocks fit an SM: 318 us for 288 at T = 55,414, M = 3,584.)
constexpr int kNormStages = 2;

__host__ __device__ constexpr bool copies_rows(int size, int vw, int nv, bool any) {
    return any || (size == 2 && vw > 1 && nv <= 2);  // with four units to a lane they do not fit
}

// The unit's piece, for rows that lie in the view.
__device__ __forceinline__ void copy_piece(uint4 *to, uint64_t p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(p) : "memory");
}

// A unit of global memory to shared memory, behind the thread's back; the hardware
// has such copies from 4 bytes on.
template <class S, int VW>
__device__ __forceinline__ void copy_unit(Unit<S, VW> *to, const S *from) {
    constexpr int bytes = int(sizeof(Unit<S, VW>));
    const uint32_t at = uint32_t(__cvta_generic_to_shared(to));
    if constexpr (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                     ::"r"(at), "l"(from), "n"(bytes >= 4 ? bytes : 4) : "memory");
}
__device__ __forceinline__ void commit_copies() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The norm's backward pass.  A block walks its rows, a.warps warps to each, with the
// weight's gradient in registers, and leaves it in a.partial.  What bounds the pass
// is the bytes in flight.  Rows of 16-bit elements are copied to shared memory (a
// thread's units to places that no other thread touches), a row ahead of the one that
// is worked on; their values take too many registers for enough of them to be
// loaded at a time (bf16, T = 55,414, M = 3,584, with grad_total: 288 us, 335 with the
// rows in registers).  Rows of float32 stay in registers (T = 55,413, M = 2,048: 271
// us, 314 through shared memory).
//
// ANY: rows at any address, in pieces, copied whatever their type; the weight's units lie in
// shared memory too, shifted once.  The rows of a block are a multiple of 8 apart where
// there is more than one round of them, so that they lie alike: a lane has the same
// columns of all.
template <class E, int VW, int NV, bool ANY>
__global__ void __launch_bounds__(512, NV <= 2 ? 2 : 1)
norm_backward_rows(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    using U = Unit<S, VW>;
    constexpr bool kCopies = copies_rows(int(sizeof(S)), VW, NV, ANY);
    static_assert(kCopies || !ANY, "rows at any address are copied");
    __shared__ float2 parts[2][32];
    // [kNormStages][h, g, more][NV][threads] units; ANY: the weight's, [VW / 4][NV][threads]
    // in float32 or [NV][threads]
    extern __shared__ uint4 dynamic[];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int part = warp % a.warps, rows = int(blockDim.x / 32 / a.warps);
    U *const ring = reinterpret_cast<U *>(dynamic) + threadIdx.x;
    const int step = int(blockDim.x);
    float dw[NV][VW] = {};
    const int64_t ahead = int64_t(gridDim.x) * rows;
    int64_t t = int64_t(blockIdx.x) * rows + warp / a.warps;
    const auto unit_of = [&](int j) { return (j * a.warps + part) * 32 + lane; };
    PieceRow first = {};                   // all of the lane's rows lie as it does
    if constexpr (ANY) first = PieceRow(a.x, t, a.T, a.M, S());
    const auto there = [&](int j) {
        return ANY ? 16 * unit_of(j) < first.span : unit_of(j) < a.units;
    };
    const auto whole = [&](int j) { return !ANY || first.whole(unit_of(j) - lane); };
    const int head = first.head / int(sizeof(S));
    const auto copy = [&](const View &view, int64_t r, int j, U *to) {
        if constexpr (ANY) {
            const PieceRow row(view, r, a.T, a.M, S());
            if (row.inside) copy_piece(&to->b, row.start + int64_t(16 * unit_of(j)));
            else to->b = row.load_slow(unit_of(j));
        } else {
            copy_unit(to, view.unit<const S, VW>(r, unit_of(j)));
        }
    };
    const auto load = [&](const View &view, int j) {
        U u;
        u.load(view.unit<const S, VW>(t, unit_of(j)));
        return u;
    };
    uint4 *const weights = dynamic + (kCopies ? kNormStages * 3 * NV * step : 0) + threadIdx.x;
    if constexpr (ANY) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[VW];
            load_weight_at<E, VW>(a, unit_of(j) * VW - head, w);
            if (a.weight32) {
#pragma unroll
                for (int i = 0; i < VW / 4; ++i)
                    memcpy(&weights[(i * NV + j) * step], w + 4 * i, 16);
            } else {
                weights[j * step] = round_unit<E, VW>(w).b;
            }
        }
    }
    const auto weight = [&](int j, float (&w)[VW]) {
        if constexpr (!ANY) {
            load_weight<E, VW>(a, int64_t(unit_of(j)) * VW, w);
        } else if (a.weight32) {
#pragma unroll
            for (int i = 0; i < VW / 4; ++i) memcpy(w + 4 * i, &weights[(i * NV + j) * step], 16);
        } else {
            widen_unit<E, VW>(U{weights[j * step]}, w);
        }
    };
    const auto fetch = [&](int64_t t, U *to) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t < a.T && there(j)) {
                copy(a.x, t, j, to + j * step);
                copy(a.grad, t, j, to + (NV + j) * step);
                if (a.grad_total.p) copy(a.grad_total, t, j, to + (2 * NV + j) * step);
            }
        }
        commit_copies();
    };
    if constexpr (kCopies)
        for (int i = 0; i < kNormStages - 1; ++i) fetch(t + i * ahead, ring + i * 3 * NV * step);
    int turn = 0, stage = 0;
    for (int64_t t0 = int64_t(blockIdx.x) * rows; t0 < a.T; t0 += ahead, t += ahead) {
        U *const here = ring + stage * 3 * NV * step;
        U held[3][NV];
        if constexpr (!kCopies) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                held[0][j].b = held[1][j].b = held[2][j].b = {};
                if (t < a.T && there(j)) {
                    held[0][j] = load(a.x, j);
                    held[1][j] = load(a.grad, j);
                    if (a.grad_total.p) held[2][j] = load(a.grad_total, j);
                }
            }
        } else {
            // the stage that was read last time takes the row that comes last
            const int free = stage == 0 ? kNormStages - 1 : stage - 1;
            fetch(t + (kNormStages - 1) * ahead, ring + free * 3 * NV * step);
            wait_copies<kNormStages - 1>();
        }
        const auto row = [&](int which, int j) {
            U u;
            if constexpr (kCopies) u = here[(which * NV + j) * step];
            else u = held[which][j];
            if constexpr (ANY)
                if (!whole(j))
                    u.b = some_bytes(u.b, first.from(unit_of(j)), first.to(unit_of(j)));
            return u;
        };
        float2 squares = make_float2(0.0f, 0.0f), dot = squares;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t >= a.T || !there(j)) continue;
            float f[VW], d[VW], w[VW];
            weight(j, w);
            widen_unit<E, VW>(row(0, j), f);
            widen_unit<E, VW>(row(1, j), d);
            dot_n<VW>(f, f, squares);
            mul_n<VW>(d, w, d);
            dot_n<VW>(d, f, dot);
        }
        const float2 both =
            row_sums(squares.x + squares.y, dot.x + dot.y, parts, turn, a.warps);
        const float r = inverse_rms(a, both.x);
        const float q = r * r * (both.y * a.inv_m);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t >= a.T || !there(j)) continue;
            float f[VW], d[VW], w[VW], m[VW] = {};
            weight(j, w);
            widen_unit<E, VW>(row(0, j), f);
            widen_unit<E, VW>(row(1, j), d);
            mul_n<VW>(d, w, w);
            fma_n<VW>(f, -q, w, w);                        // w g - h q
            mul_n<VW>(f, r, f);
            fma_n<VW>(d, f, dw[j], dw[j]);
            if (a.grad_total.p) widen_unit<E, VW>(row(2, j), m);
            fma_n<VW>(w, r, m, m);
            const U result = round_unit<E, VW>(m);
            if constexpr (ANY) {
                const uint64_t p = reinterpret_cast<uint64_t>(a.grad_x.at<S>(t, 0)) -
                                   uint64_t(first.head) + int64_t(16 * unit_of(j));
                if (whole(j)) *reinterpret_cast<uint4 *>(p) = result.b;
                else store_part(p, result.b, first.from(unit_of(j)), first.to(unit_of(j)));
            } else {
                result.store(a.grad_x.unit<S, VW>(t, unit_of(j)));
            }
        }
        turn ^= 1;
        if (++stage == kNormStages) stage = 0;
    }
    if constexpr (kCopies) wait_copies<0>();
    __syncthreads();                                       // the ring's memory is free
    float *sums = reinterpret_cast<float *>(dynamic);      // [M], with more than one row
    // the block's rows one after the other, so that the order is fixed
    float *mine = a.partial + int64_t(blockIdx.x) * a.M;
    for (int row = 0; row < rows; ++row) {
        if (row > 0) __syncthreads();
        if (warp / a.warps != row) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const int c = unit_of(j) * VW - head + i;
                if (c < 0 || c >= a.M) continue;
                const float v = row > 0 ? sums[c] + dw[j][i] : dw[j][i];
                if (row < rows - 1) sums[c] = v;
                else mine[c] = v;
            }
        }
    }
}

// The same for rows of any length and strides: a block to a row, its share of the
// weight's gradient in a.partial from the start.
template <class E>
__global__ void __launch_bounds__(256)
norm_backward_any(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    __shared__ float parts[32];
    wait_for_previous_grid();
    const int warps = int(blockDim.x >> 5);
    float *mine = a.partial + int64_t(blockIdx.x) * a.M;
    for (int64_t c = threadIdx.x; c < a.M; c += blockDim.x) mine[c] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float squares = 0.0f, dot = 0.0f;
        for (int64_t c = threadIdx.x; c < a.M; c += blockDim.x) {
            Unit<S, 1> u;
            float f[1], d[1], w[1];
            u.load(a.x.at<const S>(t, c));
            widen_unit<E, 1>(u, f);
            u.load(a.grad.at<const S>(t, c));
            widen_unit<E, 1>(u, d);
            load_weight<E, 1>(a, c, w);
            squares = fmaf(f[0], f[0], squares);
            dot = fmaf(w[0] * d[0], f[0], dot);
        }
        const float r = inverse_rms(a, row_sum(squares, parts, warps));
        const float q = r * r * (row_sum(dot, parts, warps) * a.inv_m);
        for (int64_t c = threadIdx.x; c < a.M; c += blockDim.x) {
            Unit<S, 1> u;
            float f[1], d[1], w[1], more[1] = {0.0f};
            u.load(a.x.at<const S>(t, c));
            widen_unit<E, 1>(u, f);
            u.load(a.grad.at<const S>(t, c));
            widen_unit<E, 1>(u, d);
            load_weight<E, 1>(a, c, w);
            if (a.grad_total.p) {
                u.load(a.grad_total.at<const S>(t, c));
                widen_unit<E, 1>(u, more);
            }
            mine[c] = fmaf(d[0], f[0] * r, mine[c]);
            d[0] = r * (w[0] * d[0] - f[0] * q) + more[0];
            round_unit<E, 1>(d).store(a.grad_x.at<S>(t, c));
        }
    }
}

// The weight's gradient: the blocks' shares, summed in a fixed order.  A block takes
// 32 columns, its warps every 32nd share, all of whose loads are issued at once (608
// shares of 2,048 columns: 8.4 us with four at a time).
constexpr int kNormBlocks = 608;                           // most blocks of the pass before

__global__ void __launch_bounds__(1024)
norm_weight_grad(const __grid_constant__ NormArgs a) {
    __shared__ float sums[32][33];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float share[kNormBlocks / 32], v = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormBlocks / 32; ++i) {
        const int b = warp + 32 * i;
        share[i] = c < a.M && b < a.blocks ? a.partial[int64_t(b) * a.M + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kNormBlocks / 32; ++i) v += share[i];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || c >= a.M) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    a.grad_weight[c] = v;
}

}  // namespace vf
