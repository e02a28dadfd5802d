// Device side of a layer's row-wise operators (include/vf_relayout.h, "Gated
// activation" and "Root-mean-square norm").
//
// glu            out = s(g) g u                  s(g) = 1 / (1 + exp(-g))
// glu backward   dg = s (1 + g (1 - s)) d u,  du = g s d
// norm           h = x + residual, r = 1 / sqrt(mean(h^2) + eps), y = h r w
// norm backward  dx = r (w g - h r^2 mean(w g h)) + dtotal,  dw = sum_t g h r
//
// All are bound by HBM: each element is read and written once, with some twenty
// operations in float32 between.
#pragma once

#include <cstdint>

#include "expert_kernel.cuh"

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
};

// ---- gated activation ------------------------------------------------------------

struct GluArgs {
    const int32_t *slot_of, *offsets;
    View gate, up, grad;          // read
    View out, out_up;             // glu: out; backward: the gradients of gate and up
    int32_t rows, E;
    int32_t units;                // F / VW
    int32_t col_blocks;
};

// s(g); exact enough for any type: an error of some 2^-22 of it.
template <class S>
__device__ __forceinline__ float sigmoid(float g) {
    const float e = sizeof(S) == 4 ? expf(-g) : __expf(-g);
    return __frcp_rn(1.0f + e);
}

// A thread takes one unit of columns of U rows at a time; blockDim is (columns, rows).
template <class E, int VW, bool BACKWARD>
__global__ void __launch_bounds__(256)
expert_glu_rows(const __grid_constant__ GluArgs a) {
    using S = typename E::S;
    constexpr int U = 2;
    wait_for_previous_grid();
    const int used = min(max(a.offsets[a.E], 0), a.rows);
    const int unit = int(blockIdx.x % uint32_t(a.col_blocks) * blockDim.x + threadIdx.x);
    if (unit >= a.units) return;
    const int64_t c = int64_t(unit) * VW;
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
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (there[i]) {
                gate[i].load(a.gate.at<const S>(r0 + i, c));
                up[i].load(a.up.at<const S>(r0 + i, c));
                if constexpr (BACKWARD) grad[i].load(a.grad.at<const S>(r0 + i, c));
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
            round_unit<E, VW>(y).store(a.out.at<S>(r0 + i, c));
            if constexpr (BACKWARD) round_unit<E, VW>(u).store(a.out_up.at<S>(r0 + i, c));
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
    int32_t M, units;             // units: M / VW
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

// The norm with a row held in the registers of a.warps warps, NV units of VW
// elements to a lane.  FMT: 0 writes out, else codes (VW = 8, a group is 4 to 32
// lanes).
template <class E, int VW, int NV, int FMT>
__global__ void __launch_bounds__(1024)
norm_rows(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    __shared__ float parts[32];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int part = warp % a.warps;
    const int64_t t = int64_t(blockIdx.x) * int(blockDim.x / 32 / a.warps) + warp / a.warps;
    Unit<S, VW> x[NV], other[NV];
    bool there[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int unit = (j * a.warps + part) * 32 + lane;
        there[j] = t < a.T && unit < a.units;
        x[j].b = other[j].b = {};
        if (there[j]) x[j].load(a.x.at<const S>(t, int64_t(unit) * VW));
    }
    float squares = 0.0f;
    if (a.residual.p) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            if (there[j]) other[j].load(a.residual.at<const S>(t, int64_t(unit) * VW));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            float f[VW], g[VW];
            widen_unit<E, VW>(x[j], f);
            widen_unit<E, VW>(other[j], g);
#pragma unroll
            for (int i = 0; i < VW; ++i) f[i] += g[i];
            x[j] = round_unit<E, VW>(f);
            if (there[j]) x[j].store(a.total.at<S>(t, int64_t(unit) * VW));
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float f[VW];
        widen_unit<E, VW>(x[j], f);
#pragma unroll
        for (int i = 0; i < VW; ++i) squares = fmaf(f[i], f[i], squares);
    }
    const float r = inverse_rms(a, row_sum(squares, parts, a.warps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int unit = (j * a.warps + part) * 32 + lane;
        const int64_t c = int64_t(unit) * VW;
        float f[VW], w[VW];
        widen_unit<E, VW>(x[j], f);
#pragma unroll
        for (int i = 0; i < VW; ++i) w[i] = 0.0f;
        if (there[j]) load_weight<E, VW>(a, c, w);
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = f[i] * r * w[i];
        if constexpr (FMT == 0) {
            if (there[j]) round_unit<E, VW>(f).store(a.out.at<S>(t, c));
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < VW; ++i)
                m = max(m, there[j] ? __float_as_uint(f[i]) & 0x7FFFFFFFu : 0u);
            const int lanes = a.group / VW;
            for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
            float inv, scale;
            const bool live = group_scale32(m, top_code<FMT>(), inv, scale);
            uint8_t code[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) code[i] = live ? encode32<FMT>(f[i], inv) : uint8_t(0);
            if (there[j]) {
                store_unit<uint8_t, VW>(a.codes + t * a.M + c, code);
                if (lane % lanes == 0) a.scales[t * a.groups + unit / lanes] = scale;
            }
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

// The norm's backward pass: rows in registers as in norm_rows.  A block walks its
// rows with the weight's gradient in registers and leaves it in a.partial.
template <class E, int VW, int NV>
__global__ void __launch_bounds__(512)
norm_backward_rows(const __grid_constant__ NormArgs a) {
    using S = typename E::S;
    __shared__ float parts[32];
    extern __shared__ float sums[];                        // [M], with more than one row
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int part = warp % a.warps, rows = int(blockDim.x / 32 / a.warps);
    float dw[NV][VW] = {};
    for (int64_t t0 = int64_t(blockIdx.x) * rows; t0 < a.T; t0 += int64_t(gridDim.x) * rows) {
        const int64_t t = t0 + warp / a.warps;
        Unit<S, VW> h[NV], g[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            h[j].b = g[j].b = {};
            if (t < a.T && unit < a.units) {
                h[j].load(a.x.at<const S>(t, int64_t(unit) * VW));
                g[j].load(a.grad.at<const S>(t, int64_t(unit) * VW));
            }
        }
        float squares = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            float f[VW], d[VW], w[VW] = {};
            if (unit < a.units) load_weight<E, VW>(a, int64_t(unit) * VW, w);
            widen_unit<E, VW>(h[j], f);
            widen_unit<E, VW>(g[j], d);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                squares = fmaf(f[i], f[i], squares);
                dot = fmaf(w[i] * d[i], f[i], dot);
            }
        }
        const float r = inverse_rms(a, row_sum(squares, parts, a.warps));
        const float q = r * r * (row_sum(dot, parts, a.warps) * a.inv_m);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            const int64_t c = int64_t(unit) * VW;
            const bool there = t < a.T && unit < a.units;
            float f[VW], d[VW], w[VW] = {}, more[VW] = {};
            if (unit < a.units) load_weight<E, VW>(a, c, w);
            if (there && a.grad_total.p) {
                Unit<S, VW> u;
                u.load(a.grad_total.at<const S>(t, c));
                widen_unit<E, VW>(u, more);
            }
            widen_unit<E, VW>(h[j], f);
            widen_unit<E, VW>(g[j], d);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                if (there) dw[j][i] = fmaf(d[i], f[i] * r, dw[j][i]);
                d[i] = r * (w[i] * d[i] - f[i] * q) + more[i];
            }
            if (there) round_unit<E, VW>(d).store(a.grad_x.at<S>(t, c));
        }
    }
    // the block's rows one after the other, so that the order is fixed
    float *mine = a.partial + int64_t(blockIdx.x) * a.M;
    for (int row = 0; row < rows; ++row) {
        if (row > 0) __syncthreads();
        if (warp / a.warps != row) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int unit = (j * a.warps + part) * 32 + lane;
            if (unit >= a.units) continue;
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const int c = unit * VW + i;
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
// 32 columns, its warps every 32nd share.
__global__ void __launch_bounds__(1024)
norm_weight_grad(const __grid_constant__ NormArgs a) {
    __shared__ float sums[32][33];
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (c < a.M)
#pragma unroll 4
        for (int b = warp; b < a.blocks; b += 32) v += a.partial[int64_t(b) * a.M + c];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || c >= a.M) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    a.grad_weight[c] = v;
}

}  // namespace vf
