// Device side of the expert relayouts with 8-bit checkpoints, for rows that
// take 16-byte accesses (M % 8 == 0, aligned, unit column stride).  The same
// operations as expert_kernel.cuh, which holds the forms for other rows.
//
// A checkpointed row is bound by instruction issue before HBM unless what is
// done once per group is done once per many elements, so a lane holds NV
// 16-byte vectors of one group: L = group / (8 NV) lanes share a group, and
// vector j of a lane lies j * L vectors behind its first, so that each access
// of the group's lanes covers consecutive bytes.  A group then costs log2 L
// shuffles, one table look-up and one scale for NV vectors.  A warp's tile is
// 32 NV vectors of a row.  Measured on GB300 (device time, bytes that cannot be
// avoided over it; INT8 and E4M3 differ by a few per cent):
//   pack, restore    T = 55,413, K = 2, M = 2,048   112 + 82 us   6.91 TB/s
//   merge            T = 55,414, K = 4, M = 3,584   445 us        6.11 TB/s
//   merge backward   the same                       414 us        6.57 TB/s
// The merge still issues some 125 instructions per 256 columns of a row (206
// before the lanes held whole vectors of a group), 65% of the issue slots at 72%
// of the DRAM cycles.
#pragma once

#include "expert_kernel.cuh"

namespace vf {

template <int NV, int L>
struct Tile {
    static constexpr int kGroup = 8 * NV * L;      // columns of a group
    static constexpr int kStep = 8 * L;            // between a lane's vectors
    static constexpr int kCols = 256 * NV;         // columns of a warp's tile

    static __device__ __forceinline__ int first_col(int s, int lane) {
        return s * kCols + (lane / L) * kGroup + (lane % L) * 8;
    }
};

// A lane's vectors of a row, p at its first column c; zeros past the row's end,
// and everywhere where `there` is false.
template <int NV, int L>
__device__ __forceinline__ void load_tile(const uint16_t *p, int c, int M, bool there,
                                          uint4 (&v)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (there && c + j * Tile<NV, L>::kStep < M)
            v[j] = *reinterpret_cast<const uint4 *>(p + j * Tile<NV, L>::kStep);
    }
}

template <int NV, int L>
__device__ __forceinline__ void store_tile(uint16_t *p, int c, int M, const uint4 (&v)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (c + j * Tile<NV, L>::kStep < M)
            *reinterpret_cast<uint4 *>(p + j * Tile<NV, L>::kStep) = v[j];
}

// The larger magnitude of two bfloat16 pairs, lane-wise, in one instruction; the
// signs are left as they fall.  A NaN gives a NaN (its magnitude is above an
// infinity's, which is what marks a lost group).
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The checkpoint of a lane's vectors of row `row`.  All 32 lanes are here.
template <int FMT, int NV, int L>
__device__ __forceinline__ void checkpoint_tile(const ExpertArgs &a, const ScaleTable &tab,
                                                int64_t row, int s, int lane, int c,
                                                const uint4 (&v)[NV]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        m = max_magnitude(m, v[j].x);
        m = max_magnitude(m, v[j].y);
        m = max_magnitude(m, v[j].z);
        m = max_magnitude(m, v[j].w);
    }
    m = mag2(m);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(kAll, m, o));
    m = max(m & 0xFFFFu, m >> 16);
    const float inv = group_inverse(tab, m);
    uint8_t *codes = a.codes + row * a.M + c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (c + j * Tile<NV, L>::kStep >= a.M) continue;
        uint2 code = encode8<FMT>(v[j], inv);
        if (!live_group(m)) code = make_uint2(0, 0);     // a lost group's too
        *reinterpret_cast<uint2 *>(codes + j * Tile<NV, L>::kStep) = code;
    }
    if (lane % L == 0 && c < a.M)
        a.scales[row * a.groups + s * (32 / L) + lane / L] = group_scale(tab, m);
}

// A lane's codes of row `row` and their scale (zeros as load_tile's).
template <int NV, int L>
__device__ __forceinline__ float load_codes(const ExpertArgs &a, int64_t row, int s, int lane,
                                            int c, bool there, uint2 (&q)[NV]) {
    const uint8_t *codes = a.codes + row * a.M + c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        q[j] = make_uint2(0, 0);
        if (there && c + j * Tile<NV, L>::kStep < a.M)
            q[j] = *reinterpret_cast<const uint2 *>(codes + j * Tile<NV, L>::kStep);
    }
    return there && c < a.M ? a.scales[row * a.groups + s * (32 / L) + lane / L] : 0.0f;
}

// Pack with a checkpoint of the tokens.
template <int FMT, int NV, int L>
__global__ void __launch_bounds__(kExpertThreads)
expert_pack_tiles(const __grid_constant__ ExpertArgs a) {
    __shared__ ScaleTable tab;
    fill_table<FMT>(tab);
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<uint16_t, 8>(a, a.packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int c = Tile<NV, L>::first_col(at.s, lane);
        Slots slots(a, at.t, 0, lane, false);
        uint4 v[NV];
        load_tile<NV, L>(static_cast<const uint16_t *>(a.tokens) + at.t * a.token_stride + c, c,
                         a.M, true, v);
        for (int k0 = 0; k0 < a.K; k0 += 32) {
            if (k0 > 0) slots = Slots(a, at.t, k0, lane, false);
            for (int j = 0; j < min(32, a.K - k0); ++j) {
                const int r = __shfl_sync(kAll, slots.row, j);
                if (r >= 0)
                    store_tile<NV, L>(static_cast<uint16_t *>(a.packed) + int64_t(r) * a.M + c, c,
                                      a.M, v);
            }
        }
        checkpoint_tile<FMT, NV, L>(a, tab, at.t, at.s, lane, c, v);
    }
}

// The pack of a checkpoint of the tokens.
template <int FMT, int NV, int L>
__global__ void __launch_bounds__(kExpertThreads)
expert_restore_tiles(const __grid_constant__ ExpertArgs a) {
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<uint16_t, 8>(a, a.packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31);
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int c = Tile<NV, L>::first_col(at.s, lane);
        Slots slots(a, at.t, 0, lane, false);
        uint2 q[NV];
        const float scale = load_codes<NV, L>(a, at.t, at.s, lane, c, true, q);
        uint4 v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint2 lo = decode4<FMT>(q[j].x, scale), hi = decode4<FMT>(q[j].y, scale);
            v[j] = lost_scale(scale)
                       ? make_uint4(kLostValue2, kLostValue2, kLostValue2, kLostValue2)
                       : make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        for (int k0 = 0; k0 < a.K; k0 += 32) {
            if (k0 > 0) slots = Slots(a, at.t, k0, lane, false);
            for (int j = 0; j < min(32, a.K - k0); ++j) {
                const int r = __shfl_sync(kAll, slots.row, j);
                if (r >= 0)
                    store_tile<NV, L>(static_cast<uint16_t *>(a.packed) + int64_t(r) * a.M + c, c,
                                      a.M, v);
            }
        }
    }
}

// Merge with a checkpoint of the packed rows; two rows' loads are in flight.
template <int FMT, int NV, int L>
__global__ void __launch_bounds__(kExpertThreads, kMergeResident)
expert_merge_tiles(const __grid_constant__ ExpertArgs a) {
    constexpr int KU = 2;
    __shared__ ScaleTable tab;
    fill_table<FMT>(tab);
    wait_for_previous_grid();
    const int lane = int(threadIdx.x & 31);
    const bool weighted = a.weights != nullptr;
    for (Walk at(a); at.t < a.T; at.step(a)) {
        const int c = Tile<NV, L>::first_col(at.s, lane);
        Slots slots(a, at.t, 0, lane, weighted);
        float acc[NV][8] = {};
        for (int k0 = 0; k0 < a.K; k0 += KU) {
            if (k0 > 0 && k0 % 32 == 0) slots = Slots(a, at.t, k0, lane, weighted);
            uint4 v[KU][NV];
            int r[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                r[j] = __shfl_sync(kAll, slots.row, k0 % 32 + j);
                load_tile<NV, L>(static_cast<const uint16_t *>(a.packed) + int64_t(r[j]) * a.M + c,
                                 c, a.M, r[j] >= 0, v[j]);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const float w = __shfl_sync(kAll, slots.weight, k0 % 32 + j);
                if (r[j] < 0) continue;                              // warp-uniform
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const uint32_t x[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        float f[2];
                        Bf16::widen(x[p], f);
                        const float2 sum = fma2_rn(make_float2(w, w), make_float2(f[0], f[1]),
                                                   make_float2(acc[i][2 * p],
                                                               acc[i][2 * p + 1]));
                        acc[i][2 * p] = sum.x;
                        acc[i][2 * p + 1] = sum.y;
                    }
                }
                checkpoint_tile<FMT, NV, L>(a, tab, r[j], at.s, lane, c, v[j]);
            }
        }
        uint4 out[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            out[i] = make_uint4(Bf16::round(acc[i]), Bf16::round(acc[i] + 2),
                                Bf16::round(acc[i] + 4), Bf16::round(acc[i] + 6));
        store_tile<NV, L>(static_cast<uint16_t *>(a.tokens) + at.t * a.token_stride + c, c, a.M,
                          out);
    }
}

// Gradients of the merge from a checkpoint of the packed rows (the warps of a
// token as in expert_merge_backward_rows); four rows' loads are in flight.
template <int FMT, int NV, int L>
__global__ void __launch_bounds__(kExpertThreads, 4)
expert_merge_backward_tiles(const __grid_constant__ ExpertArgs a) {
    constexpr int KU = 4;
    __shared__ float parts[kExpertWarps][KU];
    wait_for_previous_grid();
    if (blockIdx.x >= a.row_blocks) {
        zero_gaps<uint16_t, 8>(a, a.grad_packed, blockIdx.x - a.row_blocks);
        return;
    }
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    const int tokens = int(blockDim.x >> 5) / a.token_warps;
    const int part = warp % a.token_warps;
    for (int64_t t0 = int64_t(blockIdx.x) * tokens; t0 < a.T;    // block-uniform
         t0 += int64_t(a.row_blocks) * tokens) {
        const int64_t t = t0 + warp / a.token_warps;
        for (int k0 = 0; k0 < a.K; k0 += KU) {
            const Slots slots(a, t, k0, lane, true);
            float dot[KU] = {};
            for (int s = t < a.T ? part : a.spans; s < a.spans; s += a.token_warps) {
                const int c = Tile<NV, L>::first_col(s, lane);
                uint4 gv[NV];
                load_tile<NV, L>(static_cast<const uint16_t *>(a.tokens) + t * a.token_stride + c,
                                 c, a.M, true, gv);
                uint2 q[KU][NV];
                float scale[KU];
                int r[KU];
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    r[j] = __shfl_sync(kAll, slots.row, j);
                    scale[j] = load_codes<NV, L>(a, r[j], s, lane, c, r[j] >= 0, q[j]);
                }
#pragma unroll
                for (int j = 0; j < KU; ++j) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) loaded(q[j][i]);
                    loaded(scale[j]);
                }
                float g[NV][8];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    Bf16::widen(gv[i].x, g[i]);
                    Bf16::widen(gv[i].y, g[i] + 2);
                    Bf16::widen(gv[i].z, g[i] + 4);
                    Bf16::widen(gv[i].w, g[i] + 6);
                }
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    const float w = __shfl_sync(kAll, slots.weight, j);
                    if (r[j] < 0) continue;                      // warp-uniform
                    uint16_t *out = static_cast<uint16_t *>(a.grad_packed) +
                                    int64_t(r[j]) * a.M + c;
                    // each code times its scale before the gradient: a sum of g * code
                    // can leave float32 where the row's values do not (scaling
                    // the lane's sum instead took the same 414 us at the long case)
                    const float s1 = finite_or_nan(scale[j]);
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        float y[8], d[8];
                        code_values<FMT>(q[j][i], y);
#pragma unroll
                        for (int p = 0; p < 8; p += 2) {
                            const float2 v = mul2_rn(make_float2(s1, s1),
                                                     make_float2(y[p], y[p + 1]));
                            sum = fma2_rn(make_float2(g[i][p], g[i][p + 1]), v, sum);
                        }
#pragma unroll
                        for (int p = 0; p < 8; ++p) d[p] = __fmul_rn(w, g[i][p]);
                        if (c + i * Tile<NV, L>::kStep < a.M)
                            *reinterpret_cast<uint4 *>(out + i * Tile<NV, L>::kStep) =
                                make_uint4(Bf16::round(d), Bf16::round(d + 2),
                                           Bf16::round(d + 4), Bf16::round(d + 6));
                    }
                    dot[j] += sum.x + sum.y;
                }
            }
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

}  // namespace vf
