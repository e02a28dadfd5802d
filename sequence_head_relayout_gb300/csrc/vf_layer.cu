// Host side of a layer's row-wise operators (include/vf_relayout.h, "Gated
// activation" and "Root-mean-square norm"): argument checks, launch policy and
// the launches.  The kernels are in layer_kernel.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "call.h"
#include "checks.h"
#include "layer_kernel.cuh"
#include "vf_relayout.h"

namespace {

using namespace vfc;

vf::View view(const void *p, const int64_t str[2]) {
    return {const_cast<void *>(p), str[0], str[1]};
}

// Widest unit (elements) that keeps every access of the views aligned; and whether their
// rows can be taken at any address, in pieces of 16 bytes, and lie in them alike.  The stride
// of a single row counts too (where it is one, not a smaller number of no use): a norm's
// order of summing goes by all this, and is to be the same for view[:1] and view[:2].
struct Width {
    int64_t size, n, m, vw;
    bool any = true, alike = true;
    int64_t first = -1, stride = 0;            // of the first view, in a piece

    Width(int64_t size_, int64_t n_, int64_t m_) : size(size_), n(n_), m(m_), vw(16 / size_) {
        while (vw > 1 && m % vw) vw /= 2;
    }
    void take(const void *p, const int64_t str[2]) {
        if (p == nullptr) return;
        const int64_t at = int64_t(reinterpret_cast<uintptr_t>(p) % 16);
        const int64_t row = n > 1 || str[0] >= m ? str[0] : 0;
        const int64_t step = row % (16 / size);
        if (first < 0) first = at, stride = step;
        else if (at != first || step != stride) alike = false;
        if (str[1] != 1 && m > 1) vw = 1, any = false;
        while (vw > 1 && (at % (vw * size) || row % vw)) vw /= 2;
    }
    // Rows in pieces, where accesses would have at most `narrow` elements and a block holds
    // the units.  With narrow accesses and in pieces (T = 40,000, with a residual or
    // grad_total, us):
    //               norm bf16   norm fp32   backward bf16   backward fp32
    //   M = 1,421   216   108   209   138     465   174       268   239
    //   M = 1,422    86   106   132   136     222   173       240   238
    //   M = 1,420    74   103                 169   171
    bool any_pieces(int64_t narrow, int64_t most) {
        if (!any || !alike || vw > narrow || ceil_div(m + 16 / size - 1, 16 / size) > most)
            return false;
        vw = 16 / size;
        return true;
    }
    // The same in units of columns (codes, M = 1,421, 1,422 and 1,420: 566 and 257, 478 and
    // 227, 151 and 216).
    bool any_columns(int64_t narrow, int64_t most) {
        if (!any || vw > narrow || m > most) return false;
        vw = 16 / size;
        return true;
    }
    // The most units of a row.
    int64_t units(bool pieces) const { return ceil_div(m + (pieces ? 16 / size - 1 : 0), vw); }
};
// ---------------------------------------------------------------- gated activation

template <class E, int VW, bool ANY = false>
void (*glu_kernel(bool backward))(vf::GluArgs) {
    return backward ? vf::expert_glu_rows<E, VW, true, ANY>
                    : vf::expert_glu_rows<E, VW, false, ANY>;
}

template <class E>
void (*glu_kernel(bool backward, int64_t vw, bool any))(vf::GluArgs) {
    if constexpr (sizeof(typename E::S) == 2) {            // (any: 2-byte accesses otherwise)
        if (any) return glu_kernel<E, 8, true>(backward);
        if (vw == 8) return glu_kernel<E, 8>(backward);
    }
    switch (vw) {
        case 4: return glu_kernel<E, 4>(backward);
        case 2: return glu_kernel<E, 2>(backward);
        default: return glu_kernel<E, 1>(backward);
    }
}

// Two written views of the same rows that lie beside each other, as the halves of
// one buffer do.
bool side_by_side(const void *p, const int64_t sp[2], const void *q, const int64_t sq[2],
                  int64_t cols, int64_t size) {
    if (sp[0] != sq[0] || sp[1] != 1 || sq[1] != 1) return false;
    const uintptr_t lo = std::min(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(q));
    const uintptr_t hi = std::max(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(q));
    const uint64_t apart = (hi - lo) / uint64_t(size) % uint64_t(std::max<int64_t>(1, sp[0]));
    return (hi - lo) % uint64_t(size) == 0 && apart >= uint64_t(cols) &&
           apart + uint64_t(cols) <= uint64_t(sp[0]);
}

int glu(const vf_glu_desc *d, bool backward, cudaStream_t stream) {
    if (d == nullptr || d->type < VF_TYPE_BF16 || d->type > VF_TYPE_F32 || d->E < 1 ||
        d->E > kMaxExperts || d->rows < 0 || d->rows > kMaxRows || d->F < 0 || d->F > kMaxExtent)
        return VF_ERR_ARG;
    const int64_t size = type_size(d->type);
    Ranges rs;
    rs.add_view(d->gate, d->rows, d->F, d->gate_strides, size, false);
    rs.add_view(d->up, d->rows, d->F, d->up_strides, size, false);
    if (backward) {
        rs.add_view(d->grad, d->rows, d->F, d->grad_strides, size, false);
        rs.add_view(d->grad_gate, d->rows, d->F, d->grad_gate_strides, size, true);
        const int first = rs.n - 1;
        rs.add_view(d->grad_up, d->rows, d->F, d->grad_up_strides, size, true);
        if (rs.rc == VF_OK && rs.n == first + 2 &&
            side_by_side(d->grad_gate, d->grad_gate_strides, d->grad_up, d->grad_up_strides, d->F,
                         size))
            rs.join(first);
    } else {
        rs.add_view(d->out, d->rows, d->F, d->out_strides, size, true);
    }
    if (rs.rc != VF_OK) return rs.rc;
    if (d->rows == 0 || d->F == 0) return VF_OK;
    rs.add(d->slot_of, d->rows, 4, false);
    rs.add(d->offsets, d->E + 1, 4, false);
    const int rc = rs.check();
    if (rc != VF_OK) return rc;

    vf::GluArgs a;
    std::memset(&a, 0, sizeof(a));
    a.slot_of = d->slot_of;
    a.offsets = d->offsets;
    a.rows = int32_t(d->rows);
    a.E = int32_t(d->E);
    a.gate = view(d->gate, d->gate_strides);
    a.up = view(d->up, d->up_strides);
    Width w(size, d->rows, d->F);
    w.take(d->gate, d->gate_strides);
    w.take(d->up, d->up_strides);
    if (backward) {
        a.grad = view(d->grad, d->grad_strides);
        a.out = view(d->grad_gate, d->grad_gate_strides);
        a.out_up = view(d->grad_up, d->grad_up_strides);
        w.take(d->grad, d->grad_strides);
        w.take(d->grad_gate, d->grad_gate_strides);
        w.take(d->grad_up, d->grad_up_strides);
    } else {
        a.out = view(d->out, d->out_strides);
        w.take(d->out, d->out_strides);
    }
    // 2-byte accesses and units of columns (T = 40,000, bf16; us, activation and backward):
    //   F = 4,095   424 265   540 408        F = 257   41 35   54 53
    //   F = 1,421   155 101   199 160        F = 97    15 22   23 32
    const bool any = size == 2 && d->F >= 192 && w.any_columns(1, int64_t(1) << 24);
    a.F = int32_t(d->F);
    a.units = int32_t(w.units(false));
    int64_t bx = 32;
    while (bx < 256 && bx < a.units) bx *= 2;
    if (any) bx = ceil_div(ceil_div(a.units, ceil_div(a.units, 256)), 32) * 32;
    const int64_t by = 256 / bx;
    a.col_blocks = int32_t(ceil_div(a.units, bx));
    const int64_t row_blocks = std::min(ceil_div(d->rows, (any ? 1 : 2) * by),
                                        std::max<int64_t>(1, kSMs * 32 / a.col_blocks));
    auto *kernel = d->type == VF_TYPE_BF16  ? glu_kernel<vf::Bf16>(backward, w.vw, any)
                   : d->type == VF_TYPE_F16 ? glu_kernel<vf::F16>(backward, w.vw, any)
                                            : glu_kernel<vf::F32>(backward, w.vw, any);
    return launch(kernel, dim3(unsigned(row_blocks * a.col_blocks)),
                  dim3(unsigned(bx), unsigned(by)), 0, stream, a);
}

// ---------------------------------------------------------------- norm

constexpr int64_t kNormColumns = int64_t(1) << 24;         // M

// The most that the backward pass takes: stages of three rows, two units of 16 bytes to
// each of 512 threads, and the weight's units in float32.
constexpr int kNormShared = (vf::kNormStages * 3 + 2) * 2 * 16 * 512;

int64_t norm_blocks(int64_t T) { return std::min<int64_t>(T, vf::kNormBlocks); }
static_assert(vf::kNormBlocks == kSMs * 4, "four blocks to an SM");

using NormKernel = void (*)(vf::NormArgs);

template <class E, int VW, int FMT = 0, bool ANY = false>
NormKernel norm_kernel(int64_t nv) {
    switch (nv) {
        case 1: return vf::norm_rows<E, VW, 1, FMT, ANY>;
        case 2: return vf::norm_rows<E, VW, 2, FMT, ANY>;
        default: return vf::norm_rows<E, VW, 4, FMT, ANY>;
    }
}

template <int FMT>
NormKernel norm_q_kernel(int64_t vw, int64_t nv, bool any) {
    if (any)
        return nv == 1 ? vf::norm_rows<vf::Bf16, 8, 1, FMT, true>
                       : vf::norm_rows<vf::Bf16, 8, 2, FMT, true>;
    return vw == 8 ? norm_kernel<vf::Bf16, 8, FMT>(nv) : norm_kernel<vf::Bf16, 4, FMT>(nv);
}

template <class E>
NormKernel norm_kernel(int64_t vw, int64_t nv, bool any) {
    if (any) return norm_kernel<E, 16 / int(sizeof(typename E::S)), 0, true>(nv);
    if constexpr (sizeof(typename E::S) == 2)
        if (vw == 8) return norm_kernel<E, 8>(nv);
    switch (vw) {
        case 4: return norm_kernel<E, 4>(nv);
        case 2: return norm_kernel<E, 2>(nv);
        default: return norm_kernel<E, 1>(nv);
    }
}

template <class E, int VW>
NormKernel backward_kernel(int64_t nv) {
    return nv == 1   ? vf::norm_backward_rows<E, VW, 1, false>
           : nv == 2 ? vf::norm_backward_rows<E, VW, 2, false>
                     : vf::norm_backward_rows<E, VW, 4, false>;
}

template <class E>
NormKernel backward_kernel(int64_t vw, int64_t nv, bool any) {
    constexpr int kMost = 16 / int(sizeof(typename E::S));
    if (any)
        return nv == 1 ? vf::norm_backward_rows<E, kMost, 1, true>
                       : vf::norm_backward_rows<E, kMost, 2, true>;
    if constexpr (sizeof(typename E::S) == 2)
        if (vw == 8) return backward_kernel<E, 8>(nv);
    switch (vw) {
        case 4: return backward_kernel<E, 4>(nv);
        case 2: return backward_kernel<E, 2>(nv);
        default: return backward_kernel<E, 1>(nv);
    }
}

int check_norm(const vf_norm_desc *d) {
    if (d == nullptr || d->type < VF_TYPE_BF16 || d->type > VF_TYPE_F32 ||
        (d->weight_type != d->type && d->weight_type != VF_TYPE_F32) || d->T < 0 ||
        d->T > kMaxExtent || d->M < 0 || d->M > kNormColumns || !(d->eps >= 0.0f) ||
        !std::isfinite(d->eps))
        return VF_ERR_ARG;
    return VF_OK;
}

vf::NormArgs norm_args(const vf_norm_desc *d) {
    vf::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = view(d->x, d->x_strides);
    a.weight = d->weight;
    a.weight32 = d->weight_type == VF_TYPE_F32;
    a.T = d->T;
    a.M = int32_t(d->M);
    a.eps = d->eps;
    a.inv_m = 1.0f / float(d->M);
    return a;
}

// The weight as a row of the views: its units are aligned like theirs, and 16-byte
// float32 accesses where they have four elements or more.
void take_weight(Width *w, const vf_norm_desc *d) {
    if (reinterpret_cast<uintptr_t>(d->weight) % 16) w->any = false;
    const int64_t size = type_size(d->weight_type);
    while (w->vw > 1 && reinterpret_cast<uintptr_t>(d->weight) %
                            uintptr_t(std::min<int64_t>(16, w->vw * size)))
        w->vw /= 2;
}

// Units of a lane and warps of a row: by the row's units alone, so that its result does not
// depend on how many others there are.
struct RowShape {
    int64_t nv, warps, rows;       // rows of a block
};

RowShape row_shape(int64_t units, int64_t most_warps, int64_t nv) {
    RowShape s = {nv, 0, 1};
    while (s.nv < 4 && ceil_div(units, 32 * s.nv) > most_warps) s.nv *= 2;
    while (s.nv > 1 && ceil_div(units, 32) <= s.nv / 2) s.nv /= 2;
    s.warps = ceil_div(units, 32 * s.nv);
    s.rows = std::max<int64_t>(1, 8 / s.warps);
    return s;
}

// Blocks of the backward pass: their rows, shared memory and how many are to be on an SM.
struct Backward {
    int64_t resident = 0, smem = 0;
};

// The rows of a block that bring most warps onto an SM (32 have registers; at most four
// blocks, whose shares of the weight's gradient are kept).  Blocks walk their rows, so that
// each SM has to get as many: those that copy rows ask for so much shared memory that one
// more does not fit (T = 40,000, bf16, M = 1,424: 117 us with two rows to a block, of which
// an SM had three to five, 98 so; M = 2,304: 208 and 143).  The others leave it to the L1
// cache, which holds the weight (float32, M = 3,584: 375 us without, 361).
Backward backward_shape(RowShape *s, const Width &w, bool any, int64_t M, int64_t weight_size) {
    constexpr int64_t kShared = 228 * 1024, kReserved = 1024 + 512;   // (512: static)
    const bool copies = vf::copies_rows(int(w.size), int(w.vw), int(s->nv), any);
    Backward best;
    int64_t most = 0;
    for (int64_t rows = 1; rows * s->warps <= 16; ++rows) {
        const int64_t warps = rows * s->warps, units = s->nv * warps * 32;
        // the rows to come, the weight's units, and the block's sums (rows > 1: at most two
        // units to a lane)
        const int64_t smem = std::max((copies ? vf::kNormStages * 3 * units * w.vw * w.size : 0) +
                                          (any ? units * w.vw * weight_size : 0),
                                      rows > 1 ? M * 4 : 0);
        const int64_t resident =
            std::min<int64_t>({4, 32 / warps, kShared / (smem + kReserved)});
        if (smem > kNormShared || resident * warps <= most) continue;
        most = resident * warps;
        s->rows = rows;
        best.resident = resident;
        best.smem = copies ? std::max(smem, kShared / (resident + 1) - kReserved + 16) : smem;
    }
    return best;
}

int norm(const vf_norm_desc *d, cudaStream_t stream) {
    int rc = check_norm(d);
    if (rc != VF_OK) return rc;
    const bool fmt = d->format != 0, sum = d->residual != nullptr;
    if (fmt && ((d->format != VF_FORMAT_INT8 && d->format != VF_FORMAT_E4M3) ||
                d->type != VF_TYPE_BF16 ||
                (d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)))
        return VF_ERR_ARG;
    const int64_t size = type_size(d->type), T = d->T, M = d->M;
    const int64_t groups = fmt ? ceil_div(M, d->group) : 0;
    Ranges rs;
    rs.add_view(d->x, T, M, d->x_strides, size, false);
    if (sum) {
        rs.add_view(d->residual, T, M, d->residual_strides, size, false);
        rs.add_view(d->total, T, M, d->total_strides, size, true);
    }
    if (fmt) {
        rs.add(d->codes, T * M, 1, true);
        rs.add(d->scales, T * groups, 4, true);
    } else {
        rs.add_view(d->out, T, M, d->out_strides, size, true);
    }
    if (T > 0) rs.add(d->weight, M, type_size(d->weight_type), false);
    if (rs.rc != VF_OK) return rs.rc;
    if (T == 0 || M == 0) return VF_OK;
    if ((rc = rs.check()) != VF_OK) return rc;

    vf::NormArgs a = norm_args(d);
    Width w(size, T, M);
    w.take(d->x, d->x_strides);
    if (sum) {
        a.residual = view(d->residual, d->residual_strides);
        a.total = view(d->total, d->total_strides);
        w.take(d->residual, d->residual_strides);
        w.take(d->total, d->total_strides);
    }
    if (fmt) {
        a.codes = static_cast<uint8_t *>(d->codes);
        a.scales = d->scales;
        a.group = int32_t(d->group);
        a.groups = int32_t(groups);
        while (w.vw > 1 && reinterpret_cast<uintptr_t>(d->codes) % uintptr_t(w.vw)) w.vw /= 2;
    } else {
        a.out = view(d->out, d->out_strides);
        w.take(d->out, d->out_strides);
    }
    take_weight(&w, d);
    const bool any = fmt ? w.any_columns(2, 32 * 32 * 2 * 8) : w.any_pieces(1, 32 * 32 * 4);
    a.units = int32_t(w.units(any && !fmt));
    const RowShape s = row_shape(a.units, 32, any && fmt ? 2 : 4);
    a.warps = int32_t(s.warps);
    // rows that do not fit the registers of a block, and those with codes whose groups are
    // no 4 to 32 lanes
    if (s.warps > 32 || (fmt && (w.vw < 4 || d->group > 32 * w.vw))) {
        const NormKernel kernel =
            fmt ? (d->format == VF_FORMAT_INT8 ? vf::norm_any<vf::Bf16, vf::kFmtInt8>
                                               : vf::norm_any<vf::Bf16, vf::kFmtE4M3>)
            : d->type == VF_TYPE_BF16 ? vf::norm_any<vf::Bf16, 0>
            : d->type == VF_TYPE_F16  ? vf::norm_any<vf::F16, 0>
                                      : vf::norm_any<vf::F32, 0>;
        return launch(kernel, std::min<int64_t>(T, kSMs * 8), 256, 0, stream, a);
    }
    const NormKernel kernel =
        fmt ? (d->format == VF_FORMAT_INT8 ? norm_q_kernel<vf::kFmtInt8>(w.vw, s.nv, any)
                                           : norm_q_kernel<vf::kFmtE4M3>(w.vw, s.nv, any))
        : d->type == VF_TYPE_BF16 ? norm_kernel<vf::Bf16>(w.vw, s.nv, any)
        : d->type == VF_TYPE_F16  ? norm_kernel<vf::F16>(w.vw, s.nv, any)
                                  : norm_kernel<vf::F32>(w.vw, s.nv, any);
    return launch(kernel, ceil_div(T, s.rows), int(s.warps * s.rows * 32), 0, stream, a);
}

int norm_backward(const vf_norm_desc *d, cudaStream_t stream) {
    int rc = check_norm(d);
    if (rc != VF_OK) return rc;
    const int64_t size = type_size(d->type), T = d->T, M = d->M;
    const bool more = d->grad_total != nullptr;
    const int64_t words = norm_blocks(T) * M;
    Ranges rs;
    rs.add_view(d->x, T, M, d->x_strides, size, false);
    rs.add_view(d->grad, T, M, d->grad_strides, size, false);
    if (more) rs.add_view(d->grad_total, T, M, d->grad_total_strides, size, false);
    rs.add_view(d->grad_x, T, M, d->grad_x_strides, size, true);
    if (T > 0) rs.add(d->weight, M, type_size(d->weight_type), false);
    rs.add(d->grad_weight, M, 4, true);
    rs.add(d->workspace, words, 4, true);
    if (words > 0 && reinterpret_cast<uintptr_t>(d->workspace) % 16) return VF_ERR_ARG;
    if (rs.rc != VF_OK) return rs.rc;
    if (M == 0) return VF_OK;
    if ((rc = rs.check()) != VF_OK) return rc;

    vf::NormArgs a = norm_args(d);
    a.partial = static_cast<float *>(d->workspace);
    a.grad_weight = d->grad_weight;
    if (T > 0) {
        a.grad = view(d->grad, d->grad_strides);
        a.grad_x = view(d->grad_x, d->grad_x_strides);
        Width w(size, T, M);
        w.take(d->x, d->x_strides);
        w.take(d->grad, d->grad_strides);
        w.take(d->grad_x, d->grad_x_strides);
        if (more) {
            a.grad_total = view(d->grad_total, d->grad_total_strides);
            w.take(d->grad_total, d->grad_total_strides);
        }
        take_weight(&w, d);
        const bool any = w.any_pieces(2, 16 * 32 * 2);
        a.units = int32_t(w.units(any));
        RowShape s = row_shape(a.units, 16, 2);
        a.warps = int32_t(s.warps);
        if (s.warps > 16) {
            a.blocks = int32_t(norm_blocks(T));
            const NormKernel kernel = d->type == VF_TYPE_BF16  ? vf::norm_backward_any<vf::Bf16>
                                      : d->type == VF_TYPE_F16 ? vf::norm_backward_any<vf::F16>
                                                               : vf::norm_backward_any<vf::F32>;
            rc = launch(kernel, a.blocks, 256, 0, stream, a);
        } else {
            const NormKernel kernel =
                d->type == VF_TYPE_BF16  ? backward_kernel<vf::Bf16>(w.vw, s.nv, any)
                : d->type == VF_TYPE_F16 ? backward_kernel<vf::F16>(w.vw, s.nv, any)
                                         : backward_kernel<vf::F32>(w.vw, s.nv, any);
            const Backward b = backward_shape(&s, w, any, M, type_size(d->weight_type));
            const int64_t blocks =
                std::min(norm_blocks(T), std::min(ceil_div(T, s.rows), kSMs * b.resident));
            a.blocks = int32_t(blocks);
            if (b.smem > 47 * 1024 &&
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kNormShared) != cudaSuccess) {
                cudaGetLastError();
                return VF_ERR_CUDA;
            }
            rc = launch(kernel, blocks, int(s.warps * s.rows * 32), size_t(b.smem), stream, a);
        }
        if (rc != VF_OK) return rc;
    }
    return launch(vf::norm_weight_grad, ceil_div(M, 32), 1024, 0, stream, a);
}

}  // namespace

extern "C" {

int vf_expert_glu(const vf_glu_desc *d, vf_stream_t stream) {
    return glu(d, false, as_stream(stream));
}

int vf_expert_glu_backward(const vf_glu_desc *d, vf_stream_t stream) {
    return glu(d, true, as_stream(stream));
}

int64_t vf_rms_norm_workspace(int64_t T, int64_t M) {
    if (T < 0 || T > kMaxExtent || M < 0 || M > kNormColumns) return VF_ERR_ARG;
    return norm_blocks(T) * M * 4;
}

int vf_rms_norm(const vf_norm_desc *d, vf_stream_t stream) { return norm(d, as_stream(stream)); }

int vf_rms_norm_backward(const vf_norm_desc *d, vf_stream_t stream) {
    return norm_backward(d, as_stream(stream));
}

}  // extern "C"
