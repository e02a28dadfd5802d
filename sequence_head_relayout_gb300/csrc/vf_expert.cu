// Host side of the expert relayouts (include/vf_relayout.h, "Expert
// relayouts"): argument checks, launch policy and the launches.  The kernels
// are in expert_kernel.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "checks.h"
#include "expert_kernel.cuh"
#include "vf_relayout.h"

namespace {

using namespace vfc;

constexpr int64_t kMaxSlots = int64_t(1) << 30;     // T * K
constexpr int64_t kMaxExperts = 4096;
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxGrid = int64_t(1) << 28;
constexpr int64_t kTableBlocks = 152 * 8;

cudaStream_t as_stream(vf_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Launch with programmatic stream serialisation, as the other kernels do.
template <class Args>
int launch(void (*kernel)(Args), int64_t blocks, int threads, size_t smem, cudaStream_t stream,
           const Args &args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    return VF_OK;
}

// ---------------------------------------------------------------- the plan

int check_routing(int64_t T, int64_t K, int64_t E, int64_t align, int64_t *rows) {
    if (T < 0 || K < 1 || E < 1 || align < 1) return VF_ERR_ARG;
    if (T > kMaxExtent || K > kMaxExtent || E > kMaxExperts || align > kMaxExtent)
        return VF_ERR_ARG;
    if (T * K > kMaxSlots) return VF_ERR_ARG;              // both at most 2^30
    // at most 2^30 + 2^12 * 2^30
    *rows = T * K + std::min(E, T * K) * (align - 1);
    return *rows > kMaxRows ? VF_ERR_ARG : VF_OK;
}

// Blocks of the plan, the slots of each and the warps that sort.
struct PlanShape {
    int64_t blocks, tile, warps;
};

constexpr int64_t kPlanCounters = 32768;               // int32 counters in shared memory
constexpr int64_t kPlanBlocks = 152;
constexpr int64_t kPlanOneBlock = 8192;                // slots that one block sorts by itself

PlanShape plan_shape(int64_t slots, int64_t E) {
    PlanShape p;
    // a warp for every 32 slots, at most what the counters have room for
    p.warps = std::min<int64_t>(32, std::max<int64_t>(1, ceil_div(slots, 32)));
    p.warps = std::max<int64_t>(1, std::min(p.warps, kPlanCounters / E));
    const int64_t step = 32 * p.warps;
    p.blocks = slots <= kPlanOneBlock ? 1 : std::min(kPlanBlocks, ceil_div(slots, 2048));
    p.tile = std::max<int64_t>(1, ceil_div(ceil_div(slots, p.blocks), step)) * step;
    p.blocks = std::max<int64_t>(1, ceil_div(slots, p.tile));
    return p;
}

template <class I>
int launch_plan(const vf::PlanArgs &a, const PlanShape &p, cudaStream_t stream) {
    if (p.blocks > 1) {
        const int rc = launch(vf::expert_plan_counts<I>, p.blocks, vf::kPlanThreads,
                              size_t(a.E) * 4, stream, a);
        if (rc != VF_OK) return rc;
    }
    const size_t smem = size_t(p.warps + 1) * size_t(a.E) * 4;
    // above 48 KB the kernel has to be told; set on every call, so that no
    // state is kept per device
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(vf::expert_plan_rows<I>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(smem)) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    return launch(vf::expert_plan_rows<I>, p.blocks, vf::kPlanThreads, smem, stream, a);
}

// A range of `count` items of `size` bytes at p; false when it wraps.
bool make_range(const void *p, int64_t count, int64_t size, Range *r) {
    int64_t bytes;
    if (!mul_ok(count, size, &bytes)) return false;
    *r = {reinterpret_cast<uintptr_t>(p), uint64_t(bytes)};
    return r->lo <= UINTPTR_MAX - r->len;
}

// The ranges of one call: each is present, aligned, accessible, and no written
// one overlaps another.
struct Ranges {
    Range r[12];
    bool written[12];
    const void *p[12];
    int n = 0;
    int rc = VF_OK;

    void add(const void *ptr, int64_t count, int64_t size, bool is_written) {
        if (rc != VF_OK || count == 0) return;
        if (ptr == nullptr || reinterpret_cast<uintptr_t>(ptr) % uintptr_t(size)) {
            rc = VF_ERR_ARG;
            return;
        }
        if (!make_range(ptr, count, size, &r[n])) {
            rc = VF_ERR_OVERFLOW;
            return;
        }
        p[n] = ptr;
        written[n++] = is_written;
    }

    // An [n0][n1] view with element strides.
    void add_view(const void *ptr, int64_t n0, int64_t n1, const int64_t str[2], int64_t size,
                  bool is_written) {
        if (rc != VF_OK) return;
        const int64_t ext[2] = {n0, n1};
        int64_t span;
        if ((rc = max_offset(ext, str, 2, &span)) != VF_OK || n0 == 0 || n1 == 0) return;
        if (is_written && !non_overlapping(ext, str, 2)) {
            rc = VF_ERR_ARG;
            return;
        }
        if (!add_ok(span, 1, &span)) rc = VF_ERR_OVERFLOW;
        else add(ptr, span, size, is_written);
    }

    int check() {
        if (rc != VF_OK) return rc;
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j)
                if ((written[i] || written[j]) && overlap(r[i], r[j])) return VF_ERR_ALIAS;
        for (int i = 0; i < n; ++i)
            if ((rc = check_pointer(p[i])) != VF_OK) return rc;
        return VF_OK;
    }
};

// ---------------------------------------------------------------- row kernels

int64_t type_size(int type) { return type == VF_TYPE_F32 ? 4 : 2; }

enum class Call { kPack, kRestore, kMerge, kBackward };

int check_desc(const vf_expert_desc *d, Call call) {
    if (d == nullptr || d->type < VF_TYPE_BF16 || d->type > VF_TYPE_F32) return VF_ERR_ARG;
    if (d->format != 0) {
        if (d->format != VF_FORMAT_INT8 && d->format != VF_FORMAT_E4M3) return VF_ERR_ARG;
        if (d->type != VF_TYPE_BF16) return VF_ERR_ARG;
        if (d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)
            return VF_ERR_ARG;
    } else if (call == Call::kRestore) {
        return VF_ERR_ARG;
    }
    int64_t most;
    const int rc = check_routing(d->T, d->K, d->E, 1, &most);
    if (rc != VF_OK) return rc;
    if (d->align < 1 || d->align > kMaxExtent || d->M < 0 || d->M > kMaxExtent ||
        d->rows < 0 || d->rows > kMaxRows)
        return VF_ERR_ARG;
    return VF_OK;
}

// Widest unit (elements) that keeps every access of both sides aligned.
int unit_width(const vf_expert_desc *d, bool tokens, bool packed, bool codes, bool grad_packed) {
    const int64_t size = type_size(d->type);
    for (int64_t vw = 16 / size; vw > 1; vw /= 2) {
        const uintptr_t bytes = uintptr_t(vw * size);
        if (d->M % vw) continue;
        if (tokens) {
            if (d->token_strides[1] != 1 && d->M > 1) continue;
            if (d->T > 1 && d->token_strides[0] % vw) continue;
            if (reinterpret_cast<uintptr_t>(d->tokens) % bytes) continue;
        }
        if (packed && reinterpret_cast<uintptr_t>(d->packed) % bytes) continue;
        if (grad_packed && reinterpret_cast<uintptr_t>(d->grad_packed) % bytes) continue;
        if (codes && reinterpret_cast<uintptr_t>(d->codes) % uintptr_t(vw)) continue;
        return int(vw);
    }
    return 1;
}

vf::ExpertArgs make_args(const vf_expert_desc *d) {
    vf::ExpertArgs a;
    std::memset(&a, 0, sizeof(a));
    a.row_of = d->row_of;
    a.counts = d->counts;
    a.offsets = d->offsets;
    a.tokens = d->tokens;
    a.token_stride = d->token_strides[0];
    a.col_stride = d->token_strides[1];
    a.packed = d->packed;
    a.weights = d->weights;
    a.weight_stride = d->weight_strides[0];
    a.weight_col_stride = d->weight_strides[1];
    a.codes = static_cast<uint8_t *>(d->codes);
    a.scales = d->scales;
    a.grad_packed = d->grad_packed;
    a.grad_weights = d->grad_weights;
    a.T = d->T;
    a.M = int32_t(d->M);
    a.K = int32_t(d->K);
    a.rows = int32_t(d->rows);
    a.E = int32_t(d->E);
    while (d->format && (int64_t(1) << a.group_log2) < d->group) ++a.group_log2;
    a.spans = int32_t(ceil_div(d->M, vf::kSpan));
    a.groups = d->format ? int32_t(ceil_div(d->M, d->group)) : 0;
    return a;
}

// Warps that share a token in the merge's backward pass: one per span, at most
// the block's, a power of two.
int token_warps(int64_t spans) {
    int w = 1;
    while (w < vf::kExpertWarps && w < spans) w *= 2;
    return w;
}

using RowKernel = void (*)(vf::ExpertArgs);

template <class S, int VW>
RowKernel pack_kernel(int format) {
    if constexpr (sizeof(S) == 2) {
        if (format == VF_FORMAT_INT8) return vf::expert_pack_rows<S, VW, vf::kFmtInt8>;
        if (format == VF_FORMAT_E4M3) return vf::expert_pack_rows<S, VW, vf::kFmtE4M3>;
    }
    return vf::expert_pack_rows<S, VW, 0>;
}

template <int VW>
RowKernel restore_kernel(int format) {
    return format == VF_FORMAT_INT8 ? vf::expert_restore_rows<VW, vf::kFmtInt8>
                                    : vf::expert_restore_rows<VW, vf::kFmtE4M3>;
}

// Rows whose loads are in flight at a time.
template <class E, int VW, int KU>
RowKernel merge_kernel(int format) {
    if constexpr (std::is_same_v<E, vf::Bf16>) {
        if (format == VF_FORMAT_INT8) return vf::expert_merge_rows<E, VW, vf::kFmtInt8, 4>;
        if (format == VF_FORMAT_E4M3) return vf::expert_merge_rows<E, VW, vf::kFmtE4M3, 4>;
    }
    return vf::expert_merge_rows<E, VW, 0, KU>;
}

template <class E, int VW, int KU>
RowKernel backward_kernel(int format) {
    if constexpr (std::is_same_v<E, vf::Bf16>) {
        if (format == VF_FORMAT_INT8)
            return vf::expert_merge_backward_rows<E, VW, vf::kFmtInt8, 4>;
        if (format == VF_FORMAT_E4M3)
            return vf::expert_merge_backward_rows<E, VW, vf::kFmtE4M3, 4>;
    }
    return vf::expert_merge_backward_rows<E, VW, 0, KU>;
}

// The kernel of a call for a type, unit width and format.
template <class E, int VW>
RowKernel pick(Call call, int format, int64_t K) {
    constexpr bool wide = VW * sizeof(typename E::S) == 16;
    constexpr int most = wide && sizeof(typename E::S) == 2 ? 8 : 4;
    switch (call) {
        case Call::kPack: return pack_kernel<typename E::S, VW>(format);
        case Call::kRestore: return restore_kernel<VW>(format);
        case Call::kMerge:
            if constexpr (wide) {
                if (K <= 2) return merge_kernel<E, VW, 2>(format);
                if (K <= 4) return merge_kernel<E, VW, 4>(format);
            }
            return merge_kernel<E, VW, most>(format);
        default:
            if constexpr (wide) {
                if (K <= 2) return backward_kernel<E, VW, 2>(format);
                if (K <= 4) return backward_kernel<E, VW, 4>(format);
            }
            return backward_kernel<E, VW, most>(format);
    }
}

template <class E>
RowKernel pick_width(Call call, int format, int vw, int64_t K) {
    switch (vw) {
        case 8:
            if constexpr (sizeof(typename E::S) == 2) return pick<E, 8>(call, format, K);
            return pick<E, 4>(call, format, K);
        case 4: return pick<E, 4>(call, format, K);
        case 2: return pick<E, 2>(call, format, K);
        default: return pick<E, 1>(call, format, K);
    }
}

RowKernel pick_type(Call call, int type, int format, int vw, int64_t K) {
    switch (type) {
        case VF_TYPE_BF16: return pick_width<vf::Bf16>(call, format, vw, K);
        case VF_TYPE_F16: return pick_width<vf::F16>(call, format, vw, K);
        default: return pick_width<vf::F32>(call, format, vw, K);
    }
}

int run(const vf_expert_desc *d, Call call, vf_stream_t stream) {
    int rc = check_desc(d, call);
    if (rc != VF_OK) return rc;
    const bool fmt = d->format != 0;
    const bool backward = call == Call::kBackward;
    const bool tokens = call != Call::kRestore;
    const bool packed = !(backward && fmt);
    const bool writes_rows = call != Call::kMerge;
    const int64_t size = type_size(d->type);
    const int64_t groups = fmt ? ceil_div(d->M, d->group) : 0;
    // the checkpoint covers packed rows in the merge, token rows in the pack
    const int64_t kept = call == Call::kMerge || backward ? d->rows : d->T;
    int64_t n_packed, n_kept, n_scales;
    if (!mul_ok(d->rows, d->M, &n_packed) || !mul_ok(kept, d->M, &n_kept) ||
        !mul_ok(kept, groups, &n_scales))
        return VF_ERR_OVERFLOW;

    Ranges rs;
    const int64_t slots = d->T * d->K;
    if (tokens) rs.add_view(d->tokens, d->T, d->M, d->token_strides, size, call == Call::kMerge);
    if (rs.rc != VF_OK) return rs.rc;
    if ((call == Call::kMerge && d->weights) || backward)
        rs.add_view(d->weights, d->T, d->K, d->weight_strides, 4, false);
    if (rs.rc != VF_OK) return rs.rc;
    if (slots == 0 || (d->M == 0 && !backward)) return VF_OK;      // nothing to move
    rs.add(d->row_of, slots, 4, false);
    if (writes_rows && d->align > 1) {
        rs.add(d->counts, d->E, 4, false);
        rs.add(d->offsets, d->E + 1, 4, false);
    }
    if (packed) rs.add(d->packed, n_packed, size, call != Call::kMerge && !backward);
    if (fmt) {
        const bool kept_written = call == Call::kMerge || call == Call::kPack;
        rs.add(d->codes, n_kept, 1, kept_written);
        rs.add(d->scales, n_scales, 4, kept_written);
    }
    if (backward) {
        rs.add(d->grad_packed, n_packed, size, true);
        rs.add(d->grad_weights, slots, 4, true);
    }
    if ((rc = rs.check()) != VF_OK) return rc;

    vf::ExpertArgs a = make_args(d);
    const int vw = unit_width(d, tokens, packed, fmt, backward);
    const RowKernel kernel = pick_type(call, d->type, d->format, vw, d->K);
    a.token_warps = token_warps(a.spans);
    int64_t blocks = backward ? ceil_div(a.T, vf::kExpertWarps / a.token_warps)
                              : ceil_div(a.T * a.spans, vf::kExpertWarps);
    // a checkpoint's blocks fill a table of scales first: few blocks, long ones
    if (fmt && (call == Call::kMerge || call == Call::kPack))
        blocks = std::min<int64_t>(blocks, kTableBlocks);
    blocks = std::min(blocks, kMaxGrid);
    a.row_blocks = uint32_t(blocks);
    if (a.spans > 0) {
        a.step_tokens = int32_t(blocks * vf::kExpertWarps / a.spans);
        a.step_spans = int32_t(blocks * vf::kExpertWarps % a.spans);
    }
    const bool gaps = writes_rows && d->align > 1 && n_packed > 0;
    return launch(kernel, blocks + (gaps ? int64_t(a.E) * vf::kGapBlocks : 0),
                  vf::kExpertThreads, 0, as_stream(stream), a);
}

}  // namespace

extern "C" {

int64_t vf_expert_rows(int64_t T, int64_t K, int64_t E, int64_t align) {
    int64_t rows;
    const int rc = check_routing(T, K, E, align, &rows);
    return rc != VF_OK ? rc : rows;
}

int64_t vf_expert_workspace(int64_t T, int64_t K, int64_t E) {
    int64_t rows;
    const int rc = check_routing(T, K, E, 1, &rows);
    if (rc != VF_OK) return rc;
    const PlanShape p = plan_shape(T * K, E);
    return p.blocks > 1 ? p.blocks * E * 4 : 0;
}

int vf_expert_plan(const void *experts, int index_bytes, const int64_t expert_strides[2],
                   int64_t T, int64_t K, int64_t E, int64_t align, int32_t *row_of,
                   int32_t *slot_of, int32_t *counts, int32_t *offsets, void *workspace,
                   vf_stream_t stream) {
    int64_t rows;
    int rc = check_routing(T, K, E, align, &rows);
    if (rc != VF_OK) return rc;
    if (expert_strides == nullptr || (index_bytes != 4 && index_bytes != 8)) return VF_ERR_ARG;
    const PlanShape p = plan_shape(T * K, E);
    Ranges rs;
    rs.add_view(experts, T, K, expert_strides, index_bytes, false);
    rs.add(row_of, T * K, 4, true);
    rs.add(slot_of, rows, 4, true);
    rs.add(counts, E, 4, true);
    rs.add(offsets, E + 1, 4, true);
    if (p.blocks > 1) rs.add(workspace, p.blocks * E, 4, true);
    if ((rc = rs.check()) != VF_OK) return rc;

    vf::PlanArgs a;
    std::memset(&a, 0, sizeof(a));
    a.experts = experts;
    a.token_stride = expert_strides[0];
    a.slot_stride = expert_strides[1];
    a.row_of = row_of;
    a.slot_of = slot_of;
    a.counts = counts;
    a.offsets = offsets;
    a.block_counts = p.blocks > 1 ? static_cast<int32_t *>(workspace) : nullptr;
    a.K = int32_t(K);
    a.E = int32_t(E);
    a.align = int32_t(align);
    a.slots = int32_t(T * K);
    a.rows = int32_t(rows);
    a.tile = int32_t(p.tile);
    a.warps = int32_t(p.warps);
    return index_bytes == 8 ? launch_plan<int64_t>(a, p, as_stream(stream))
                            : launch_plan<int32_t>(a, p, as_stream(stream));
}

int vf_expert_pack(const vf_expert_desc *d, vf_stream_t stream) {
    return run(d, Call::kPack, stream);
}

int vf_expert_restore(const vf_expert_desc *d, vf_stream_t stream) {
    return run(d, Call::kRestore, stream);
}

int vf_expert_merge(const vf_expert_desc *d, vf_stream_t stream) {
    return run(d, Call::kMerge, stream);
}

int vf_expert_merge_backward(const vf_expert_desc *d, vf_stream_t stream) {
    return run(d, Call::kBackward, stream);
}

}  // extern "C"
