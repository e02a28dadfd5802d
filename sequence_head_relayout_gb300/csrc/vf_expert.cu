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
#include "expert_q_kernel.cuh"
#include "vf_relayout.h"

namespace {

using namespace vfc;

constexpr int64_t kMaxSlots = int64_t(1) << 30;     // T * K
constexpr int64_t kMaxExperts = 4096;
// K of the row calls, which walk a token's slots in turn: at T = 1, K = 65,536,
// M = 4,096 the merge takes 12 ms and its backward pass 40; 2^30 slots of one token
// would hold the GPU for minutes.
constexpr int64_t kMaxChoices = 65536;
constexpr int64_t kMaxAlign = 65536;
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxGrid = int64_t(1) << 27;   // a grid's warps fit 31 bits
constexpr int64_t kSMs = 152;

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
    if (T > kMaxExtent || K > kMaxExtent || E > kMaxExperts || align > kMaxAlign)
        return VF_ERR_ARG;
    if (T * K > kMaxSlots) return VF_ERR_ARG;              // both at most 2^30
    // at most 2^30 + 2^12 * 2^16
    *rows = T * K + std::min(E, T * K) * (align - 1);
    return *rows > kMaxRows ? VF_ERR_ARG : VF_OK;
}

// Blocks of the plan, the slots of each, the warps that sort and the threads.
struct PlanShape {
    int64_t blocks, tile, warps, threads;
};

constexpr int64_t kPlanCounters = 24576;               // 8-byte counters in shared memory
// Slots that one block sorts by itself (E = 256: 7.8 us at 4,096 slots, 11.7 at
// 8,192); more are spread over the SMs (10.2 us at 4,104 slots, 11.6 at 262,144).
constexpr int64_t kPlanOneBlock = 6144;

PlanShape plan_shape(int64_t slots, int64_t E) {
    PlanShape p;
    p.blocks = slots <= kPlanOneBlock ? 1 : std::min(kSMs, ceil_div(slots, 2048));
    // a warp for every 32 slots, at most what the counters have room for
    p.warps = std::min<int64_t>(32, std::max<int64_t>(1, ceil_div(ceil_div(slots, p.blocks), 32)));
    p.warps = std::max<int64_t>(1, std::min(p.warps, kPlanCounters / E));
    const int64_t step = 32 * p.warps;
    p.tile = std::max<int64_t>(1, ceil_div(ceil_div(slots, p.blocks), step)) * step;
    p.blocks = std::max<int64_t>(1, ceil_div(slots, p.tile));
    p.threads = std::max(step, std::min<int64_t>(vf::kPlanThreads, ceil_div(E, 32) * 32));
    return p;
}

// int32 numbers of workspace: the blocks' counts and their warps' first ranks.
int64_t plan_workspace(const PlanShape &p, int64_t E) {
    return p.blocks > 1 ? p.blocks * (p.warps * E + vf::counts_stride(E)) : 0;
}

// The most that a plan's kernel takes: (2 * 6 + 2) arrays of 4,096 experts.
constexpr int kPlanShared = 14 * 4096 * 4;

int launch_plan_kernel(void (*kernel)(vf::PlanArgs), const vf::PlanArgs &a, const PlanShape &p,
                       int64_t arrays, cudaStream_t stream) {
    const size_t smem = size_t(arrays) * size_t(a.E) * 4;
    // above 48 KB, the kernel's own arrays included, it has to be told; on every
    // call, so that no state is kept per device, and always the same number, since
    // another thread may be between this and its launch
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPlanShared) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    return launch(kernel, p.blocks, int(p.threads), smem, stream, a);
}

template <class I>
int launch_plan(const vf::PlanArgs &a, const PlanShape &p, cudaStream_t stream) {
    if (p.blocks == 1)
        return launch_plan_kernel(vf::expert_plan_one<I>, a, p, 2 * p.warps + 2, stream);
    const int rc = launch_plan_kernel(vf::expert_plan_rank<I>, a, p, 2 * p.warps, stream);
    return rc != VF_OK ? rc : launch_plan_kernel(vf::expert_plan_place<I>, a, p, p.warps + 3,
                                                 stream);
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
    if (d->K > kMaxChoices || d->align < 1 || d->align > kMaxAlign || d->M < 0 ||
        d->M > kMaxExtent || d->rows < 0 || d->rows > kMaxRows)
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

using RowKernel = void (*)(vf::ExpertArgs);

// The kernels of expert_kernel.cuh: any unit width, checkpoints below 16 bytes.
template <class E, int VW, int FMT>
RowKernel row_kernel(Call call) {
    switch (call) {
        case Call::kPack: return vf::expert_pack_rows<typename E::S, VW, FMT>;
        case Call::kRestore:
            if constexpr (FMT != 0) return vf::expert_restore_rows<VW, FMT>;
            return nullptr;                                // refused by check_desc
        case Call::kMerge: return vf::expert_merge_rows<E, VW, FMT>;
        default: return vf::expert_merge_backward_rows<E, VW, FMT>;
    }
}

template <class E, int FMT>
RowKernel row_kernel(Call call, int vw) {
    constexpr int widest = 16 / int(sizeof(typename E::S));
    if constexpr (widest == 8 && FMT == 0)
        if (vw == 8) return row_kernel<E, 8, FMT>(call);
    switch (vw) {
        case 4: return row_kernel<E, 4, FMT>(call);
        case 2: return row_kernel<E, 2, FMT>(call);
        default: return row_kernel<E, 1, FMT>(call);
    }
}

// The kernels of expert_q_kernel.cuh, NV vectors per lane.  Measured on GB300:
// the pack and the restore take NV = 4 (112 + 82 us at T = 55,413, K = 2,
// M = 2,048, INT8; NV = 2 113 + 85, NV = 1 136 + 95), the merge and its backward
// pass NV = 2 (45 and 40 us at T = 4,096, K = 4, M = 4,096, E4M3; NV = 4 47 and
// 43), which leaves them registers for more rows at once.
template <int FMT, int GROUP>
RowKernel tile_kernel(Call call) {
    switch (call) {
        case Call::kPack: return vf::expert_pack_tiles<FMT, 4, GROUP / 32>;
        case Call::kRestore: return vf::expert_restore_tiles<FMT, 4, GROUP / 32>;
        case Call::kMerge: return vf::expert_merge_tiles<FMT, 2, GROUP / 16>;
        default: return vf::expert_merge_backward_tiles<FMT, 2, GROUP / 16>;
    }
}

int64_t tile_columns(Call call) {
    return call == Call::kPack || call == Call::kRestore ? 1024 : 512;
}

template <int FMT>
RowKernel tile_kernel(Call call, int64_t group) {
    switch (group) {
        case 32: return tile_kernel<FMT, 32>(call);
        case 64: return tile_kernel<FMT, 64>(call);
        case 128: return tile_kernel<FMT, 128>(call);
        default: return tile_kernel<FMT, 256>(call);
    }
}

RowKernel pick_kernel(const vf_expert_desc *d, Call call, int vw, bool tiles) {
    if (tiles)
        return d->format == VF_FORMAT_INT8 ? tile_kernel<vf::kFmtInt8>(call, d->group)
                                           : tile_kernel<vf::kFmtE4M3>(call, d->group);
    switch (d->format) {                                   // bfloat16 with a format
        case VF_FORMAT_INT8: return row_kernel<vf::Bf16, vf::kFmtInt8>(call, vw);
        case VF_FORMAT_E4M3: return row_kernel<vf::Bf16, vf::kFmtE4M3>(call, vw);
        default: break;
    }
    switch (d->type) {
        case VF_TYPE_BF16: return row_kernel<vf::Bf16, 0>(call, vw);
        case VF_TYPE_F16: return row_kernel<vf::F16, 0>(call, vw);
        default: return row_kernel<vf::F32, 0>(call, vw);
    }
}

// Warps that share a token in the merge's backward pass.  A warp needs some 16
// spans of rows (8 tiles) to hide the block's start and the sum over its warps:
// at M = 2,048, K = 2 (16 spans) one warp takes 181 us at T = 55,414, eight 264;
// at M = 4,096, K = 8 (128) one takes 364 us at T = 16,384, eight 331.  They get
// the same number of spans, or nearly: with a checkpoint at M = 3,584, K = 4
// (7 tiles) one warp takes 475 us, three 540.  Few tokens are spread over more
// warps, even or not.
int token_warps(const vf::ExpertArgs &a, bool tiles) {
    const int64_t spans = std::max(a.spans, 1);
    int64_t w = std::min<int64_t>({spans * a.K / (tiles ? 8 : 16), spans, vf::kExpertWarps});
    while (w > 1 && 10 * spans < 9 * w * ceil_div(spans, w)) --w;
    w = std::max<int64_t>(w, 1);
    while (w < vf::kExpertWarps && w < spans && a.T * w < kSMs * 32) ++w;
    return int(ceil_div(spans, ceil_div(spans, w)));
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
    if (call == Call::kMerge && a.rows == 0) a.K = 0;      // no rows: every slot is dropped
    const int vw = unit_width(d, tokens, packed, fmt, backward);
    const bool tiles = fmt && vw == 8;
    if (tiles) a.spans = int32_t(ceil_div(d->M, tile_columns(call)));
    int64_t warps = vf::kExpertWarps, blocks;
    if (backward) {
        a.token_warps = token_warps(a, tiles);
        warps -= warps % a.token_warps;
        blocks = ceil_div(a.T, warps / a.token_warps);
    } else {
        blocks = ceil_div(a.T * a.spans, warps);
    }
    // The merge reads each token's rows from K places, and goes fastest with the
    // resident blocks walking the tokens side by side: at T = 55,414, K = 8,
    // M = 3,584 499 us, against 565 with a block for every 8 items and 650 with
    // 5 blocks per SM, which do not all fit; with a checkpoint (K = 4) 442-447 in
    // 2-3 rounds, 462 in one, 489 in short blocks.  The other calls run best in
    // short blocks (the pack 510 us, 590 and more in rounds).  Rows of smaller units
    // have as many blocks, in two rounds where their registers leave room for two:
    // at T = 20,000, K = 4, M = 2,052 75 us with 4 to an SM, 120 with 2, 77 with 8;
    // at M = 2,049 154, 152 and 153; with an E4M3 checkpoint 303, 313 and 258, and
    // 542, 539 and 543.
    if (call == Call::kMerge)
        blocks = std::min(blocks, kSMs * vf::kMergeResident * (tiles ? 2 : 1));
    blocks = std::min(blocks, kMaxGrid);
    a.row_blocks = uint32_t(blocks);
    if (a.spans > 0) {
        a.step_tokens = int32_t(blocks * warps / a.spans);
        a.step_spans = int32_t(blocks * warps % a.spans);
    }
    // Blocks that zero an expert's gap, fewer than align rows: 16 tokens, K = 8,
    // E = 128, M = 4,096, align = 128 packed in 14 us with 16 to an expert, 27 with 4;
    // with 64 tokens, E = 256, M = 2,048, align = 16 8 to an expert 4.0, 16 5.3.
    if (writes_rows && d->align > 1 && n_packed > 0)
        a.gap_blocks = int32_t(std::min<int64_t>(16, d->align / 2));
    return launch(pick_kernel(d, call, vw, tiles), blocks + int64_t(a.E) * a.gap_blocks,
                  int(warps) * 32, 0, as_stream(stream), a);
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
    return plan_workspace(p, E) * 4;
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
    const int64_t words = plan_workspace(p, E);
    rs.add(workspace, words, 4, true);
    if (words > 0 && reinterpret_cast<uintptr_t>(workspace) % 16) return VF_ERR_ARG;
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
    a.block_counts = static_cast<int32_t *>(workspace);
    if (p.blocks > 1) a.warp_first = a.block_counts + p.blocks * vf::counts_stride(E);
    a.K = int32_t(K);
    a.E = int32_t(E);
    a.align = int32_t(align);
    a.slots = int32_t(T * K);
    a.rows = int32_t(rows);
    a.tile = int32_t(p.tile);
    a.warps = int32_t(p.warps);
    a.flat = expert_strides[1] == 1 && (expert_strides[0] == K || T <= 1);
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
