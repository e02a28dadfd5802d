// Host side of the experts' products (include/vf_relayout.h, "Expert products"):
// argument checks, the choice of a form, the tensor maps and the launches.  The
// kernel is in product_kernel.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "call.h"
#include "checks.h"
#include "product_kernel.cuh"
#include "vf_relayout.h"

namespace {

using namespace vfc;

constexpr int64_t kMaxFeatures = int64_t(1) << 20;       // N and M
constexpr int64_t kMaxAlign = 65536;
constexpr int64_t kSharedMemory = 227 * 1024;

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder; it has no device state, and is looked up once.
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return EncodeTiled(nullptr);
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A map of 16-bit elements, innermost dimension contiguous; strides in elements
// from the second dimension on; boxes of 64 elements (128 bytes, swizzled), n_slabs of
// them along dimension `slabs`, where that is not 0.
int make_map(CUtensorMap *map, bool bf16, int nd, const void *base, const int64_t *ext,
             const int64_t *str, int64_t box1, int slabs = 0, int64_t n_slabs = 2) {
    const EncodeTiled fn = encoder();
    if (fn == nullptr) return VF_ERR_CUDA;
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4] = {64, cuuint32_t(box1), 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    if (slabs) box[slabs] = cuuint32_t(n_slabs);
    for (int i = 0; i < nd; ++i) {
        dims[i] = cuuint64_t(ext[i]);
        if (i > 0) strides[i - 1] = cuuint64_t(str[i]) * 2;
    }
    const CUresult r =
        fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
           cuuint32_t(nd), const_cast<void *>(base), dims, strides, box, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? VF_OK : VF_ERR_CUDA;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// A stride (elements) that a map takes; those of one item are not used.
bool map_stride(int64_t ext, int64_t *str, int64_t row) {
    if (ext <= 1) {
        *str = ceil_div(row, 8) * 8;
        return true;
    }
    return *str > 0 && *str % 8 == 0 && *str < (int64_t(1) << 39);
}

int check_desc(const vf_product_desc *d) {
    if (d == nullptr || (d->type != VF_TYPE_BF16 && d->type != VF_TYPE_F16)) return VF_ERR_ARG;
    if (d->E < 1 || d->E > kMaxExperts || d->rows < 0 || d->rows > kMaxRows || d->slots < 0 ||
        d->slots > kMaxSlots || d->align < 1 || d->align > kMaxAlign || d->N < 0 ||
        d->N > kMaxFeatures || d->M < 0 || d->M > kMaxFeatures)
        return VF_ERR_ARG;
    return VF_OK;
}

// The dimensions of one of the kernel's forms.
struct Form {
    int64_t ctas, tile_n, box;
    bool weights = false;
    int64_t split = 1;            // CTAs that share a tile's sums

    int64_t cluster() const { return ctas * split; }
};

// Rows that an expert has on average.
int64_t mean_rows(const vf_product_desc *d) {
    return ceil_div(d->slots > 0 ? d->slots : d->rows, d->E);
}

void set_form(vfp::ProductArgs *a, const Form &f) {
    const int64_t b_rows = f.tile_n / f.ctas;
    a->tile_n = int32_t(f.tile_n);
    a->box = int32_t(f.box);
    a->split = int32_t(f.split);
    a->stage_bytes = int32_t(vfp::kStageA + b_rows * 128);
    a->stages = 0;
    while (a->stages < vfp::kMaxStages &&
           vfp::shared_bytes(f.weights, f.split > 1, a->stages + 1, a->stage_bytes) <=
               kSharedMemory)
        ++a->stages;
    a->acc_stride = int32_t(std::max<int64_t>(32, f.tile_n));
    a->tmem_cols = 64;
    while (a->tmem_cols < 2 * a->acc_stride) a->tmem_cols *= 2;
    a->feat_tiles = int32_t(ceil_div(a->feat, vfp::kTileM * f.ctas));
    a->col_tiles = int32_t(ceil_div(a->cols, f.tile_n));
}

using Kernel = void (*)(vfp::ProductArgs);

int launch_product(Kernel kernel, vfp::ProductArgs &a, const Form &f, int64_t tiles,
                   cudaStream_t stream) {
    if (tiles == 0) return VF_OK;
    const int64_t ctas = f.cluster();
    const int64_t groups = std::min(kSMs / ctas, tiles);
    if (a.col_tiles > 0) {
        a.step_experts = int32_t(groups / (int64_t(a.feat_tiles) * a.col_tiles));
        a.step_tiles = int32_t(groups % (int64_t(a.feat_tiles) * a.col_tiles));
    }
    // on every call, so that no state is kept per device, and always the same number
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kSharedMemory)) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * ctas), 1, 1);
    cfg.blockDim = dim3(vfp::kThreads, 1, 1);
    cfg.dynamicSmemBytes =
        size_t(vfp::shared_bytes(f.weights, f.split > 1, a.stages, a.stage_bytes));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    return VF_OK;
}

// Adds the workspace of `need` bytes (or a status) to the call's ranges.
int add_workspace(Ranges *rs, const vf_product_desc *d, int64_t need) {
    if (need < 0) return int(need);
    if (need == 0) return VF_OK;
    if (d->workspace == nullptr) return VF_ERR_CAPACITY;
    if (!aligned16(d->workspace)) return VF_ERR_ARG;
    rs->add(d->workspace, need, 1, true);
    return rs->rc;
}

vfp::ProductArgs make_args(const vf_product_desc *d) {
    vfp::ProductArgs a;
    std::memset(&a, 0, sizeof(a));
    a.counts = d->counts;
    a.offsets = d->offsets;
    a.E = int32_t(d->E);
    a.rows = int32_t(d->rows);
    a.feat = int32_t(d->N);
    a.bf16 = d->type == VF_TYPE_BF16;
    a.gaps = d->align > 1;
    return a;
}

int64_t pad8(int64_t n) { return ceil_div(n, 8) * 8; }

// An operand as a tensor map takes it, [outer][lines][len] with strides in elements, or
// as the workspace gets a copy of it that one does.
struct Operand {
    const void *p;
    int64_t outer, lines, len;
    int64_t s_outer, s_line, s_el;
    bool copied = false;

    Operand(const void *p_, int64_t outer_, int64_t lines_, int64_t len_, int64_t s_outer_,
            int64_t s_line_, int64_t s_el_)
        : p(p_), outer(outer_), lines(lines_), len(len_), s_outer(s_outer_), s_line(s_line_),
          s_el(s_el_) {
        int64_t so = s_outer, sl = s_line;
        copied = len > 0 && !((s_el == 1 || len == 1) && aligned16(p) &&
                              map_stride(outer, &so, 8) && map_stride(lines, &sl, 8));
        if (!copied) {
            map_stride(lines, &s_line, len);
            map_stride(outer, &s_outer, len);
        }
    }

    // Bytes of the workspace; the extents are at most 2^31, 2^20 and 2^12.
    int64_t bytes() const {
        int64_t n;
        if (!copied) return 0;
        return mul_ok(outer * lines, pad8(len) * 2, &n) ? n : -1;
    }

    // Copies it to `at`; `span`: elements from p to behind the last.
    int copy(void *at, int64_t span, const int32_t *counts, const int32_t *limit,
             cudaStream_t stream) {
        vfp::PadArgs a;
        std::memset(&a, 0, sizeof(a));
        a.src = static_cast<const uint16_t *>(p);
        a.end = a.src + span;
        a.s_outer = s_outer;
        a.s_line = s_line;
        a.s_el = len == 1 ? 1 : s_el;
        a.dst = static_cast<uint16_t *>(at);
        a.outer = outer;
        a.lines = lines;
        a.len = len;
        a.pitch = pad8(len);
        a.counts = counts;
        a.limit = limit;
        p = at;
        s_line = a.pitch;
        s_outer = lines * a.pitch;
        s_el = 1;
        const int64_t blocks = std::min(ceil_div(outer * lines, 8), kSMs * 8);
        a.step_outer = blocks * 8 / lines;
        a.step_lines = blocks * 8 % lines;
        return launch(vfp::pad_lines, blocks, 256, 0, stream, a);
    }
};

// The weights along m, or along n where their unit stride is.
bool along_n(const vf_product_desc *d) {
    return d->weight_strides[2] != 1 && d->M != 1 && (d->weight_strides[1] == 1 || d->N == 1);
}

Operand weights_of(const vf_product_desc *d) {
    const int64_t *s = d->weight_strides;
    return along_n(d) ? Operand(d->weights, d->E, d->M, d->N, s[0], s[2], s[1])
                      : Operand(d->weights, d->E, d->N, d->M, s[0], s[1], s[2]);
}

Operand rows_of(const void *p, int64_t rows, int64_t len) {
    return Operand(p, 1, rows, len, 0, len, 1);
}

// Bytes of workspace for two operands, or a status.
int64_t workspace_of(const Operand &a, const Operand &b) {
    const int64_t n = a.bytes(), m = b.bytes();
    int64_t sum;
    return n < 0 || m < 0 || !add_ok(n, m, &sum) ? VF_ERR_OVERFLOW : sum;
}

// The longest sum of one accumulation.  The tensor cores cut off what lies below an
// accumulator's last bit, always towards zero, so that a sum's error grows with its length:
// terms of one sign lose some 2 units of 2^-23 with every 16, 4.5e-6 of the result at 768
// terms, 3e-5 at 4,096, 2.4e-4 at 32,768 (terms of both signs a tenth of that and less).
// Longer sums are taken in parts that are added with rounding.  Of a 16-bit result a part
// loses an eighth of the smallest half unit at most (fp16 2^-12, bf16 2^-9); a float32
// result is as near as parts of 768 make it: T = 4,096, K = 8, E = 32, N = 4,096, M = 2,048
// takes 384 us in one part, 397 in parts of 768 rows, 415 in parts of 512.
int64_t part_of(const vf_product_desc *d, bool out32) {
    return out32 ? 768 : d->type == VF_TYPE_F16 ? 4096 : 32768;
}

// The form by the rows that an expert has on average.  Measured with E = 64,
// N = 4,096, M = 2,048 (us; forms by CTAs and rows of a tile):
//   rows    1 x 32   1 x 64   1 x 128   2 x 128   2 x 256
//      8       162      159       163       159       166
//     32       174      164       167       164       171
//     64       222      179       174       169       174
//    128       367      239       198       187       185
//    192       520      305       237       217       201
// A pair would have no feature to store in its second CTA with N at most 128.
Form rows_form(const vf_product_desc *d) {
    const int64_t mean = mean_rows(d);
    if (mean <= 32) return {1, 64, 16};
    if (d->N <= vfp::kTileM) return {1, 128, 32};
    return mean <= 112 ? Form{2, 128, 16} : Form{2, 256, 32};
}

template <int CTAS>
Kernel rows_kernel(bool mn, bool parts) {
    return parts ? (mn ? vfp::expert_product<CTAS, false, true, true>
                       : vfp::expert_product<CTAS, false, false, true>)
                 : (mn ? vfp::expert_product<CTAS, false, true>
                       : vfp::expert_product<CTAS, false, false>);
}

int product(const vf_product_desc *d, cudaStream_t stream) {
    int rc = check_desc(d);
    if (rc != VF_OK) return rc;
    int64_t n_packed, n_out, span;
    const int64_t ext[3] = {d->E, d->N, d->M};
    if (!mul_ok(d->rows, d->M, &n_packed) || !mul_ok(d->rows, d->N, &n_out))
        return VF_ERR_OVERFLOW;
    if ((rc = max_offset(ext, d->weight_strides, 3, &span)) != VF_OK) return rc;
    if (!add_ok(span, 1, &span)) return VF_ERR_OVERFLOW;
    if (n_out == 0) return VF_OK;                          // nothing to write
    Ranges rs;
    rs.add(d->counts, d->E, 4, false);
    rs.add(d->offsets, d->E + 1, 4, false);
    rs.add(d->packed, n_packed, 2, false);
    if (d->M > 0) rs.add(d->weights, span, 2, false);
    rs.add(d->out, n_out, 2, true);
    if (rs.rc != VF_OK) return rs.rc;
    Operand w = weights_of(d), x = rows_of(d->packed, d->rows, d->M);
    if ((rc = add_workspace(&rs, d, d->M > 0 ? workspace_of(w, x) : 0)) != VF_OK) return rc;
    if ((rc = rs.check(true)) != VF_OK) return rc;

    vfp::ProductArgs a = make_args(d);
    a.red = int32_t(d->M);
    a.out = d->out;
    a.vec = d->N % 8 == 0 && aligned16(d->out);
    const Form f = rows_form(d);
    set_form(&a, f);
    const bool mn = along_n(d);
    if (d->M > 0) {                                        // else sums of nothing: zeros
        char *const space = static_cast<char *>(d->workspace);
        if (w.copied && (rc = w.copy(space, span, d->counts, nullptr, stream)) != VF_OK) return rc;
        if (x.copied && (rc = x.copy(space + w.bytes(), n_packed, nullptr, d->offsets + d->E,
                                     stream)) != VF_OK)
            return rc;
        a.a_slabs = mn && d->N % 64 == 0 ? 2 : 0;
        if (a.a_slabs) {
            const int64_t dims[4] = {64, w.lines, d->N / 64, d->E};
            const int64_t str[4] = {1, w.s_line, 64, w.s_outer};
            rc = make_map(&a.a_map, a.bf16, 4, w.p, dims, str, 64, 2);
        } else {
            const int64_t dims[3] = {w.len, w.lines, d->E}, str[3] = {1, w.s_line, w.s_outer};
            rc = make_map(&a.a_map, a.bf16, 3, w.p, dims, str, mn ? 64 : 128);
        }
        const int64_t dims[2] = {d->M, d->rows}, str[2] = {1, x.s_line};
        for (int i = 0; i < vfp::kBoxes && rc == VF_OK; ++i)
            if (i * f.box < f.tile_n / f.ctas)
                rc = make_map(&a.b_maps[i], a.bf16, 2, x.p, dims, str, (i + 1) * f.box);
        if (rc != VF_OK) return rc;
    }
    const int64_t part = part_of(d, false);
    a.part = int32_t(part);
    const Kernel kernel = f.ctas == 2 ? rows_kernel<2>(mn, d->M > part)
                                      : rows_kernel<1>(mn, d->M > part);
    const int64_t most = std::min(d->E, d->rows);          // experts that have rows
    return launch_product(kernel, a, f, a.feat_tiles * (most + d->rows / f.tile_n), stream);
}

// The map of packed rows for the weights' gradient: the second dimension steps over
// the rows as the third does (see the kernel); columns by 64 where they are whole.
int make_row_map(CUtensorMap *map, bool bf16, const Operand &x, int64_t slabs) {
    if (x.len % 64) {
        const int64_t dims[3] = {x.len, 64, x.lines}, str[3] = {1, x.s_line, x.s_line};
        return make_map(map, bf16, 3, x.p, dims, str, 64);
    }
    const int64_t dims[4] = {64, 64, x.lines, x.len / 64}, str[4] = {1, x.s_line, x.s_line, 64};
    return make_map(map, bf16, 4, x.p, dims, str, 64, 3, slabs);
}

// Pairs, unless half of a pair would have no feature to store, they would leave half of
// the SMs idle, or experts have few rows: then a tile is mostly its stores, for which
// the CTAs of a pair wait for each other (E = 64, N = 2,048, M = 1,024, bf16, us):
//   rows             64    128    192    256    384    512   1,024
//   pairs          76.1   83.9   90.4   97.1  109.8  122.5   198.9
//   single CTAs    54.1   65.8   77.1   88.5  114.1  140.2   258.3
// Tiles that are still few are made smaller, and the CTAs of a cluster
// share their rows: N = M = 512, E = 2 with 27,707 rows each takes 199 us with
// 16 tiles of 256 columns, 71 with four CTAs to each (102 with eight, whose clusters do
// not all find room at once), 47 with 32 tiles of 128 columns and four CTAs to each.
// Below some 24 blocks to a CTA its sums cost more than they save (1,500 rows: 8.1 us,
// 11.9 with two CTAs).
Form weights_form(const vf_product_desc *d) {
    const int64_t columns = d->E * ceil_div(d->M, 256), features = ceil_div(d->N, vfp::kTileM);
    if (features > 1 && 4 * columns * ceil_div(features, 2) > kSMs && mean_rows(d) > 352)
        return {2, 256, 0, true};
    const bool few = 4 * columns * features < kSMs;
    Form f = {1, few ? 128 : 256, 0, true};
    const int64_t tiles = d->E * ceil_div(d->M, f.tile_n) * features;
    const int64_t blocks = ceil_div(mean_rows(d), vfp::kBlockK);
    while (f.split < 4 && 2 * f.split * tiles <= kSMs && blocks >= 48 * f.split) f.split *= 2;
    return f;
}

template <int CTAS, bool SPLIT>
Kernel weights_kernel(bool parts, bool out32) {
    return out32   ? vfp::expert_product<CTAS, true, true, true, SPLIT, true>
           : parts ? vfp::expert_product<CTAS, true, true, true, SPLIT>
                   : vfp::expert_product<CTAS, true, true, false, SPLIT>;
}

int weight_grad(const vf_product_desc *d, cudaStream_t stream) {
    int rc = check_desc(d);
    if (rc != VF_OK) return rc;
    if (d->out_type != d->type && d->out_type != VF_TYPE_F32) return VF_ERR_ARG;
    const int64_t size = type_size(d->out_type);
    int64_t n_packed, n_grad, n_out;
    if (!mul_ok(d->rows, d->M, &n_packed) || !mul_ok(d->rows, d->N, &n_grad) ||
        !mul_ok(d->N * d->M, d->E, &n_out))                // N * M at most 2^40
        return VF_ERR_OVERFLOW;
    if (n_out == 0) return VF_OK;
    Ranges rs;
    rs.add(d->counts, d->E, 4, false);
    rs.add(d->offsets, d->E + 1, 4, false);
    rs.add(d->packed, n_packed, 2, false);
    rs.add(d->grad, n_grad, 2, false);
    rs.add(d->grad_weights, n_out, size, true);
    if (rs.rc != VF_OK) return rs.rc;
    Operand g = rows_of(d->grad, d->rows, d->N), x = rows_of(d->packed, d->rows, d->M);
    if ((rc = add_workspace(&rs, d, d->rows > 0 ? workspace_of(g, x) : 0)) != VF_OK) return rc;
    if ((rc = rs.check(true)) != VF_OK) return rc;

    vfp::ProductArgs a = make_args(d);
    a.cols = int32_t(d->M);
    a.out = d->grad_weights;
    const bool out32 = d->out_type == VF_TYPE_F32;
    // Where an expert can have more rows than a part, the sums are taken in parts.
    const int64_t part = part_of(d, out32);
    const bool parts = out32 || d->rows > part;
    a.part = int32_t(part);
    a.vec = d->M % (16 / size) == 0 && aligned16(d->grad_weights);
    const Form f = weights_form(d);
    set_form(&a, f);
    a.a_slabs = d->N % 64 ? 0 : 2;
    a.b_slabs = d->M % 64 ? 0 : int32_t(f.tile_n / f.ctas / 64);
    if (d->rows > 0) {                                     // else sums of nothing: zeros
        char *const space = static_cast<char *>(d->workspace);
        const int32_t *const used = d->offsets + d->E;
        if (g.copied && (rc = g.copy(space, n_grad, nullptr, used, stream)) != VF_OK) return rc;
        if (x.copied && (rc = x.copy(space + g.bytes(), n_packed, nullptr, used, stream)) != VF_OK)
            return rc;
        if ((rc = make_row_map(&a.a_map, a.bf16, g, 2)) != VF_OK ||
            (rc = make_row_map(&a.b_maps[0], a.bf16, x, a.b_slabs)) != VF_OK)
            return rc;
    }
    const Kernel kernel =
        f.ctas == 2    ? weights_kernel<2, false>(parts, out32)
        : f.split == 1 ? weights_kernel<1, false>(parts, out32)
                       : weights_kernel<1, true>(parts, out32);
    return launch_product(kernel, a, f, int64_t(a.feat_tiles) * a.col_tiles * a.E, stream);
}

}  // namespace

extern "C" {

int64_t vf_expert_product_workspace(const vf_product_desc *d) {
    const int rc = check_desc(d);
    if (rc != VF_OK) return rc;
    for (int i = 0; i < 3; ++i)
        if (d->weight_strides[i] < 0) return VF_ERR_ARG;
    return d->M > 0 ? workspace_of(weights_of(d), rows_of(d->packed, d->rows, d->M)) : 0;
}

int64_t vf_expert_weight_grad_workspace(const vf_product_desc *d) {
    const int rc = check_desc(d);
    if (rc != VF_OK) return rc;
    return workspace_of(rows_of(d->grad, d->rows, d->N), rows_of(d->packed, d->rows, d->M));
}

int vf_expert_product(const vf_product_desc *d, vf_stream_t stream) {
    return product(d, as_stream(stream));
}

int vf_expert_weight_grad(const vf_product_desc *d, vf_stream_t stream) {
    return weight_grad(d, as_stream(stream));
}

}  // extern "C"
