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
// from the second dimension on; boxes of 64 elements (128 bytes, swizzled), two of
// them along dimension `slabs`.
int make_map(CUtensorMap *map, bool bf16, int nd, const void *base, const int64_t *ext,
             const int64_t *str, int64_t box1, int slabs = 0) {
    const EncodeTiled fn = encoder();
    if (fn == nullptr) return VF_ERR_CUDA;
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4] = {64, cuuint32_t(box1), 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    if (slabs) box[slabs] = 2;
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
};

void set_form(vfp::ProductArgs *a, const Form &f, bool fill) {
    const int64_t b_rows = f.tile_n / f.ctas;
    a->tile_n = int32_t(f.tile_n);
    a->box = int32_t(f.box);
    a->stage_bytes = int32_t(vfp::kStageA + (fill ? vfp::kTileM : b_rows) * 128);
    a->stages = 0;
    while (a->stages < vfp::kMaxStages &&
           vfp::shared_bytes(a->stages + 1, a->stage_bytes) <= kSharedMemory)
        ++a->stages;
    a->acc_stride = int32_t(std::max<int64_t>(32, f.tile_n));
    a->tmem_cols = 64;
    while (a->tmem_cols < 2 * a->acc_stride) a->tmem_cols *= 2;
    a->feat_tiles = int32_t(ceil_div(a->feat, vfp::kTileM * f.ctas));
    a->col_tiles = int32_t(ceil_div(a->cols, f.tile_n));
}

using Kernel = void (*)(vfp::ProductArgs);

int launch_product(Kernel kernel, vfp::ProductArgs &a, int64_t ctas, int64_t tiles,
                   cudaStream_t stream, int threads = vfp::kThreads) {
    if (tiles == 0) return VF_OK;
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
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = size_t(vfp::shared_bytes(a.stages, a.stage_bytes));
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

// How tensor maps take the operands of a product: 0 not at all, 1 the weights with
// unit stride along m, 2 along n.
int weight_maps(const vf_product_desc *d) {
    if (d->M == 0 || d->M % 8 || !aligned16(d->packed) || !aligned16(d->weights)) return 0;
    int64_t e = d->weight_strides[0], n = d->weight_strides[1], m = d->weight_strides[2];
    if (!map_stride(d->E, &e, 8)) return 0;
    if ((m == 1 || d->M == 1) && map_stride(d->N, &n, 8)) return 1;
    if ((n == 1 || d->N == 1) && map_stride(d->M, &m, 8)) return 2;
    return 0;
}

// Rows of a tile, by the rows that an expert has on average.
Form rows_form(const vf_product_desc *d, bool maps) {
    if (!maps) return {1, 128, 0};
    const int64_t mean = ceil_div(d->slots, d->E);
    if (mean <= 8) return {1, 32, 16};
    if (mean <= 32) return {1, 64, 16};
    if (mean <= 96 || d->N <= 128) return {1, 128, 32};
    return {2, 256, 32};
}

int product(const vf_product_desc *d, cudaStream_t stream) {
    int rc = check_desc(d);
    if (rc != VF_OK) return rc;
    int64_t n_packed, n_out, w_span;
    const int64_t ext[3] = {d->E, d->N, d->M};
    if (!mul_ok(d->rows, d->M, &n_packed) || !mul_ok(d->rows, d->N, &n_out))
        return VF_ERR_OVERFLOW;
    if ((rc = max_offset(ext, d->weight_strides, 3, &w_span)) != VF_OK) return rc;
    if (n_out == 0) return VF_OK;                          // nothing to write
    Ranges rs;
    rs.add(d->counts, d->E, 4, false);
    rs.add(d->offsets, d->E + 1, 4, false);
    rs.add(d->packed, n_packed, 2, false);
    if (!add_ok(w_span, 1, &w_span)) return VF_ERR_OVERFLOW;
    if (d->M > 0) rs.add(d->weights, w_span, 2, false);
    rs.add(d->out, n_out, 2, true);
    if ((rc = rs.check(true)) != VF_OK) return rc;

    vfp::ProductArgs a = make_args(d);
    a.red = int32_t(d->M);
    a.out = d->out;
    a.vec = d->N % 8 == 0 && aligned16(d->out);
    const int64_t most = std::min(d->E, d->rows);          // experts that have rows
    a.a = static_cast<const uint16_t *>(d->weights);
    a.b = static_cast<const uint16_t *>(d->packed);
    a.a_expert = d->weight_strides[0];
    a.a_i = d->weight_strides[1];
    a.a_k = d->weight_strides[2];
    a.b_i = d->M;
    a.b_k = 1;
    const int maps = weight_maps(d);
    const Form f = rows_form(d, maps != 0);
    set_form(&a, f, maps == 0);
    const int64_t tiles = a.feat_tiles * (most + d->rows / f.tile_n);
    if (maps == 0)
        return launch_product(vfp::expert_product<1, false, false, true>, a, f.ctas, tiles,
                              stream, vfp::kFillThreads);
    const bool mn = maps == 2;
    const int64_t dims[3] = {mn ? d->N : d->M, mn ? d->M : d->N, d->E};
    int64_t str[3] = {1, d->weight_strides[mn ? 2 : 1], d->weight_strides[0]};
    map_stride(dims[1], &str[1], dims[0]);
    map_stride(dims[2], &str[2], dims[0]);
    a.a_slabs = mn && d->N % 64 == 0;
    if (a.a_slabs) {
        const int64_t dims4[4] = {64, dims[1], d->N / 64, d->E}, str4[4] = {1, str[1], 64, str[2]};
        rc = make_map(&a.a_map, a.bf16, 4, d->weights, dims4, str4, 64, 2);
    } else {
        rc = make_map(&a.a_map, a.bf16, 3, d->weights, dims, str, mn ? 64 : 128);
    }
    if (rc != VF_OK) return rc;
    const int64_t b_dims[2] = {d->M, d->rows}, b_str[2] = {1, d->M};
    for (int i = 0; i < vfp::kBoxes && rc == VF_OK; ++i)
        if (i * f.box < f.tile_n / f.ctas)
            rc = make_map(&a.b_maps[i], a.bf16, 2, d->packed, b_dims, b_str, (i + 1) * f.box);
    if (rc != VF_OK) return rc;
    const Kernel kernel =
        f.ctas == 2 ? (mn ? vfp::expert_product<2, false, true, false>
                          : vfp::expert_product<2, false, false, false>)
                    : (mn ? vfp::expert_product<1, false, true, false>
                          : vfp::expert_product<1, false, false, false>);
    return launch_product(kernel, a, f.ctas, tiles, stream);
}

// The map of packed rows for the weights' gradient: the second dimension steps over
// the rows as the third does (see the kernel); columns by 64 where they are whole.
int make_row_map(CUtensorMap *map, bool bf16, const void *p, int64_t cols, int64_t rows) {
    if (cols % 64) {
        const int64_t dims[3] = {cols, 64, rows}, str[3] = {1, cols, cols};
        return make_map(map, bf16, 3, p, dims, str, 64);
    }
    const int64_t dims[4] = {64, 64, rows, cols / 64}, str[4] = {1, cols, cols, 64};
    return make_map(map, bf16, 4, p, dims, str, 64, 3);
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
    if ((rc = rs.check(true)) != VF_OK) return rc;

    vfp::ProductArgs a = make_args(d);
    a.cols = int32_t(d->M);
    a.out = d->grad_weights;
    a.out32 = d->out_type == VF_TYPE_F32;
    // The tensor cores cut off what lies below an accumulator's last bit, always towards
    // the same side, so that a sum's error grows with its length: 1.2e-6 of the result
    // at 1,024 rows.  Sums in float32 are therefore taken in parts, which are added with
    // rounding.  (The 16-bit types round a thousand times as coarsely.)
    a.part_rows = a.out32 ? 256 : INT32_MAX;
    a.vec = d->M % (16 / size) == 0 && aligned16(d->grad_weights);
    a.a = static_cast<const uint16_t *>(d->grad);
    a.b = static_cast<const uint16_t *>(d->packed);
    a.a_i = a.b_i = 1;
    a.a_k = d->N;
    a.b_k = d->M;
    const bool maps = d->rows > 0 && d->N % 8 == 0 && d->M % 8 == 0 && aligned16(d->grad) &&
                      aligned16(d->packed);
    const Form f = maps ? Form{2, 256, 0} : Form{1, 128, 0};
    set_form(&a, f, !maps);
    const int64_t tiles = int64_t(a.feat_tiles) * a.col_tiles * a.E;
    if (!maps)
        return launch_product(vfp::expert_product<1, true, false, true>, a, f.ctas, tiles,
                              stream, vfp::kFillThreads);
    a.a_slabs = d->N % 64 == 0;
    a.b_slabs = d->M % 64 == 0;
    if ((rc = make_row_map(&a.a_map, a.bf16, d->grad, d->N, d->rows)) != VF_OK ||
        (rc = make_row_map(&a.b_maps[0], a.bf16, d->packed, d->M, d->rows)) != VF_OK)
        return rc;
    const Kernel kernel = a.out32 ? vfp::expert_product<2, true, true, false, true>
                                  : vfp::expert_product<2, true, true, false>;
    return launch_product(kernel, a, f.ctas, tiles, stream);
}

}  // namespace

extern "C" {

int vf_expert_product(const vf_product_desc *d, vf_stream_t stream) {
    return product(d, as_stream(stream));
}

int vf_expert_weight_grad(const vf_product_desc *d, vf_stream_t stream) {
    return weight_grad(d, as_stream(stream));
}

}  // extern "C"
