// What the host sides of the row operators share (the expert relayouts, the
// experts' products and the layer's row-wise operators): the limits of a plan,
// the ranges of a call and the launch.  Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "checks.h"
#include "vf_relayout.h"

namespace vfc {

constexpr int64_t kMaxSlots = int64_t(1) << 30;     // T * K
constexpr int64_t kMaxExperts = 4096;
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kSMs = 152;

inline cudaStream_t as_stream(vf_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Launch with programmatic stream serialisation, as the other kernels do.
template <class Args>
int launch(void (*kernel)(Args), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
           const Args &args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
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

template <class Args>
int launch(void (*kernel)(Args), int64_t blocks, int threads, size_t smem, cudaStream_t stream,
           const Args &args) {
    return launch(kernel, dim3(unsigned(blocks)), dim3(unsigned(threads)), smem, stream, args);
}

inline int64_t type_size(int type) { return type == VF_TYPE_F32 ? 4 : 2; }

// A range of `count` items of `size` bytes at p; false when it wraps.
inline bool make_range(const void *p, int64_t count, int64_t size, Range *r) {
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

    // Ranges i and i + 1 interleave without a common element.
    void join(int i) { joined = i; }
    int joined = -1;

    int check(bool device = false) {
        if (rc != VF_OK) return rc;
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j)
                if (!(i == joined && j == i + 1) &&
                    (written[i] || written[j]) && overlap(r[i], r[j]))
                    return VF_ERR_ALIAS;
        for (int i = 0; i < n; ++i)
            if ((rc = check_pointer(p[i], device)) != VF_OK) return rc;
        return VF_OK;
    }
};

}  // namespace vfc
