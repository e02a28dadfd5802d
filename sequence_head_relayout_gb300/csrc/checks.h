// Host-side argument checks shared by every entry point of the C ABI: checked
// 64-bit arithmetic, strided-view geometry, byte ranges and pointer queries.
// Nothing here enqueues work.  Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "vf_relayout.h"

namespace vfc {

constexpr int64_t kMaxExtent = int64_t(1) << 30;        // limit of every tensor extent

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    return !__builtin_mul_overflow(a, b, out);
}
inline bool add_ok(int64_t a, int64_t b, int64_t *out) {
    return !__builtin_add_overflow(a, b, out);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return a == 0 ? 0 : (a - 1) / b + 1; }

// Largest element offset a strided view addresses (all strides >= 0).
inline int max_offset(const int64_t *ext, const int64_t *str, int nd, int64_t *out) {
    int64_t m = 0;
    for (int i = 0; i < nd; ++i) {
        if (str[i] < 0) return VF_ERR_ARG;
        if (ext[i] <= 1) continue;
        int64_t term;
        if (!mul_ok(ext[i] - 1, str[i], &term) || !add_ok(m, term, &m)) return VF_ERR_OVERFLOW;
    }
    *out = m;
    return VF_OK;
}

// True when a write view never maps two logical elements to one address:
// sorted by stride, each stride must exceed the span of the smaller ones.
inline bool non_overlapping(const int64_t *ext, const int64_t *str, int nd) {
    int idx[4] = {0, 0, 0, 0};
    int k = 0;
    for (int i = 0; i < nd; ++i)
        if (ext[i] > 1) idx[k++] = i;
    for (int j = 1; j < k; ++j)                 // insertion sort by stride, k <= 4
        for (int m = j; m > 0 && str[idx[m]] < str[idx[m - 1]]; --m) std::swap(idx[m], idx[m - 1]);
    int64_t span = 0;
    for (int j = 0; j < k; ++j) {
        const int i = idx[j];
        if (str[i] <= span) return false;
        span += str[i] * (ext[i] - 1);      // bounded by max_offset, no overflow
    }
    return true;
}

// A byte range [lo, lo + len).
struct Range {
    uintptr_t lo;
    uint64_t len;
};

inline bool overlap(const Range &a, const Range &b) {
    if (a.len == 0 || b.len == 0) return false;
    return a.lo < b.lo + b.len && b.lo < a.lo + a.len;
}

inline int check_pointer(const void *p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return VF_ERR_CUDA;
    }
    if (at.type == cudaMemoryTypeUnregistered) return VF_ERR_ARG;
    // page-locked host memory must be mapped at the same address on the device
    if (at.type == cudaMemoryTypeHost && at.devicePointer != p) return VF_ERR_ARG;
    if (at.type == cudaMemoryTypeDevice) {
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            return VF_ERR_CUDA;
        }
        if (at.device != dev) return VF_ERR_ARG;       // another GPU's memory
    }
    return VF_OK;
}

}  // namespace vfc
