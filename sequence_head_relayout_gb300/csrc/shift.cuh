// Rows at any address: what lies across two 16-byte pieces.
#pragma once

#include <cstdint>

namespace vf {

// The 16 bytes from byte `shift` (even) of lo and hi on.
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, int shift) {
    uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) x[j] = shift & 8 ? x[j + 2] : x[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) x[j] = shift & 4 ? x[j + 1] : x[j];
    const int bits = shift & 2 ? 16 : 0;
    return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                      __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

}  // namespace vf
