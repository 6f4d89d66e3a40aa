// work_split.h -- how the attention kernels share the units of a call among CTAs.
//
// The U units (key tiles) of a call lie on a line; CTA c of n takes
// [c U / n, (c + 1) U / n). The part of item w that CTA c computes goes to
// slot w + c: along the line each step raises w or c, so slots are distinct.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SC_HOST_DEVICE static inline
#endif

namespace sc {

// Divisions are made in 32 bits where both numbers fit. U n < 2^63.
SC_HOST_DEVICE int64_t share_begin(int64_t c, int64_t U, int64_t n) {
    const int64_t x = c * U;
    return x <= UINT32_MAX ? (int64_t)((uint32_t)x / (uint32_t)n) : x / n;
}
// The CTA that takes unit u (u < U).
SC_HOST_DEVICE int share_of(int64_t u, int64_t U, int64_t n) {
    const int64_t x = (u + 1) * n - 1;
    if (x <= UINT32_MAX && U <= UINT32_MAX) return (int)((uint32_t)x / (uint32_t)U);
    return (int)(x / U);
}

}  // namespace sc
