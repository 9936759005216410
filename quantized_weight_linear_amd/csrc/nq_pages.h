// What the kernels that write rows into the paged cache share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nq_device.h"

namespace nq {

// The sequence that packed row t belongs to: the last b with cu[b] <= t.
__device__ __forceinline__ int owner(const int32_t* cu, int seqs, int64_t t) {
    int lo = 0, hi = seqs;                               // cu[lo] <= t < cu[hi] where cu is in order
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The page and slot of token `at` of a sequence, or page -1 where the table
// has none inside the pool.
__device__ __forceinline__ int64_t page_of(const int32_t* table, int64_t width, int64_t pages, int shift, int64_t at) {
    if (at < 0 || (at >> shift) >= width) return -1;
    const int64_t p = table[at >> shift];
    return p < 0 || p >= pages ? -1 : p;
}

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if (fabsf(a) < 448.f && fabsf(b) < 448.f && fabsf(c) < 448.f && fabsf(d) < 448.f) return f32x4_to_e4m3_hw(a, b, c, d);
    return f32_to_e4m3_sat(a) | f32_to_e4m3_sat(b) << 8 | f32_to_e4m3_sat(c) << 16 | f32_to_e4m3_sat(d) << 24;
}

}  // namespace nq
