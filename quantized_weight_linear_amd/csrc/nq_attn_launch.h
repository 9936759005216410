// Launchers of the attention and cache kernels, and what their entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "nq_launch.h"

namespace nq {

// Raises a kernel's limit of dynamic LDS, once per device (one object a
// kernel).  Two threads may both do it; that is harmless.
class LdsLimit {
public:
    hipError_t raise(const void* kernel, int bytes) {
        int dev = 0;
        if (hipError_t e = hipGetDevice(&dev); e != hipSuccess) return e;
        const uint64_t bit = 1ull << (dev & 63);
        if (dev < 64 && (done_.load(std::memory_order_relaxed) & bit)) return hipSuccess;
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == hipSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }

private:
    std::atomic<uint64_t> done_{0};
};

// Attention and the paged cache (see nq.h for the arguments; everything is
// validated by the callers).
hipError_t launch_attn_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int64_t seqs, int64_t tq,
                              int64_t tk, int64_t hq, int64_t hkv, int64_t d, float scale, bool bf16_out, void* o,
                              float* lse, hipStream_t stream);
int64_t attn_tree_workspace_bytes(int64_t seqs, int64_t max_q, int64_t hq, int64_t hkv, int64_t d, int64_t max_len);
hipError_t launch_attn_tree(int kv_fmt, const uint16_t* q, int64_t q_stride, const void* k_pages, const void* v_pages,
                            const float* k_scale, const float* v_scale, const int32_t* table, int64_t width,
                            const int32_t* lens, const int32_t* cu_q, const uint64_t* masks, int64_t seqs, int64_t max_q,
                            int64_t t, int64_t hq, int64_t hkv, int64_t d, int64_t page_size, int64_t pages,
                            int64_t max_len, float scale, bool bf16_out, void* o, float* lse, void* workspace,
                            int64_t workspace_bytes, hipStream_t stream);
hipError_t launch_kv_append(bool fp8, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                            const float* k_scale, const float* v_scale, const int32_t* table, int64_t width,
                            const int32_t* lens, const int32_t* cu, int64_t seqs, int64_t t, int64_t hkv, int64_t d,
                            int64_t page_size, int64_t pages, void* k_pages, void* v_pages, hipStream_t stream);
hipError_t launch_kv_reserve(int32_t* refs, int64_t pages, int32_t* table, int64_t width, const int32_t* lens,
                             const int32_t* new_lens, int64_t seqs, int64_t page_size, int32_t* free_list,
                             int32_t* shortfall, hipStream_t stream);
hipError_t launch_kv_release(int32_t* refs, int64_t pages, int32_t* table, int64_t width, const int32_t* keep, int64_t seqs,
                             int64_t page_size, hipStream_t stream);
hipError_t launch_kv_fork(int32_t* refs, int64_t pages, const int32_t* table, int64_t width, const int32_t* lens, int64_t seqs,
                          const int32_t* parents, int64_t children, int64_t page_size, int32_t* child_table, int32_t* copies,
                          int32_t* free_list, int32_t* shortfall, hipStream_t stream);
hipError_t launch_kv_copy_pages(void* pool, int64_t planes, int64_t plane_bytes, int64_t page_bytes, int64_t pages,
                                const int32_t* copies, int64_t n, hipStream_t stream);
hipError_t launch_kv_compact(void* pool, int64_t planes, int64_t plane_bytes, int64_t hkv, int64_t page_size,
                             int64_t row_bytes, int64_t pages, const int32_t* table, int64_t width, const int32_t* lens,
                             const int32_t* accept, const int32_t* cu_accept, int64_t seqs, int64_t accepted,
                             hipStream_t stream);

}  // namespace nq
