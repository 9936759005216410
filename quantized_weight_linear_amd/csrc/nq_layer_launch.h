// Launchers of the norm, the block-scaled FP8 product and the rotated append
// (see nq.h for the arguments; everything is validated by the callers).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nq {

hipError_t launch_rmsnorm(int act_fmt, const uint16_t* x, int64_t x_stride, const uint16_t* residual, uint16_t* residual_out,
                          const uint16_t* weight, float bias, float eps, int64_t t, int64_t k, void* y, float* y_scale,
                          hipStream_t stream);
hipError_t launch_quantize_fp8_b128(const uint16_t* x, int64_t t, int64_t k, uint8_t* codes, float* scale, hipStream_t stream);

int64_t gemm_fp8_b128_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_gemm_fp8_b128(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int64_t m,
                                int64_t n, int64_t k, bool bf16_out, void* y, void* workspace, int64_t workspace_bytes,
                                hipStream_t stream);

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;                  // elements between tokens
    const uint16_t *q_weight, *k_weight; // [D], or NULL: the heads are not normalised
    float bias, eps;
    const int32_t* positions;
    const float* freq;                   // [rot / 2]
    int rot;
    bool pairs;
    float *k_scale, *v_scale;            // per head, or per page, head and slot
    const int32_t *table, *lens, *cu;
    int64_t width, pages, t;
    int seqs, hq, hkv, d, shift;
    uint16_t *q_out, *k_out;             // k_out may be NULL
    int64_t qos, kos;
    void *k_pages, *v_pages;
};
hipError_t launch_kv_append_rope(int kv_fmt, const RopeArgs& a, hipStream_t stream);

}  // namespace nq
