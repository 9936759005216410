// Host-side launchers for the HIP kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

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

// Weight formats, same values as nq_wfmt plus the row-scaled FP8 format.
enum WFmt { W_Q4G64 = 0, W_Q8G32 = 1, W_Q8G64 = 2, W_MXFP8 = 3, W_BF16 = 4, W_Q3G64 = 5, W_Q5G64 = 6, W_Q6G64 = 7,
            W_FP8ROW = 8 };

hipError_t launch_decode_mxfp8(const uint32_t* words, const uint8_t* e8, int64_t N, int64_t K, bool bf16_out,
                               void* out, hipStream_t stream);
hipError_t launch_decode_mlx_affine_int8(const uint8_t* codes, const uint16_t* scales, const uint16_t* biases,
                                         int64_t N, int64_t K, bool bf16_out, void* out, hipStream_t stream);
hipError_t launch_unpack_q4_to_int8(const uint8_t* codes, int64_t N, int64_t K, int8_t* out, hipStream_t stream);
hipError_t launch_reencode_block128(const uint8_t* codes, const float* wsi, int64_t N, int64_t K, int64_t gc,
                                    int64_t r0, int64_t r1, uint8_t* out_codes, uint16_t* out_scale,
                                    hipStream_t stream);
hipError_t launch_encode_fp8row_bf16(const uint16_t* w, int64_t N, int64_t K, uint8_t* out_codes,
                                     uint16_t* out_scale, hipStream_t stream);
hipError_t launch_quantize_int8_g64(const uint16_t* x, int64_t T, int64_t K, int8_t* q, float* scale,
                                    hipStream_t stream);
hipError_t launch_quantize_fp8_row(const uint16_t* x, int64_t M, int64_t K, uint8_t* codes, float* scale,
                                   hipStream_t stream);

// Decode GEMV for every weight format.  `scales` is the per-format scale
// array (row scales for W_FP8ROW).  `workspace` (may be NULL) enables split-K
// across workgroups when it is large enough (gemv_workspace_bytes).
int64_t gemv_workspace_bytes(int fmt, int64_t T, int64_t N, int64_t K);
// `packed`: weights in the layout written by launch_pack_weights (requires K % 128 == 0).
hipError_t launch_gemv(int fmt, const void* w, const void* scales, const uint16_t* x, int64_t T, int64_t N,
                       int64_t K, bool bf16_out, void* y, void* workspace, int64_t workspace_bytes,
                       hipStream_t stream, bool packed);
int64_t packed_weight_bytes(int fmt, int64_t N, int64_t K);
// launch_gemv with the library's own per-device scratch array instead of a
// caller workspace (no allocation); the caller checks gemv_workspace_bytes
// against GEMV_STATIC_SCRATCH_BYTES first.
constexpr int64_t GEMV_STATIC_SCRATCH_BYTES = (int64_t)8 << 20;
hipError_t launch_gemv_noalloc(int fmt, const void* w, const void* scales, const uint16_t* x, int64_t T, int64_t N,
                               int64_t K, bool bf16_out, void* y, hipStream_t stream, bool packed);
hipError_t launch_pack_weights(int fmt, const void* src, int64_t N, int64_t K, void* dst, hipStream_t stream);

// A8 decode GEMV (int8 activation codes and scales from launch_quantize_int8_g64,
// Q8 or Q4 group-64 weights, row-major or packed as for launch_gemv).
int64_t gemv_a8_workspace_bytes(int64_t T, int64_t N, int64_t K);
hipError_t launch_gemv_a8(int fmt, const void* w, const uint16_t* w_scale, const int8_t* aq, const float* asc,
                          int64_t T, int64_t N, int64_t K, bool bf16_out, void* y, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream, bool packed);

// Q3 / Q5 / Q6 group-64 (dense little-endian bit streams): the BF16-activation
// GEMV (row-major or packed), the packing, and the widening to int8.
int qbits_of(int fmt);   // 3, 5, 6, or 0 for other formats
int64_t gemv_qbits_workspace_bytes(int64_t T, int64_t N, int64_t K);
hipError_t launch_gemv_qbits(int fmt, const void* w, const uint16_t* w_scale, const uint16_t* x, int64_t T, int64_t N,
                             int64_t K, bool bf16_out, void* y, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream, bool packed);
hipError_t launch_pack_qbits(int fmt, const void* src, int64_t N, int64_t K, void* dst, hipStream_t stream);
hipError_t launch_unpack_qbits_to_int8(int fmt, const uint8_t* codes, int64_t N, int64_t K, int8_t* out,
                                       hipStream_t stream);

hipError_t launch_gemm_w8a8(const int8_t* a_q, const float* a_scale, const int8_t* w_q, const uint16_t* w_scale,
                            int64_t M, int64_t N, int64_t K, bool bf16_out, void* y, int32_t* group_sums,
                            hipStream_t stream);
hipError_t launch_gemm_fp8(const uint8_t* a_codes, const float* a_scale, const uint8_t* w, const uint16_t* w_scale,
                           int64_t M, int64_t N, int64_t K, bool bf16_out, void* y, hipStream_t stream);

// Attention and the paged cache (see nq.h for the arguments; everything is
// validated by the callers).
hipError_t launch_attn_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int64_t seqs, int64_t tq,
                              int64_t tk, int64_t hq, int64_t hkv, int64_t d, float scale, bool bf16_out, void* o,
                              float* lse, hipStream_t stream);
int64_t attn_tree_workspace_bytes(int64_t seqs, int64_t max_q, int64_t hq, int64_t hkv, int64_t d, int64_t max_len);
hipError_t launch_attn_tree(bool fp8, const uint16_t* q, int64_t q_stride, const void* k_pages, const void* v_pages,
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

int device_cu_count();

// Plain streaming read of `bytes` (a multiple of 16) from src; one word per
// workgroup (stream_read_blocks() of them) goes to sink.
int stream_read_blocks();
hipError_t launch_stream_read(const void* src, int64_t bytes, uint32_t* sink, hipStream_t stream);

}  // namespace nq
