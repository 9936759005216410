// RMS norm with the residual's addition (nq_rmsnorm) and the E4M3 quantizer
// with a scale for each 128 columns (nq_quantize_act_fp8_b128).
//
//   h = bf16(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = (h r) (w + bias)
//
// A row stays in registers between its two passes (the sum of squares, then
// the output), so every byte is read and written once.  Bound by HBM where
// rows are many (16383 x 5120 in BF16: 66.2 us, 5.1 TB/s; 1792 with the residual
// and E4M3 out: 15.9 us, 4.1 TB/s), by latency where they are few (one row: 3.9 us),
// and by the FP64 arithmetic beside the loads where 8-bit outputs come without a
// residual (16383 x 5120 to E4M3 83 us, to int8 86, for 50 of bytes).
//   h is rounded to BF16 before it is normalised: it is what the next layer
// adds to, so the norm is that of the stored residual, fused or not.  Squares
// are summed in FP64, which costs nothing beside the loads and neither
// overflows nor loses bits at any BF16 input; h r is one rounding to FP32.
//   The 8-bit outputs are quantized from the FP32 values of y, without a
// rounding to BF16 between.
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_device.h"
#include "nq_layer_launch.h"

namespace nq {
namespace {

struct NormArgs {
    const uint16_t* x;
    int64_t xs;                     // elements between rows of x
    const uint16_t* residual;       // [T][K], or NULL
    uint16_t* residual_out;
    const uint16_t* weight;         // [K], or NULL (ones)
    float bias;
    double eps;
    int64_t t;
    int k;
    void* y;
    float* y_scale;
};

__device__ __forceinline__ void unpack8(v4u w, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

// The largest |f| as FP32 bits; a NaN is larger than everything.
__device__ __forceinline__ uint32_t top_bits(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    return m;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
    for (int off = 1; off < LANES; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    return m;
}

// Eight E4M3 codes of f / s (s = amax / 448 of the group they belong to): a
// group of zeros keeps its signed zeros, a NaN scale gives NaN codes.
__device__ __forceinline__ v2u codes_e4m3(const float (&f)[8], float s) {
    const double r = s == 0.f ? 1.0 : 1.0 / (double)s;
    float g[8];
    bool plain = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        g[j] = div_via_recip64(f[j], r);
        plain = plain && __builtin_fabsf(g[j]) < 464.f;
    }
    if (plain) return v2u{f32x4_to_e4m3_hw(g[0], g[1], g[2], g[3]), f32x4_to_e4m3_hw(g[4], g[5], g[6], g[7])};
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= f32_to_e4m3_sat(g[j]) << (8 * (j & 3));
    return v2u{w[0], w[1]};
}

__device__ __forceinline__ v2u codes_i8(const float (&f)[8], float s) {
    const double r = 1.0 / (double)s;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= ((uint32_t)f32_to_i8_sat(s == 0.f ? 0.f : div_via_recip64(f[j], r)) & 0xFFu) << (8 * (j & 3));
    return v2u{w[0], w[1]};
}

// A row a workgroup of THREADS, PIECES pieces of 8 columns a thread, piece i of
// thread n at 8 (i THREADS + n): a scale's columns lie in 8 or 16 neighbouring
// lanes.
template <int FMT, int THREADS, int PIECES, bool RESIDUAL>
__global__ __launch_bounds__(THREADS) void rmsnorm_kernel(NormArgs a) {
    constexpr int WAVES = THREADS / 64;
    __shared__ double part[WAVES];
    const int mine = threadIdx.x;
    const int64_t t = blockIdx.x, row = t * a.k;
    const uint16_t* x = a.x + t * a.xs;
    v4u h[PIECES], w[PIECES], r[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int col = (i * THREADS + mine) * 8;
        h[i] = r[i] = w[i] = v4u{0u, 0u, 0u, 0u};
        if (col < a.k) {
            h[i] = *reinterpret_cast<const v4u*>(x + col);
            if (RESIDUAL) r[i] = *reinterpret_cast<const v4u*>(a.residual + row + col);
            w[i] = a.weight ? *reinterpret_cast<const v4u*>(a.weight + col) : v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int col = (i * THREADS + mine) * 8;
        float f[8];
        unpack8(h[i], f);
        if (RESIDUAL) {
            float g[8];
            unpack8(r[i], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] = f32_to_bf16_rne(f[2 * j] + g[2 * j]) | f32_to_bf16_rne(f[2 * j + 1] + g[2 * j + 1]) << 16;
            if (col < a.k) *reinterpret_cast<v4u*>(a.residual_out + row + col) = h[i];
            unpack8(h[i], f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)f[j], (double)f[j], sum);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) part[mine / 64] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) sum += part[i];
    }
    const double rstd = 1.0 / __builtin_sqrt(sum / (double)a.k + a.eps);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int col = (i * THREADS + mine) * 8;
        float f[8], g[8];
        unpack8(h[i], f);
        unpack8(w[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)((double)f[j] * rstd) * (g[j] + a.bias);
        const bool store = col < a.k;
        if constexpr (FMT == NQ_ACT_BF16) {
            v4u o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = f32_to_bf16_rne(f[2 * j]) | f32_to_bf16_rne(f[2 * j + 1]) << 16;
            if (store) *reinterpret_cast<v4u*>((uint16_t*)a.y + row + col) = o;
        } else {
            constexpr int GROUP = FMT == NQ_ACT_INT8_G64 ? 64 : 128;
            if (col >= a.k) {                            // past the row: nothing of the last group's
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = 0.f;
            }
            const float top = __uint_as_float(lanes_max<GROUP / 8>(top_bits(f)));
            const float s = top / (FMT == NQ_ACT_INT8_G64 ? 127.0f : 448.0f);
            const v2u c = FMT == NQ_ACT_INT8_G64 ? codes_i8(f, s) : codes_e4m3(f, s);
            if (store) *reinterpret_cast<v2u*>((uint8_t*)a.y + row + col) = c;
            if (store && mine % (GROUP / 8) == 0) a.y_scale[t * ((a.k + GROUP - 1) / GROUP) + col / GROUP] = s;
        }
    }
}

// Eight columns a thread, sixteen lanes a scale.  s = fp32(amax / 448), codes
// e4m3_rne_sat(fp32(x / s)): exact, see div_via_recip64.  Bound by HBM (1792 x 17408
// 23.1 us, 4.1 TB/s; 16384 x 5120 57, 4.4), by latency for few rows (33 x 17408 2.6 us).
__global__ __launch_bounds__(256) void quantize_fp8_b128_kernel(const uint16_t* x, int64_t t, int k, int groups, uint8_t* codes,
                                                                float* scale) {
    const int64_t g = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16, row = g / groups;
    const int col = (int)(g % groups) * 128 + threadIdx.x % 16 * 8;
    const bool store = row < t && col < k;
    const v4u w = store ? *reinterpret_cast<const v4u*>(x + row * k + col) : v4u{0u, 0u, 0u, 0u};
    float f[8];
    unpack8(w, f);
    const float s = __uint_as_float(lanes_max<16>(top_bits(f))) / 448.0f;
    const v2u c = codes_e4m3(f, s);
    if (!store) return;
    *reinterpret_cast<v2u*>(codes + row * k + col) = c;
    if (threadIdx.x % 16 == 0) scale[g] = s;
}

template <int FMT, int THREADS, int PIECES>
hipError_t go_norm(const NormArgs& a, hipStream_t stream) {
    const unsigned blocks = (unsigned)a.t;
    if (a.residual) rmsnorm_kernel<FMT, THREADS, PIECES, true><<<blocks, THREADS, 0, stream>>>(a);
    else rmsnorm_kernel<FMT, THREADS, PIECES, false><<<blocks, THREADS, 0, stream>>>(a);
    return hipGetLastError();
}

// Few rows: as few pieces a thread as there are, since a row waits for its sum
// and its pieces come one after another.  Many: workgroups half as large, of
// which a CU holds more rows.  Microseconds with the residual, E4M3 output, three
// sets of inputs in turn; (int8) where that output's order is another:
//                     1 row    1792    3000    4096   16384   65536
//   512:   64 x 1      2.5      3.7     4.5     5.1    13.1    45.8
//   1024: 128 x 1      2.7      4.9     7.0     9.2    21.3    85.3 (93.3)
//          64 x 2      3.2      5.0     7.3     9.3    22.5    86.9 (87.9)
//   2048: 256 x 1      2.8      8.1    11.0    13.2    47.0 (51.0)   166 (176)
//         128 x 2      3.4      8.8    12.1    14.2    47.0 (48.6)   165 (166)
//   4096: 512 x 1      3.2     12.3    17.4    21.9    86.7
//         256 x 2      3.6     13.3    18.2    22.7    86.0
//   5120: 512 x 2      4.0     17.3    25.6    35.4   127
//         256 x 3      4.5     16.4    23.4    31.3   108
//   8192: 512 x 2      4.2     20.7    35.0    47.6   165
//         256 x 4      5.5     23.5    41.4    54.7   185
//        1024 x 1      4.2     21.8    36.2    48.5   182
//   12288: 512 x 3     5.4     31.7    54.1    69.8
//         1024 x 2     5.8     42.8    69.3    89.9
//   16384: 1024 x 2    6.0     52.1    82.4   106
//          512 x 4     6.4     45.5    71.1    91.7
//   24576: 1024 x 3    7.6     79.1   121     162
//   32768: 1024 x 4    9.2    106     166     217
// Between 2049 and some 10000 rows of 1024 to 4096 the larger workgroups are up to
// 11 % faster; without a residual the smaller ones gain most (65536 x 1024 E4M3
// 55.7 / 47.2).  BF16 outputs are within 8 % either way, also at 16384 columns
// (1024 x 2 47.2, 512 x 4 48.4 for 1792 rows), whose form was chosen for few rows.
template <int FMT>
hipError_t go_norm(const NormArgs& a, hipStream_t stream) {
    const bool few = a.t <= 2048;
    if (a.k <= 64 * 8) return go_norm<FMT, 64, 1>(a, stream);
    if (a.k <= 128 * 8) return few ? go_norm<FMT, 128, 1>(a, stream) : go_norm<FMT, 64, 2>(a, stream);
    if (a.k <= 256 * 8) return few ? go_norm<FMT, 256, 1>(a, stream) : go_norm<FMT, 128, 2>(a, stream);
    if (a.k <= 512 * 8) return few ? go_norm<FMT, 512, 1>(a, stream) : go_norm<FMT, 256, 2>(a, stream);
    if (a.k <= 256 * 24) return a.t <= 1024 ? go_norm<FMT, 512, 2>(a, stream) : go_norm<FMT, 256, 3>(a, stream);
    if (a.k <= 512 * 16) return go_norm<FMT, 512, 2>(a, stream);
    if (a.k <= 512 * 24) return go_norm<FMT, 512, 3>(a, stream);
    if (a.k <= 1024 * 16) return go_norm<FMT, 1024, 2>(a, stream);
    if (a.k <= 1024 * 24) return go_norm<FMT, 1024, 3>(a, stream);
    return go_norm<FMT, 1024, 4>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(int act_fmt, const uint16_t* x, int64_t x_stride, const uint16_t* residual, uint16_t* residual_out,
                          const uint16_t* weight, float bias, float eps, int64_t t, int64_t k, void* y, float* y_scale,
                          hipStream_t stream) {
    const NormArgs a{x, x_stride, residual, residual_out, weight, bias, (double)eps, t, (int)k, y, y_scale};
    switch (act_fmt) {
        case NQ_ACT_BF16: return go_norm<NQ_ACT_BF16>(a, stream);
        case NQ_ACT_INT8_G64: return go_norm<NQ_ACT_INT8_G64>(a, stream);
        default: return go_norm<NQ_ACT_E4M3_B128>(a, stream);
    }
}

hipError_t launch_quantize_fp8_b128(const uint16_t* x, int64_t t, int64_t k, uint8_t* codes, float* scale, hipStream_t stream) {
    const int64_t groups = (k + 127) / 128;
    quantize_fp8_b128_kernel<<<(unsigned)((t * groups + 15) / 16), 256, 0, stream>>>(x, t, (int)k, (int)groups, codes, scale);
    return hipGetLastError();
}

}  // namespace nq
