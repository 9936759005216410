// RMS norm with the residual's addition (nq_rmsnorm) and the E4M3 quantizer
// with a scale for each 128 columns (nq_quantize_act_fp8_b128).
//
//   h = bf16(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = (h r) (w + bias)
//
// A row stays in registers between its two passes (the sum of squares, then
// the output), so every byte is read and written once.  Bound by HBM where
// rows are many (16383 x 5120 in BF16: 69.7 us, 4.8 TB/s; 1792 with the residual
// and E4M3 out: 15.6 us, 4.1 TB/s), by latency where they are few (one row: 3.8 us).
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
// e4m3_rne_sat(fp32(x / s)): exact, see div_via_recip64.
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
// which a CU holds more rows.  Microseconds, E4M3 output (the residual but for *):
//                     1 row    1792   16384   65536 *
//   512:   64 x 1      2.3      3.5    13.0    31
//          64 x 2      2.8      4.3    17.3    42
//   1024: 128 x 1      2.5      5.0    23.7    63
//          64 x 2      3.1      5.2    23.6    52
//   2048: 256 x 1      2.6      8.1    43.7    64 (32768)
//         128 x 2      3.3      8.8    40.4    59
//   4096: 512 x 1      2.9     12.8    85.7
//         256 x 2      3.4     13.6    74.8
//   5120: 512 x 2      3.8     17.4   129
//         256 x 3      4.3     16.6   112
//   8192: 512 x 2      4.1     22.8   167
//         256 x 4      5.4     26.6   189
//   12288: 512 x 3     5.2     36.0
//         1024 x 2     5.6     44.3
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
