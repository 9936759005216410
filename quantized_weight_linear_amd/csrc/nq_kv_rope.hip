// A step's queries, keys and values: heads normalised (where the model does
// that) and turned by their tokens' positions, keys and values written into
// the paged cache (nq_kv_append_rope).
//
//   angle_i = position * freq_i,  (a, b) -> (a cos - b sin, a sin + b cos)
//
// for the pair (a, b) = columns (i, i + rot / 2), or (2 i, 2 i + 1).  A
// workgroup has one token (or some heads of it): its angles' cosines and sines are worked
// out once, in FP64 up to the fraction of a turn, since an FP32 angle of a far
// position is off by more than a thousandth, and all heads read them from LDS.
//   Each element is read once and written once; bound by HBM for prompts (12800
// tokens of 32 / 8 heads of 128 in BF16: 65 us, 4.8 TB/s; with a head's scale and
// E4M3 64.6, with one a row 71.8) and by latency for steps (one token: 4.1 us).  Heads'
// norms in FP64 come on top where there are many tokens: 93, 94 and 102 us.
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_device.h"
#include "nq_layer_launch.h"
#include "nq_pages.h"

namespace nq {
namespace {

constexpr int MOST_ROT = 256;

__device__ __forceinline__ void unpack8(v4u w, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ v4u pack8(const float (&f)[8]) {
    v4u o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = f32_to_bf16_rne(f[2 * j]) | f32_to_bf16_rne(f[2 * j + 1]) << 16;
    return o;
}

// Eight columns of a head into its cache row.  With a scale for the token:
// that of the row's largest finite value, so that a scale is always finite;
// infinities saturate like everything beyond 448 s, NaN stays NaN.
template <int FMT, int D>
__device__ __forceinline__ void keep(const float (&f)[8], void* pages, float* scale, int64_t row, int head, int col) {
    const int64_t to = row * D + col;
    if constexpr (FMT == NQ_KV_BF16) {
        if (row >= 0) *reinterpret_cast<v4u*>((uint16_t*)pages + to) = pack8(f);
    } else {
        double r;
        if constexpr (FMT == NQ_KV_E4M3) {
            r = 1.0 / (double)scale[head];
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(f[j]) & 0x7FFFFFFFu;
                top = u < 0x7F800000u ? max(top, u) : top;
            }
#pragma unroll
            for (int off = 1; off < D / 8; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
            const float s = __uint_as_float(top) / 448.0f;
            r = s == 0.f ? 1.0 : 1.0 / (double)s;
            if (row >= 0 && col == 0) scale[row] = s;
        }
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = div_via_recip64(f[j], r);
        if (row >= 0) *reinterpret_cast<v2u*>((uint8_t*)pages + to) = v2u{encode4(g[0], g[1], g[2], g[3]), encode4(g[4], g[5], g[6], g[7])};
    }
}

// One token a workgroup: D / 8 lanes a head, eight columns a lane.
template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_append_rope_kernel(RopeArgs a) {
    constexpr int LANES = D / 8;
    __shared__ __align__(16) float cos_s[MOST_ROT / 2], sin_s[MOST_ROT / 2];
    const int64_t t = blockIdx.x;
    const int b = owner(a.cu, a.seqs, t);
    const int64_t first = a.cu[b];
    if (t < first || t >= a.cu[b + 1]) return;          // no sequence's token
    const int half = a.rot / 2;
    if ((int)threadIdx.x < half) {
        const double turns = (double)a.positions[t] * (double)a.freq[threadIdx.x] * 0.15915494309189533577;
        const float x = (float)(2.0 * (turns - __builtin_rint(turns)));
        cos_s[threadIdx.x] = cospif(x);
        sin_s[threadIdx.x] = sinpif(x);
    }
    const int64_t at = (int64_t)a.lens[b] + (t - first);
    const int64_t page = a.lens[b] < 0 ? -1 : page_of(a.table + b * a.width, a.width, a.pages, a.shift, at);
    __syncthreads();
    const int heads = a.hq + 2 * a.hkv, col = threadIdx.x % LANES * 8;
    const int step = 256 / LANES * gridDim.y;
    for (int head = blockIdx.y * (256 / LANES) + threadIdx.x / LANES; head < heads; head += step) {     // a head's lanes go together
        const bool is_q = head < a.hq, is_v = head >= a.hq + a.hkv;
        const int h = is_q ? head : is_v ? head - a.hq - a.hkv : head - a.hq;
        const uint16_t* x = is_q ? a.q + t * a.qs : is_v ? a.v + t * a.vs : a.k + t * a.ks;
        const v4u mine = *reinterpret_cast<const v4u*>(x + h * D + col);
        float f[8];
        unpack8(mine, f);
        if (!is_v) {
            const bool turned = col < a.rot;
            // the other column of each pair: this lane's own, or a lane rot / 16 away
            const int lane = threadIdx.x & 63, away = a.pairs || !turned ? 0 : col < half ? half / 8 : -(half / 8);
            const uint16_t* w = is_q ? a.q_weight : a.k_weight;
            v4u other;
#pragma unroll
            for (int j = 0; j < 4; ++j) other[j] = __shfl((int)mine[j], lane + away, 64);
            float g[8];
            unpack8(other, g);
            if (w) {
                double sum = 0.0;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)f[j], (double)f[j], sum);
#pragma unroll
                for (int off = 1; off < LANES; off <<= 1) sum += __shfl_xor(sum, off, 64);
                const double rstd = 1.0 / __builtin_sqrt(sum / D + (double)a.eps);
                float u[8], v[8];
                unpack8(*reinterpret_cast<const v4u*>(w + col), u);
                unpack8(*reinterpret_cast<const v4u*>(w + col + 8 * away), v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] = (float)((double)f[j] * rstd) * (u[j] + a.bias);
                    g[j] = (float)((double)g[j] * rstd) * (v[j] + a.bias);
                }
            }
            if (turned) {
                if (a.pairs) {
                    const v4f c = *reinterpret_cast<const v4f*>(cos_s + col / 2), s = *reinterpret_cast<const v4f*>(sin_s + col / 2);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = f[2 * j], q = f[2 * j + 1];
                        f[2 * j] = fmaf(p, c[j], -(q * s[j]));
                        f[2 * j + 1] = fmaf(p, s[j], q * c[j]);
                    }
                } else {
                    const int i = col < half ? col : col - half;
                    const float sign = col < half ? -1.0f : 1.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = fmaf(f[j], cos_s[i + j], sign * (g[j] * sin_s[i + j]));
                }
            }
        }
        if (is_q) {
            *reinterpret_cast<v4u*>(a.q_out + t * a.qos + h * D + col) = pack8(f);
            continue;
        }
        if (!is_v && a.k_out) *reinterpret_cast<v4u*>(a.k_out + t * a.kos + h * D + col) = pack8(f);
        const int64_t row = page < 0 ? -1 : ((page * a.hkv + h) << a.shift) + (at & ((1 << a.shift) - 1));
        keep<FMT, D>(f, is_v ? a.v_pages : a.k_pages, is_v ? a.v_scale : a.k_scale, row, h, col);
    }
}

// Few tokens: a workgroup for each round of heads; many: one for all heads of a
// token, which works its angles out once.  24 / 4 heads of 256, normalised, into
// E4M3 rows with a scale each (us): 1 token 4.2 / 7.4, 64 4.6 / 7.8, 512 9.7 /
// 10.4, 700 11.7 / 12.4, 1024 15.5 / 14.9, 4096 45 / 39 (24.5 as bytes); 32 / 8
// heads of 128 in BF16: 1 token 2.7 / 3.7, 512 5.2 / 5.2, 700 6.9 / 6.6, 4096
// 23.9 / 19.5.
template <int FMT>
hipError_t go_rope(const RopeArgs& a, hipStream_t stream) {
    const int at_once = 256 * 8 / a.d, rounds = (a.hq + 2 * a.hkv + at_once - 1) / at_once;
    const dim3 grid((unsigned)a.t, (unsigned)(a.t <= 512 ? rounds : 1));
    if (a.d == 64) kv_append_rope_kernel<FMT, 64><<<grid, 256, 0, stream>>>(a);
    else if (a.d == 128) kv_append_rope_kernel<FMT, 128><<<grid, 256, 0, stream>>>(a);
    else kv_append_rope_kernel<FMT, 256><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_rope(int kv_fmt, const RopeArgs& a, hipStream_t stream) {
    switch (kv_fmt) {
        case NQ_KV_BF16: return go_rope<NQ_KV_BF16>(a, stream);
        case NQ_KV_E4M3: return go_rope<NQ_KV_E4M3>(a, stream);
        default: return go_rope<NQ_KV_E4M3_TOKEN>(a, stream);
    }
}

}  // namespace nq
