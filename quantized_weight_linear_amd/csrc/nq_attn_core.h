// Attention tiles on the BF16 matrix cores, shared by the prompt and the tree
// kernels.
//
// A wave holds 32 query rows per block (QB blocks) as the columns of its
// products.  For 32 keys at a time it forms S^T = K Q^T, so that lane l has
// the logits of query row l % 32 in its own registers (16 of the 32 keys, the
// other half in lane l ^ 32): the running maximum and sum of the softmax are
// one value per lane, and one exchange between the wave's halves joins them.
// P^T, rounded to BF16 in those same registers, is already the right operand
// of O^T += V^T P^T: the products sum over the keys in whatever order both
// operands give them, so V^T is read in the order that S^T's rows come in.
// V^T comes out of the row-major V tile through the LDS's transposing reads.
//
//   x_j = c <q, k_j> (c = scale log2 e),  p_j = 2^(x_j - m),  l = sum p_j,
//   o = sum p_j v_j / l,  log-sum-exp = (m + log2 l) ln 2
//
// m is a running upper reference, not the exact maximum: it moves only when a
// new logit passes it by more than RESCALE_LOG2 (p then stays below
// 2^RESCALE_LOG2, far from FP32's and BF16's range, and every rounding is
// relative), so the accumulators are rescaled a few times per row and not once
// per tile.  Sums, m and l are FP32.  P is rounded once to BF16 (2^-8
// relative at most, as a BF16 output is); for FP32 outputs SPLITP makes it
// three BF16 terms (2^-22), for three products with V instead of one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nq_device.h"

namespace nq {
namespace attn {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char* lds_ptr;
typedef __attribute__((address_space(3))) const unsigned char* lds_cptr;

constexpr float RESCALE_LOG2 = 8.0f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.44269504088896340736f;
constexpr int BUF_RAW = 0x00027000;      // raw buffer, no format conversion: loads past num_records give zeros

// A tile's rows in LDS: key-major, ROW bytes a key, in 16-byte chunks whose
// place in the row is permuted by the key's low four bits (XOR), so that the
// 16-byte reads of K (one chunk of 8 .. 16 neighbouring keys) and the
// transposing 8-byte reads of V (32 or 64 bytes of 4 or 8 keys) both spread
// over all banks.
template <int D, bool FP8>
struct Tile {
    static constexpr int ROW = D * (FP8 ? 1 : 2);
    static constexpr int CH = ROW / 16;                 // chunks a row: 4 .. 32
    static constexpr int RPI = 64 / CH;                 // rows one 1 KiB load instruction of a wave fills
    static constexpr int LOADS16 = CH / 4;              // load instructions for 16 rows
    // XOR-linear in the key's bits 0..3.
    __device__ static constexpr int sw(int key) {
        const int b0 = key & 1, b1 = (key >> 1) & 1, b2 = (key >> 2) & 1, b3 = (key >> 3) & 1;
        if (!FP8) return CH >= 16 ? (b0 << 2 | b1 << 3 | b2 | b3 << 1) : (b1 << 2 | b2 | b3 << 1);
        return CH >= 16 ? (b0 << 1 | b1 << 2 | b3 << 3 | b2) : CH == 8 ? (b1 << 1 | b3 << 2 | b2) : (b2 | b3 << 1);
    }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int rows, int stride_bytes, int row_bytes) {
    const int n = rows > 0 ? (rows - 1) * stride_bytes + row_bytes : 0;
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, n, BUF_RAW);
}

// 16 rows (keys 16-aligned in the tile) from memory into LDS at dst, no
// registers between; rows past the descriptor's range become zeros.  The wave
// waits with vmcnt before anyone reads them.
template <int D, bool FP8>
struct Stager {
    using T = Tile<D, FP8>;
    int row0, chunk0;                                    // this lane's row and chunk (already permuted) in the first load
    __device__ __forceinline__ explicit Stager(int lane) {
        row0 = lane / T::CH;
        chunk0 = (lane % T::CH) ^ T::sw(row0);
    }
    __device__ __forceinline__ void rows16(__amdgpu_buffer_rsrc_t r, int stride_bytes, lds_ptr dst) const {
#pragma unroll
        for (int i = 0; i < T::LOADS16; ++i) {
            const int off = (row0 + i * T::RPI) * stride_bytes + ((chunk0 ^ T::sw(i * T::RPI)) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) uint32_t*)(dst + i * 1024), 16,
                                                     off, 0, 0, 0);
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ float max2(float a, float b) { return __builtin_fmaxf(a, b); }

// x of this lane and of lane ^ 32, joined.
__device__ __forceinline__ float halves_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ v8bf as_frag(v4u x) { return __builtin_bit_cast(v8bf, x); }

// Eight E4M3 codes -> eight BF16 values, exact.
__device__ __forceinline__ v8bf e4m3x8_to_frag(uint32_t a, uint32_t b) {
    return as_frag(v4u{e4m3x2_to_bf16x2<false>(a, 1.0f), e4m3x2_to_bf16x2<true>(a, 1.0f),
                       e4m3x2_to_bf16x2<false>(b, 1.0f), e4m3x2_to_bf16x2<true>(b, 1.0f)});
}

// Whether a dword of the cache holds an infinity or a NaN (BF16 pair), or a
// NaN (four E4M3 codes): the field's all-ones exponent (E4M3: all-ones code)
// carries into the bit above it.
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    if (FP8) return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// Whether any of 16 staged rows at p holds such a value.
template <int D, bool FP8>
__device__ __forceinline__ bool rows16_not_finite(lds_cptr p, int lane) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < Tile<D, FP8>::LOADS16; ++i) {
        const v4u x = *(__attribute__((address_space(3))) const v4u*)(p + i * 1024 + lane * 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) bad |= not_finite<FP8>(x[w]);
    }
    return __ballot(bad != 0) != 0;
}

// One wave's rows and their running results.
template <int D, int QB, bool FP8, bool SPLITP>
struct Rows {
    using T = Tile<D, FP8>;
    static constexpr int NS = D / 16;                   // steps of 16 columns in K Q^T
    static constexpr int ND = D / 32;                   // blocks of 32 output columns
    static constexpr int TERMS = SPLITP ? 3 : 1;        // BF16 terms of P
    static constexpr int KA = FP8 ? ND : (NS < 8 ? NS : 8);
    static constexpr int VA = FP8 ? ND : (ND < 4 ? ND : 4);

    v8bf q[QB][NS];
    v16f o[QB][ND];
    float m[QB], l[QB];                                 // reference (unscaled logit units), this lane's half of the sum
    float c;                                            // scale log2 e (> 0)
    int ka[KA], va[FP8 ? 1 : 2][VA];                    // byte offsets of this lane's reads in a K and a V tile
    int lane;

    __device__ __forceinline__ void init(int lane_, float c_) {
        lane = lane_;
        c = c_;
        const int n = lane & 31, h = lane >> 5, g = lane >> 4, r = lane & 15;
#pragma unroll
        for (int s = 0; s < KA; ++s) ka[s] = n * T::ROW + (((2 * s + h) ^ T::sw(n)) << 4);
        if constexpr (FP8) {
            const int key = 4 * h + ((r >> 1) & 3) + 8 * (r >> 3);
#pragma unroll
            for (int b = 0; b < VA; ++b) va[0][b] = key * T::ROW + (((2 * b + (g & 1)) ^ T::sw(key)) << 4) + (r & 1) * 8;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = 4 * h + (r >> 2) + 8 * e;
#pragma unroll
                for (int b = 0; b < VA; ++b)
                    va[e][b] = key * T::ROW + (((4 * b + 2 * (g & 1) + ((r & 3) >> 1)) ^ T::sw(key)) << 4) + (r & 1) * 8;
            }
        }
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            m[b] = -INFINITY;
            l[b] = 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][d][i] = 0.f;
        }
    }

    // The query row of this lane in block b (NULL: no such row, zeros).  The
    // columns of step s are those that K's reads give it.
    __device__ __forceinline__ void load_q(int b, const uint16_t* row) {
        const int h = lane >> 5;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int col = FP8 ? 32 * (s >> 1) + 16 * h + 8 * (s & 1) : 16 * s + 8 * h;
            q[b][s] = as_frag(row ? *reinterpret_cast<const v4u*>(row + col) : v4u{0u, 0u, 0u, 0u});
        }
    }

    __device__ __forceinline__ v8bf v_frag(lds_cptr v, int t, int d) const {
        if constexpr (FP8) {
            const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(v + va[0][d] + t * 16 * T::ROW));
            return e4m3x8_to_frag(x[0], x[1]);
        } else {
            const int at = (d >> 2) * 256 + t * 16 * T::ROW;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) v4s*)(v + va[0][d & 3] + at));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) v4s*)(v + va[1][d & 3] + at));
            const v2u a = __builtin_bit_cast(v2u, lo), b = __builtin_bit_cast(v2u, hi);
            return as_frag(v4u{a[0], a[1], b[0], b[1]});
        }
    }

    // S^T of KB blocks of 32 keys at k.
    template <int KB>
    __device__ __forceinline__ void logits(lds_cptr k, v16f (&s)[QB][KB]) const {
#pragma unroll
        for (int b = 0; b < QB; ++b)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][kb][i] = 0.f;
        if constexpr (FP8) {
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const v4u x = *(__attribute__((address_space(3))) const v4u*)(k + ka[d] + kb * 32 * T::ROW);
                    const v8bf f0 = e4m3x8_to_frag(x[0], x[1]), f1 = e4m3x8_to_frag(x[2], x[3]);
#pragma unroll
                    for (int b = 0; b < QB; ++b) {
                        s[b][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f0, q[b][2 * d], s[b][kb], 0, 0, 0);
                        s[b][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f1, q[b][2 * d + 1], s[b][kb], 0, 0, 0);
                    }
                }
        } else {
#pragma unroll
            for (int st = 0; st < NS; ++st)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const v8bf f = as_frag(*(__attribute__((address_space(3))) const v4u*)(
                        k + ka[st & 7] + (st >> 3) * 256 + kb * 32 * T::ROW));
#pragma unroll
                    for (int b = 0; b < QB; ++b)
                        s[b][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[b][st], s[b][kb], 0, 0, 0);
                }
        }
    }

    // Logits of keys that the row does not see become -infinity.  seen: bit j
    // = key j of these KB blocks.
    template <int KB>
    __device__ __forceinline__ void hide(v16f (&s)[KB], uint64_t seen) const {
        const uint64_t mine = seen >> (4 * (lane >> 5));
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const uint32_t w = (uint32_t)(mine >> (32 * kb));
#pragma unroll
            for (int i = 0; i < 16; ++i) s[kb][i] = (w >> (8 * (i >> 2) + (i & 3))) & 1u ? s[kb][i] : -INFINITY;
        }
    }

    // S^T -> P^T (in place), with m, l and o brought along.
    template <int KB>
    __device__ __forceinline__ void softmax(int b, v16f (&s)[KB]) {
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max2(top, s[kb][i]);
        top = halves_max(top);
        if (__ballot((top - m[b]) * c > RESCALE_LOG2 || (m[b] == -INFINITY && top > -INFINITY)) != 0) {
            const float to = max2(m[b], top);
            const float a = m[b] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[b] - to) * c);
            m[b] = to;
            l[b] *= a;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][d][i] *= a;
        }
        const float mc = m[b] == -INFINITY ? 0.f : m[b] * c;
        float sum = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], c, -mc));
                sum += s[kb][i];
            }
        l[b] += sum;
    }

    // The operand of 16 keys: registers i0 .. i0 + 7 of S^T, as BF16.  SPLITP:
    // as three BF16 terms, each but the last rounded from (1 - 2^-8) of what
    // is left, so that it stays below it and all terms are positive: an
    // infinite value times them gives infinity, not infinity - infinity.
    __device__ __forceinline__ static void p_frag(const v16f& p, int i0, v8bf (&out)[TERMS]) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = p[i0 + j];
#pragma unroll
        for (int e = 0; e < TERMS; ++e) {
            const float f = e + 1 < TERMS ? 0.99609375f : 1.0f;
            v4u a;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                a[w] = f32x2_to_bf16x2(x[2 * w] * f, x[2 * w + 1] * f);
                if (e + 1 < TERMS) {
                    x[2 * w] -= __uint_as_float(a[w] << 16);
                    x[2 * w + 1] -= __uint_as_float(a[w] & 0xFFFF0000u);
                }
            }
            out[e] = as_frag(a);
        }
    }

    // O^T += V^T P^T over KB blocks of 32 keys at v.
    template <int KB>
    __device__ __forceinline__ void values(lds_cptr v, const v16f (&p)[QB][KB]) {
#pragma unroll
        for (int t = 0; t < 2 * KB; ++t) {
            v8bf pf[QB][TERMS];
#pragma unroll
            for (int b = 0; b < QB; ++b) p_frag(p[b][t >> 1], 8 * (t & 1), pf[b]);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const v8bf f = v_frag(v, t, d);
#pragma unroll
                for (int e = 0; e < TERMS; ++e)
#pragma unroll
                    for (int b = 0; b < QB; ++b)
                        o[b][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, pf[b][e], o[b][d], 0, 0, 0);
            }
        }
    }

    // The same where some rows must not see keys whose values are not finite:
    // a product over 16 keys would give 0 x infinity = NaN, so one key at a
    // time is summed and kept by the rows that see it.
    template <int KB>
    __device__ void values_one_by_one(lds_cptr v, const v16f (&p)[QB][KB], const uint64_t (&seen)[QB]) {
        const int h = lane >> 5;
#pragma unroll
        for (int t = 0; t < 2 * KB; ++t) {
            v8bf pf[QB][TERMS];
#pragma unroll
            for (int b = 0; b < QB; ++b) p_frag(p[b][t >> 1], 8 * (t & 1), pf[b]);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const v4u f = __builtin_bit_cast(v4u, v_frag(v, t, d));
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {           // key 16 t + k sits in half (k >> 2) & 1, element 4 (k >> 3) + (k & 3)
                    const int e = 4 * (k >> 3) + (k & 3);
                    const uint32_t keep = ((k >> 2) & 1) == h ? (e & 1 ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
                    v4u a;
#pragma unroll
                    for (int w = 0; w < 4; ++w) a[w] = w == (e >> 1) ? f[w] & keep : 0u;
#pragma unroll
                    for (int b = 0; b < QB; ++b) {
                        v16f next = o[b][d];
#pragma unroll
                        for (int term = 0; term < TERMS; ++term) {
                            v4u x = __builtin_bit_cast(v4u, pf[b][term]);
#pragma unroll
                            for (int w = 0; w < 4; ++w) x[w] = w == (e >> 1) ? x[w] & keep : 0u;
                            next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(a), as_frag(x), next, 0, 0, 0);
                        }
                        const bool sees = (seen[b] >> (16 * t + k)) & 1u;
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[b][d][i] = sees ? next[i] : o[b][d][i];
                    }
                }
            }
        }
    }

    // This lane's output column block: o[b][d][4 e + j] is column 32 d + 8 e + 4 h + j.
    __device__ __forceinline__ int column(int d, int e) const { return 32 * d + 8 * e + 4 * (lane >> 5); }
};

// Four outputs at out[0..3], FP32 or BF16.
template <bool BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, float a, float b, float c, float d) {
    if constexpr (BF16) {
        *reinterpret_cast<v2u*>(reinterpret_cast<uint16_t*>(out) + at) = v2u{f32x2_to_bf16x2(a, b), f32x2_to_bf16x2(c, d)};
    } else {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + at) = v4f{a, b, c, d};
    }
}

// 1 / sum, or 0 for a row that saw nothing (its outputs are zeros); a NaN sum stays NaN.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }
__device__ __forceinline__ float log_sum_exp(float mc, float l) {
    return l == 0.f ? -INFINITY : (mc + __builtin_log2f(l)) * LN2;
}

}  // namespace attn
}  // namespace nq
