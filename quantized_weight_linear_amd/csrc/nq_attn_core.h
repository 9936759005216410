// Attention tiles on the BF16 matrix cores, shared by the prompt and the tree
// kernels.
//
// A wave holds 32 query rows as the columns of its products.  For 32 keys at a
// time it forms S^T = K Q^T, so that lane l has the logits of query row l % 32
// in its own registers (16 of the 32 keys, the other half in lane l ^ 32): the
// reference and sum of the softmax are one value per lane, and one exchange
// between the wave's halves joins the maxima.
// P^T, rounded to BF16 in those same registers, is already the right operand
// of O^T += V^T P^T: the products sum over the keys in whatever order both
// operands give them, so V^T is read in the order that S^T's rows come in.
// V^T comes out of the row-major V tile through the LDS's transposing reads.
//
//   x_j = c <q, k_j> (c = scale log2 e),  p_j = 2^(x_j - r),  l = sum p_j,
//   o = sum p_j v_j / l,  log-sum-exp = (r + log2 l) ln 2
//
// r = m + RESCALE_LOG2, where m is a running reference, not the exact maximum:
// it moves only when a logit passes it by more than RESCALE_LOG2, so the
// accumulators are rescaled a few times per row and not once per tile.  No
// weight is above 1 (sums of p v stay finite where those of a softmax under the
// exact maximum do), the largest is at least 2^-RESCALE_LOG2, and every
// rounding is relative (of values below 2^-118 in size, products may lose bits
// to FP32's smallest numbers).  Sums, m and l are FP32.
//
// P's bits: one BF16 term for BF16 outputs, whose own rounding is as coarse
// (2^-9 relative at most, each); l sums the weights as they were before it.
// Against 64 bits the outputs of 16384 tokens of 24 heads of 256 are then
// 2.0e-3 off (Frobenius), 1.5e-3 with the output's rounding alone.  For FP32
// outputs SPLITP makes P three BF16 terms (2^-22: 2e-7 off), for three products
// with V instead of one: 8192 tokens of 32 heads of 128 take 927 us so and 520
// with one term.
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
constexpr float FAR_LOG2 = 536870912.0f; // references beyond it (2^29): see factor()
constexpr float FLT_TOP = 3.40282347e38f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.44269504088896340736f;
constexpr int BUF_RAW = 0x00027000;      // raw buffer, no format conversion

// Arrays that the kernel reading them does not write (an earlier one may have:
// the scalar cache is empty when a kernel starts), read at uniform places: by
// scalar loads, which no wait for vector loads in flight holds up.
typedef __attribute__((address_space(4))) const int32_t* uniform_ints;
__device__ __forceinline__ int uniform(const int32_t* p, int64_t i) { return ((uniform_ints)(uintptr_t)p)[i]; }

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

// A raw buffer of `rows` rows from base on: loads past it give zeros.
__device__ __forceinline__ v4i rows_rsrc(const void* base, int rows, int stride_bytes, int row_bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    return v4i{(int)(uint32_t)at, (int)(uint32_t)(at >> 32) & 0xFFFF, rows > 0 ? (rows - 1) * stride_bytes + row_bytes : 0, BUF_RAW};
}

// 16 bytes a lane from the buffer at `off` to LDS at dst + 16 lane.  Written
// as one instruction, not as the builtin: the compiler would wait for every
// such load in flight before any LDS read that it cannot tell from their
// targets.  Whoever reads the rows waits with wait_vm.  (No register is
// written; the wait state between M0 and its use is part of the block.)
__device__ __forceinline__ void load_to_lds(v4i r, int off, lds_ptr dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"((uint32_t)(uintptr_t)dst), "v"(off), "s"(r)
                 : "memory", "m0");
}

// 16 rows (keys 16-aligned in the tile) from memory into LDS at dst, no
// registers between; rows past the descriptor's range become zeros.  The wave
// waits with vmcnt before anyone reads them.
template <int D, bool FP8>
struct Stager {
    using T = Tile<D, FP8>;
    int stride, first, chunk0;                           // bytes between rows; this lane's row, and its place in it, in the first load
    __device__ __forceinline__ Stager(int lane, int stride_bytes) {
        stride = stride_bytes;
        first = lane / T::CH * stride;
        chunk0 = ((lane % T::CH) ^ T::sw(lane / T::CH)) << 4;
    }
    __device__ __forceinline__ void rows16(v4i r, lds_ptr dst) const {
        int at = chunk0;
        asm volatile("" : "+v"(at));                     // offsets are formed as they are needed, not kept in registers
#pragma unroll
        for (int i = 0; i < T::LOADS16; ++i)
            load_to_lds(r, (at ^ (T::sw(i * T::RPI) << 4)) + first + i * T::RPI * stride, dst + i * 1024);
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

// The staged rows at p that hold such a value, as bits: N pieces of 1 KiB (RPI
// rows each) that this wave has loaded.
template <int D, bool FP8, int N>
__device__ __forceinline__ uint32_t rows_not_finite(lds_cptr p, int lane) {
    using T = Tile<D, FP8>;
    uint32_t rows = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const v4u x = *(__attribute__((address_space(3))) const v4u*)(p + i * 1024 + lane * 16);
        uint32_t bad = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) bad |= not_finite<FP8>(x[w]);
        const uint64_t lanes = __ballot(bad != 0);
        if (lanes) {
            for (int r = 0; r < T::RPI; ++r)
                if (lanes >> (r * T::CH) & ((1ull << T::CH) - 1)) rows |= 1u << (i * T::RPI + r);
        }
    }
    return rows;
}

// ... and zeros in the place of such values.
template <int D, bool FP8, int N>
__device__ __forceinline__ void rows_made_finite(lds_ptr p, int lane) {
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        auto* at = (__attribute__((address_space(3))) v4u*)(p + i * 1024 + lane * 16);
        v4u x = *at;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t top = not_finite<FP8>(x[w]);                      // the bit above each such field
            x[w] &= FP8 ? ~((top >> 7) * 0xFFu) : ~((top >> 15) * 0xFFFFu);
        }
        *at = x;
    }
}

// One wave's 32 rows and their running results; a lane has one row (lane % 32).
template <int D, bool FP8, bool SPLITP>
struct Rows {
    using T = Tile<D, FP8>;
    static constexpr int NS = D / 16;                   // steps of 16 columns in K Q^T
    static constexpr int ND = D / 32;                   // blocks of 32 output columns
    static constexpr int TERMS = SPLITP ? 3 : 1;        // BF16 terms of P

    v8bf q[NS];
    v16f o[ND];
    float m, l;                                         // reference m (unscaled logit units), this lane's half of the sum
    bool far;                                           // some row's |m c| is beyond FAR_LOG2 (the same in all lanes)
    float c;                                            // scale log2 e, made positive
    uint32_t q_and, q_xor;                              // what that makes of the queries' bits
    int ka, va;                                         // byte offsets of this lane's first read in a K and a V tile
    int lane;

    __device__ __forceinline__ void init(int lane_, float c_) {
        lane = lane_;
        // A negative scale becomes the queries' sign, and with a scale of zero
        // they are zeros, so that larger logits are larger ones of c <q, k>
        // and -infinity (a hidden key) stays what it is.
        c = c_ == 0.f ? 1.0f : __builtin_fabsf(c_);
        q_and = c_ == 0.f ? 0u : ~0u;
        q_xor = c_ < 0.f ? 0x80008000u : 0u;
        const int n = lane & 31, h = lane >> 5, g = lane >> 4, r = lane & 15;
        ka = n * T::ROW + ((h ^ T::sw(n)) << 4);
        if constexpr (FP8) {
            const int key = 4 * h + ((r >> 1) & 3) + 8 * (r >> 3);
            va = key * T::ROW + (((g & 1) ^ T::sw(key)) << 4) + (r & 1) * 8;
        } else {
            const int key = 4 * h + (r >> 2);
            va = key * T::ROW + (((2 * (g & 1) + ((r & 3) >> 1)) ^ T::sw(key)) << 4) + (r & 1) * 8;
        }
        m = -INFINITY;
        l = 0.f;
        far = false;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    }

    // The query row of this lane (NULL: no such row, zeros).  The columns of
    // step s are those that K's reads give it.
    __device__ __forceinline__ void load_q(const uint16_t* row) {
        const int h = lane >> 5;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int col = FP8 ? 32 * (s >> 1) + 16 * h + 8 * (s & 1) : 16 * s + 8 * h;
            q[s] = as_frag(row ? (*reinterpret_cast<const v4u*>(row + col) & q_and) ^ q_xor : v4u{0u, 0u, 0u, 0u});
        }
    }
    // Waits for the queries here, once: a wait at their first use would stand
    // in the loop over the keys and hold up its loads in every turn.
    __device__ __forceinline__ void queries_ready() {
#pragma unroll
        for (int s = 0; s < NS; ++s) asm volatile("" : "+v"(q[s]));
    }

    // The reads' places: a chunk number is XORed into the row's permuted place
    // (low four chunk bits), further chunks and rows are added.  LEAN: formed
    // anew each time (one instruction a read) instead of being kept in registers.
    static constexpr bool LEAN = D == 256;
    __device__ __forceinline__ int fresh(int at) const {
        if (LEAN) asm volatile("" : "+v"(at));
        return at;
    }
    __device__ __forceinline__ static int chunk(int at, int c) { return (at ^ ((c & 15) << 4)) + (c >> 4) * 256; }

    // The raw operand of V^T: 16 keys from 16 t on, columns 32 d ..
    __device__ __forceinline__ v4u read_v(lds_cptr v, int at, int t, int d) const {
        if constexpr (FP8) {
            const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(v + chunk(at, 2 * d) + t * 16 * T::ROW));
            return v4u{(uint32_t)x[0], (uint32_t)x[1], 0u, 0u};
        } else {
            const lds_cptr rows = v + t * 16 * T::ROW;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(rows + chunk(at, 4 * d)));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) v4s*)(rows + chunk(at, (4 * d) ^ T::sw(8)) + 8 * T::ROW));
            const v2u a = __builtin_bit_cast(v2u, lo), b = __builtin_bit_cast(v2u, hi);
            return v4u{a[0], a[1], b[0], b[1]};
        }
    }
    __device__ __forceinline__ static v8bf v_frag(v4u x) {
        if constexpr (FP8) return e4m3x8_to_frag(x[0], x[1]);
        else return as_frag(x);
    }

    // Keeps LDS reads and products in the order written (the vector and scalar
    // unit's other work may cross).  Left to itself the compiler reads each
    // operand right before its product, and every product waits for LDS; so
    // the operands are read AHEAD products before their use.  AHEAD is what the
    // registers bear beside the rest.
    __device__ __forceinline__ static void in_order() { __builtin_amdgcn_sched_barrier(0x406); }

    // S^T of the 32 keys at k.
    __device__ __forceinline__ void logits(lds_cptr k, v16f& s) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
        const int at = fresh(ka);
        constexpr int READS = FP8 ? ND : NS, AHEAD = FP8 ? 3 : 4;          // 16 bytes a read: 16 codes or 8 values
        v4u x[AHEAD];
        auto read = [&](int i) { return *(__attribute__((address_space(3))) const v4u*)(k + chunk(at, 2 * i)); };
#pragma unroll
        for (int i = 0; i < AHEAD && i < READS; ++i) x[i] = read(i);
        in_order();
#pragma unroll
        for (int i = 0; i < READS; ++i) {
            const v4u w = x[i % AHEAD];
            if constexpr (FP8) {
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_frag(w[0], w[1]), q[2 * i], s, 0, 0, 0);
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_frag(w[2], w[3]), q[2 * i + 1], s, 0, 0, 0);
            } else {
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(w), q[i], s, 0, 0, 0);
            }
            if (i + AHEAD < READS) x[i % AHEAD] = read(i + AHEAD);
            in_order();
        }
    }

    // Logits of keys that the row does not see become -infinity.  seen: bit j
    // = key j of these 32.
    __device__ __forceinline__ void hide(v16f& s, uint64_t seen) const {
        const uint32_t w = (uint32_t)(seen >> (4 * (lane >> 5)));
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = (w >> (8 * (i >> 2) + (i & 3))) & 1u ? s[i] : -INFINITY;
    }

    // r, in log2 units, kept finite (-infinity is the reference of a row that
    // has seen nothing).
    __device__ __forceinline__ float reference() const {
        return __builtin_fminf(max2(m * c + RESCALE_LOG2, -FLT_TOP), FLT_TOP);
    }
    // The logits' factor in the weights.  fma(s, c, -r) sees s c exactly and r
    // rounded: one factor for all weights of the row, of 2^32 at most up to |m c|
    // = 2^29 and beyond FP32's range soon after.  There the logits' own steps are
    // 32 and more, so that all weights but those of the largest logit vanish
    // (2^-32), and they still do under the factor that brings |m| to 2^29.
    __device__ __forceinline__ bool is_far() const { return m > -INFINITY && __builtin_fabsf(m) * c > FAR_LOG2; }
    __device__ __forceinline__ float factor() const {
        float f = c;
        if (far && is_far()) f = FAR_LOG2 / __builtin_fabsf(m);
        return f;
    }

    // P^T of the 32 keys at k, with m, l and o brought along.
    template <bool HIDE>
    __device__ __forceinline__ void weights(lds_cptr k, uint64_t seen, v16f& s) {
        logits(k, s);
        if (HIDE) hide(s, seen);
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = max2(top, s[i]);
        top = halves_max(top);
        if (__ballot((top - m) * c > RESCALE_LOG2) != 0) {
            const float to = max2(m, top);
            const float a = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - to) * c);
            m = to;
            far = __ballot(is_far()) != 0;
            l *= a;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= a;
        }
        const float f = factor(), r = m == -INFINITY ? 0.f : m * f + RESCALE_LOG2;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], f, -r));
            sum += s[i];
        }
        l += sum;
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

    // O^T += V^T P^T over the 32 keys at v.
    __device__ __forceinline__ void values(lds_cptr v, const v16f& p) {
        const int at = fresh(va);
        constexpr int AHEAD = FP8 ? 4 : 2;
        v4u x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = read_v(v, at, i / ND, i % ND);
        in_order();
        v8bf pf[TERMS];
#pragma unroll
        for (int i = 0; i < 2 * ND; ++i) {
            if (i % ND == 0) p_frag(p, 8 * (i / ND), pf);
            const v8bf f = v_frag(x[i % AHEAD]);
#pragma unroll
            for (int e = 0; e < TERMS; ++e) o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, pf[e], o[i % ND], 0, 0, 0);
            if (i + AHEAD < 2 * ND) x[i % AHEAD] = read_v(v, at, (i + AHEAD) / ND, (i + AHEAD) % ND);
            in_order();
        }
    }

    // Values that are not finite, of keys that some rows do not see: a product
    // over 16 keys would give 0 x infinity = NaN there.  They are added to the
    // rows that see them (a positive weight makes the sum infinite or NaN by
    // them whatever it is; one of 0, under a logit far below the others or of
    // -infinity, is not told apart), and then count as zeros in the products.
    // bad: the keys of the 32 at v that hold such values; seen: as in hide().
    __device__ __forceinline__ void add_not_finite(lds_cptr v, uint32_t bad, uint64_t seen) {
        while (bad) {
            const int key = __builtin_ctz(bad);
            const bool sees = (seen >> key) & 1u;
            bad &= bad - 1;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
                    read4(v, key, column(d, e), x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = __builtin_isfinite(x[j]) ? 0.f : x[j];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[d][4 * e + j] += sees ? x[j] : 0.f;
                }
        }
    }
    // Four neighbouring values of a row in a staged tile.
    __device__ __forceinline__ static void read4(lds_cptr tile, int key, int col, float (&x)[4]) {
        const int byte = col * (FP8 ? 1 : 2);
        const lds_cptr at = tile + key * T::ROW + (((byte >> 4) ^ T::sw(key)) << 4) + (byte & 15);
        if constexpr (FP8) {
            e4m3x4_to_f32(*(__attribute__((address_space(3))) const uint32_t*)at, x);
        } else {
            const v2u w = *(__attribute__((address_space(3))) const v2u*)at;
            x[0] = bf16_bits_to_f32(w[0] & 0xFFFFu), x[1] = bf16_bits_to_f32(w[0] >> 16);
            x[2] = bf16_bits_to_f32(w[1] & 0xFFFFu), x[3] = bf16_bits_to_f32(w[1] >> 16);
        }
    }

    // A row without weights (sum 0): no outputs either, whatever its values
    // were (0 x infinity, or a value added by add_not_finite).
    __device__ __forceinline__ void drop_if_empty(float sum) {
        if (sum != 0.f) return;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    }

    // o[d][4 e + j] is this lane's output column 32 d + 8 e + 4 h + j.
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
__device__ __forceinline__ float log_sum_exp(float r, float l) {
    return l == 0.f ? -INFINITY : (r + __builtin_log2f(l)) * LN2;
}

}  // namespace attn
}  // namespace nq
