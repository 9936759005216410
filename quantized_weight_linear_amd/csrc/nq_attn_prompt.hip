// Causal attention over packed prompts (nq_attn_prompt).
//
// One workgroup per (128 or 256 query tokens of a sequence, query head): the
// keys and values that tile sees are read from LDS, where the workgroup's
// waves share them; grouped query heads read the same K and V through L2.
// Bound by the matrix cores: 4 D flops per (row, visible key).
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_attn_rows.h"
#include "nq_launch.h"

namespace nq {
namespace attn {

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;             // elements between tokens
    const int32_t *cu_q, *cu_k;
    int seqs;
    int64_t tq, tk;
    int hq, hkv;
    float c;
    void* o;
    float* lse;
};

// A packed offset, kept inside [0, total] and in order whatever the array holds.
__device__ __forceinline__ int64_t offset_of(const int32_t* cu, int i, int64_t total) {
    const int64_t x = uniform(cu, i);
    return x < 0 ? 0 : x > total ? total : x;
}

struct PackedRows {                 // K or V rows of one sequence and KV head
    const uint16_t *k, *v;
    int k_stride, v_stride;         // bytes
    int n, row_bytes;
    __device__ __forceinline__ v4i k_rows(int key) const {
        const int rows = n - key < 16 ? n - key : 16;
        return rows_rsrc((const char*)k + (rows > 0 ? (int64_t)key * k_stride : 0), rows, k_stride, row_bytes);
    }
    __device__ __forceinline__ v4i v_rows(int key) const {
        const int rows = n - key < 16 ? n - key : 16;
        return rows_rsrc((const char*)v + (rows > 0 ? (int64_t)key * v_stride : 0), rows, v_stride, row_bytes);
    }
};

template <int QB>
struct CausalSees {
    int clean;                      // every row of the workgroup sees the keys below it
    int none;                       // no row of the wave sees keys from it on
    int limit[QB];                  // this lane's rows see the keys below it
    __device__ __forceinline__ int all_before() const { return clean; }
    __device__ __forceinline__ int none_from() const { return none; }
    __device__ __forceinline__ uint64_t seen(int b, int key) const { return bits_below(limit[b] - key); }
};

template <int D, int QB, int NW, int RING, int PER_SIMD, bool BF16OUT>
__global__ __launch_bounds__(NW * 64, PER_SIMD) void attn_prompt_kernel(PromptArgs a) {
    constexpr int BM = NW * QB * 32;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.hq;
    int tile = blockIdx.x / a.hq;
    // which sequence, which tile of it (the last one, with the most keys, first)
    int64_t q0 = 0, q1 = 0;
    int b = 0, tiles = 0;
    for (; b < a.seqs; ++b) {
        q0 = offset_of(a.cu_q, b, a.tq);
        q1 = offset_of(a.cu_q, b + 1, a.tq);
        tiles = q1 > q0 ? (int)((q1 - q0 + BM - 1) / BM) : 0;
        if (tile < tiles) break;
        tile -= tiles;
    }
    if (b == a.seqs) return;
    tile = tiles - 1 - tile;
    const int64_t k0 = offset_of(a.cu_k, b, a.tk), k1 = offset_of(a.cu_k, b + 1, a.tk);
    const int nq = (int)(q1 - q0), nk = k1 > k0 ? (int)(k1 - k0) : 0, ahead = nk - nq;
    const int first = tile * BM, last = first + BM < nq ? first + BM : nq;      // rows [first, last)
    const int kvh = head / (a.hq / a.hkv);

    Rows<D, QB, false, !BF16OUT> R;
    R.init(lane, a.c);
    CausalSees<QB> sees;
    sees.clean = first + 1 + ahead;
    sees.none = first + (wave + 1) * QB * 32 + ahead;
    int row[QB];
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        row[i] = first + (wave * QB + i) * 32 + (lane & 31);
        sees.limit[i] = row[i] + 1 + ahead;
    }
    PackedRows src;
    src.k = a.k + k0 * a.ks + kvh * D;
    src.v = a.v + k0 * a.vs + kvh * D;
    src.k_stride = (int)(a.ks * 2);
    src.v_stride = (int)(a.vs * 2);
    src.n = nk;
    src.row_bytes = D * 2;
    const int end = last + ahead;                       // keys that the tile's last row sees
    auto queries = [&] {
#pragma unroll
        for (int i = 0; i < QB; ++i) R.load_q(i, row[i] < nq ? a.q + (q0 + row[i]) * a.qs + head * D : nullptr);
    };
    attend_rows<RING, NW>(R, (lds_ptr)smem, 0, end, src, sees, queries, wave, lane);
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const float l = halves_sum(R.l[i]), inv = inverse_sum(l);
        if (row[i] < nq) {
            const int64_t at = ((q0 + row[i]) * a.hq + head) * D;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    store4<BF16OUT>(a.o, at + R.column(d, e), R.o[i][d][4 * e] * inv, R.o[i][d][4 * e + 1] * inv,
                                    R.o[i][d][4 * e + 2] * inv, R.o[i][d][4 * e + 3] * inv);
            if (a.lse && lane < 32) a.lse[(q0 + row[i]) * a.hq + head] = log_sum_exp(l == 0.f ? 0.f : R.m[i] * a.c, l);
        }
    }
}

template <int D, int QB, int NW, int RING, int PER_SIMD, bool BF16OUT>
hipError_t go(const PromptArgs& a, hipStream_t stream) {
    constexpr int BM = NW * QB * 32, LDS = RowsLds<D, false, NW, RING>::BYTES;
    auto kernel = attn_prompt_kernel<D, QB, NW, RING, PER_SIMD, BF16OUT>;
    static LdsLimit limit;
    if (hipError_t e = limit.raise((const void*)kernel, LDS); e != hipSuccess) return e;
    // every sequence may end in a part of a tile
    const int64_t tiles = a.tq / BM + (a.seqs < a.tq ? a.seqs : a.tq);
    kernel<<<(unsigned)(tiles * a.hq), NW * 64, LDS, stream>>>(a);
    return hipGetLastError();
}

}  // namespace attn

hipError_t launch_attn_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int64_t seqs, int64_t tq,
                              int64_t tk, int64_t hq, int64_t hkv, int64_t d, float scale, bool bf16_out, void* o,
                              float* lse, hipStream_t stream) {
    using namespace attn;
    const PromptArgs a{q, k, v, q_stride, k_stride, v_stride, cu_q, cu_k, (int)seqs, tq, tk, (int)hq, (int)hkv,
                       scale * LOG2E, o, lse};
    switch (d) {
        case 64: return bf16_out ? go<64, 1, 4, 2, 4, true>(a, stream) : go<64, 1, 4, 2, 4, false>(a, stream);
        case 128: return bf16_out ? go<128, 1, 4, 2, 3, true>(a, stream) : go<128, 1, 4, 2, 3, false>(a, stream);
        default: return bf16_out ? go<256, 1, 4, 2, 2, true>(a, stream) : go<256, 1, 4, 2, 2, false>(a, stream);
    }
}

}  // namespace nq
