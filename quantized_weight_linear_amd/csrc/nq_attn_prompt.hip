// Causal attention over packed prompts (nq_attn_prompt).
//
// One workgroup per (128 or 32 query tokens of a sequence, query head): the
// keys and values that tile sees are read from LDS, where the workgroup's
// waves share them; grouped query heads read the same K and V through L2.
// Bound by the matrix cores: 4 D flops per (row, visible key).  Neighbouring
// workgroups are heads of one tile, so that one round of them reads the same
// keys; 1792 tokens on top of 8192 keys, 24 heads of 256, take 0.45 ms (336
// workgroups for 512 places: 880 TFLOP/s).
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_attn_keys.h"
#include "nq_attn_launch.h"

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

// A packed offset, kept inside [0, total] whatever the array holds.
__device__ __forceinline__ int cut_offset(int x, int64_t total) { return x < 0 ? 0 : x > (int)total ? (int)total : x; }

struct PackedRows {                 // K or V rows of one sequence and KV head
    static constexpr bool SCALED = false;
    const uint16_t *k, *v;
    int k_stride, v_stride;         // bytes
    int n, row_bytes;
    struct At {
        int key, rows;
    };
    __device__ __forceinline__ At find(int key) const { return At{key, n - key < 16 ? n - key : 16}; }
    __device__ __forceinline__ v4i rows(const uint16_t* base, int stride, const At& at) const {
        return rows_rsrc((const char*)base + (at.rows > 0 ? (int64_t)at.key * stride : 0), at.rows, stride, row_bytes);
    }
    __device__ __forceinline__ v4i k_rows(const At& at) const { return rows(k, k_stride, at); }
    __device__ __forceinline__ v4i v_rows(const At& at) const { return rows(v, v_stride, at); }
};

struct CausalSees {
    int clean;                      // every row of the workgroup sees the keys below it
    int none;                       // no row of the wave sees keys from it on
    int limit;                      // this lane's row sees the keys below it
    __device__ __forceinline__ int all_before() const { return clean; }
    __device__ __forceinline__ int none_from() const { return none; }
    __device__ __forceinline__ uint64_t seen(int key) const { return bits_below(limit - key); }
};

// The tile of bm query rows that workgroup `index` of a head has: the
// sequences in order, in each its last tile, which sees most keys, first.  A
// wave looks through 256 sequences at a time (1000 of 1 .. 33 tokens, 24 heads
// of 256: one after another 5.4 ms, 64 at a time 0.86, so 0.75).
struct QueryTile {
    int64_t q0, k0;                 // the sequence's first query and key
    int nq, nk, first, last;        // its lengths; rows [first, last) of it
    bool real;
    __device__ __forceinline__ static uint32_t tiles_of(int q0, int q1, int bm) { return q1 > q0 ? ((uint32_t)(q1 - q0) + bm - 1) / bm : 0u; }
    __device__ __forceinline__ QueryTile(const PromptArgs& a, uint32_t index, int bm) {
        constexpr int PER = 4;      // sequences a lane
        int b = 0;
        real = a.seqs == 1;
        if (!real) {
            const int lane = threadIdx.x & 63;
            for (int b0 = 0; b0 < a.seqs && !real; b0 += 64 * PER) {
                int edge[PER + 1];
#pragma unroll
                for (int e = 0; e <= PER; ++e) {
                    const int at = b0 + lane * PER + e;
                    edge[e] = a.cu_q[at < a.seqs ? at : a.seqs];
                }
                uint32_t n[PER], mine = 0;              // (a tile count is below 2^26; in 64 bits for offsets out of order)
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    n[e] = tiles_of(cut_offset(edge[e], a.tq), cut_offset(edge[e + 1], a.tq), bm);
                    mine += n[e];
                }
                uint64_t upto = mine;
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    const uint64_t y = __shfl_up(upto, off, 64);
                    if (lane >= off) upto += y;
                }
                const uint64_t past = __ballot(upto > index);
                real = past != 0;
                if (!real) {
                    index -= __builtin_amdgcn_readlane((uint32_t)upto, 63);
                    continue;
                }
                const int which = __builtin_ctzll(past);
                index -= __builtin_amdgcn_readlane((uint32_t)upto - mine, which);
                b = b0 + which * PER;
#pragma unroll
                for (int e = 0; e + 1 < PER; ++e) {     // past the lane's first sequences
                    const uint32_t here = __builtin_amdgcn_readlane(n[e], which);
                    if (b != b0 + which * PER + e || index < here) continue;
                    index -= here;
                    ++b;
                }
            }
            if (!real) return;
        }
        q0 = cut_offset(uniform(a.cu_q, b), a.tq);
        const int64_t q1 = cut_offset(uniform(a.cu_q, b + 1), a.tq);
        const uint32_t tiles = tiles_of((int)q0, (int)q1, bm);
        real = index < tiles;
        if (!real) return;
        k0 = cut_offset(uniform(a.cu_k, b), a.tk);
        const int64_t k1 = cut_offset(uniform(a.cu_k, b + 1), a.tk);
        nq = (int)(q1 - q0);
        nk = k1 > k0 ? (int)(k1 - k0) : 0;
        first = (int)(tiles - 1 - index) * bm;
        last = first + bm < nq ? first + bm : nq;
    }
};

template <int D>
__device__ __forceinline__ PackedRows packed_rows(const PromptArgs& a, const QueryTile& t, int kvh, int keys) {
    PackedRows src;
    src.k = a.k + t.k0 * a.ks + kvh * D;
    src.v = a.v + t.k0 * a.vs + kvh * D;
    src.k_stride = (int)(a.ks * 2);
    src.v_stride = (int)(a.vs * 2);
    src.n = keys;
    src.row_bytes = D * 2;
    return src;
}

// Few tiles: 32 rows a workgroup, whose four waves take different keys (167
// tokens of 24 heads of 256: 12.6 us, latency).
template <int D, bool BF16OUT>
__global__ __launch_bounds__(256) void attn_prompt_keys_kernel(PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.hq;
    const QueryTile t(a, blockIdx.x / a.hq, 32);
    if (!t.real) return;
    const int ahead = t.nk - t.nq, row = t.first + (lane & 31);
    Rows<D, false, !BF16OUT> R;
    R.init(lane, a.c);
    CausalSees sees;
    sees.clean = t.first + 1 + ahead;
    sees.none = t.last + ahead;
    sees.limit = row + 1 + ahead;
    const int keys = t.last + ahead > 0 ? t.last + ahead : 0;
    const PackedRows src = packed_rows<D>(a, t, head / (a.hq / a.hkv), keys);
    auto queries = [&] { R.load_q(row < t.nq ? a.q + (t.q0 + row) * a.qs + head * D : nullptr); };
    auto emit = [&](int i, int col, const v4f& x, float ref, float l) {
        const int64_t out = (t.q0 + t.first + i) * a.hq + head;
        const float f = inverse_sum(l);
        store4<BF16OUT>(a.o, out * D + col, x[0] * f, x[1] * f, x[2] * f, x[3] * f);
        if (col == 0 && a.lse) a.lse[out] = log_sum_exp(ref, l);
    };
    attend_keys(R, smem, 0, keys, t.last - t.first, src, sees, queries, emit, wave, lane);
}

// Many tiles: 128 rows a workgroup (16384 tokens of 24 heads of 256: 1120
// to 1140 TFLOP/s).
template <int D, bool BF16OUT>
__global__ __launch_bounds__(256, D == 256 ? 2 : D == 128 ? 3 : 4) void attn_prompt_rows_kernel(PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.hq;
    const QueryTile t(a, blockIdx.x / a.hq, 128);
    if (!t.real) return;
    const int ahead = t.nk - t.nq, row = t.first + wave * 32 + (lane & 31);
    Rows<D, false, !BF16OUT> R;
    R.init(lane, a.c);
    CausalSees sees;
    sees.clean = t.first + 1 + ahead;
    sees.none = t.first + (wave + 1) * 32 + ahead;
    sees.limit = row + 1 + ahead;
    const PackedRows src = packed_rows<D>(a, t, head / (a.hq / a.hkv), t.nk);
    auto queries = [&] { R.load_q(row < t.nq ? a.q + (t.q0 + row) * a.qs + head * D : nullptr); };
    attend_rows(R, (lds_ptr)smem, 0, t.last + ahead, src, sees, queries, wave, lane);
    const float l = halves_sum(R.l), inv = inverse_sum(l);
    R.drop_if_empty(l);
    if (row >= t.nq) return;
    const int64_t out = (t.q0 + row) * a.hq + head;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            store4<BF16OUT>(a.o, out * D + R.column(d, e), R.o[d][4 * e] * inv, R.o[d][4 * e + 1] * inv,
                            R.o[d][4 * e + 2] * inv, R.o[d][4 * e + 3] * inv);
    if (a.lse && lane < 32) a.lse[out] = log_sum_exp(l == 0.f ? 0.f : R.reference(), l);
}

// Tiles of bm rows at most: every sequence may end in a part of one.
int64_t tiles_of(const PromptArgs& a, int bm) { return a.tq / bm + (a.seqs < a.tq ? a.seqs : a.tq); }

template <int D, bool BF16OUT>
hipError_t go(const PromptArgs& a, bool few, hipStream_t stream) {
    constexpr int KEYS_LDS = KeysLds<D, false>::BYTES, ROWS_LDS = RowsLds<D, false>::BYTES;
    static LdsLimit keys_limit, rows_limit;
    hipError_t e;
    if (few) {
        auto kernel = attn_prompt_keys_kernel<D, BF16OUT>;
        if ((e = keys_limit.raise((const void*)kernel, KEYS_LDS)) != hipSuccess) return e;
        kernel<<<(unsigned)(tiles_of(a, 32) * a.hq), 256, KEYS_LDS, stream>>>(a);
    } else {
        auto kernel = attn_prompt_rows_kernel<D, BF16OUT>;
        if ((e = rows_limit.raise((const void*)kernel, ROWS_LDS)) != hipSuccess) return e;
        kernel<<<(unsigned)(tiles_of(a, 128) * a.hq), 256, ROWS_LDS, stream>>>(a);
    }
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
    // Few tiles of 128 rows: 32 rows a workgroup, so that more CUs have one and
    // each row's keys are walked four at a time; 512 tokens of 24 heads of 256
    // take 24.5 us so and 35.7 the other way, of 32 heads of 128 11.2 and 17.6,
    // 2048 of 14 heads of 64 22.4 and 35.7.  With two key tiles there is little to
    // share out: 33 tokens of 32 heads of 128 6.9 and 5.8 us (of 24 of 256 11.1
    // and 12.1).  Past the bound for rows of 256 the first form is still the
    // faster one at 1024 tokens of 24 heads (47.1 and 57.7 us) and at 16 prompts
    // of up to 300 of 8 heads (20.7 and 27.6).
    const bool few = tiles_of(a, 128) * hq * (d == 256 ? 2 : 1) <= device_cu_count() && tk > 64 * seqs;
    switch (d) {
        case 64: return bf16_out ? go<64, true>(a, few, stream) : go<64, false>(a, few, stream);
        case 128: return bf16_out ? go<128, true>(a, few, stream) : go<128, false>(a, few, stream);
        default: return bf16_out ? go<256, true>(a, few, stream) : go<256, false>(a, few, stream);
    }
}

}  // namespace nq
