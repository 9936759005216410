// Attention of drafted tokens over a paged cache (nq_attn_tree).
//
// The rows of one (sequence, KV head) are its drafted tokens times the query
// heads that share the head, so every cached byte is read once for all of
// them.  Few rows (up to 32: one token, or a few): the waves of a workgroup
// take different keys, each through LDS of its own without barriers, and join
// at the end.  More rows: the waves take different rows of the same keys.
// Either way a sequence's keys are split over workgroups and the parts are
// joined by a second small kernel, so that one long context uses every CU.
// Bound by HBM, the cache's bytes once, while the rows are few; from about 64
// rows a KV head by the products.  First kernel and join, 24 / 4 heads of 256:
//   one context of 131072 keys, one token   BF16 93.6 + 5.8 us   E4M3 46.9 + 5.1
//   one of 32768, one token                      27.1 + 4.5           18.0 + 4.6
//   one of 32768, 33 drafts                      53.2 + 12.2          50.4 + 12.0
// (the longest: 5.7 and 5.7 TB/s of keys and values).
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_attn_keys.h"
#include "nq_attn_launch.h"

namespace nq {
namespace attn {

struct TreeArgs {
    const uint16_t* q;
    int64_t qs;                     // elements between tokens
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale; // per KV head (E4M3 caches), or NULL
    const int32_t* table;
    int width;
    const int32_t *lens, *cu;
    const uint64_t* masks;
    int seqs, max_q;
    int64_t t;
    int hq, hkv, group;
    int page_shift;
    int64_t pages;
    float scale;
    void* o;
    float* lse;
    float* parts;                   // parts' outputs, then their (r, l) pairs, then each sequence's (first part, parts)
    int want;                       // ranges to split all sequences' keys into, about (0: one a sequence)
    int least, step;                // keys of a range: at least, and a multiple of
    int row_tiles;
};

// One sequence as the call describes it, kept inside its arrays.
struct Seq {
    int64_t t0;
    int n, len, total;
    // `b` is the same in all lanes: scalar loads
    __device__ __forceinline__ Seq(const TreeArgs& a, int b) : Seq(a, uniform(a.cu, b), uniform(a.cu, b + 1), uniform(a.lens, b)) {}
    __device__ __forceinline__ Seq(const TreeArgs& a, int64_t x0, int64_t x1, int64_t ln) {
        x0 = x0 < 0 ? 0 : x0 > a.t ? a.t : x0;
        x1 = x1 < x0 ? x0 : x1 > a.t ? a.t : x1;
        t0 = x0;
        n = (int)(x1 - x0 < a.max_q ? x1 - x0 : a.max_q);
        const int64_t cap = (int64_t)a.width << a.page_shift;
        ln = ln < 0 ? 0 : ln > cap ? cap : ln;
        len = (int)ln;
        total = (int)(ln + n < cap ? ln + n : cap);
    }
};

// How the keys of all sequences are split into ranges: ranges of one length,
// so that there are about a.want of them whatever the sequences' lengths are,
// numbered through the sequences in order.  Every workgroup works this out for
// itself from the lengths (a wave reads 64 sequences at a time).
constexpr int MOST_PARTS = 128;     // of a sequence
struct Range {
    int b, first, parts, key0, key1;                    // its sequence, number of the sequence's first range and of ranges
    __device__ __forceinline__ static int64_t keys_of(const TreeArgs& a, int b) {
        if (b >= a.seqs) return 0;
        const Seq s(a, a.cu[b], a.cu[b + 1], a.lens[b]);
        return s.n > 0 ? s.total : -1;                  // -1: nothing to do
    }
    // Keys of a range, for `all` keys in `busy` sequences, `top` in the longest.
    __device__ __forceinline__ static int64_t length(const TreeArgs& a, int64_t all, int64_t top, int busy) {
        if (a.want == 0) return (int64_t)1 << 30;
        // the last range of each sequence is a part of one: aim at `busy` fewer
        const int aim = a.want - busy > a.want / 2 ? a.want - busy : (a.want + 1) / 2;
        int64_t chunk = (all + aim - 1) / aim;
        if (chunk < (top + MOST_PARTS - 1) / MOST_PARTS) chunk = (top + MOST_PARTS - 1) / MOST_PARTS;
        if (chunk < a.least) chunk = a.least;
        return (chunk + a.step - 1) / a.step * a.step;
    }
    // Range `index`; b = -1 where there is none.
    __device__ __forceinline__ Range(const TreeArgs& a, int index) {
        const int lane = threadIdx.x & 63;
        if (a.seqs == 1) {                              // the same without the lanes' exchanges (a third of a short decode step)
            const Seq s(a, 0);
            const int64_t c = length(a, s.total, s.total, s.total > 0);
            first = 0;
            parts = s.n == 0 ? 0 : s.total == 0 ? 1 : (int)((s.total + c - 1) / c);
            b = index < parts ? 0 : -1;
            key0 = (int)(index * c < s.total ? index * c : s.total);
            key1 = (int)(key0 + c < s.total ? key0 + c : s.total);
            return;
        }
        int64_t all = 0, top = 0;
        int busy = 0;
        for (int b0 = 0; b0 < a.seqs; b0 += 64) {
            const int64_t t = keys_of(a, b0 + lane);
            all += t > 0 ? t : 0;
            top = t > top ? t : top;
            busy += t > 0;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            all += __shfl_xor(all, off, 64);
            const int64_t o = __shfl_xor(top, off, 64);
            top = o > top ? o : top;
            busy += __shfl_xor(busy, off, 64);
        }
        const int64_t chunk = length(a, all, top, busy);
        b = -1;
        int before = 0;
        for (int b0 = 0; b0 < a.seqs && b < 0; b0 += 64) {
            const int64_t t = keys_of(a, b0 + lane);
            const int n = b0 + lane >= a.seqs || t < 0 ? 0 : t == 0 ? 1 : (int)((t + chunk - 1) / chunk);
            int upto = n;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int y = __shfl_up(upto, off, 64);
                if (lane >= off) upto += y;
            }
            const uint64_t past = __ballot(before + upto > index);
            if (past) {
                const int at = __builtin_ctzll(past);
                b = b0 + at;
                parts = __shfl(n, at, 64);
                first = before + __shfl(upto, at, 64) - parts;
            }
            before += __shfl(upto, 63, 64);
        }
        if (b < 0) return;
        b = __builtin_amdgcn_readfirstlane(b);
        parts = __builtin_amdgcn_readfirstlane(parts);
        first = __builtin_amdgcn_readfirstlane(first);
        const int64_t total = keys_of(a, b), from = (index - first) * chunk;
        key0 = __builtin_amdgcn_readfirstlane((int)from);
        key1 = __builtin_amdgcn_readfirstlane((int)(from + chunk < total ? from + chunk : total));
    }
};

// K or V rows of one sequence and KV head in pages of (1 << page_shift) rows.
// A page number outside the pool gives rows of zeros.
template <int D, bool FP8>
struct PagedRows {
    const char *k, *v;
    const int32_t* table;           // this sequence's row
    int64_t pages;
    int64_t page_bytes, head_bytes; // bytes of a page; of the heads before this one
    int page_shift, total;
    static constexpr int k_stride = Tile<D, FP8>::ROW, v_stride = Tile<D, FP8>::ROW;
    __device__ __forceinline__ v4i rows(const char* base, int key) const {
        int rows = total - key < 16 ? total - key : 16;
        const int64_t page = rows > 0 ? uniform(table, key >> page_shift) : -1;
        if (page < 0 || page >= pages) rows = 0;
        const int64_t at = rows > 0 ? page * page_bytes + head_bytes + (int64_t)(key & ((1 << page_shift) - 1)) * k_stride : 0;
        return rows_rsrc(base + at, rows, k_stride, k_stride);
    }
    __device__ __forceinline__ v4i k_rows(int key) const { return rows(k, key); }
    __device__ __forceinline__ v4i v_rows(int key) const { return rows(v, key); }
};

struct TreeSees {
    int len;                        // committed keys: seen by every row
    int none = 1 << 30;             // 0: the wave has no rows
    uint64_t mask;                  // drafted keys that this lane's row sees
    __device__ __forceinline__ int all_before() const { return len; }
    __device__ __forceinline__ int none_from() const { return none; }
    __device__ __forceinline__ uint64_t seen(int key) const {
        const int at = len - key;   // where the drafted keys start among these 64
        const uint64_t drafted = at >= 64 ? 0ull : at >= 0 ? mask << at : at > -64 ? mask >> -at : 0ull;
        return bits_below(at) | drafted;
    }
};

// Parts are numbered as the ranges are; row: max_q group of them a KV head.
__device__ __forceinline__ int64_t part_row(const TreeArgs& a, int range, int kvh, int row) {
    return ((int64_t)range * a.hkv + kvh) * ((int64_t)a.max_q * a.group) + row;
}
__device__ __forceinline__ float2* part_sums(const TreeArgs& a, int d) {
    return reinterpret_cast<float2*>(a.parts + part_row(a, a.want + a.seqs, 0, 0) * d);
}
__device__ __forceinline__ int2* part_ranges(const TreeArgs& a, int d) {
    return reinterpret_cast<int2*>(part_sums(a, d) + part_row(a, a.want + a.seqs, 0, 0));
}

// Rows [0, n group) of (b, kvh): token row / group, query head kvh group + row % group.
__device__ __forceinline__ TreeSees tree_sees(const TreeArgs& a, const Seq& s, int row) {
    TreeSees sees;
    sees.len = s.len;
    sees.mask = row < s.n * a.group ? a.masks[s.t0 + row / a.group] & bits_below(s.total - s.len) : ~0ull;
    return sees;
}
__device__ __forceinline__ const uint16_t* tree_query(const TreeArgs& a, const Seq& s, int kvh, int row, int d) {
    if (row >= s.n * a.group) return nullptr;
    return a.q + (s.t0 + row / a.group) * a.qs + (int64_t)(kvh * a.group + row % a.group) * d;
}
__device__ __forceinline__ int64_t tree_out(const TreeArgs& a, const Seq& s, int kvh, int row) {
    return (s.t0 + row / a.group) * a.hq + kvh * a.group + row % a.group;
}

template <int D, bool FP8>
__device__ __forceinline__ PagedRows<D, FP8> paged_rows(const TreeArgs& a, const Seq& s, int b, int kvh) {
    PagedRows<D, FP8> src;
    src.k = (const char*)a.k_pages;
    src.v = (const char*)a.v_pages;
    src.table = a.table + (int64_t)b * a.width;
    src.pages = a.pages;
    src.head_bytes = ((int64_t)kvh << a.page_shift) * Tile<D, FP8>::ROW;
    src.page_bytes = ((int64_t)a.hkv << a.page_shift) * Tile<D, FP8>::ROW;
    src.page_shift = a.page_shift;
    src.total = s.total;
    return src;
}

// More than 32 rows: 128 a workgroup.  Bound by the vector ALU and the products,
// and by the parts it writes: 33 drafts of 24 / 4 heads of 256 over 32768 keys
// 50 us in an E4M3 cache (10 vector instructions a product, 4 of them the
// decode; 52 MB of parts, and the join below reads them in 12 us).  With half as
// many parts, one workgroup a CU, 53 + 9 us.
template <int D, bool FP8, bool BF16OUT>
__global__ __launch_bounds__(256, D == 256 ? 2 : D == 128 ? 3 : 4) void attn_tree_rows_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the row tiles of one range are 8 apart: on the same XCD, whose L2 gives all but the first their keys
    const int rt = blockIdx.x / 8 % a.row_tiles, unit = blockIdx.x / (8 * a.row_tiles) * 8 + blockIdx.x % 8;
    const int kvh = unit % a.hkv, range = unit / a.hkv;
    const Range r(a, range);
    if (r.b < 0) return;
    const Seq s(a, r.b);
    if (rt * 128 >= s.n * a.group) return;
    if (r.first == range && kvh == 0 && rt == 0 && threadIdx.x == 0 && a.want > 0) part_ranges(a, D)[r.b] = make_int2(r.first, r.parts);
    Rows<D, FP8, !BF16OUT> R;
    R.init(lane, a.scale * (FP8 ? a.k_scale[kvh] : 1.0f) * LOG2E);
    const int row = (rt * 4 + wave) * 32 + (lane & 31);
    TreeSees sees = tree_sees(a, s, row);
    if ((rt * 4 + wave) * 32 >= s.n * a.group) sees.none = 0;
    const PagedRows<D, FP8> src = paged_rows<D, FP8>(a, s, r.b, kvh);
    auto queries = [&] { R.load_q(tree_query(a, s, kvh, row, D)); };
    attend_rows(R, (lds_ptr)smem, r.key0, r.key1, src, sees, queries, wave, lane);
    const float l = halves_sum(R.l), ref = R.m == -INFINITY ? 0.f : R.reference();
    R.drop_if_empty(l);
    if (row >= s.n * a.group) return;
    const bool only = r.parts == 1;
    const int64_t out = tree_out(a, s, kvh, row), part = part_row(a, range, kvh, row);
    const float f = only ? inverse_sum(l) * (FP8 ? a.v_scale[kvh] : 1.0f) : 1.0f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = R.o[d][4 * e] * f, x1 = R.o[d][4 * e + 1] * f, x2 = R.o[d][4 * e + 2] * f, x3 = R.o[d][4 * e + 3] * f;
            if (only) store4<BF16OUT>(a.o, out * D + R.column(d, e), x0, x1, x2, x3);
            else store4<false>(a.parts, part * D + R.column(d, e), x0, x1, x2, x3);
        }
    if (lane < 32) {
        if (!only) part_sums(a, D)[part] = make_float2(ref, l);
        else if (a.lse) a.lse[out] = log_sum_exp(ref, l);
    }
}

// Up to 32 rows: the waves take different keys.  Bound by HBM; 40 sequences of
// up to 8191 keys, 32 / 8 heads of 128, 34 us for 120 MB.
template <int D, bool FP8, bool BF16OUT>
__global__ __launch_bounds__(256) void attn_tree_keys_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = blockIdx.x % a.hkv, range = blockIdx.x / a.hkv;
    const Range r(a, range);
    if (r.b < 0) return;
    const Seq s(a, r.b);
    if (r.first == range && kvh == 0 && threadIdx.x == 0 && a.want > 0) part_ranges(a, D)[r.b] = make_int2(r.first, r.parts);
    Rows<D, FP8, !BF16OUT> R;
    R.init(lane, a.scale * (FP8 ? a.k_scale[kvh] : 1.0f) * LOG2E);
    const int row = lane & 31;
    const TreeSees sees = tree_sees(a, s, row);
    PagedRows<D, FP8> src = paged_rows<D, FP8>(a, s, r.b, kvh);
    src.total = r.key1;                                 // keys past the range: no rows, zeros
    auto queries = [&] { R.load_q(tree_query(a, s, kvh, row, D)); };
    const bool only = r.parts == 1;
    const float vs = FP8 ? a.v_scale[kvh] : 1.0f;
    auto emit = [&](int i, int col, const v4f& x, float ref, float l) {
        const int64_t out = tree_out(a, s, kvh, i);
        if (only) {
            const float f = inverse_sum(l) * vs;
            store4<BF16OUT>(a.o, out * D + col, x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            if (col == 0 && a.lse) a.lse[out] = log_sum_exp(ref, l);
        } else {
            const int64_t part = part_row(a, range, kvh, i);
            store4<false>(a.parts, part * D + col, x[0], x[1], x[2], x[3]);
            if (col == 0) part_sums(a, D)[part] = make_float2(ref, l);
        }
    };
    attend_keys(R, smem, r.key0, r.key1, s.n * a.group, src, sees, queries, emit, wave, lane);
}

// The parts of a row, joined in the order of their keys (one result whatever
// the order in which the parts were made).  WAVES waves a row, each summing
// every WAVES-th part; then the waves are added.  Bound by the parts' bytes, 52
// MB in 12 us, and by latency where there is little to join, 7 us: the ranges
// are loaded beside the lengths and the parts beside their references.
template <int D, int WAVES, bool BF16OUT>
__global__ __launch_bounds__(WAVES * 64) void attn_tree_join_kernel(TreeArgs a) {
    __shared__ float sum_s[WAVES];
    __shared__ __align__(16) float o_s[WAVES][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = a.max_q * a.group;
    const int row = blockIdx.x % rows, kvh = blockIdx.x / rows % a.hkv, b = blockIdx.x / rows / a.hkv;
    // (loaded beside the lengths: a sequence without drafts has left nothing there)
    const int* ranges = reinterpret_cast<const int*>(part_ranges(a, D));
    const int first = uniform(ranges, 2 * b), parts = uniform(ranges, 2 * b + 1);
    const Seq s(a, b);
    if (row >= s.n * a.group || parts <= 1) return;
    const float2* ml = part_sums(a, D);
    constexpr int W = D / 64, BATCH = 16;               // columns a lane; parts whose loads are in flight together
    typedef float vw __attribute__((ext_vector_type(W)));
    float2 tops[MOST_PARTS / 64];                       // this lane's parts (a part twice does no harm)
#pragma unroll
    for (int i = 0; i < MOST_PARTS / 64; ++i)
        tops[i] = ml[part_row(a, first + (i * 64 + lane < parts ? i * 64 + lane : 0), kvh, row)];
    auto highest = [&] {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < MOST_PARTS / 64; ++i)
            if (tops[i].y != 0.f) top = max2(top, tops[i].x);
        return wave_max(top);
    };
    float top = -INFINITY, sum = 0.f, x[W];
#pragma unroll
    for (int j = 0; j < W; ++j) x[j] = 0.f;
    bool have = false;
    for (int i0 = wave; i0 < parts; i0 += WAVES * BATCH) {
        float2 p[BATCH];
        vw y[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const int64_t at = part_row(a, first + (i0 + WAVES * e < parts ? i0 + WAVES * e : i0), kvh, row);
            p[e] = ml[at];
            y[e] = *reinterpret_cast<const vw*>(a.parts + at * D + lane * W);
        }
        if (!have) top = highest();                     // (beside the first loads)
        have = true;
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const bool real = i0 + WAVES * e < parts && p[e].y != 0.f;        // (a part that saw nothing has neither)
            const float f = real ? __builtin_amdgcn_exp2f(p[e].x - top) : 0.f;
            sum += real ? p[e].y * f : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) x[j] += real ? y[e][j] * f : 0.f;
        }
    }
    if (!have) top = highest();
    if constexpr (WAVES > 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) o_s[wave][lane * W + j] = x[j];
        if (lane == 0) sum_s[wave] = sum;
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            sum += sum_s[w];
#pragma unroll
            for (int j = 0; j < W; ++j) x[j] += o_s[w][lane * W + j];
        }
    }
    const float f = inverse_sum(sum) * (a.v_scale ? a.v_scale[kvh] : 1.0f);
    const int64_t out = tree_out(a, s, kvh, row);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const int col = lane * W + j;
        const float y = x[j] * f;
        if constexpr (BF16OUT) reinterpret_cast<uint16_t*>(a.o)[out * D + col] = (uint16_t)f32_to_bf16_rne(y);
        else reinterpret_cast<float*>(a.o)[out * D + col] = y;
    }
    if (lane == 0 && a.lse) a.lse[out] = log_sum_exp(top == -INFINITY ? 0.f : top, sum);
}

// Rows a workgroup of the launch holds.  (Eight waves with 256 rows, one
// workgroup a CU, took the same time for 198 rows of 256 over 32768 E4M3 keys
// as two workgroups of four.)
constexpr int tile_rows(int64_t rows) { return rows <= 32 ? 32 : 128; }

template <int D, bool FP8, bool BF16OUT>
hipError_t go_tree(const TreeArgs& a, hipStream_t stream) {
    const unsigned units = (unsigned)(a.want + a.seqs) * a.hkv;
    hipError_t e;
    if (tile_rows(a.max_q * a.group) == 32) {
        constexpr int LDS = KeysLds<D, FP8>::BYTES;
        auto kernel = attn_tree_keys_kernel<D, FP8, BF16OUT>;
        static LdsLimit limit;
        if ((e = limit.raise((const void*)kernel, LDS)) != hipSuccess) return e;
        kernel<<<units, 256, LDS, stream>>>(a);
    } else {
        constexpr int LDS = RowsLds<D, FP8>::BYTES;
        auto kernel = attn_tree_rows_kernel<D, FP8, BF16OUT>;
        static LdsLimit limit;
        if ((e = limit.raise((const void*)kernel, LDS)) != hipSuccess) return e;
        kernel<<<(units + 7) / 8 * 8 * a.row_tiles, 256, LDS, stream>>>(a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.want > 0) {
        // four waves a row where rows are few; one where they fill the CUs by themselves (most have one part then)
        const unsigned rows = (unsigned)a.seqs * a.hkv * a.max_q * a.group;
        if (rows < 2048) attn_tree_join_kernel<D, 4, BF16OUT><<<rows, 256, 0, stream>>>(a);
        else attn_tree_join_kernel<D, 1, BF16OUT><<<rows, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace attn

namespace {

struct TreePlan {
    int want, least, step, row_tiles;
    int64_t bytes;
};

// Workspace of one range: the results and sums of every row.
int64_t range_bytes(int64_t max_q, int64_t hq, int64_t d) { return max_q * hq * (d * 4 + 8); }

// Ranges of 128 keys (four waves of 32) or, with more rows and so more to
// write for each part, 256, and up.  Few sequences: as many
// workgroups as run at once.  Many: about four times as many, short enough
// that the last ones to run do not leave most CUs idle.
TreePlan tree_plan(int64_t seqs, int64_t max_q, int64_t hq, int64_t hkv, int64_t d, int64_t max_len, int64_t cus) {
    const int64_t rows = max_q * (hq / hkv), tile = attn::tile_rows(rows), tiles = (rows + tile - 1) / tile;
    const int64_t least = rows <= 32 ? 128 : 256, units = seqs * hkv * tiles;
    TreePlan p{0, (int)least, rows <= 32 ? 128 : 32, (int)tiles, 0};
    if (max_len > (int64_t)1 << 30) max_len = (int64_t)1 << 30;          // the most that a table holds
    // Short contexts: one range a sequence and one launch.  Microseconds in a
    // graph, one range against several joined, BF16:
    //                                      200 keys     450          768
    //   24 / 4 of 256, 1 sequence, 1 token  10.6 13.6    13.4 13.7    16.4 13.8
    //     8 drafts                          15.6 17.8    23.5 20.2    33.4 22.5
    //     64 sequences, 1 token             12.2 27.0    15.7 30.1    19.9 36.8
    //   32 / 8 of 128, 1 sequence, 1 token   7.5 10.3     9.6 10.4    11.8 10.7
    //     64 sequences, 1 token             10.2 19.7    12.0 21.6    16.0 24.9
    // One bound for all is a middle: for one sequence the two meet near 450 keys,
    // for 64 past 768.  (Callers choose through max_len.)
    if (max_len <= 768) return p;
    const int64_t slots = cus * (tile == 32 && d == 256 ? 1 : 2);        // workgroups that run at once
    int64_t want = (2 * units <= slots ? slots : 4 * cus) / (hkv * tiles);
    const int64_t most = seqs * ((max_len + least - 1) / least) + seqs;
    if (want > most) want = most;
    if (want < 1) want = 1;
    p.want = (int)want;
    p.bytes = (want + seqs) * range_bytes(max_q, hq, d) + seqs * 8;
    return p;
}

}  // namespace

// What any call up to these sizes needs: fewer drafts may need more, since they
// have fewer row tiles and are split further.
int64_t attn_tree_workspace_bytes(int64_t seqs, int64_t max_q, int64_t hq, int64_t hkv, int64_t d, int64_t max_len) {
    const int64_t cus = device_cu_count();
    int64_t most = 0;
    for (int64_t q = 1; q <= max_q; ++q) {
        const int64_t bytes = tree_plan(seqs, q, hq, hkv, d, max_len, cus).bytes;
        if (bytes > most) most = bytes;
    }
    return most;
}

hipError_t launch_attn_tree(bool fp8, const uint16_t* q, int64_t q_stride, const void* k_pages, const void* v_pages,
                            const float* k_scale, const float* v_scale, const int32_t* table, int64_t width,
                            const int32_t* lens, const int32_t* cu_q, const uint64_t* masks, int64_t seqs, int64_t max_q,
                            int64_t t, int64_t hq, int64_t hkv, int64_t d, int64_t page_size, int64_t pages,
                            int64_t max_len, float scale, bool bf16_out, void* o, float* lse, void* workspace,
                            int64_t workspace_bytes, hipStream_t stream) {
    using namespace attn;
    TreePlan p = tree_plan(seqs, max_q, hq, hkv, d, max_len, device_cu_count());
    if (workspace_bytes < p.bytes) {        // as many ranges as fit, each sequence's last one beside them
        const int64_t fit = (workspace_bytes - seqs * 8) / range_bytes(max_q, hq, d) - seqs;
        p.want = fit > 0 ? (int)fit : 0;
    }
    const TreeArgs a{q, q_stride, k_pages, v_pages, fp8 ? k_scale : nullptr, fp8 ? v_scale : nullptr, table, (int)width, lens,
                     cu_q, masks, (int)seqs, (int)max_q, t, (int)hq, (int)hkv, (int)(hq / hkv), __builtin_ctzll(page_size),
                     pages, scale, o, lse, reinterpret_cast<float*>(workspace), p.want, p.least, p.step, p.row_tiles};
    switch (d) {
        case 64:
            return fp8 ? (bf16_out ? go_tree<64, true, true>(a, stream) : go_tree<64, true, false>(a, stream))
                       : (bf16_out ? go_tree<64, false, true>(a, stream) : go_tree<64, false, false>(a, stream));
        case 128:
            return fp8 ? (bf16_out ? go_tree<128, true, true>(a, stream) : go_tree<128, true, false>(a, stream))
                       : (bf16_out ? go_tree<128, false, true>(a, stream) : go_tree<128, false, false>(a, stream));
        default:
            return fp8 ? (bf16_out ? go_tree<256, true, true>(a, stream) : go_tree<256, true, false>(a, stream))
                       : (bf16_out ? go_tree<256, false, true>(a, stream) : go_tree<256, false, false>(a, stream));
    }
}

}  // namespace nq
