// Pages of a K/V cache: rows appended, pages counted, shared, copied, rows of
// an accepted path moved together (nq_kv_*).  Nothing is computed: the row and
// page moves are bound by HBM (each byte read once and written once), the
// accounting by launch latency and, for large pools, by one pass over the
// counts.
//
// Accounting: refs[page] counts the table entries that name the page; a page
// is free when its count is 0.  Free pages are handed out lowest first, in the
// order of the requests, by one workgroup (a scan, no races), so the result
// does not depend on timing.
#include <hip/hip_runtime.h>

#include "nq.h"
#include "nq_attn_launch.h"
#include "nq_device.h"
#include "nq_pages.h"

namespace nq {
namespace {

constexpr int POOL_THREADS = 1024;

struct AppendArgs {
    const uint16_t *k, *v;
    int64_t ks, vs;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens, *cu;
    int64_t width, pages, t;
    int seqs, hkv, d, shift;
    void *k_pages, *v_pages;
};

// Eight values a thread: K (blockIdx.y = 0) or V.  Bound by latency at a
// step's sizes (33 tokens of 4 heads of 256: 5 us), by HBM for a prompt (16384
// tokens 22.8 us, 5.9 TB/s read and written; as E4M3 codes, whose divisions
// count too, 24.8 us, 4.1 TB/s).
template <bool FP8>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a) {
    const int per = a.hkv * a.d / 8;                     // threads a token
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / per;
    if (t >= a.t) return;
    const int piece = (int)(i % per), head = piece / (a.d / 8), col = piece % (a.d / 8) * 8;
    const int b = owner(a.cu, a.seqs, t);
    const int64_t first = a.cu[b];
    if (t < first || t >= a.cu[b + 1]) return;
    const int64_t at = a.lens[b] + (t - first);
    const int64_t page = page_of(a.table + b * a.width, a.width, a.pages, a.shift, at);
    if (a.lens[b] < 0 || page < 0) return;
    const bool value = blockIdx.y != 0;
    const uint16_t* x = (value ? a.v + t * a.vs : a.k + t * a.ks) + head * a.d + col;
    const int64_t to = (((page * a.hkv + head) << a.shift) + (at & ((1 << a.shift) - 1))) * a.d + col;
    const v4u w = *reinterpret_cast<const v4u*>(x);
    void* pages = value ? a.v_pages : a.k_pages;
    if constexpr (FP8) {
        const double r = 1.0 / (double)(value ? a.v_scale : a.k_scale)[head];
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = div_via_recip64(bf16_bits_to_f32(w[j] & 0xFFFFu), r);
            f[2 * j + 1] = div_via_recip64(bf16_bits_to_f32(w[j] >> 16), r);
        }
        *reinterpret_cast<v2u*>((uint8_t*)pages + to) = v2u{encode4(f[0], f[1], f[2], f[3]), encode4(f[4], f[5], f[6], f[7])};
    } else {
        *reinterpret_cast<v4u*>((uint16_t*)pages + to) = w;
    }
}

// Sum over the lanes before this one in the workgroup, and the workgroup's
// total; `part` is LDS for one value a wave.
__device__ __forceinline__ int before_in_block(int x, int* part, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(incl, off, 64);
        if (lane >= off) incl += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < POOL_THREADS / 64; ++w) {
        if (w < wave) base += part[w];
        all += part[w];
    }
    *total = all;
    return base + incl - x;
}

// The lowest free pages, as many as wanted at most, into list; returns how
// many there are.  16 counts a thread and step, read before any are handed on.
__device__ int collect_free(const int32_t* refs, int64_t pages, int wanted, int32_t* list, int* part) {
    int found = 0;
    for (int64_t at = 0; at < pages && found < wanted; at += POOL_THREADS * 16) {
        const int64_t mine = at + threadIdx.x * 16;
        uint32_t free = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (mine + j < pages && refs[mine + j] == 0) free |= 1u << j;
        int total;
        int rank = found + before_in_block(__builtin_popcount(free), part, &total);
        for (; free; free &= free - 1, ++rank)
            if (rank < wanted) list[rank] = (int32_t)(mine + __builtin_ctz(free));
        found += total;
    }
    __syncthreads();
    return found < wanted ? found : wanted;
}

__device__ __forceinline__ int64_t ceil_pages(int64_t n, int shift) { return n <= 0 ? 0 : (n + (1 << shift) - 1) >> shift; }

// One workgroup: entries [lens >> shift, ceil(new_lens)) of each table row that
// are negative get pages, rows in order.  A thread takes a row with up to FEW
// such entries (a decode step), a wave a longer one (a prompt); the rows'
// counts, then first ranks, are in `rank` (LDS).  Latency: 1 row 3 us, 100 9 us.
constexpr int FEW = 4;
__global__ __launch_bounds__(POOL_THREADS) void kv_reserve_kernel(int32_t* refs, int64_t pages, int32_t* table, int64_t width,
                                                                  const int32_t* lens, const int32_t* new_lens, int seqs,
                                                                  int shift, int32_t* list, int32_t* shortfall) {
    extern __shared__ int rank[];                        // [seqs]; -1 in the first pass: a wave counts the row
    __shared__ int part[POOL_THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto range = [&](int b, int64_t& e0, int64_t& e1) {
        e0 = lens[b] > 0 ? lens[b] >> shift : 0;
        e1 = ceil_pages(new_lens[b], shift);
        if (e1 > width) e1 = width;
    };
    auto few = [&](int b, int64_t e0, int64_t e1) {      // the missing ones of a short row's entries, as bits
        uint32_t missing = 0;
#pragma unroll
        for (int j = 0; j < FEW; ++j)
            if (e0 + j < e1 && table[b * width + e0 + j] < 0) missing |= 1u << j;
        return missing;
    };
    for (int b = threadIdx.x; b < seqs; b += POOL_THREADS) {
        int64_t e0, e1;
        range(b, e0, e1);
        rank[b] = e1 - e0 > FEW ? -1 : __builtin_popcount(few(b, e0, e1));
    }
    __syncthreads();
    for (int b = wave; b < seqs; b += POOL_THREADS / 64) {
        if (rank[b] >= 0) continue;
        int64_t e0, e1;
        range(b, e0, e1);
        int n = 0;
        for (int64_t e = e0; e < e1; e += 64)
            n += __builtin_popcountll(__ballot(e + lane < e1 && table[b * width + e + lane] < 0));
        if (lane == 0) rank[b] = n;
    }
    __syncthreads();
    int wanted = 0;
    for (int b0 = 0; b0 < seqs; b0 += POOL_THREADS) {
        const int b = b0 + threadIdx.x, n = b < seqs ? rank[b] : 0;
        int total;
        const int first = wanted + before_in_block(n, part, &total);
        if (b < seqs) rank[b] = first;
        wanted += total;
    }
    const int found = wanted ? collect_free(refs, pages, wanted, list, part) : 0;
    auto give = [&](int64_t entry, int at) {
        if (at >= found) return;
        const int32_t page = list[at];
        table[entry] = page;
        refs[page] = 1;
    };
    __syncthreads();
    for (int b = threadIdx.x; b < seqs && wanted; b += POOL_THREADS) {
        int64_t e0, e1;
        range(b, e0, e1);
        if (e1 - e0 > FEW) continue;
        int at = rank[b];
        for (uint32_t missing = few(b, e0, e1); missing; missing &= missing - 1)
            give(b * width + e0 + __builtin_ctz(missing), at++);
    }
    for (int b = wave; b < seqs && wanted; b += POOL_THREADS / 64) {
        int64_t e0, e1;
        range(b, e0, e1);
        if (e1 - e0 <= FEW) continue;
        int r = rank[b];
        for (int64_t e = e0; e < e1; e += 64) {
            const bool mine = e + lane < e1 && table[b * width + e + lane] < 0;
            const uint64_t all = __ballot(mine);
            if (mine) give(b * width + e + lane, r + __builtin_popcountll(all & ((1ull << lane) - 1)));
            r += __builtin_popcountll(all);
        }
    }
    if (threadIdx.x == 0) *shortfall = wanted - found;
}

// A thread an entry: entries past the kept ones are given back.  A count that
// is already 0 stays 0.  Latency: 1 to 5 us.
__global__ __launch_bounds__(256) void kv_release_kernel(int32_t* refs, int64_t pages, int32_t* table, int64_t width,
                                                         const int32_t* keep, int shift) {
    const int64_t e = (int64_t)blockIdx.y * 256 + threadIdx.x;
    const int b = blockIdx.x;
    if (e >= width || e < ceil_pages(keep[b], shift)) return;
    const int32_t page = table[b * width + e];
    if (page < 0) return;
    table[b * width + e] = -1;
    if (page < pages && atomicSub(&refs[page], 1) <= 0) atomicAdd(&refs[page], 1);
}

struct ForkArgs {
    int32_t* refs;
    int64_t pages;
    const int32_t* table;
    int64_t width;
    const int32_t* lens;
    int seqs;
    const int32_t* parents;
    int children, shift;
    int32_t *child, *copies, *list, *shortfall;
};

// A child's parent row, whole pages and whether a part of a page follows.
struct Branch {
    const int32_t* row;
    int64_t full;
    int32_t last;                                        // the partly filled page, or -1
    __device__ __forceinline__ Branch(const ForkArgs& a, int c) {
        const int p = a.parents[c];
        const bool real = p >= 0 && p < a.seqs;
        const int64_t len = real && a.lens[p] > 0 ? a.lens[p] : 0;
        row = a.table + (real ? p : 0) * a.width;
        full = len >> a.shift;
        last = -1;
        if (full > a.width) full = a.width;
        else if ((len & ((1 << a.shift) - 1)) && full < a.width) last = row[full];
        if (last >= a.pages) last = -1;
    }
};

// Entry e of child c: whole pages are shared and counted.
__device__ __forceinline__ void share_entry(const ForkArgs& a, const Branch& br, int c, int64_t e) {
    int32_t page = e < br.full ? br.row[e] : e == br.full ? a.copies[2 * c + 1] : -1;
    if (page >= a.pages) page = -1;
    if (e < br.full && page >= 0) atomicAdd(&a.refs[page], 1);
    a.child[c * a.width + e] = page < 0 ? -1 : page;
}

// One workgroup: a page for every child whose parent ends inside a page.
// `share`: the entries too (few of them; otherwise the next kernel's work).
// Latency: 4 children 7 us, entries included; 128 8 us, and 5 for the entries.
__global__ __launch_bounds__(POOL_THREADS) void kv_fork_pages_kernel(ForkArgs a, bool share) {
    __shared__ int part[POOL_THREADS / 64];
    int wanted = 0, total;
    for (int c0 = 0; c0 < a.children; c0 += POOL_THREADS) {
        const int c = c0 + threadIdx.x;
        before_in_block(c < a.children && Branch(a, c).last >= 0, part, &total);
        wanted += total;
    }
    const int found = wanted ? collect_free(a.refs, a.pages, wanted, a.list, part) : 0;
    __syncthreads();
    int first = 0;
    for (int c0 = 0; c0 < a.children; c0 += POOL_THREADS) {
        const int c = c0 + threadIdx.x;
        const int32_t last = c < a.children ? Branch(a, c).last : -1;
        const int at = first + before_in_block(last >= 0, part, &total);
        first += total;
        if (c < a.children) {
            const bool got = last >= 0 && at < found;
            const int32_t page = got ? a.list[at] : -1;
            a.copies[2 * c] = got ? last : -1;
            a.copies[2 * c + 1] = page;
            if (got) a.refs[page] = 1;
        }
    }
    if (threadIdx.x == 0) *a.shortfall = wanted - found;
    if (!share) return;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.children * a.width; i += POOL_THREADS) {
        const int c = (int)(i / a.width);
        share_entry(a, Branch(a, c), c, i % a.width);
    }
}

__global__ __launch_bounds__(256) void kv_fork_share_kernel(ForkArgs a) {
    const int64_t e = (int64_t)blockIdx.y * 256 + threadIdx.x;
    const int c = blockIdx.x;
    if (e < a.width) share_entry(a, Branch(a, c), c, e);
}

// 16 KiB of one page a workgroup.  Bound by HBM: 128 pages of 128 KiB in 32
// planes 162 us, 6.6 TB/s read and written.
constexpr int COPY_BYTES = 16384;
__global__ __launch_bounds__(256) void kv_copy_kernel(char* pool, int64_t plane_bytes, int64_t page_bytes, int64_t pages,
                                                      const int32_t* copies, int pieces) {
    const int c = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    const int64_t src = copies[2 * c], dst = copies[2 * c + 1];
    if (src < 0 || dst < 0 || src >= pages || dst >= pages || src == dst) return;
    char* plane = pool + blockIdx.y * plane_bytes;
    const int64_t at = (int64_t)piece * COPY_BYTES + threadIdx.x * 16;
    v4u x[COPY_BYTES / 4096];
#pragma unroll
    for (int j = 0; j < COPY_BYTES / 4096; ++j)
        if (at + j * 4096 < page_bytes) x[j] = *reinterpret_cast<const v4u*>(plane + src * page_bytes + at + j * 4096);
#pragma unroll
    for (int j = 0; j < COPY_BYTES / 4096; ++j)
        if (at + j * 4096 < page_bytes) *reinterpret_cast<v4u*>(plane + dst * page_bytes + at + j * 4096) = x[j];
}

// The accepted rows of a (sequence, head) in PLANES planes, one wave: the
// places are worked out once for all planes, and the rows of a batch are all
// read before any is written, since a row may be both.  Later batches never
// read what an earlier one wrote: accepted tokens ascend, so the place that
// row i moves to lies below every row read after it.  100 sequences of up to 64
// drafts, 32 planes of 4 heads of 256 in BF16: 19 us; one 5 us.  Rows of 4 bytes, the
// scales of an E4M3 cache: 4.9 us; one 3.6.
constexpr int MOVE_ROWS = 64, MOVE_PLANES = 4, MOVE_BATCH = 4;
template <class Piece>               // 16 bytes, or the 4 of a scale's row
__global__ __launch_bounds__(256) void kv_compact_kernel(char* pool, int64_t plane_bytes, int planes, int hkv, int shift,
                                                         int row_bytes, int64_t pages, const int32_t* table, int64_t width,
                                                         const int32_t* lens, const int32_t* accept, const int32_t* cu,
                                                         int64_t accepted) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % hkv, b = blockIdx.x / hkv, plane0 = (blockIdx.y * 4 + wave) * MOVE_PLANES;
    const int32_t* row = table + b * width;
    int64_t a0 = cu[b], a1 = cu[b + 1];
    a0 = a0 < 0 ? 0 : a0 > accepted ? accepted : a0;
    a1 = a1 < a0 ? a0 : a1 > accepted ? accepted : a1;
    const int n = (int)(a1 - a0 > MOVE_ROWS ? MOVE_ROWS : a1 - a0), len = lens[b], per = row_bytes / (int)sizeof(Piece);
    if (len < 0 || plane0 >= planes) return;
    pool += plane0 * plane_bytes;
    auto place = [&](int64_t at) -> int64_t {
        const int64_t page = page_of(row, width, pages, shift, at);
        return page < 0 ? -1 : (((page * hkv + head) << shift) + (at & ((1 << shift) - 1))) * row_bytes;
    };
    for (int p0 = 0; p0 < n * per; p0 += 64 * MOVE_BATCH) {
        int64_t src[MOVE_BATCH], dst[MOVE_BATCH];
        Piece x[MOVE_BATCH][MOVE_PLANES];
#pragma unroll
        for (int j = 0; j < MOVE_BATCH; ++j) {
            const int p = p0 + j * 64 + lane, i = p / per;
            const int from = i < n ? accept[a0 + i] : i;
            src[j] = dst[j] = -1;
            if (from != i && from >= 0 && from < MOVE_ROWS) {
                src[j] = place((int64_t)len + from);
                dst[j] = place((int64_t)len + i);
                if (src[j] < 0) dst[j] = -1;
                src[j] += p % per * (int)sizeof(Piece);
                if (dst[j] >= 0) dst[j] += p % per * (int)sizeof(Piece);
            }
        }
#pragma unroll
        for (int j = 0; j < MOVE_BATCH; ++j)
#pragma unroll
            for (int q = 0; q < MOVE_PLANES; ++q)
                if (dst[j] >= 0 && plane0 + q < planes) x[j][q] = *reinterpret_cast<const Piece*>(pool + q * plane_bytes + src[j]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int j = 0; j < MOVE_BATCH; ++j)
#pragma unroll
            for (int q = 0; q < MOVE_PLANES; ++q)
                if (dst[j] >= 0 && plane0 + q < planes) *reinterpret_cast<Piece*>(pool + q * plane_bytes + dst[j]) = x[j][q];
    }
}

int shift_of(int64_t page_size) { return __builtin_ctzll(page_size); }

}  // namespace

hipError_t launch_kv_append(bool fp8, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                            const float* k_scale, const float* v_scale, const int32_t* table, int64_t width,
                            const int32_t* lens, const int32_t* cu, int64_t seqs, int64_t t, int64_t hkv, int64_t d,
                            int64_t page_size, int64_t pages, void* k_pages, void* v_pages, hipStream_t stream) {
    const AppendArgs a{k, v, k_stride, v_stride, k_scale, v_scale, table, lens, cu, width, pages, t, (int)seqs, (int)hkv,
                       (int)d, shift_of(page_size), k_pages, v_pages};
    const dim3 grid((unsigned)((t * hkv * d / 8 + 255) / 256), 2);
    if (fp8) kv_append_kernel<true><<<grid, 256, 0, stream>>>(a);
    else kv_append_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_reserve(int32_t* refs, int64_t pages, int32_t* table, int64_t width, const int32_t* lens,
                             const int32_t* new_lens, int64_t seqs, int64_t page_size, int32_t* free_list,
                             int32_t* shortfall, hipStream_t stream) {
    kv_reserve_kernel<<<1, POOL_THREADS, (size_t)seqs * 4, stream>>>(refs, pages, table, width, lens, new_lens, (int)seqs,
                                                                     shift_of(page_size), free_list, shortfall);
    return hipGetLastError();
}

hipError_t launch_kv_release(int32_t* refs, int64_t pages, int32_t* table, int64_t width, const int32_t* keep, int64_t seqs,
                             int64_t page_size, hipStream_t stream) {
    kv_release_kernel<<<dim3((unsigned)seqs, (unsigned)((width + 255) / 256)), 256, 0, stream>>>(refs, pages, table, width, keep,
                                                                                               shift_of(page_size));
    return hipGetLastError();
}

hipError_t launch_kv_fork(int32_t* refs, int64_t pages, const int32_t* table, int64_t width, const int32_t* lens, int64_t seqs,
                          const int32_t* parents, int64_t children, int64_t page_size, int32_t* child_table, int32_t* copies,
                          int32_t* free_list, int32_t* shortfall, hipStream_t stream) {
    const ForkArgs a{refs, pages, table, width, lens, (int)seqs, parents, (int)children, shift_of(page_size), child_table,
                     copies, free_list, shortfall};
    // a few rounds of one workgroup take less than another launch
    const bool share = children * width <= 4 * POOL_THREADS;
    kv_fork_pages_kernel<<<1, POOL_THREADS, 0, stream>>>(a, share);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || share) return e;
    kv_fork_share_kernel<<<dim3((unsigned)children, (unsigned)((width + 255) / 256)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_copy_pages(void* pool, int64_t planes, int64_t plane_bytes, int64_t page_bytes, int64_t pages,
                                const int32_t* copies, int64_t n, hipStream_t stream) {
    const int pieces = (int)((page_bytes + COPY_BYTES - 1) / COPY_BYTES);
    kv_copy_kernel<<<dim3((unsigned)(n * pieces), (unsigned)planes), 256, 0, stream>>>((char*)pool, plane_bytes, page_bytes,
                                                                                      pages, copies, pieces);
    return hipGetLastError();
}

hipError_t launch_kv_compact(void* pool, int64_t planes, int64_t plane_bytes, int64_t hkv, int64_t page_size,
                             int64_t row_bytes, int64_t pages, const int32_t* table, int64_t width, const int32_t* lens,
                             const int32_t* accept, const int32_t* cu_accept, int64_t seqs, int64_t accepted,
                             hipStream_t stream) {
    const dim3 grid((unsigned)(seqs * hkv), (unsigned)((planes + 4 * MOVE_PLANES - 1) / (4 * MOVE_PLANES)));
    auto kernel = row_bytes == 4 ? kv_compact_kernel<uint32_t> : kv_compact_kernel<v4u>;
    kernel<<<grid, 256, 0, stream>>>((char*)pool, plane_bytes, (int)planes, (int)hkv, shift_of(page_size), (int)row_bytes, pages,
                                     table, width, lens, accept, cu_accept, accepted);
    return hipGetLastError();
}

}  // namespace nq
