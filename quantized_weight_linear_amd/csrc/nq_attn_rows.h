// The workgroup form with many query rows: NW waves with 32 QB rows each walk
// the keys together, 32 at a time.  Every 32-key tile of K and V is loaded
// into LDS once per workgroup, into rings of RING tiles: the loads of tile
// i + RING - 1 are issued when tile i is complete.  The matrix work of one
// wave runs beside the softmax of the others on its SIMD.
#pragma once

#include <type_traits>

#include "nq_attn_core.h"

namespace nq {
namespace attn {

constexpr int KEYS = 32;        // keys a step

template <int D, bool FP8, int NW, int RING>
struct RowsLds {
    static constexpr int TILE = KEYS * Tile<D, FP8>::ROW;
    static constexpr int FLAGS = 2 * RING * TILE;        // [2] steps x NW words: the staged values that are not finite
    static constexpr int BYTES = FLAGS + 2 * NW * 4;
};

// Bits below n (0 .. 64 and beyond either end).
__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Source: k_rows(key) / v_rows(key) give the descriptor of 16 keys from a
// 16-aligned key on (keys past the last one are outside it), k_stride /
// v_stride the bytes between rows.
// Sees: all_before() = every row of the workgroup sees all keys below it;
// none_from() = no row of this wave sees keys from it on; seen(b, key) = the
// 64 keys from `key` on as bits, for this lane's row of block b.
// Queries: loads the rows' queries; called once the first keys are on their way.
template <int RING, int NW, int D, int QB, bool FP8, bool SPLITP, class Source, class Sees, class Queries>
__device__ __forceinline__ void attend_rows(Rows<D, QB, FP8, SPLITP>& R, lds_ptr lds, int key0, int key1,
                                            const Source& src, const Sees& sees, const Queries& queries,
                                            int wave, int lane) {
    using L = RowsLds<D, FP8, NW, RING>;
    using T = Tile<D, FP8>;
    constexpr int ROW = T::ROW, LOADS = 4 * T::LOADS16 / NW;          // a wave's load instructions a step
    static_assert((NW == 4 || NW == 8) && LOADS * NW == 4 * T::LOADS16, "a step stages four groups of 16 rows");
    const int group = wave & 3, part = (group & 1) * 16;             // groups 0, 1: K; 2, 3: V
    const Stager<D, FP8> st(lane, group < 2 ? src.k_stride : src.v_stride);
    const lds_ptr k_ring = lds, v_ring = lds + RING * L::TILE;
    auto load = [&](v4i r, lds_ptr dst) {
        if (NW == 4 || wave < 4) st.template pieces<0, LOADS>(r, dst);
        else st.template pieces<NW == 4 ? 0 : LOADS, LOADS>(r, dst);
    };
    auto stage = [&](int i, int slot) {
        const int key = key0 + i * KEYS + part;
        if (group < 2) load(src.k_rows(key), k_ring + slot * L::TILE + part * ROW);
        else load(src.v_rows(key), v_ring + slot * L::TILE + part * ROW);
    };
    if (key0 >= key1) return;
    const int n = (key1 - key0 + KEYS - 1) / KEYS;
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) stage(i, i);
    queries();
    R.queries_ready();
    auto step = [&](int i, int slot, auto partly) {
        constexpr bool PARTLY = decltype(partly)::value;
        const int key = key0 + i * KEYS;
        const lds_ptr k = k_ring + slot * L::TILE, v = v_ring + slot * L::TILE;
        auto* flags = (__attribute__((address_space(3))) uint32_t*)(lds + L::FLAGS) + (i & 1) * NW;
        wait_vm<(RING - 2) * LOADS>();
        if (PARTLY) {
            uint32_t rows = 0;
            if (group >= 2) {
                const lds_cptr p = v + part * ROW + (wave >> 2) * LOADS * 1024;
                rows = rows_not_finite<D, FP8, LOADS>(p, lane) << (part + (wave >> 2) * LOADS * T::RPI);
            }
            if (lane == 0) flags[wave] = rows;
        }
        lds_barrier();
        stage(i + RING - 1, slot == 0 ? RING - 1 : slot - 1);
        uint32_t bad = 0;
        bool some = true;
        uint64_t seen[QB];
        if (PARTLY) {
            some = key < sees.none_from();
#pragma unroll
            for (int w = 0; w < NW; ++w) bad |= flags[w];
            bad = __builtin_amdgcn_readfirstlane(bad);
#pragma unroll
            for (int b = 0; b < QB; ++b) seen[b] = sees.seen(b, key);
        }
        v16f s[QB];
        if (some) R.template weights<PARTLY>(k, seen, s);
        if (PARTLY && bad) {
            if (some) R.add_not_finite(v, bad, seen);
            lds_barrier();
            if (group >= 2) rows_made_finite<D, FP8, LOADS>(v + part * ROW + (wave >> 2) * LOADS * 1024, lane);
            lds_barrier();
        }
        if (some) R.values(v, s);
    };
    const int clean = sees.all_before() - key0 < 0 ? 0 : (sees.all_before() - key0) / KEYS;
    int i = 0, slot = 0;
    for (const int whole = (clean < n ? clean : n) - RING; i <= whole; i += RING) {
#pragma unroll
        for (int j = 0; j < RING; ++j) step(i + j, j, std::false_type{});
    }
    for (; i < n; ++i) {
        step(i, slot, std::true_type{});
        slot = slot == RING - 1 ? 0 : slot + 1;
    }
    wait_vm<0>();                                        // nothing may land in LDS after the workgroup has gone
}

}  // namespace attn
}  // namespace nq
