// The workgroup form with many query rows: four waves with 32 rows each walk
// the keys together, 32 at a time.  Every 32-key tile of K and V is loaded
// into LDS once per workgroup, two tiles deep: the loads of the next one are
// issued when a tile is complete.  Two to four workgroups run on a CU (by the
// registers), and the matrix work of one wave runs beside the softmax of the
// others on its SIMD.
//   Bound by the matrix cores and the vector ALU beside them: 16384 causal
// tokens of 24 heads of 256 take 2.9 ms, 1120 to 1140 TFLOP/s; 8192 of 24 of 256
// 1050 TFLOP/s, of 32 of 128 1060, of 32 of 64 880, of 32 of 128 with FP32 outputs
// 590 (three products with V).  At 16384 tokens eight waves a workgroup are 3 %
// slower, rings of three 2 %; logits of the next tile beside the softmax of
// this one within a wave, with fewer waves, 30 %.
//   E4M3 rows become BF16 as operands are read, in every wave: 33 drafts of 24
// heads of 256 over 32768 keys take 50 us.  Decoded once a workgroup into
// BF16 tiles, by the wave that loaded them, they took 58: the decode then
// stands between a tile's loads and its products.
#pragma once

#include <type_traits>

#include "nq_attn_core.h"

namespace nq {
namespace attn {

constexpr int KEYS = 32;        // keys a step

template <int D, bool FP8>
struct RowsLds {
    static constexpr int TILE = KEYS * Tile<D, FP8>::ROW;
    static constexpr int FLAGS = 4 * TILE;               // [2] steps x 4 waves: the staged rows that are not finite
    static constexpr int BYTES = FLAGS + 2 * 4 * 4;
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
// none_from() = no row of this wave sees keys from it on; seen(key) = the
// 64 keys from `key` on as bits, for this lane's row.
// Queries: loads the rows' queries; called once the first keys are on their way.
template <int D, bool FP8, bool SPLITP, class Source, class Sees, class Queries>
__device__ __forceinline__ void attend_rows(Rows<D, FP8, SPLITP>& R, lds_ptr lds, int key0, int key1, const Source& src,
                                            const Sees& sees, const Queries& queries, int wave, int lane) {
    using L = RowsLds<D, FP8>;
    constexpr int ROW = Tile<D, FP8>::ROW, LOADS = Tile<D, FP8>::LOADS16;
    // waves 0, 1 stage K's rows, 2, 3 V's, 16 each
    const bool is_k = wave < 2;
    const int part = (wave & 1) * 16;
    const Stager<D, FP8> st(lane, is_k ? src.k_stride : src.v_stride);
    const lds_ptr k_ring = lds, v_ring = lds + 2 * L::TILE;
    auto stage = [&](int i, int slot) {
        const int key = key0 + i * KEYS + part;
        if (is_k) st.rows16(src.k_rows(key), k_ring + slot * L::TILE + part * ROW);
        else st.rows16(src.v_rows(key), v_ring + slot * L::TILE + part * ROW);
    };
    if (key0 >= key1) return;
    const int n = (key1 - key0 + KEYS - 1) / KEYS;
    stage(0, 0);
    queries();
    R.queries_ready();
    auto step = [&](int i, int slot, auto partly) {
        constexpr bool PARTLY = decltype(partly)::value;
        const int key = key0 + i * KEYS;
        const lds_ptr k = k_ring + slot * L::TILE, v = v_ring + slot * L::TILE;
        auto* flags = (__attribute__((address_space(3))) uint32_t*)(lds + L::FLAGS) + (i & 1) * 4;
        wait_vm<0>();
        if (PARTLY) {
            const uint32_t rows = is_k ? 0u : rows_not_finite<D, FP8, LOADS>(v + part * ROW, lane) << part;
            if (lane == 0) flags[wave] = rows;
        }
        lds_barrier();
        stage(i + 1, slot ^ 1);
        uint32_t bad = 0;
        bool some = true;
        uint64_t seen = 0;
        if (PARTLY) {
            some = key < sees.none_from();
            bad = __builtin_amdgcn_readfirstlane(flags[2] | flags[3]);
            seen = sees.seen(key);
        }
        v16f s;
        if (some) R.template weights<PARTLY>(k, seen, s);
        if (PARTLY && bad) {
            if (some) R.add_not_finite(v, bad, seen);
            lds_barrier();
            if (!is_k) rows_made_finite<D, FP8, LOADS>(v + part * ROW, lane);
            lds_barrier();
        }
        if (some) R.values(v, s);
    };
    const int clean = sees.all_before() - key0 < 0 ? 0 : (sees.all_before() - key0) / KEYS;
    int i = 0;
    for (const int whole = (clean < n ? clean : n) - 2; i <= whole; i += 2) {       // by two: the slots' places are constants
        step(i, 0, std::false_type{});
        step(i + 1, 1, std::false_type{});
    }
    for (; i < n; ++i) step(i, i & 1, std::true_type{});
    wait_vm<0>();                                        // nothing may land in LDS after the workgroup has gone
}

}  // namespace attn
}  // namespace nq
