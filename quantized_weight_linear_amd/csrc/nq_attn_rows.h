// The workgroup form with many query rows: NW waves with 32 QB rows each walk
// the keys together, 64 at a time.  Every K and V tile is loaded into LDS once
// per workgroup, two tiles deep: the loads of the next tile are issued when
// the current one is complete and land while it is computed on.
#pragma once

#include "nq_attn_core.h"

namespace nq {
namespace attn {

constexpr int KEYS = 64;        // keys a tile

template <int D, bool FP8, int NW>
struct RowsLds {
    static constexpr int TILE = KEYS * Tile<D, FP8>::ROW;
    static constexpr int FLAGS = 4 * TILE;               // [2] tiles x NW words: a value that is not finite was staged
    static constexpr int BYTES = FLAGS + 2 * NW * 4;
};

// Source: k_rows(key) / v_rows(key) give the descriptor of 16 keys from a
// 16-aligned key on (keys past the last one are outside it), k_stride /
// v_stride the bytes between rows.
// Sees: all_before() = every row of the workgroup sees all keys below it;
// seen(b, key) = the 64 keys from `key` on as bits, for this lane's row of
// block b.
template <int D, int QB, int KB, bool FP8, bool SPLITP, int NW, class Source, class Sees>
__device__ __forceinline__ void attend_rows(Rows<D, QB, FP8, SPLITP>& R, lds_ptr lds, int key0, int key1,
                                            const Source& src, const Sees& sees, int wave, int lane) {
    using L = RowsLds<D, FP8, NW>;
    constexpr int GROUPS = 2 * KEYS / 16;                // groups of 16 rows to stage: 4 of K, 4 of V
    const Stager<D, FP8> st(lane);
    auto flags = [&](int buf) { return (__attribute__((address_space(3))) uint32_t*)(lds + L::FLAGS) + buf * NW; };
    auto stage = [&](int key, int buf) {
        const lds_ptr k = lds + buf * 2 * L::TILE, v = k + L::TILE;
#pragma unroll
        for (int i = 0; i < GROUPS / NW; ++i) {
            const int g = wave + NW * i, part = (g & 3) * 16;
            if (g < 4) st.rows16(src.k_rows(key + part), src.k_stride, k + part * Tile<D, FP8>::ROW);
            else st.rows16(src.v_rows(key + part), src.v_stride, v + part * Tile<D, FP8>::ROW);
        }
    };
    if (key0 < key1) stage(key0, 0);
    int buf = 0;
    for (int key = key0; key < key1; key += KEYS, buf ^= 1) {
        const lds_ptr k = lds + buf * 2 * L::TILE, v = k + L::TILE;
        const bool partly = key + KEYS > sees.all_before();
        wait_vm<0>();
        if (partly) {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < GROUPS / NW; ++i) {
                const int g = wave + NW * i;
                if (g >= 4) bad |= rows16_not_finite<D, FP8>(v + (g & 3) * 16 * Tile<D, FP8>::ROW, lane);
            }
            if (lane == 0) flags(buf)[wave] = bad;
        }
        __syncthreads();
        if (key + KEYS < key1) stage(key + KEYS, buf ^ 1);
#pragma unroll
        for (int sub = 0; sub < KEYS / (32 * KB); ++sub) {
            const lds_cptr ks = k + sub * KB * 32 * Tile<D, FP8>::ROW, vs = v + sub * KB * 32 * Tile<D, FP8>::ROW;
            v16f s[QB][KB];
            R.template logits<KB>(ks, s);
            uint64_t seen[QB];
            if (partly) {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    seen[b] = sees.seen(b, key) >> (sub * KB * 32 & 63);
                    R.template hide<KB>(s[b], seen[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < QB; ++b) R.template softmax<KB>(b, s[b]);
            bool bad = false;
            if (partly) {
#pragma unroll
                for (int w = 0; w < NW; ++w) bad |= flags(buf)[w] != 0;
            }
            if (bad) R.template values_one_by_one<KB>(vs, s, seen);
            else R.template values<KB>(vs, s);
        }
    }
}

// Bits below n (0 .. 64 and beyond either end).
__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

}  // namespace attn
}  // namespace nq
