// The workgroup form with up to 32 query rows: four waves take different keys
// of the same rows, every fourth tile of 32, each through LDS of its own
// without barriers, and join at the end.  Bound by HBM: four contexts of
// 71494 to 131000 keys, 24 / 4 heads of 256, BF16, up to 4 drafts, 281 us, 5.9
// TB/s of keys and values; by latency where they are few: 701 keys 16.5 us, a
// prompt of 167 tokens 12.6 us.
#pragma once

#include "nq_attn_rows.h"

namespace nq {
namespace attn {

// A ring of RING tiles a wave; K and V of a tile are waited for separately,
// and each slot is loaded again as soon as it has been read.
constexpr int KEY_WAVES = 4;

template <int D, bool FP8>
struct KeysLds {
    static constexpr int TILE = 32 * Tile<D, FP8>::ROW;
    static constexpr int RING = TILE >= 8192 ? 1 : TILE >= 4096 ? 2 : 4;
    static constexpr int WAVE = 2 * RING * TILE;                    // 16 KiB (BF16 rows of 256: 32 KiB)
    static constexpr int PITCH = D + 4;                             // floats a row of the waves' results at the end
    static constexpr int JOIN = KEY_WAVES * 32 * PITCH * 4;
    static constexpr int BYTES = KEY_WAVES * WAVE > JOIN ? KEY_WAVES * WAVE : JOIN;
};

// Source, Sees and Queries as for attend_rows (keys from key1 on are outside
// the source's descriptors).  emit(row, column, x, r, l): four neighbouring
// columns of a row's sum of p v, its reference in log2 units and its sum of p;
// once for each of the first `rows` rows and every fourth column.
template <int D, bool FP8, bool SPLITP, class Source, class Sees, class Queries, class Emit>
__device__ __forceinline__ void attend_keys(Rows<D, FP8, SPLITP>& R, unsigned char* smem, int key0, int key1, int rows,
                                            const Source& src, const Sees& sees, const Queries& queries, const Emit& emit,
                                            int wave, int lane) {
    using L = KeysLds<D, FP8>;
    constexpr int LOADS = 2 * Tile<D, FP8>::LOADS16, LATER = (2 * L::RING - 1) * LOADS, STEP = KEY_WAVES * 32;
    const Stager<D, FP8> st_k(lane, src.k_stride), st_v(lane, src.v_stride);
    const lds_ptr mine = (lds_ptr)smem + wave * L::WAVE;
    auto load_k = [&](int key, int slot) {
        st_k.rows16(src.k_rows(key), mine + slot * 2 * L::TILE);
        st_k.rows16(src.k_rows(key + 16), mine + slot * 2 * L::TILE + L::TILE / 2);
    };
    auto load_v = [&](int key, int slot) {
        st_v.rows16(src.v_rows(key), mine + slot * 2 * L::TILE + L::TILE);
        st_v.rows16(src.v_rows(key + 16), mine + slot * 2 * L::TILE + L::TILE + L::TILE / 2);
    };
    const int from = key0 + wave * 32;
#pragma unroll
    for (int i = 0; i < L::RING; ++i) {
        load_k(from + i * STEP, i);
        load_v(from + i * STEP, i);
    }
    queries();
    R.queries_ready();
    auto step = [&](int key, int slot, auto partly) {
        constexpr bool PARTLY = decltype(partly)::value;
        const lds_ptr k = mine + slot * 2 * L::TILE, v = k + L::TILE;
        v16f x;
        uint64_t seen = 0;
        if (PARTLY) seen = sees.seen(key);
        wait_vm<LATER>();
        R.template weights<PARTLY>(k, seen, x);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");          // K is read: its slot is free
        load_k(key + L::RING * STEP, slot);
        wait_vm<LATER>();
        if (PARTLY) {
            if (const uint32_t bad = rows_not_finite<D, FP8, LOADS>(v, lane)) {
                R.add_not_finite(v, bad, seen);
                rows_made_finite<D, FP8, LOADS>(v, lane);
            }
        }
        R.values(v, x);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load_v(key + L::RING * STEP, slot);
    };
    const int clean = (sees.all_before() < key1 ? sees.all_before() : key1) - 32;
    int key = from, slot = 0;
    for (; key <= clean; key += STEP) {
        step(key, slot, std::false_type{});
        slot = slot + 1 == L::RING ? 0 : slot + 1;
    }
    for (; key < key1; key += STEP) {
        step(key, slot, std::true_type{});
        slot = slot + 1 == L::RING ? 0 : slot + 1;
    }
    wait_vm<0>();
    __syncthreads();
    // The waves' results go to LDS, and the workgroup's threads finish the rows.
    float* join = reinterpret_cast<float*>(smem);
    const float l = halves_sum(R.l);
    float* at = join + (wave * 32 + (lane & 31)) * L::PITCH;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<v4f*>(at + R.column(d, e)) =
                v4f{R.o[d][4 * e], R.o[d][4 * e + 1], R.o[d][4 * e + 2], R.o[d][4 * e + 3]};
    if (lane < 32) {
        at[D] = R.m == -INFINITY ? -INFINITY : R.reference();
        at[D + 1] = l;
    }
    __syncthreads();
    constexpr int LANES = D / 4;                        // threads a row
    for (int i = threadIdx.x / LANES; i < rows; i += KEY_WAVES * 64 / LANES) {
        const int col = threadIdx.x % LANES * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < KEY_WAVES; ++w) top = max2(top, join[(w * 32 + i) * L::PITCH + D]);
        v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < KEY_WAVES; ++w) {
            const float* p = join + (w * 32 + i) * L::PITCH;
            const float lw = p[D + 1];
            // a wave without weights has neither sum nor outputs (which may be infinity or NaN there)
            const float f = lw == 0.f ? 0.f : __builtin_amdgcn_exp2f(p[D] == -INFINITY ? 0.f : p[D] - top);
            const v4f y = *reinterpret_cast<const v4f*>(p + col);
            sum += lw * f;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += lw == 0.f ? 0.f : y[j] * f;
        }
        emit(i, col, x, top == -INFINITY ? 0.f : top, sum);
    }
}

}  // namespace attn
}  // namespace nq
