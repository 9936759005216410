// E4M3 activations times E4M3 weights with block scales (nq_gemm_fp8_b128):
//
//   y[m][n] = sum_g (a_scale[m][g] w_scale[n / 128][g]) P[m][n][g],
//   P[m][n][g] = sum over the 128 columns k of block g of a[m][k] w[n][k]
//
// P is formed on the matrix cores, each block from zero, and the blocks are
// summed in FP32.  Weight rows are the rows of the products and tokens their
// columns, so that a lane has one token: the two scales make one factor a lane
// for all rows it holds, and a block costs one FMA an output.
//
// Two arithmetics.  BF16 outputs take the FP8 matrix instructions, which cut
// products at 2^-13 of the largest of eight (1.3e-5 to 1.8e-5 off a block's exact
// sum, Frobenius, and up to 8.5e-4 of a block's sum of sizes where few products
// outweigh the others; a BF16 output's own rounding is 1.7e-3, Frobenius).  FP32 outputs keep to the 1e-5 of this
// library's FP32 results: codes become BF16, exactly, as operands are read,
// and go through the BF16 instructions at half the rate.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "nq_attn_launch.h"
#include "nq_device.h"
#include "nq_launch.h"
#include "nq_layer_launch.h"

namespace nq {
namespace {

constexpr int BLOCK = 128;               // columns of a scale
constexpr int64_t MOST_BLOCKS = (int64_t)1 << 24;        // of 256 threads a launch (the callers' limits give no more of 64 rows)

struct B128Args {
    const uint8_t* a;
    const float* as;
    const uint8_t* w;
    const float* ws;
    int m, n, k, groups;
    int per;                             // blocks a workgroup, of the tile kernels
    void* y;
};

__device__ __forceinline__ v8i join(v4u x, v4u y) {
    return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
}
__device__ __forceinline__ v8bf eight_bf16(uint32_t x, uint32_t y) {
    return __builtin_bit_cast(v8bf, v4u{e4m3x2_to_bf16x2<false>(x, 1.0f), e4m3x2_to_bf16x2<true>(x, 1.0f),
                                        e4m3x2_to_bf16x2<false>(y, 1.0f), e4m3x2_to_bf16x2<true>(y, 1.0f)});
}

// p[i], the same in all lanes, by a scalar load (no wait for vector loads in flight).
typedef __attribute__((address_space(4))) const float* uniform_floats;
__device__ __forceinline__ float uniform(const float* p, int64_t i) { return ((uniform_floats)(uintptr_t)p)[i]; }

// Two values as BF16, rounded as f32_to_bf16_rne does.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) { return f32_to_bf16_rne(a) | f32_to_bf16_rne(b) << 16; }

template <bool BF16OUT>
__device__ __forceinline__ void store(void* y, int64_t at, float x) {
    if constexpr (BF16OUT) reinterpret_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16_rne(x);
    else reinterpret_cast<float*>(y)[at] = x;
}

typedef __attribute__((address_space(3))) unsigned char* lds_ptr;
constexpr int PAST = 0x40000000;         // an offset outside every buffer here: reads as zeros

__device__ __forceinline__ v4i buffer(const void* base, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    return v4i{(int)(uint32_t)at, (int)(uint32_t)(at >> 32) & 0xFFFF, (int)bytes, 0x00027000};
}
// 16 (4) bytes a lane into LDS at dst + 16 (4) lane, no registers between;
// whoever reads them waits for the loads himself.
__device__ __forceinline__ void lds_load16(v4i r, int off, lds_ptr dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"((uint32_t)(uintptr_t)dst), "v"(off), "s"(r) : "memory", "m0");
}
template <bool STREAM>                   // bytes that are read once: past the caches
__device__ __forceinline__ void lds_load16_as(v4i r, int off, lds_ptr dst) {
    if constexpr (STREAM)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                     ::"s"((uint32_t)(uintptr_t)dst), "v"(off), "s"(r) : "memory", "m0");
    else lds_load16(r, off, dst);
}
__device__ __forceinline__ void lds_load4(v4i r, int off, lds_ptr dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"((uint32_t)(uintptr_t)dst), "v"(off), "s"(r) : "memory", "m0");
}

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn; each XCD
// takes a contiguous range of tiles, in bands of BAND token tiles, tokens first,
// so that those that share an L2 read few different rows (8192 x 8192 x 8192:
// 555 us without bands, 495 with).
constexpr int BAND = 8;
struct Place {
    int m, n;
    __device__ __forceinline__ Place(int tiles_m, int tiles_n) {
        const int each = (int)gridDim.x / 8, more = (int)gridDim.x % 8, xcd = blockIdx.x % 8;
        const int tile = xcd * each + min(xcd, more) + blockIdx.x / 8;
        const int band = tile / (BAND * tiles_n), high = min(BAND, tiles_m - band * BAND), inside = tile - band * BAND * tiles_n;
        m = band * BAND + inside % high;
        n = inside / high;
    }
};

// ---- few tokens: every wave streams its own blocks ------------------------------------------------------------------

// A workgroup has 16 RF weight rows and up to 8 TL tokens, and all blocks of 128
// columns or a run of them; its waves split these between them and join in LDS, in
// the order of the waves.
// Each wave streams its blocks (weights, tokens and the tokens' scales) through a ring of RING
// slots of its own in LDS, without barriers: from memory straight into LDS, since
// there eight neighbouring lanes read a row's 128 bytes, where operand order
// (neighbouring lanes on different rows) asks for four times the requests.
// Bound by HBM: the weights once; the tokens come from L2, once for 16 RF rows.
//   The scales of a token's blocks lie side by side: they come four at a time,
// 16 bytes a token, in windows of four blocks (two slots of their own).
template <int TL, int RF, int WAVES, int RING>
struct Few {
    static constexpr int NT = (TL + 1) / 2;
    static constexpr int TOKENS = 16 * RF * BLOCK, SLOT = TOKENS + TL * 1024;    // the tokens' place in a slot
    static constexpr int WINDOWS = RING * SLOT, WAVE = WINDOWS + 2 * 1024;
    static constexpr int LOADS = 2 * RF + TL;
    // Loads that may be on their way when block v of a window is needed: those of the RING - 1 blocks after it.
    static constexpr int later(int v) {
        int n = LOADS * (RING - 1);
        for (int d = 1; d < RING; ++d) n += (v + d) % 4 == 0;
        return n;
    }
    static constexpr int JOIN = WAVES * RF * NT * 1024;
    // (the last 16 tokens' operands may reach 8 rows past the last slot's tokens)
    static constexpr int STREAM = WAVES * WAVE, LDS = STREAM > JOIN ? STREAM : JOIN;
    static_assert(TL <= 8 && LOADS * (RING - 1) + 1 < 64 && RING <= 4, "");
};

template <int TL, int RF, int WAVES, int RING, bool ONCE, bool FP8, bool BF16OUT>
__global__ __launch_bounds__(WAVES * 64) void b128_few_kernel(B128Args a) {
    using L = Few<TL, RF, WAVES, RING>;
    constexpr int NT = L::NT;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const lds_ptr mine = (lds_ptr)smem + wave * L::WAVE;
    const Place place((a.m + 8 * TL - 1) / (8 * TL), (a.n + 16 * RF - 1) / (16 * RF));
    const int n0 = place.n * 16 * RF, m0 = place.m * 8 * TL;
    const int rows_w = min(a.n - n0, 16 * RF), rows_a = min(a.m - m0, 8 * TL);
    const v4i buf_w = buffer(a.w + (int64_t)n0 * a.k, (int64_t)rows_w * a.k), buf_a = buffer(a.a + (int64_t)m0 * a.k, (int64_t)rows_a * a.k);
    const v4i buf_s = buffer(a.as + (int64_t)m0 * a.groups, (int64_t)rows_a * a.groups * 4);
    const int first_block = blockIdx.y * a.per, blocks = max(0, min(a.per, a.groups - first_block));    // this workgroup's blocks
    const int per = (blocks + WAVES - 1) / WAVES, from = first_block + min(wave * per, blocks), upto = first_block + min((wave + 1) * per, blocks);
    // Load i: rows 8 i .. 8 i + 7 of a panel.
    int col[2], off[2];                  // the lane's piece, and its place, for even and odd i
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        col[p] = 16 * ((lane & 7) ^ ((4 * p + (lane >> 4)) & 7));
        off[p] = (lane >> 3) * a.k + col[p];
    }
    // A window never reaches past its row: the last one starts earlier.  Rows of
    // fewer than four scales (a block a wave) come a scale a token.
    const bool narrow = a.groups < 4;
    const int scale_off = lane * a.groups * 4, scale_step = narrow ? 4 : 16;
    auto window = [&](int s) { return max(0, min(s, a.groups - 4)); };
    auto issue = [&](int s, int slot, int v) {
        const lds_ptr at = mine + slot * L::SLOT;
        const int left = s < upto ? a.k - s * BLOCK : 0;                 // columns from this block on
        const int here[2] = {col[0] < left ? off[0] + s * BLOCK : PAST, col[1] < left ? off[1] + s * BLOCK : PAST};
        if (v == 0) {
            const lds_ptr to = mine + L::WINDOWS + ((s - from) / 4 & 1) * 1024;
            const int from_row = s < upto ? scale_off + (narrow ? s : window(s)) * 4 : PAST;
            if (narrow) lds_load4(buf_s, from_row, to);
            else lds_load16(buf_s, from_row, to);
        }
#pragma unroll
        for (int i = 0; i < 2 * RF; ++i) lds_load16_as<ONCE>(buf_w, here[i & 1] + 8 * i * a.k, at + i * 1024);
#pragma unroll
        for (int i = 0; i < TL; ++i) lds_load16(buf_a, here[i & 1] + 8 * i * a.k, at + L::TOKENS + i * 1024);
    };
    const int n = lane & 15, g = lane >> 4;
    const int first = n * BLOCK + ((g ^ (n >> 1)) << 4);                 // of this lane's pieces g and 4 + g of its row
    auto read = [&](lds_ptr row, v4u (&x)[2]) {
        x[0] = *(__attribute__((address_space(3))) const v4u*)(row + first);
        x[1] = *(__attribute__((address_space(3))) const v4u*)(row + (first ^ 64));
    };
    const float* ws = a.ws + (int64_t)(n0 / BLOCK) * a.groups;           // (16 RF rows lie in one block of 128)
    v4f acc[RF][NT];
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < RING; ++d) issue(from + d, d, d % 4);
    int slot = 0;
    auto block = [&](int s, auto nth) {
        constexpr int V = decltype(nth)::value;                          // its number in the window
        const lds_ptr at = mine + slot * L::SLOT;
        const lds_ptr scales = mine + L::WINDOWS + ((s - from) / 4 & 1) * 1024 + (narrow ? 0 : s - window(s - V)) * 4;
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L::later(V)) : "memory");
        v4u w[RF][2], x[NT][2];
        float f[NT];
#pragma unroll
        for (int i = 0; i < RF; ++i) read(at + 16 * i * BLOCK, w[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            read(at + L::TOKENS + 16 * t * BLOCK, x[t]);
            f[t] = *(__attribute__((address_space(3))) const float*)(scales + (16 * t + n) * scale_step);
        }
        const float by = uniform(ws, s);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");               // the slot is read
        issue(s + RING, slot, (V + RING) % 4);
        slot = slot + 1 == RING ? 0 : slot + 1;
        v8bf wide[RF][FP8 ? 1 : 4];
        if constexpr (!FP8) {
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h) wide[i][h] = eight_bf16(w[i][h >> 1][2 * (h & 1)], w[i][h >> 1][2 * (h & 1) + 1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            v4f p[RF];
#pragma unroll
            for (int i = 0; i < RF; ++i) p[i] = v4f{0.f, 0.f, 0.f, 0.f};
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < RF; ++i)
                    p[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w[i][0], w[i][1]), join(x[t][0], x[t][1]), p[i], 0, 0, 0,
                                                                            0, 0, 0);
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const v8bf y = eight_bf16(x[t][h >> 1][2 * (h & 1)], x[t][h >> 1][2 * (h & 1) + 1]);
#pragma unroll
                    for (int i = 0; i < RF; ++i) p[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[i][h], y, p[i], 0, 0, 0);
                }
            }
            const float to = f[t] * by;
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(p[i][e], to, acc[i][t][e]);
        }
    };
    for (int s = from; s < upto; s += 4) {
        block(s, std::integral_constant<int, 0>{});
        if (s + 1 < upto) block(s + 1, std::integral_constant<int, 1>{});
        if (s + 2 < upto) block(s + 2, std::integral_constant<int, 2>{});
        if (s + 3 < upto) block(s + 3, std::integral_constant<int, 3>{});
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");                     // nothing is on its way into LDS any more
    __syncthreads();
    char* const y = (char*)a.y + (int64_t)blockIdx.y * a.m * a.n * 4;    // (several workgroups an output: FP32 parts, one after another)
    auto* part = (__attribute__((address_space(3))) v4f*)smem;           // [WAVES][RF NT][64]
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[(wave * RF * NT + i * NT + t) * 64 + lane] = acc[i][t];
    __syncthreads();
    for (int c = wave; c < RF * NT; c += WAVES) {
        v4f sum = part[c * 64 + lane];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) {
            const v4f z = part[(v * RF * NT + c) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += z[e];
        }
        const int t = c % NT * 16 + n, row = n0 + c / NT * 16 + 4 * g;
        if (t >= rows_a) continue;
        const int64_t to = (int64_t)(m0 + t) * a.n + row;
        if (a.n % 4 == 0) {
            if (row >= a.n) continue;
            if constexpr (BF16OUT) *reinterpret_cast<v2u*>((uint16_t*)y + to) = v2u{bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
            else *reinterpret_cast<v4f*>((float*)y + to) = sum;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row + e < a.n) store<BF16OUT>(y, to + e, sum[e]);
        }
    }
}

template <int TL, int RF, int WAVES, int RING, bool ONCE, bool FP8, bool BF16OUT>
hipError_t go_few(const B128Args& a, int splits, hipStream_t stream) {
    using L = Few<TL, RF, WAVES, RING>;
    auto kernel = b128_few_kernel<TL, RF, WAVES, RING, ONCE, FP8, BF16OUT>;
    static LdsLimit limit;
    if (hipError_t e = limit.raise((const void*)kernel, L::LDS); e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)(a.n + 16 * RF - 1) / (16 * RF)) * ((a.m + 8 * TL - 1) / (8 * TL));
    kernel<<<dim3((unsigned)tiles, (unsigned)splits), WAVES * 64, L::LDS, stream>>>(a);
    return hipGetLastError();
}

// ---- many tokens: tiles through LDS ---------------------------------------------------------------------------------

// WR x WT waves of FI x FT products of 16 x 16: a workgroup has 16 WR FI weight
// rows and 16 WT FT tokens.  A stage is one block of 128 columns of both, in two
// slots: row r of a panel at byte 128 r, its 16-byte piece c in place
// c ^ (r / 2 % 8), so that operand reads (16 rows, one piece each) cover all
// banks once.  The tokens' scales come in windows of four blocks, 16 bytes a
// token (one at a time, each load asks for 64 lines: 173 us instead of 160 for
// 1792 x 17408 x 5120), in two slots of their own.
template <int WR, int WT, int FI, int FT>
struct Tile {
    static constexpr int WAVES = WR * WT, ROWS = 16 * WR * FI, TOKENS = 16 * WT * FT;
    static constexpr int LOADS_W = ROWS / 8 / WAVES, LOADS_T = TOKENS / 8 / WAVES;          // of 8 rows, a wave
    static constexpr int STAGE = (ROWS + TOKENS) * BLOCK;
    static constexpr int WINDOWS = 2 * STAGE, WINDOW = TOKENS * 16, LDS = WINDOWS + 2 * WINDOW;
    static_assert(ROWS % (8 * WAVES) == 0 && TOKENS % (8 * WAVES) == 0 && TOKENS % 64 == 0 && TOKENS / 64 <= WAVES && FT % 2 == 0, "");
    static_assert(BLOCK % (16 * FI) == 0, "a wave's rows lie in one block of the weights' scales");
};

// A wave's outputs in LDS on their way out, a row of them a token.
template <int FI, int FT, bool BF16OUT>
struct Output {
    static constexpr int SIZE = BF16OUT ? 2 : 4, EACH = 16 / SIZE, ROWS = 16 * FI, TOKENS = 16 * FT, PIECES = ROWS / EACH;
    static constexpr int PITCH = ROWS * SIZE + 16, BYTES = TOKENS * PITCH;
};

// The products run some steps ahead of the rescales, so that no rescale waits for
// its product.  Operands are read a column of products ahead, also across stages.
template <int WR, int WT, int FI, int FT, bool FP8, bool BF16OUT, bool NARROW>
__global__ __launch_bounds__(WR * WT * 64, 2) void b128_tile_kernel(B128Args a) {
    using T = Tile<WR, WT, FI, FT>;
    extern __shared__ __align__(16) unsigned char smem[];
    const lds_ptr lds = (lds_ptr)smem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place place((a.m + T::TOKENS - 1) / T::TOKENS, (a.n + T::ROWS - 1) / T::ROWS);
    const int m0 = place.m * T::TOKENS, n0 = place.n * T::ROWS;
    const int rows_w = min(a.n - n0, T::ROWS), rows_a = min(a.m - m0, T::TOKENS);
    const int from = blockIdx.y * a.per, upto = min(from + a.per, a.groups);     // this workgroup's blocks

    const v4i buf_w = buffer(a.w + (int64_t)n0 * a.k, (int64_t)rows_w * a.k), buf_a = buffer(a.a + (int64_t)m0 * a.k, (int64_t)rows_a * a.k);
    const v4i buf_s = buffer(a.as + (int64_t)m0 * a.groups, (int64_t)rows_a * a.groups * 4);
    // A window never reaches past its row: the last one starts earlier.  NARROW: rows
    // of fewer than four scales come at once, 4 bytes a token and block.
    auto window = [&](int s) { return min(s - ((s - from) & 3), a.groups - 4); };
    auto issue_window = [&](int s) {     // that of blocks s .. s + 3
        if (wave >= T::TOKENS / 64 || s >= upto) return;
        const int row = (64 * wave + lane) * a.groups;
        if constexpr (NARROW)
            for (int g = 0; g < a.groups; ++g) lds_load4(buf_s, (row + g) * 4, lds + T::WINDOWS + g * T::TOKENS * 4 + wave * 256);
        else lds_load16(buf_s, (row + window(s)) * 4, lds + T::WINDOWS + ((s - from) / 4 & 1) * T::WINDOW + wave * 1024);
    };
    auto scales_of = [&](int s) {
        return T::WINDOWS + (NARROW ? s * T::TOKENS * 4 : ((s - from) / 4 & 1) * T::WINDOW + (s - window(s)) * 4);
    };

    // Load i of this wave: rows 8 q .. 8 q + 7 of a panel, q = i WAVES + wave.  No
    // branches: past the last block, and of what lies past the last column, nothing
    // is read and zeros arrive.
    const int col = 16 * ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)), off = (8 * wave + (lane >> 3)) * a.k + col;
    auto issue = [&](v4i buf, int panel, int s, int i) {
        const int at = s < upto && col < a.k - s * BLOCK ? off : PAST;
        lds_load16(buf, at + (8 * T::WAVES * i * a.k + s * BLOCK), lds + ((s - from) & 1) * T::STAGE + panel + (i * T::WAVES + wave) * 1024);
    };
    auto issue_w = [&](int s, int i) { issue(buf_w, 0, s, i); };
    auto issue_t = [&](int s, int i) { issue(buf_a, T::ROWS * BLOCK, s, i); };

    const int wr = wave % WR * FI * 16, wt = wave / WR * FT * 16;
    const int n = lane & 15, g = lane >> 4;
    const int first = n * BLOCK + ((g ^ (n >> 1)) << 4);                 // of this lane's pieces g and 4 + g of its row
    auto read = [&](lds_ptr row, v4u (&x)[2]) {
        x[0] = *(__attribute__((address_space(3))) const v4u*)(row + first);
        x[1] = *(__attribute__((address_space(3))) const v4u*)(row + (first ^ 64));
    };
    auto read_scale = [&](int at, int j) { return *(__attribute__((address_space(3))) const float*)(lds + at + (wt + 16 * j + n) * (NARROW ? 4 : 16)); };
    auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    v4f acc[FI][FT];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto rescale = [&](v4f& c, const v4f& x, float by) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = fmaf(x[e], by, c[e]);
    };
    const float* ws = a.ws + (int64_t)min((n0 + wr) / BLOCK, (a.n - 1) / BLOCK) * a.groups;
    // A stage has Q steps of one product.  Its weight rows are in registers once
    // the first FI steps are done: from a barrier there on the weights of the stage
    // after the next go out, with almost two stages to arrive (weights come from
    // memory more often than tokens do; with all loads after step TURN 1792 x 17408 x
    // 5120 took 171 us instead of 151, 1024 x 7168 x 5120 57 instead of 48, and half
    // the tokens' loads from a third barrier on gained nothing).  The reads of its last
    // tokens are out before step TURN (they are read one column ahead, two for FP32
    // outputs): at the barrier there they are done, the next stage has arrived, and
    // the tokens of the one after it go out.  One load in GAP steps (all at once, the
    // waves would queue at the address unit with no products on their way).
    constexpr int Q = FI * FT, TURN = FP8 ? Q - FI - 2 : Q - 2 * FI, GAP = FP8 && FT > 4 ? 2 : 1;
    static_assert(FI + (T::LOADS_W - 1) * GAP < TURN && TURN + T::LOADS_T <= Q, "");
    auto barriers = [&](int q) {
        if (q == FI) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        if (q == TURN) {                 // (all but the weights of the stage after the next have arrived)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(T::LOADS_W) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
    };
    auto issue_at = [&](int s, int q) {
#pragma unroll
        for (int i = 0; i < T::LOADS_W; ++i)
            if (q == FI + i * GAP) issue_w(s + 2, i);
#pragma unroll
        for (int i = 0; i < T::LOADS_T; ++i)
            if (q == TURN + i) issue_t(s + 2, i);
    };
    if (from < upto) {
        issue_window(from);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < T::LOADS_W; ++i) issue_w(from + s, i);
#pragma unroll
            for (int i = 0; i < T::LOADS_T; ++i) issue_t(from + s, i);
            if (s == 0) arrived();
        }
    }
    const lds_ptr tokens = lds + (T::ROWS + wt) * BLOCK, rows = lds + wr * BLOCK;
    if constexpr (FP8) {
        constexpr int LAG = 3;
        v4f p[LAG + 1];
#pragma unroll
        for (int i = 0; i <= LAG; ++i) p[i] = v4f{0.f, 0.f, 0.f, 0.f};
        v4u w[2][FI][2], t[2][2];                                        // of even and odd stages; of even and odd columns
        float raw = 0.f, f = 0.f, f_last = 0.f;
        if (from < upto) {
#pragma unroll
            for (int i = 0; i < FI; ++i) read(rows + 16 * i * BLOCK, w[0][i]);
            read(tokens, t[0]);
            raw = read_scale(scales_of(from), 0);
        }
        auto stage = [&](int s, auto odd) {
            constexpr int ODD = decltype(odd)::value;
            int here = ODD * T::STAGE, next = T::STAGE - here;
            asm volatile("" : "+s"(here), "+s"(next));                   // (addresses are formed as they are needed, not all kept in registers)
            const float by = uniform(ws, s);
            const int scales = scales_of(s), scales_next = scales_of(min(s + 1, upto - 1));
            if (((s + 2 - from) & 3) == 0) issue_window(s + 2);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = q % FI, j = q / FI;
                barriers(q);
                if (i == 0) {
                    f_last = f;
                    f = raw * by;
                    const int slot = j + 1 < FT ? here : next;           // (past the last stage: bytes that no one uses)
                    read(tokens + slot + 16 * ((j + 1) % FT) * BLOCK, t[(j + 1) & 1]);
                    raw = read_scale(j + 1 < FT ? scales : scales_next, (j + 1) % FT);
                }
                if (q >= TURN && q < TURN + FI) read(rows + next + 16 * (q - TURN) * BLOCK, w[1 - ODD][q - TURN]);
                __builtin_amdgcn_sched_barrier(0);
                p[q % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    join(w[ODD][i][0], w[ODD][i][1]), join(t[j & 1][0], t[j & 1][1]), v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                const int e = (q + Q - LAG) % Q;
                rescale(acc[e % FI][e / FI], p[(q + 1) % (LAG + 1)], i < LAG ? f_last : f);
                asm volatile("" : "+v"(acc[e % FI][e / FI]));            // (here, not beside its next use)
                issue_at(s, q);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        static_assert(FI == 4 && FT % 2 == 0, "");
        for (int s = from; s < upto; s += 2) {
            stage(s, std::integral_constant<int, 0>{});
            if (s + 1 < upto) stage(s + 1, std::integral_constant<int, 1>{});
        }
#pragma unroll
        for (int q = Q - LAG; q < Q; ++q) rescale(acc[q % FI][q / FI], p[q % (LAG + 1)], f);
    } else {
        // Codes become BF16 a column ahead of their products, a quarter a step, and
        // are read another column before that; a weight row's right after its last
        // use in the stage.
        static_assert(FI == 4 && FT % 2 == 0, "");
        auto wide = [&](const v4u (&x)[2], int e) { return eight_bf16(x[e >> 1][2 * (e & 1)], x[e >> 1][2 * (e & 1) + 1]); };
        v8bf w[FI][4], t[2][4];
        v4u wn[FI][2], tn[2][2];
        v4f last[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        float raw[2], f = 0.f, f_last = 0.f;
        if (from < upto) {
#pragma unroll
            for (int i = 0; i < FI; ++i) {
                read(rows + 16 * i * BLOCK, wn[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = wide(wn[i], e);
            }
            read(tokens, tn[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) t[0][e] = wide(tn[0], e);
            read(tokens + 16 * BLOCK, tn[1]);
            raw[0] = read_scale(scales_of(from), 0);
            raw[1] = read_scale(scales_of(from), 1);
        }
        for (int s = from; s < upto; ++s) {
            const int here = ((s - from) & 1) * T::STAGE, next = T::STAGE - here;
            const float by = uniform(ws, s);
            const int scales = scales_of(s), scales_next = scales_of(min(s + 1, upto - 1));
            if (((s + 2 - from) & 3) == 0) issue_window(s + 2);
#pragma unroll
            for (int q = 0; q < Q; q += 2) {                             // two products at once: neither waits for its own sum
                const int i = q % FI, j = q / FI;
                barriers(q);
                if (i == 0) {
                    f_last = f;
                    f = raw[j & 1] * by;
                    const int slot = j + 2 < FT ? here : next;
                    read(tokens + slot + 16 * ((j + 2) % FT) * BLOCK, tn[j & 1]);
                    raw[j & 1] = read_scale(j + 2 < FT ? scales : scales_next, (j + 2) % FT);
                }
                if (q >= Q - 2 * FI && q < Q - FI) {
                    read(rows + next + 16 * i * BLOCK, wn[i]);
                    read(rows + next + 16 * (i + 1) * BLOCK, wn[i + 1]);
                }
                __builtin_amdgcn_sched_barrier(0);
                v4f x[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i + h][e], t[j & 1][e], x[h], 0, 0, 0);
                        if (j + 1 == FT) w[i + h][e] = wide(wn[i + h], e);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    t[(j + 1) & 1][i + h] = wide(tn[(j + 1) & 1], i + h);
                    const int e = (q + Q - 2 + h) % Q;
                    rescale(acc[e % FI][e / FI], last[h], i == 0 ? f_last : f);
                    last[h] = x[h];
                    issue_at(s, q + h);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) rescale(acc[FI - 2 + h][FT - 1], last[h], f);
    }
    // A lane's outputs lie a token apart: through LDS they become pieces of whole
    // cache lines.  Each wave has a place of its own there, once all have read
    // their last stage and nothing is on its way into it.
    arrived();
    char* const y = (char*)a.y + (int64_t)blockIdx.y * a.m * a.n * 4;    // (several workgroups a tile: FP32 parts, one after another)
    using Out = Output<FI, FT, BF16OUT>;
    const lds_ptr mine = lds + wave * Out::BYTES;
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const lds_ptr to = mine + (16 * j + n) * Out::PITCH + (16 * i + 4 * g) * Out::SIZE;
            const v4f& c = acc[i][j];
            if constexpr (BF16OUT) *(__attribute__((address_space(3))) v2u*)to = v2u{bf16_pair(c[0], c[1]), bf16_pair(c[2], c[3])};
            else *(__attribute__((address_space(3))) v4f*)to = c;
        }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (a.n % Out::EACH == 0) {          // whole 16-byte pieces
#pragma unroll 4
        for (int b = lane; b < Out::TOKENS * Out::PIECES; b += 64) {
            const int m = m0 + wt + b / Out::PIECES, row = n0 + wr + b % Out::PIECES * Out::EACH;
            const v4u x = *(__attribute__((address_space(3))) const v4u*)(mine + b / Out::PIECES * Out::PITCH + b % Out::PIECES * 16);
            if (m < a.m && row < a.n) *reinterpret_cast<v4u*>(y + ((int64_t)m * a.n + row) * Out::SIZE) = x;
        }
    } else {
#pragma unroll 4
        for (int b = lane; b < Out::TOKENS * Out::ROWS; b += 64) {
            const int m = m0 + wt + b / Out::ROWS, row = n0 + wr + b % Out::ROWS;
            const lds_ptr x = mine + b / Out::ROWS * Out::PITCH + b % Out::ROWS * Out::SIZE;
            if (m >= a.m || row >= a.n) continue;
            if constexpr (BF16OUT) reinterpret_cast<uint16_t*>(y)[(int64_t)m * a.n + row] = *(__attribute__((address_space(3))) const uint16_t*)x;
            else reinterpret_cast<float*>(y)[(int64_t)m * a.n + row] = *(__attribute__((address_space(3))) const float*)x;
        }
    }
}

// The parts of each output, added in their order.
template <bool BF16OUT>
__global__ __launch_bounds__(256) void b128_join_kernel(const float* parts, int count, int64_t outputs, void* y) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at + 4 <= outputs && outputs % 4 == 0) {         // (parts stay 16-byte aligned)
        v4f sum = *reinterpret_cast<const v4f*>(parts + at);
        for (int i = 1; i < count; ++i) {
            const v4f z = *reinterpret_cast<const v4f*>(parts + i * outputs + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += z[e];
        }
        if constexpr (BF16OUT) *reinterpret_cast<v2u*>((uint16_t*)y + at) = v2u{bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
        else *reinterpret_cast<v4f*>((float*)y + at) = sum;
        return;
    }
    for (int64_t e = at; e < outputs && e < at + 4; ++e) {
        float sum = parts[e];
        for (int i = 1; i < count; ++i) sum += parts[i * outputs + e];
        store<BF16OUT>(y, e, sum);
    }
}

template <int WR, int WT, int FI, int FT, bool FP8, bool BF16OUT, bool NARROW = false>
hipError_t go_tile(const B128Args& a, int splits, hipStream_t stream) {
    using T = Tile<WR, WT, FI, FT>;
    constexpr int OUT = T::WAVES * Output<FI, FT, BF16OUT>::BYTES, LDS = OUT > T::LDS ? OUT : T::LDS;
    static_assert(LDS <= 160 * 1024, "");
    auto kernel = b128_tile_kernel<WR, WT, FI, FT, FP8, BF16OUT, NARROW>;
    static LdsLimit limit;
    if (hipError_t e = limit.raise((const void*)kernel, LDS); e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)(a.m + T::TOKENS - 1) / T::TOKENS) * ((a.n + T::ROWS - 1) / T::ROWS);
    kernel<<<dim3((unsigned)tiles, (unsigned)splits), T::WAVES * 64, LDS, stream>>>(a);
    return hipGetLastError();
}

struct Plan {
    enum { FEW, SMALL, MID, BIG } form;
    int rows;                            // FEW: blocks of 16 weight rows a workgroup
    int splits;                          // FEW, SMALL: workgroups an output
};

// Up to 64 tokens: FEW, with 16 rows a workgroup while that gives no more
// workgroups than CUs (or for up to 4 tokens, where the tokens' bytes do not
// count), else 32; or K split over the CUs that this leaves idle, with 16 or 64
// rows, where the blocks that a wave saves (nanoseconds each, by rows and tokens)
// are worth the join.  Microseconds unsplit with 16 / 32 rows, FP32, K = 5120: 33
// tokens, N = 2048 7.5 / 8.8, 7168 13.4 / 10.8, 17408 32.7 / 28.3; one token, N =
// 17408 17.0 / 18.2.  Split / not: 5120 x 17408, 64 rows three times, 16 tokens
// 20.4 / 22.4, 33 23.4 / 29.6, 64 27.8 / 39.7; 5120 x 6144, 33 tokens 11.9 / 10.4;
// 256 x 7168, 16 rows four times, 16 tokens 5.7 / 6.0, 64 7.9 / 10.9; 2048 x 5120,
// 16 rows twice, 33 tokens 7.7 / 7.5.
//   More tokens: the form with the least time by what a block of 128 columns
// takes each and what a workgroup takes beside them (nanoseconds, fitted), times
// the rounds in which its workgroups fill the CUs.  Over 125 sizes of 65 .. 16384
// tokens, N 100 .. 17408, K 128 .. 17408, both outputs, it takes a form within 2 % of
// the best one in 230 of 250 cases, and one more than 10 % behind in 10 (200 x 5120 x
// 512 BF16 9.7 for 7.0, 512 x 17408 x 5120 FP32 143 for 111, 1792 x 5120 x 5120 FP32
// 129 for 108).  Measured against each other (us):
//                             FEW 16   32    64   SMALL (splits)    MID    BIG
//   300 x 1024 x 2048          8.1   5.8   7.9   13.5, 11.5 (4)    16.9   27.1
//   96 x 7168 x 5120          28.3  19.3  15.8   30.2, 17.2 (4)    42.5   58.1
//   512 x 5120 x 17408         230   138   110    103, 67 (3)       132    187
//   4800 x 600 x 2896         61.4  40.6  31.6   20.1              25.8   37.9
//   1024 x 7168 x 5120         208   128    95   48.3              45.6   62.8
//   2048 x 7168 x 5120         414   252   185   92.2              91.8   69.3
//   1792 x 5120 x 128, FP32   77.5  51.7  38.3   13.9
//   512 x 5120 x 5120, FP32   75.4  48.5  42.3   45.1, 39.4 (3)
constexpr int64_t MOST_SPLITS = 8, JOIN = 2500, JOIN_RATE = 625, TWO_F32 = 1900;
Plan plan(int64_t m, int64_t n, int64_t k, bool bf16_out, int64_t cus, int64_t most_splits = MOST_SPLITS) {
    auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    const int64_t groups = up(k, BLOCK);
    Plan best{Plan::FEW, 1, 1};
    int64_t least = INT64_MAX;
    auto consider = [&](const Plan& p, int64_t ns) {
        if (ns < least) least = ns, best = p;
    };
    if (m <= 64) {
        const bool small = up(n, 16) <= cus;
        const int64_t tl = m <= 48 ? up(m, 8) : 8;                       // (eights of tokens: the kernel's TL)
        if (small || m <= 4) consider({Plan::FEW, 1, 1}, up(groups, 4) * (150 + 55 * tl));
        else consider({Plan::FEW, 2, 1}, up(groups, 4) * (400 + 85 * tl));
        const int rows = small ? 1 : 4;
        for (int64_t z = 2; z <= most_splits && 4 * z <= groups && up(n, 16 * rows) * z <= cus && (small || m > 4); ++z)
            consider({Plan::FEW, rows, (int)z}, up(up(groups, z), 4) * (small ? 150 + 55 * tl : 1000 + 110 * tl) + 2200 + 400 * z + z * (m * n / 1000));
        return best;
    }
    const int64_t few[3] = {170, 230, 360}, start[3] = {550, 750, 1550};
    for (int i = 0; i < 3; ++i) {
        const int64_t blocks = up(n, 16 << i) * up(m, 64);
        if (i == 2 || blocks < MOST_BLOCKS) consider({Plan::FEW, 1 << i, 1}, (groups * few[i] + start[i]) * up(blocks, cus));
    }
    const int64_t tiles = up(n, 128) * up(m, 128);
    for (int64_t z = 1; z <= most_splits && (z == 1 || 4 * z <= groups); ++z) {
        const int64_t one = bf16_out ? 900 : 1100, two = bf16_out ? 1450 : TWO_F32;         // workgroups on a CU
        const int64_t join = z == 1 ? 0 : JOIN + z * (m * n / JOIN_RATE);                    // its launch, and the parts at 5 TB/s
        const int64_t per = up(groups, z);
        consider({Plan::SMALL, 0, (int)z}, (tiles * z <= cus ? per * one + 1500 : (per * two + 2250) * up(tiles * z, 2 * cus)) + join);
    }
    if (bf16_out && groups >= 4) {       // (fewer scales a row: SMALL alone has that form)
        consider({Plan::MID, 0, 1}, (groups * 1400 + 1700) * up(up(n, 256) * up(m, 128), cus));
        consider({Plan::BIG, 0, 1}, (groups * 2300 + 3400) * up(up(n, 256) * up(m, 256), cus));
    }
    return best;
}

template <int TL, bool FP8, bool BF16OUT>
hipError_t go_few(const B128Args& a, const Plan& p, hipStream_t stream) {
    // Weights that are read once, and fill a good part of the caches, go past them (us through them / past them: one token, 17408 x
    // 5120 18.6 / 17.1; 5120 x 6144, which stays in the last cache from call to call, 7.7 / 8.2).  Not so in the split forms of 64 rows
    // and of the FP8 units: 33 tokens, 5120 x 17408, 64 rows three times 21.2 / 22.3 where three such weights take turns (267 MB, about
    // the last cache's size), 23.3 / 22.6 where seven do.
    const bool once = a.m <= 8 * TL && (int64_t)a.n * a.k >= (64 << 20);
    constexpr bool PARTS = FP8 && !BF16OUT;                              // of K split: 16 or 64 rows, through the caches
    if constexpr (!BF16OUT || TL == 8) {
        if (p.rows == 4) return go_few<TL, 4, 4, 2, false, FP8, BF16OUT>(a, p.splits, stream);
    }
    if constexpr (!PARTS) {
        if (p.rows == 2)
            return once ? go_few<TL, 2, 4, 2, true, FP8, BF16OUT>(a, p.splits, stream) : go_few<TL, 2, 4, 2, false, FP8, BF16OUT>(a, p.splits, stream);
        if (once) return go_few<TL, 1, 4, 2, true, FP8, BF16OUT>(a, p.splits, stream);
    }
    return go_few<TL, 1, 4, 2, false, FP8, BF16OUT>(a, p.splits, stream);
}

template <bool FP8, bool BF16OUT>
hipError_t go_few(const B128Args& a, const Plan& p, hipStream_t stream) {
    if (a.m <= 8) return go_few<1, FP8, BF16OUT>(a, p, stream);
    if (a.m <= 16) return go_few<2, FP8, BF16OUT>(a, p, stream);
    if (a.m <= 24) return go_few<3, FP8, BF16OUT>(a, p, stream);
    if (a.m <= 32) return go_few<4, FP8, BF16OUT>(a, p, stream);
    if (a.m <= 40) return go_few<5, FP8, BF16OUT>(a, p, stream);
    if (a.m <= 48) return go_few<6, FP8, BF16OUT>(a, p, stream);
    return go_few<8, FP8, BF16OUT>(a, p, stream);
}

template <bool BF16OUT>
hipError_t go(B128Args a, const Plan& p, float* parts, hipStream_t stream) {
    if constexpr (BF16OUT) {
        if (p.form == Plan::BIG) return go_tile<4, 2, 4, 8, true, true>(a, 1, stream);
        if (p.form == Plan::MID) return go_tile<4, 2, 4, 4, true, true>(a, 1, stream);
    }
    const bool few = p.form == Plan::FEW;
    if (!few && a.groups < 4) return go_tile<2, 2, 4, 4, BF16OUT, BF16OUT, true>(a, 1, stream);
    if (p.splits == 1) return few ? go_few<BF16OUT, BF16OUT>(a, p, stream) : go_tile<2, 2, 4, 4, BF16OUT, BF16OUT>(a, 1, stream);
    void* y = a.y;
    a.y = parts;
    a.per = (a.groups + p.splits - 1) / p.splits;
    if (hipError_t e = few ? go_few<BF16OUT, false>(a, p, stream) : go_tile<2, 2, 4, 4, BF16OUT, false>(a, p.splits, stream); e != hipSuccess) return e;
    const int64_t outputs = (int64_t)a.m * a.n;
    b128_join_kernel<BF16OUT><<<(unsigned)((outputs + 1023) / 1024), 256, 0, stream>>>(parts, p.splits, outputs, y);
    return hipGetLastError();
}

}  // namespace

// The most bytes of parts that any size up to m takes.  From one of the sizes
// below to the next all costs but the join's stay as they are, and that grows with
// m and the splits: the first of them has the most splits.  Above 64 tokens a split
// saves less than a round of two workgroups a CU, so no size splits once two
// parts cost as much, and no parts cost more; that stands for what is not searched
// of few rows with more than half a million tokens.
int64_t gemm_fp8_b128_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    const int64_t cus = device_cu_count(), groups = (k + BLOCK - 1) / BLOCK, round = TWO_F32 * groups;
    if (groups < 8) return 0;
    int64_t most = 0, from = 1;
    for (int i = 0; from <= m && (from <= 64 || 2 * (from * n / JOIN_RATE) < round); ++i) {
        if (i == 8192) return std::max(most, 4 * std::min(MOST_SPLITS * m * n, JOIN_RATE * (round + MOST_SPLITS)));
        const int64_t upto = from < 5 ? 4 : from < 49 ? (from + 7) / 8 * 8 : (from + 63) / 64 * 64;
        const int splits = std::max(plan(from, n, k, true, cus).splits, plan(from, n, k, false, cus).splits);
        if (splits > 1) most = std::max(most, splits * std::min(upto, m) * n * 4);
        from = upto + 1;
    }
    return most;
}

hipError_t launch_gemm_fp8_b128(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int64_t m,
                                int64_t n, int64_t k, bool bf16_out, void* y, void* workspace, int64_t workspace_bytes,
                                hipStream_t stream) {
    const int groups = (int)((k + BLOCK - 1) / BLOCK);
    const B128Args args{a, a_scale, w, w_scale, (int)m, (int)n, (int)k, groups, groups, y};
    const int64_t fit = workspace_bytes / (m * n * 4);                   // parts
    const Plan p = plan(m, n, k, bf16_out, device_cu_count(), std::clamp(fit, (int64_t)1, MOST_SPLITS));
    return bf16_out ? go<true>(args, p, (float*)workspace, stream) : go<false>(args, p, (float*)workspace, stream);
}

}  // namespace nq
