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
// Two arithmetics.  BF16 outputs take the FP8 matrix instructions, whose sums
// drop low bits (1.3e-5 to 1.8e-5 off a block's exact sum, Frobenius; a BF16
// output's own rounding is 1.7e-3).  FP32 outputs keep to the 1e-5 of this
// library's FP32 results: codes become BF16, exactly, as operands are read,
// and go through the BF16 instructions at half the rate.
#include <hip/hip_runtime.h>

#include "nq_attn_launch.h"
#include "nq_device.h"
#include "nq_launch.h"
#include "nq_layer_launch.h"

namespace nq {
namespace {

constexpr int BLOCK = 128;               // columns of a scale
constexpr int ONE_E8M0 = 0x7F7F7F7F;     // the instructions' own block scales: 1

struct B128Args {
    const uint8_t* a;
    const float* as;
    const uint8_t* w;
    const float* ws;
    int m, n, k, groups;
    void* y;
};

__device__ __forceinline__ v8i join(v4u x, v4u y) {
    return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
}
__device__ __forceinline__ v8bf eight_bf16(uint32_t x, uint32_t y) {
    return __builtin_bit_cast(v8bf, v4u{e4m3x2_to_bf16x2<false>(x, 1.0f), e4m3x2_to_bf16x2<true>(x, 1.0f),
                                        e4m3x2_to_bf16x2<false>(y, 1.0f), e4m3x2_to_bf16x2<true>(y, 1.0f)});
}

template <bool BF16OUT>
__device__ __forceinline__ void store(void* y, int64_t at, float x) {
    if constexpr (BF16OUT) reinterpret_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16_rne(x);
    else reinterpret_cast<float*>(y)[at] = x;
}

// ---- few tokens: weights straight from memory into registers --------------------------------------------------------

// A workgroup has 16 weight rows and up to 16 NT tokens; its waves take every
// WAVES-th block of 128 columns and join in LDS, in the order of the waves.
// Bound by HBM: the weights once.
constexpr int FEW_TOKENS = 64;

template <int NT, int WAVES, bool BF16OUT>
__global__ __launch_bounds__(WAVES * 64) void b128_few_kernel(B128Args a) {
    __shared__ __align__(16) v4f part[WAVES][NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * FEW_TOKENS;
    const uint8_t* w = a.w + (int64_t)(n0 + r < a.n ? n0 + r : a.n - 1) * a.k;
    const float* ws = a.ws + (int64_t)(n0 / BLOCK) * a.groups;
    const uint8_t* x[NT];
    const float* xs[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int m = m0 + 16 * t + r < a.m ? m0 + 16 * t + r : a.m - 1;
        x[t] = a.a + (int64_t)m * a.k;
        xs[t] = a.as + (int64_t)m * a.groups;
    }
    v4f acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    struct Part {
        v4u w[2], x[NT][2];
        float xs[NT], ws;
    };
    // The lane's two pieces of a block: columns 16 g and 64 + 16 g on (zeros past the last column).
    auto load = [&](int b, Part& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = b * BLOCK + 64 * h + 16 * g;
            const bool in = col < a.k;
            p.w[h] = in ? __builtin_nontemporal_load(reinterpret_cast<const v4u*>(w + col)) : v4u{0u, 0u, 0u, 0u};
#pragma unroll
            for (int t = 0; t < NT; ++t) p.x[t][h] = in ? *reinterpret_cast<const v4u*>(x[t] + col) : v4u{0u, 0u, 0u, 0u};
        }
        p.ws = ws[b];
#pragma unroll
        for (int t = 0; t < NT; ++t) p.xs[t] = xs[t][b];
    };
    auto add = [&](const Part& p) {
        v4f s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (BF16OUT) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                s[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(p.w[0], p.w[1]), join(p.x[t][0], p.x[t][1]), s[t], 0, 0, 0,
                                                                        ONE_E8M0, 0, ONE_E8M0);
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const v8bf wf = eight_bf16(p.w[h >> 1][2 * (h & 1)], p.w[h >> 1][2 * (h & 1) + 1]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        wf, eight_bf16(p.x[t][h >> 1][2 * (h & 1)], p.x[t][h >> 1][2 * (h & 1) + 1]), s[t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float f = p.xs[t] * p.ws;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(s[t][e], f, acc[t][e]);
        }
    };
    for (int b = wave; b < a.groups; b += WAVES) {
        Part p;
        load(b, p);
        add(p);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 64; i += WAVES * 64) {
        v4f sum = part[0][i / 64][i % 64];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) {
            const v4f z = part[v][i / 64][i % 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += z[e];
        }
        const int m = m0 + i / 64 * 16 + i % 16, n = n0 + i % 64 / 16 * 4;
        if (m >= a.m) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.n) store<BF16OUT>(a.y, (int64_t)m * a.n + n + e, sum[e]);
    }
}

template <int NT, bool BF16OUT>
hipError_t go_few(const B128Args& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)((a.m + FEW_TOKENS - 1) / FEW_TOKENS));
    b128_few_kernel<NT, 8, BF16OUT><<<grid, 512, 0, stream>>>(a);
    return hipGetLastError();
}

// ---- many tokens: tiles through LDS ---------------------------------------------------------------------------------

// WR x WT waves of TI x TJ products of 32 x 32: a workgroup has 32 WR TI weight
// rows and 32 WT TJ tokens.  A stage is one block of 128 columns of both, in two
// slots: row r of a panel at byte 128 r, its 16-byte piece c in place
// c ^ (r / 2 % 8), so that operand reads (32 rows, two pieces) spread over all
// banks; and the tokens' scales of the block.
template <int WR, int WT, int TI, int TJ>
struct Tile {
    static constexpr int WAVES = WR * WT, ROWS = 32 * WR * TI, TOKENS = 32 * WT * TJ;
    static constexpr int LOADS = (ROWS + TOKENS) / 8 / WAVES;            // of 8 rows, a wave
    static constexpr int SCALES = (ROWS + TOKENS) * BLOCK;               // their place in a stage
    static constexpr int STAGE = SCALES + TOKENS * 4;
    static_assert((ROWS + TOKENS) % (8 * WAVES) == 0 && TOKENS % 64 == 0 && TOKENS / 64 <= WAVES && TJ % 2 == 0, "");
};

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
__device__ __forceinline__ void lds_load4(v4i r, int off, lds_ptr dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"((uint32_t)(uintptr_t)dst), "v"(off), "s"(r) : "memory", "m0");
}

template <int WR, int WT, int TI, int TJ, bool BF16OUT>
__global__ __launch_bounds__(WR * WT * 64, 2) void b128_tile_kernel(B128Args a) {
    using T = Tile<WR, WT, TI, TJ>;
    extern __shared__ __align__(16) unsigned char smem[];
    const lds_ptr lds = (lds_ptr)smem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous range of
    // tiles, tokens first, so that those that share an L2 read the same rows.
    const int tiles_m = (a.m + T::TOKENS - 1) / T::TOKENS;
    const int each = (int)gridDim.x / 8, more = (int)gridDim.x % 8, xcd = blockIdx.x % 8;
    const int tile = xcd * each + min(xcd, more) + blockIdx.x / 8;
    const int m0 = tile % tiles_m * T::TOKENS, n0 = tile / tiles_m * T::ROWS;
    const int rows_w = min(a.n - n0, T::ROWS), rows_a = min(a.m - m0, T::TOKENS);
    const v4i buf_w = buffer(a.w + (int64_t)n0 * a.k, (int64_t)rows_w * a.k), buf_a = buffer(a.a + (int64_t)m0 * a.k, (int64_t)rows_a * a.k);
    const v4i buf_s = buffer(a.as + (int64_t)m0 * a.groups, (int64_t)rows_a * a.groups * 4);
    const int steps = a.groups;

    // Load i of this wave: rows 8 q .. 8 q + 7 of the panels (weights first), q = wave LOADS + i.
    int place[2];                        // the lane's piece for even and odd q, as a column
#pragma unroll
    for (int p = 0; p < 2; ++p) place[p] = 16 * ((lane & 7) ^ ((4 * p + (lane >> 4)) & 7));
    const int row_off = (lane >> 3) * a.k;
    auto issue = [&](int s) {
        const lds_ptr at = lds + (s & 1) * T::STAGE;
        const int col = s * BLOCK;
#pragma unroll
        for (int i = 0; i < T::LOADS; ++i) {
            const int q = wave * T::LOADS + i;
            const bool is_w = q < T::ROWS / 8;
            const int mine = col + place[q & 1];
            int off = row_off + 8 * (is_w ? q : q - T::ROWS / 8) * a.k + mine;
            if (mine >= a.k) off = PAST;
            lds_load16(is_w ? buf_w : buf_a, off, at + q * 1024);
        }
        if (wave < T::TOKENS / 64) lds_load4(buf_s, ((64 * wave + lane) * a.groups + s) * 4, at + T::SCALES + wave * 256);
    };

    const int wr = wave % WR * TI * 32, wt = wave / WR * TJ * 32;
    const int n = lane & 31, h = lane >> 5;
    const int first = n * BLOCK + ((h ^ ((n >> 1) & 7)) << 4);           // of this lane's pieces h, 2 + h, 4 + h, 6 + h of its row
    auto read = [&](lds_ptr panel, int row, v4u (&x)[4]) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
            x[p] = *(__attribute__((address_space(3))) const v4u*)(panel + row * BLOCK + (first ^ (p << 5)));
    };
    auto product = [&](const v4u (&w)[4], const v4u (&t)[4]) {
        v16f p;
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0.f;
        if constexpr (BF16OUT) {
            p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(w[0], w[1]), join(t[0], t[1]), p, 0, 0, 0, ONE_E8M0, 0, ONE_E8M0);
            p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(w[2], w[3]), join(t[2], t[3]), p, 0, 0, 0, ONE_E8M0, 0, ONE_E8M0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(eight_bf16(w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1]),
                                                            eight_bf16(t[i >> 1][2 * (i & 1)], t[i >> 1][2 * (i & 1) + 1]), p, 0, 0, 0);
        }
        return p;
    };
    v16f acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    auto rescale = [&](v16f& c, const v16f& p, float f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) c[e] = fmaf(p[e], f, c[e]);
    };
    v4u w[TI][4], t[2][4];
    float f[TJ];
    const float* ws = a.ws + (int64_t)((n0 + wr) / BLOCK) * a.groups;    // (32 TI rows of a wave lie in one block of 128)
    const bool busy = n0 + wr < a.n;
    auto scales = [&](int s, lds_ptr at) {
        const float by = busy ? ws[s] : 0.f;
#pragma unroll
        for (int j = 0; j < TJ; ++j) f[j] = by * *(__attribute__((address_space(3))) const float*)(at + T::SCALES + (wt + 32 * j + n) * 4);
    };

    auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    if (steps > 0) issue(0);
    for (int s = 0; s < steps; ++s) {
        const lds_ptr at = lds + (s & 1) * T::STAGE;
        arrived();
        if (s + 1 < steps) issue(s + 1);
        scales(s, at);
#pragma unroll
        for (int i = 0; i < TI; ++i) read(at, wr + 32 * i, w[i]);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            read(at + T::ROWS * BLOCK, wt + 32 * j, t[0]);
#pragma unroll
            for (int i = 0; i < TI; ++i) rescale(acc[i][j], product(w[i], t[0]), f[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int m = m0 + wt + 32 * j + n;
        if (m >= a.m) continue;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = n0 + wr + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3);
                if (row < a.n) store<BF16OUT>(a.y, (int64_t)m * a.n + row, acc[i][j][e]);
            }
    }
}

template <int WR, int WT, int TI, int TJ, bool BF16OUT>
hipError_t go_tile(const B128Args& a, hipStream_t stream) {
    using T = Tile<WR, WT, TI, TJ>;
    constexpr int LDS = 2 * T::STAGE;
    auto kernel = b128_tile_kernel<WR, WT, TI, TJ, BF16OUT>;
    static LdsLimit limit;
    if (hipError_t e = limit.raise((const void*)kernel, LDS); e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)(a.m + T::TOKENS - 1) / T::TOKENS) * ((a.n + T::ROWS - 1) / T::ROWS);
    kernel<<<(unsigned)tiles, T::WAVES * 64, LDS, stream>>>(a);
    return hipGetLastError();
}

template <bool BF16OUT>
hipError_t go(const B128Args& a, hipStream_t stream) {
    if (a.m > 128) return go_tile<4, 2, 2, 4, BF16OUT>(a, stream);
    if (a.m <= 16) return go_few<1, BF16OUT>(a, stream);
    if (a.m <= 32) return go_few<2, BF16OUT>(a, stream);
    if (a.m <= 48) return go_few<3, BF16OUT>(a, stream);
    return go_few<4, BF16OUT>(a, stream);
}

}  // namespace

int64_t gemm_fp8_b128_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_fp8_b128(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int64_t m,
                                int64_t n, int64_t k, bool bf16_out, void* y, void*, int64_t, hipStream_t stream) {
    const B128Args args{a, a_scale, w, w_scale, (int)m, (int)n, (int)k, (int)((k + BLOCK - 1) / BLOCK), y};
    return bf16_out ? go<true>(args, stream) : go<false>(args, stream);
}

}  // namespace nq
