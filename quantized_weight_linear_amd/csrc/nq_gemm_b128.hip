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

#include <type_traits>

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

// WR x WT waves of FI x FT products of 16 x 16: a workgroup has 16 WR FI weight
// rows and 16 WT FT tokens.  A stage is one block of 128 columns of both, in two
// slots: row r of a panel at byte 128 r, its 16-byte piece c in place
// c ^ (r / 2 % 8), so that operand reads (16 rows, one piece each) cover all
// banks once; and the tokens' scales of the block.
template <int WR, int WT, int FI, int FT>
struct Tile {
    static constexpr int WAVES = WR * WT, ROWS = 16 * WR * FI, TOKENS = 16 * WT * FT;
    static constexpr int LOADS = (ROWS + TOKENS) / 8 / WAVES;            // of 8 rows, a wave
    static constexpr int SCALES = (ROWS + TOKENS) * BLOCK;               // their place in a stage
    static constexpr int SINK = SCALES + TOKENS * 4;                     // of the waves that have no scales to load
    static constexpr int STAGE = SINK + 256;
    static_assert((ROWS + TOKENS) % (8 * WAVES) == 0 && TOKENS % 64 == 0 && TOKENS / 64 <= WAVES && FT % 2 == 0, "");
    static_assert(BLOCK % (16 * FI) == 0, "a wave's rows lie in one block of the weights' scales");
};

// A wave's outputs in LDS on their way out, a row of them a token.
template <int FI, int FT, bool BF16OUT>
struct Output {
    static constexpr int SIZE = BF16OUT ? 2 : 4, EACH = 16 / SIZE, ROWS = 16 * FI, TOKENS = 16 * FT, PIECES = ROWS / EACH;
    static constexpr int PITCH = ROWS * SIZE + 16, BYTES = TOKENS * PITCH;
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

// The products run LAG steps ahead of the rescales, so that no rescale waits for
// its product.  Operands are read one column of products ahead, also across
// stages: the barrier at which the next stage has arrived (and this one has been
// read by all) stands before the last column.
template <int WR, int WT, int FI, int FT, bool BF16OUT>
__global__ __launch_bounds__(WR * WT * 64, 2) void b128_tile_kernel(B128Args a) {
    using T = Tile<WR, WT, FI, FT>;
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
    const int from = blockIdx.y * a.per, upto = min(from + a.per, a.groups);     // this workgroup's blocks

    const v4i buf_w = buffer(a.w + (int64_t)n0 * a.k, (int64_t)rows_w * a.k), buf_a = buffer(a.a + (int64_t)m0 * a.k, (int64_t)rows_a * a.k);
    const bool has_scales = wave < T::TOKENS / 64;
    const v4i buf_s = buffer(a.as + (int64_t)m0 * a.groups, has_scales ? (int64_t)rows_a * a.groups * 4 : 0);
    const int scales_at = has_scales ? T::SCALES + wave * 256 : T::SINK, scales_off = (64 * wave + lane) * a.groups * 4;

    // Load i of this wave: rows 8 q .. 8 q + 7 of the panels (weights first), q =
    // wave LOADS + i.  No branches: past the last block, and of what lies past the
    // last column, nothing is read and zeros arrive.
    int col[2], off[2];                  // the lane's piece, and its place, for even and odd q
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        col[p] = 16 * ((lane & 7) ^ ((4 * p + (lane >> 4)) & 7));
        off[p] = (lane >> 3) * a.k + col[p];
    }
    auto issue = [&](int s, int lo, int hi) {
        const lds_ptr at = lds + ((s - from) & 1) * T::STAGE;
        const int left = s < upto ? a.k - s * BLOCK : 0;                 // columns from this block on
        const int mine[2] = {col[0] < left ? off[0] : PAST, col[1] < left ? off[1] : PAST};
#pragma unroll
        for (int i = 0; i < T::LOADS; ++i) {
            if (i < lo || i >= hi) continue;
            const int q = wave * T::LOADS + i;
            const bool is_w = q < T::ROWS / 8;
            lds_load16(is_w ? buf_w : buf_a, mine[q & 1] + (8 * (is_w ? q : q - T::ROWS / 8) * a.k + s * BLOCK), at + q * 1024);
        }
        if (lo == 0) lds_load4(buf_s, s < upto ? scales_off + s * 4 : PAST, at + scales_at);
    };

    const int wr = wave % WR * FI * 16, wt = wave / WR * FT * 16;
    const int n = lane & 15, g = lane >> 4;
    const int first = n * BLOCK + ((g ^ (n >> 1)) << 4);                 // of this lane's pieces g and 4 + g of its row
    auto read = [&](lds_ptr row, v4u (&x)[2]) {
        x[0] = *(__attribute__((address_space(3))) const v4u*)(row + first);
        x[1] = *(__attribute__((address_space(3))) const v4u*)(row + (first ^ 64));
    };
    auto read_scale = [&](lds_ptr at, int j) { return *(__attribute__((address_space(3))) const float*)(at + T::SCALES + (wt + 16 * j + n) * 4); };
    auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    constexpr int Q = FI * FT, LAG = BF16OUT ? 3 : 1;
    v4f acc[FI][FT], p[LAG + 1];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i <= LAG; ++i) p[i] = v4f{0.f, 0.f, 0.f, 0.f};
    // Operands: codes as they are, or (FP32 outputs) as BF16, a block's 128 columns in four steps.
    struct Codes {
        v4u x[2];
    };
    struct Wide {
        v8bf x[4];
    };
    using Operand = std::conditional_t<BF16OUT, Codes, Wide>;
    auto operand = [&](const v4u (&x)[2]) {
        Operand o;
        if constexpr (BF16OUT) {
            o.x[0] = x[0], o.x[1] = x[1];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o.x[e] = eight_bf16(x[e >> 1][2 * (e & 1)], x[e >> 1][2 * (e & 1) + 1]);
        }
        return o;
    };
    auto product = [&](const Operand& w, const Operand& t) {
        v4f x = {0.f, 0.f, 0.f, 0.f};
        if constexpr (BF16OUT) {
            x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w.x[0], w.x[1]), join(t.x[0], t.x[1]), x, 0, 0, 0, ONE_E8M0, 0, ONE_E8M0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.x[e], t.x[e], x, 0, 0, 0);
        }
        return x;
    };
    auto rescale = [&](v4f& c, const v4f& x, float by) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = fmaf(x[e], by, c[e]);
    };
    const float* ws = a.ws + (int64_t)min((n0 + wr) / BLOCK, (a.n - 1) / BLOCK) * a.groups;
    Operand w[FI], t;
    v4u wn[FI][2], tn[2];
    float raw = 0.f, f = 0.f, f_last = 0.f;
    if (from < upto) {
        issue(from, 0, T::LOADS);
        arrived();
        issue(from + 1, 0, T::LOADS);
#pragma unroll
        for (int i = 0; i < FI; ++i) read(lds + (wr + 16 * i) * BLOCK, wn[i]);
        read(lds + (T::ROWS + wt) * BLOCK, tn);
        raw = read_scale(lds, 0);
    }
    for (int s = from; s < upto; ++s) {
        const lds_ptr at = lds + ((s - from) & 1) * T::STAGE, next = lds + ((s - from + 1) & 1) * T::STAGE;
        const float by = uniform(ws, s);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int i = q % FI, j = q / FI;
            if (i == 0) {
                t = operand(tn);
                if (j + 1 == FT) arrived();
                f_last = f;
                f = raw * by;
                read((j + 1 < FT ? at : next) + (T::ROWS + wt + 16 * ((j + 1) % FT)) * BLOCK, tn);    // (past the last stage: bytes that no one uses)
                raw = read_scale(j + 1 < FT ? at : next, (j + 1) % FT);
            }
            if (j == 0) w[i] = operand(wn[i]);
            __builtin_amdgcn_sched_barrier(0);
            p[q % (LAG + 1)] = product(w[i], t);
            {
                const int e = (q + Q - LAG) % Q;
                rescale(acc[e % FI][e / FI], p[(q + 1) % (LAG + 1)], i < LAG ? f_last : f);
            }
            if (j + 1 == FT) {
                read(next + (wr + 16 * i) * BLOCK, wn[i]);
                issue(s + 2, T::LOADS * i / FI, T::LOADS * (i + 1) / FI);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int q = Q - LAG; q < Q; ++q) rescale(acc[q % FI][q / FI], p[q % (LAG + 1)], f);
    // A lane's outputs lie a token apart: through LDS they become pieces of whole
    // cache lines.  Each wave has a place of its own there, once all have read
    // their last stage and nothing is on its way into it.
    arrived();
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
            if (m < a.m && row < a.n) *reinterpret_cast<v4u*>((char*)a.y + ((int64_t)m * a.n + row) * Out::SIZE) = x;
        }
    } else {
#pragma unroll 4
        for (int b = lane; b < Out::TOKENS * Out::ROWS; b += 64) {
            const int m = m0 + wt + b / Out::ROWS, row = n0 + wr + b % Out::ROWS;
            const lds_ptr x = mine + b / Out::ROWS * Out::PITCH + b % Out::ROWS * Out::SIZE;
            if (m >= a.m || row >= a.n) continue;
            if constexpr (BF16OUT) reinterpret_cast<uint16_t*>(a.y)[(int64_t)m * a.n + row] = *(__attribute__((address_space(3))) const uint16_t*)x;
            else reinterpret_cast<float*>(a.y)[(int64_t)m * a.n + row] = *(__attribute__((address_space(3))) const float*)x;
        }
    }
}

template <int WR, int WT, int FI, int FT, bool BF16OUT>
hipError_t go_tile(const B128Args& a, hipStream_t stream) {
    using T = Tile<WR, WT, FI, FT>;
    constexpr int OUT = T::WAVES * Output<FI, FT, BF16OUT>::BYTES, LDS = OUT > 2 * T::STAGE ? OUT : 2 * T::STAGE;
    static_assert(LDS <= 160 * 1024, "");
    auto kernel = b128_tile_kernel<WR, WT, FI, FT, BF16OUT>;
    static LdsLimit limit;
    if (hipError_t e = limit.raise((const void*)kernel, LDS); e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)(a.m + T::TOKENS - 1) / T::TOKENS) * ((a.n + T::ROWS - 1) / T::ROWS);
    kernel<<<(unsigned)tiles, T::WAVES * 64, LDS, stream>>>(a);
    return hipGetLastError();
}

template <bool BF16OUT>
hipError_t go(const B128Args& a, hipStream_t stream) {
    if (a.m > 128) {
        if constexpr (BF16OUT) return go_tile<4, 2, 4, 8, BF16OUT>(a, stream);
        else return go_tile<4, 2, 4, 4, BF16OUT>(a, stream);
    }
    if (a.m <= 16) return go_few<1, BF16OUT>(a, stream);
    if (a.m <= 32) return go_few<2, BF16OUT>(a, stream);
    if (a.m <= 48) return go_few<3, BF16OUT>(a, stream);
    return go_few<4, BF16OUT>(a, stream);
}

}  // namespace

int64_t gemm_fp8_b128_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_fp8_b128(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int64_t m,
                                int64_t n, int64_t k, bool bf16_out, void* y, void*, int64_t, hipStream_t stream) {
    const B128Args args{a, a_scale, w, w_scale, (int)m, (int)n, (int)k, (int)((k + BLOCK - 1) / BLOCK), (int)((k + BLOCK - 1) / BLOCK), y};
    return bf16_out ? go<true>(args, stream) : go<false>(args, stream);
}

}  // namespace nq
