// Block-scaled 8-bit floating-point linears on the matrix cores of gfx950
// (v_mfma_f32_16x16x128_f8f6f4): y[t][j] = sum_b xd[t][b] wd[j/128][b] sum_{i in b} xq[t][i] wq[j][i].
//
// Tile: BN weight rows x BM activation rows, WN x WM waves, TN x TM fragments of 16 x 16 a wave.  A K
// step is one block of 128 inputs, 128 bytes a row: weight rows are the instruction's A (so a lane ends
// up with four neighbouring outputs of one row), activation rows its B.  One instruction is a whole
// block of a fragment; its sum starts at zero and joins the accumulators as acc += (xd * wd) * sum, the
// factor being one number a lane (the lane's activation row) and fragment, since a fragment's weight
// rows lie in one block of 128.  (Fragments of 32 x 32, two instructions a block, read their operands half as often, and
// measured 263 us where these take 237, 4096 rows of 8192 x 8192: their sums are four times as long on
// the way.)
//
// The instruction aligns the products of eight inputs at the largest of them and cuts them off
// 2^-13 below it before they join its float32 sum (measured with pairs of products).  Random codes lose 2e-5
// of an output's size so, whatever k (in the norm; 8e-5 where one activation in 128 is 60 times the others), where the
// rounding of a binary16 result is 2.1e-4 and of a bf16 one 1.7e-3.  At worst it is 7 * 2^-13 of the largest product
// of every eight, less than half a step of bf16 (2^-8) and more than one of binary16 (2^-11) even where nothing
// cancels; where large products cancel, it may be all that is left.  Both 16-bit types take it for the rate.  A
// float32 result does not: its codes are widened to bf16, which holds them exactly, and multiplied by
// v_mfma_f32_16x16x32_bf16, at half the rate, whose sums of them are off by 2^-26.
//
// Tile rows reach LDS by direct copies of 16 bytes a lane, two stages.  Within a row the eight
// 16-byte chunks are stored at chunk ^ (row % 8), so that the fragments' reads (16 rows, one chunk of
// each) fall on all banks; lane group g reads chunks g and g + 4 of its row, the same for both operands,
// which makes the order of the inputs within a block immaterial.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "f8_tile.h"
#include "q8_internal.h"

namespace q8k {

namespace {

struct F8LinearArgs {
    const uint8_t* w;
    const float* wd;
    const uint8_t* x;
    const float* xd;
    void* y;
    void* gu;  // gate and up products of the fused call, or NULL
    int64_t ldy, ldgu;
    int n_out, m, k, kb;
    int m_tiles, n_tiles;
    bool vec, vec_gu;  // rows of y (gu) are aligned to four elements
};

// The 32 codes of a row that a lane supplies, and a block's sums of a fragment.
struct F8Codes {
    f8_i32x8 v;
    __device__ __forceinline__ void set(f8_i32x4 lo, f8_i32x4 hi) { v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
struct F8Widened {
    f8_bf16x8 v[4];
    __device__ __forceinline__ void set(f8_i32x4 lo, f8_i32x4 hi) {
        v[0] = f8_widen(lo[0], lo[1]);
        v[1] = f8_widen(lo[2], lo[3]);
        v[2] = f8_widen(hi[0], hi[1]);
        v[3] = f8_widen(hi[2], hi[3]);
    }
};
__device__ __forceinline__ f8_f32x4 f8_block_sum(const F8Codes& a, const F8Codes& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f8_f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f8_f32x4 f8_block_sum(const F8Widened& a, const F8Widened& b) {
    f8_f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], t, 0, 0, 0);
    return t;
}

// Four neighbouring outputs of a row from column n on: the products, or SiLU(gate) * up of the two.
template <bool SILU, class T>
__device__ __forceinline__ void f8_store_outputs(const F8LinearArgs& a, int row, int n, f8_f32x4 v, f8_f32x4 u) {
    const int inside = a.n_out - n;
    if constexpr (SILU) {
        if (a.gu) {
            T* gu = static_cast<T*>(a.gu) + (int64_t)row * a.ldgu + n;
            f8_store4(gu, v, inside, a.vec_gu);
            f8_store4(gu + a.n_out, u, inside, a.vec_gu && a.n_out % 4 == 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] / (1.0f + __expf(-v[e])) * u[e];
    }
    f8_store4(static_cast<T*>(a.y) + (int64_t)row * a.ldy + n, v, inside, a.vec);
}

// Words of a stage of scales, which every wave copies 64 of: the first BM / 64 waves (of eight waves the
// first four) the tile's rows', the others, all alike, those of its weight blocks.
template <int WN, int WM, int TM>
constexpr int f8_scale_rows() {
    return WN * WM == 8 ? 256 : (WM * TM * 16 + 63) / 64 * 64;
}
template <int WN, int WM, int TM>
constexpr int f8_scale_words() {
    return f8_scale_rows<WN, WM, TM>() + 64;
}
// Stages of rows and of scales (the turns of eight waves free the rows earlier than the scales).
template <int WN, int WM, int D>
constexpr int f8_scale_stages() {
    return WN * WM == 8 ? 4 : D;
}
template <int WN, int WM, int TN, int TM, int D>
constexpr size_t f8_linear_lds_bytes() {
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    return D * (size_t)(BN + BM) * 128 + f8_scale_stages<WN, WM, D>() * (size_t)f8_scale_words<WN, WM, TM>() * 4;
}

template <int WN, int WM, int TN, int TM, int D, bool SILU, class T>
__global__ __launch_bounds__(64 * WN * WM) void f8_linear_kernel(F8LinearArgs a) {
    constexpr int W = WN * WM, BN = WN * TN * 16, BM = WM * TM * 16, ROWS = BN + BM;
    constexpr int COPIES = ROWS / 8 / W;  // of a wave and step, eight rows each, and one of scales
    constexpr int SCALE_STAGES = f8_scale_stages<WN, WM, D>();
    constexpr int OUT = SILU ? TN * 8 : TN * 16;  // outputs of a wave
    using Codes = std::conditional_t<sizeof(T) == 4, F8Widened, F8Codes>;
    // Where a wave's weight rows do not divide a block, fragment i's block is its first or its last one's.
    constexpr bool CROSSES = 128 % (TN * 16) != 0;
    static_assert(!SILU || (!CROSSES && TN % 2 == 0), "a wave's gate rows lie in one block, and its up rows");
    static_assert(TN * 16 <= 128, "a wave's weight rows lie in two blocks at most");
    constexpr int FACTORS = CROSSES ? TN : SILU ? 2 : 1;  // of an activation row
    static_assert(ROWS / 8 % W == 0 && f8_scale_rows<WN, WM, TM>() / 64 < W && (W != 8 || D == 2),
                  "every wave has the same number of copies");
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;

    const F8Tile tile = f8_tile_of_block((int)blockIdx.x, a.m_tiles, a.n_tiles);
    if (!tile.inside) return;  // block-uniform, before any barrier
    const int n0 = tile.col * (SILU ? BN / 2 : BN), m0 = tile.row * BM;

    // Copy j of a wave: rows r .. r + 7 of the stage (weights, then activations), r = stage_row(j); lane l
    // the stage's chunk l % 8 of row l / 8.  Eight waves take turns (f8_turns): first the copies of the
    // piece X, the weights and each group's first activation rows, then those of Y, the groups' others.
    constexpr int PARTS = W == 8 ? 2 : 1, PM = TM / PARTS;
    constexpr int YC = W == 8 ? WM * PM * 2 / W : 0, XC = COPIES - YC;
    static_assert(W != 8 || (WM == 2 && TM % 2 == 0 && WM * 2 * PM % W == 0 && ROWS / 8 % W == 0), "pieces divide evenly");
    auto stage_row = [&](int j) __attribute__((always_inline)) {
        const int c = wave + W * (j < XC ? j : j - XC);
        if (W != 8 || c * 8 < BN && j < XC) return c * 8;
        constexpr int OF = 2 * PM;  // copies a group
        const int q = j < XC ? c - BN / 8 : c;
        return BN + q / OF * (TM * 16) + q % OF * 8 + (j < XC ? 0 : PM * 16);
    };
    const uint8_t* base[COPIES];
    uint32_t off[COPIES];
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
        const int r = stage_row(j);
        int first, rows;
        bool up = false;
        const uint8_t* from = a.w;
        if (r < BN) {
            const int wv = r / (TN * 16), in = r % (TN * 16);  // the wave whose rows these are
            rows = a.n_out;
            if constexpr (SILU) {
                up = in >= TN * 8;
                first = n0 + wv * (TN * 8) + (up ? in - TN * 8 : in);
            } else {
                first = n0 + wv * (TN * 16) + in;
            }
        } else {
            from = a.x;
            rows = a.m;
            first = m0 + r - BN;
        }
        // rows past the operand's end are its last row again
        const int start = first < rows ? first : rows - 1;
        const int row = first + lr < rows ? first + lr - start : rows - 1 - start;
        base[j] = from + (int64_t)(start + (up ? a.n_out : 0)) * a.k;
        off[j] = (uint32_t)row * (uint32_t)a.k + 16u * lc;
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const uint32_t lds_sx = lds + D * ROWS * 128;
    // Scales, a copy of four bytes a lane: the waves w < SX / 64 those of rows 64w .., the others word i the
    // scale of a weight block of wave i / 2 (gate's and up's where they are fused, else the first and the last
    // fragment's); past the matrix: the last block, of rows that are not stored.
    constexpr int SX = f8_scale_rows<WN, WM, TM>(), SW = f8_scale_words<WN, WM, TM>();
    const int last_block = (a.n_out - 1) / 128;
    auto weight_scale = [&](int i) __attribute__((always_inline)) {
        const int b = (n0 + (i / 2 % WN) * OUT + (!SILU && i % 2 ? OUT - 16 : 0)) / 128;
        return (uint32_t)((b < last_block ? b : last_block) + (SILU && i % 2 ? last_block + 1 : 0));
    };
    const int sx_row = m0 + 64 * wave + lane;
    const bool of_rows = 64 * wave < SX;
    const float* sc_base = of_rows ? a.xd + (int64_t)m0 * a.kb : a.wd;
    const uint32_t sc_off =
        4u * (of_rows ? (uint32_t)((sx_row < a.m ? sx_row : a.m - 1) - m0) * (uint32_t)a.kb : weight_scale(lane) * (uint32_t)a.kb);
    auto scale_stage = [&](int s) __attribute__((always_inline)) { return lds_sx + (uint32_t)(s % SCALE_STAGES) * SW * 4; };
    auto copy_scales = [&](int s) __attribute__((always_inline)) {
        f8_copy4(reinterpret_cast<const uint8_t*>(sc_base + s), sc_off, scale_stage(s) + (uint32_t)(of_rows ? 256 * wave : SX * 4));
    };

    // copy j of step s into stage `to`; copy COPIES is the wave's of the scales
    auto copy = [&](int s, int j, int to) __attribute__((always_inline)) {
        if (j == COPIES) copy_scales(s);
        else f8_copy16(base[j] + (int64_t)s * 128, off[j], lds + (uint32_t)(to * ROWS + stage_row(j)) * 128);
    };
    // the step of a cut block into stage 0, zeros past its inputs
    auto copy_cut = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < COPIES; ++j)
            f8_copy16_or_zeros(base[j] + (int64_t)s * 128, off[j], lc * 16 < (a.k & 127),
                               lds + (uint32_t)stage_row(j) * 128);
        copy_scales(s);
    };

    const int l16 = lane & 15, g = lane >> 4;
    // fragment i of the rows from `row` of stage `from` on
    const uint32_t lane_at = (uint32_t)l16 * 128 + 16u * (uint32_t)(g ^ (l16 & 7));
    auto fragment = [&](int from, int row, int i) __attribute__((always_inline)) {
        const uint8_t* at = f8_smem + (from * ROWS + row + i * 16) * 128;
        Codes c;
        c.set(*reinterpret_cast<const f8_i32x4*>(at + lane_at), *reinterpret_cast<const f8_i32x4*>(at + (lane_at ^ 64u)));
        return c;
    };

    const int out0 = n0 + wn * OUT;
    f8_f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f8_f32x4{0.f, 0.f, 0.f, 0.f};

    // A step's products in PARTS parts of its activation rows; the weights' fragments serve them all.
    Codes av[TN], bv[PM];
    float factor[FACTORS][PM] = {};
    float sx[PM], w0 = 0.f, w1 = 0.f;
    const int in_first = (128 - out0 % 128) / 16;  // fragments in the wave's first block
    auto load_from = [&](int s, int h, int from) __attribute__((always_inline)) {
        if (h == 0)
#pragma unroll
            for (int i = 0; i < TN; ++i) av[i] = fragment(from, wn * TN * 16, i);
#pragma unroll
        for (int j = 0; j < PM; ++j) bv[j] = fragment(from, BN + wm * TM * 16, h * PM + j);
        const float* at = reinterpret_cast<const float*>(f8_smem + D * ROWS * 128) + (s % SCALE_STAGES) * SW;
#pragma unroll
        for (int j = 0; j < PM; ++j) sx[j] = at[(wm * TM + h * PM + j) * 16 + l16];
        w0 = at[SX + 2 * wn];
        if (FACTORS > 1) w1 = at[SX + 2 * wn + 1];
    };
    auto ready = [&](int, int) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PM; ++j)
#pragma unroll
            for (int i = 0; i < FACTORS; ++i)
                factor[i][j] = sx[j] * (CROSSES ? (i < in_first ? w0 : w1) : i ? w1 : w0);
    };
    // A sum joins the accumulators LAG instructions after it was asked for, in this order
    // (scheduling fences): the lanes then work while the matrix cores do.  The last LAG join in finish().
    constexpr int LAG = TN * PM < 3 ? TN * PM : 3;
    f8_f32x4 t[LAG + 1] = {};
    auto join = [&](int h, int p) __attribute__((always_inline)) {
        const int i = p / PM, j = p % PM;
        const float c = factor[CROSSES ? i : SILU ? i / (TN / 2) : 0][j];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[i][h * PM + j][e] = __builtin_fmaf(c, t[p % (LAG + 1)][e], acc[i][h * PM + j][e]);
    };
    auto multiply = [&](int h, auto&& side) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < TN * PM; ++p) {
            t[p % (LAG + 1)] = f8_block_sum(av[p / PM], bv[p % PM]);
            if (p >= LAG) join(h, p - LAG);
            side(p);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto finish = [&](int h) __attribute__((always_inline)) {
#pragma unroll
        for (int p = TN * PM - LAG; p < TN * PM; ++p) join(h, p);
    };
    const int whole = a.k >> 7;  // steps; a cut block is a step of its own behind them
    if constexpr (W == 8) {
        if (whole)
            f8_turns<XC + 1, YC>(
                wave >> 2, whole,
                [&](int s, int i, int to) __attribute__((always_inline)) { if (i >= 0) copy(s, i < XC ? i : COPIES, to); },
                [&](int s, int i, int to) __attribute__((always_inline)) { if (i >= 0) copy(s, XC + i, to); },
                [&](int s, int h) __attribute__((always_inline)) { load_from(s, h, s & 1); }, finish, ready, multiply);
    } else {
        f8_ring<D, COPIES + 1>(
            whole,
            [&](int s, int to) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j <= COPIES; ++j) copy(s, j, to);
            },
            [&](int s, int from) __attribute__((always_inline)) {
                load_from(s, 0, from);
                ready(s, 0);
                multiply(0, [](int) {});
                finish(0);
            });
    }
    if (a.k & 127) {
        copy_cut(whole);
        wait_vmcnt_mem<0>();
        __syncthreads();
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
            load_from(whole, h, 0);
            ready(whole, h);
            multiply(h, [](int) {});
            finish(h);
        }
    }

    // element e of fragment (i, j): output 16i + 4g + e of the wave, row 16j + l16
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int row = m0 + (wm * TM + j) * 16 + l16;
        if (row >= a.m) continue;
#pragma unroll
        for (int i = 0; i < (SILU ? TN / 2 : TN); ++i)
            f8_store_outputs<SILU, T>(a, row, out0 + 16 * i + 4 * g, acc[i][j], acc[SILU ? i + TN / 2 : i][j]);
    }
}

template <int WN, int WM, int TN, int TM, int D, bool SILU, class T>
hipError_t launch_tile(F8LinearArgs a, hipStream_t stream) {
    constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
    auto kernel = f8_linear_kernel<WN, WM, TN, TM, D, SILU, T>;
    constexpr size_t lds = f8_linear_lds_bytes<WN, WM, TN, TM, D>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    constexpr int COLS = SILU ? BN / 2 : BN;
    a.m_tiles = (a.m + BM - 1) / BM;
    a.n_tiles = (a.n_out + COLS - 1) / COLS;
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    if (f8_grid(tiles) * (64 * WN * WM) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)f8_grid(tiles)), dim3(64 * WN * WM), lds, stream, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------------- few activation rows
//
// Bound by the weights' bytes.  A workgroup owns R x 16 weight rows (fused: half of them gate rows, half
// their up rows) and all activation rows (MT fragments of 16; rows past the call's are its last one); its
// WK waves share the blocks of inputs, block b to wave b % WK, and their sums meet in LDS and are added in
// the order of the waves.  A wave has D stages of LDS of its own, filled D blocks ahead by direct copies:
// loads into the instruction's registers, whose neighbouring lanes are rows apart, reached a sixth of
// the rate at 64 rows (4096 x 24576: 88 us).
template <int WK, int R, int MT, int D>
constexpr size_t f8_rows_stage_bytes() {
    return (size_t)(R + MT) * 2048 + (MT * 16 + R <= 64 ? 1 : 2) * 256;
}
template <int WK, int R, int MT, int D>
constexpr size_t f8_rows_lds_bytes() {
    const size_t ring = WK * D * f8_rows_stage_bytes<WK, R, MT, D>(), sums = (size_t)WK * MT * R * 64 * 16;
    return ring > sums ? ring : sums;
}

template <int WK, int R, int MT, int D, bool SILU, class T>
__global__ __launch_bounds__(64 * WK) void f8_rows_kernel(F8LinearArgs a) {
    constexpr int HALF = SILU ? R / 2 : R;  // fragments of outputs
    constexpr int STAGE = f8_rows_stage_bytes<WK, R, MT, D>();
    constexpr int SCALES = MT * 16 + R <= 64 ? 1 : 2, COPIES = 2 * (R + MT) + SCALES;  // of a stage
    static_assert(R <= 64 && MT <= 4 && (D - 1) * COPIES < 64 && (!SILU || R % 2 == 0), "copies are counted");
    using Codes = std::conditional_t<sizeof(T) == 4, F8Widened, F8Codes>;
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * (16 * HALF);

    // copy c of a stage: rows 8(c % 2) .. + 7 of fragment c / 2 (weights, then activations), lane l the
    // chunk l % 8 of row l / 8 as in the tiles; past the operand: its last row
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
    uint32_t off[2 * (R + MT)];
#pragma unroll
    for (int c = 0; c < 2 * (R + MT); ++c) {
        const int f = c / 2, rows = f < R ? a.n_out - n0 : a.m;
        const int row = (f < R ? 16 * (f % HALF) : 16 * (f - R)) + 8 * (c % 2) + lr;
        off[c] = (uint32_t)(row < rows ? row : rows - 1) * (uint32_t)a.k + 16u * lc;
    }
    const uint8_t* w[2] = {a.w + (int64_t)n0 * a.k, a.w + (int64_t)(n0 + (SILU ? a.n_out : 0)) * a.k};
    // word i of a stage's scales: row i's, then those of the weights' fragments
    auto scale_word = [&](int i) __attribute__((always_inline)) {
        const int f = i - MT * 16;
        const int blocks = (a.n_out + 127) / 128, at = (n0 + 16 * (f % HALF)) / 128;
        const int b = (at < blocks ? at : blocks - 1) + (SILU && f >= HALF ? blocks : 0);
        return i < MT * 16 ? a.xd + (int64_t)(i < a.m ? i : a.m - 1) * a.kb : a.wd + (int64_t)(f < R ? b : 0) * a.kb;
    };
    const float* scale_at[SCALES];
#pragma unroll
    for (int i = 0; i < SCALES; ++i) scale_at[i] = scale_word(64 * i + lane);

    // Workgroups start at different blocks: rows are often a multiple of 4 KB apart, and all of them in step
    // would ask the same few channels of the L2 (24576 x 4096 fused, 8 rows: 24.4 us, so 21.4).
    const int whole = a.k >> 7;
    const int turns = (whole - wave + WK - 1) / WK;  // whole blocks of this wave
    const int first = turns > 0 ? blockIdx.x % turns : 0;
    const uint32_t lds = f8_lds_address(f8_smem) + (uint32_t)(wave * D * STAGE);
    auto copy_scales = [&](int b, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SCALES; ++i) f8_copy4_from(scale_at[i] + b, to + (uint32_t)((R + MT) * 2048 + 256 * i));
    };
    auto copies = [&](int turn, int slot) __attribute__((always_inline)) {
        const int from = turn + first - (turn + first < turns ? 0 : turns), b = from * WK + wave;
        const uint32_t to = lds + (uint32_t)(slot * STAGE);
#pragma unroll
        for (int c = 0; c < 2 * (R + MT); ++c)
            f8_copy16((c / 2 < R ? w[c / 2 / HALF] : a.x) + (int64_t)b * 128, off[c], to + (uint32_t)(c * 1024));
        copy_scales(b, to);
    };
    f8_f32x4 acc[MT][R];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[j][r] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t lane_at = (uint32_t)l16 * 128 + 16u * (uint32_t)(g ^ (l16 & 7));
    struct Stage {
        f8_i32x4 w[R][2], x[MT][2];
        float wd[R], xd[MT];
    };
    auto read = [&](int slot) __attribute__((always_inline)) {
        const uint8_t* at = f8_smem + (wave * D + slot) * STAGE;
        const float* scales = reinterpret_cast<const float*>(at + (R + MT) * 2048);
        Stage v;
#pragma unroll
        for (int f = 0; f < R + MT; ++f) {
            f8_i32x4(&to)[2] = f < R ? v.w[f < R ? f : 0] : v.x[f < R ? 0 : f - R];
            to[0] = *reinterpret_cast<const f8_i32x4*>(at + f * 2048 + lane_at);
            to[1] = *reinterpret_cast<const f8_i32x4*>(at + f * 2048 + (lane_at ^ 64u));
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) v.xd[j] = scales[16 * j + l16];
#pragma unroll
        for (int r = 0; r < R; ++r) v.wd[r] = scales[16 * MT + r];
        return v;
    };
    auto multiply = [&](const Stage& v) __attribute__((always_inline)) {
        Codes wc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) wc[r].set(v.w[r][0], v.w[r][1]);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            Codes xc;
            xc.set(v.x[j][0], v.x[j][1]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const f8_f32x4 t = f8_block_sum(wc[r], xc);
                const float c = v.xd[j] * v.wd[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][r][e] = __builtin_fmaf(c, t[e], acc[j][r][e]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < turns) copies(d, d);
    int t = 0, slot = 0;
    for (; t + D < turns; ++t) {
        wait_vmcnt_mem<(D - 1) * COPIES>();
        const Stage v = read(slot);
        wait_lgkmcnt_mem<0>();  // read before it is copied over
        copies(t + D, slot);
        multiply(v);
        slot = slot + 1 < D ? slot + 1 : 0;
    }
    auto drain = [&](auto dc) __attribute__((always_inline)) {
        constexpr int d = decltype(dc)::value;
        if (turns - t > d) {
            wait_vmcnt_mem<d * COPIES>();
            multiply(read(slot));
            ++t;
            slot = slot + 1 < D ? slot + 1 : 0;
        }
    };
    if constexpr (D > 2) drain(std::integral_constant<int, 2>{});
    if constexpr (D > 1) drain(std::integral_constant<int, 1>{});
    drain(std::integral_constant<int, 0>{});
    static_assert(D <= 3, "stages are drained one by one");
    if ((a.k & 127) && whole % WK == wave) {  // the cut block, zeros past its inputs
        wait_lgkmcnt_mem<0>();
#pragma unroll
        for (int c = 0; c < 2 * (R + MT); ++c)
            f8_copy16_or_zeros((c / 2 < R ? w[c / 2 / HALF] : a.x) + (int64_t)whole * 128, off[c],
                               16 * lc < (a.k & 127), lds + (uint32_t)(c * 1024));
        copy_scales(whole, lds);
        wait_vmcnt_mem<0>();
        multiply(read(0));
    }

    __syncthreads();  // every wave is done with its stages
    f8_f32x4* sums = reinterpret_cast<f8_f32x4*>(f8_smem);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) sums[((wave * MT + j) * R + r) * 64 + lane] = acc[j][r];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * HALF * 64; i += 64 * WK) {
        const int at = i & 63, r = (i >> 6) % HALF, j = (i >> 6) / HALF;
        auto sum = [&](int r) __attribute__((always_inline)) {
            f8_f32x4 v = sums[(j * R + r) * 64 + at];
#pragma unroll
            for (int o = 1; o < WK; ++o) v += sums[((o * MT + j) * R + r) * 64 + at];
            return v;
        };
        const int row = 16 * j + (at & 15);
        if (row < a.m) f8_store_outputs<SILU, T>(a, row, n0 + 16 * r + 4 * (at >> 4), sum(r), sum(SILU ? r + HALF : r));
    }
}

template <int WK, int R, int MT, int D, bool SILU, class T>
hipError_t launch_rows(const F8LinearArgs& a, hipStream_t stream) {
    auto kernel = f8_rows_kernel<WK, R, MT, D, SILU, T>;
    constexpr size_t lds = f8_rows_lds_bytes<WK, R, MT, D>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    constexpr int COLS = 16 * (SILU ? R / 2 : R);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.n_out + COLS - 1) / COLS)), dim3(64 * WK), lds, stream, a);
    return hipGetLastError();
}

template <bool SILU, class T>
hipError_t launch_type(const DeviceInfo& dev, const F8LinearArgs& a, hipStream_t stream) {
    const int64_t cus = dev.cu_count, cols = SILU ? 2 : 1;
    const bool few = (a.n_out + 31) / 32 < cus;  // 16 outputs a workgroup then, not 32
    if (a.m <= 16) return launch_rows<8, SILU ? 2 : 1, 1, SILU ? 3 : 2, SILU, T>(a, stream);
    if constexpr (!SILU) {
        if (a.m <= 32 && few) return launch_rows<8, 1, 2, 2, SILU, T>(a, stream);
        if (a.m <= 48 && few) return launch_rows<8, 1, 3, 2, SILU, T>(a, stream);
        if (a.m <= 64 && few) return launch_rows<4, 1, 4, 3, SILU, T>(a, stream);
    }
    if (a.m <= 32) return launch_rows<4, 2, 2, 2, SILU, T>(a, stream);
    if (a.m <= 48) return launch_rows<4, 2, 3, 3, SILU, T>(a, stream);
    if (a.m <= 64) return launch_rows<4, 2, 4, 3, SILU, T>(a, stream);
    // The tile whose rounds (a workgroup a CU) cost least, a round by its measured time for 32 blocks of
    // inputs, in us: 16-bit results 59, 30, 23 and 16; float32 results 57, 46, 29 and 19.  Measured for
    // 6144 x 4096 in bfloat16, in that order of tiles: 128 rows 49.6, 30.4, 23.4, 16.9; 256 rows 58.6, 30.5,
    // 23.3, 30.9; 512 rows 58.3, 30.9, 44.2, 45.4; 4096 rows 121, 176, 254, 333.
    // A fifth tile of 192 weight rows (16-bit products; a wave's 48 rows lie in two blocks, so with factors for each
    // fragment) costs 53, more than three quarters of the largest's 59 as it reads more for a product; it is for
    // calls that end between whole rounds of that one: 6144 x 4096, 4096 rows, 384 tiles 120 us, 512 of these 112;
    // 4096 x 12288, 2048 rows, 128 tiles 153 us, 176 of these 131; 10240 x 4096, 2048 rows 120 us, so 103.
    constexpr bool WIDE = sizeof(T) == 4;
    constexpr int BIG = WIDE ? 4 : 8;
    constexpr bool THIRD = !WIDE && !SILU;
    const int64_t bn[5] = {256, 128, 128, 64, 192}, bm[5] = {32 * BIG, 128, 64, 64, 256};
    const int64_t cost[5] = {WIDE ? 57 : 59, WIDE ? 46 : 30, WIDE ? 29 : 23, WIDE ? 19 : 16, 53};
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < (THIRD ? 5 : 4); ++i) {
        const int64_t tiles = (a.n_out * cols + bn[i] - 1) / bn[i] * ((a.m + bm[i] - 1) / bm[i]);
        const int64_t time = (tiles + cus - 1) / cus * cost[i];
        if (time < least) {
            least = time;
            best = i;
        }
    }
    switch (best) {
        case 0: return launch_tile<4, 2, 4, BIG, 2, SILU, T>(a, stream);
        case 1: return launch_tile<2, 2, 4, 4, 4, SILU, T>(a, stream);
        case 2: return launch_tile<4, 1, 2, 4, 6, SILU, T>(a, stream);
        case 3: return launch_tile<2, 2, 2, 2, 6, SILU, T>(a, stream);
        default: break;
    }
    if constexpr (THIRD) return launch_tile<4, 2, 3, 8, 2, SILU, T>(a, stream);
    return hipErrorInvalidValue;  // not reached
}

template <class T>
bool aligned4(const void* p, int64_t ld) {
    return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

template <class T>
hipError_t launch_any(const DeviceInfo& dev, bool silu, F8LinearArgs a, hipStream_t stream) {
    a.vec = aligned4<T>(a.y, a.ldy);
    a.vec_gu = aligned4<T>(a.gu, a.ldgu);
    return silu ? launch_type<true, T>(dev, a, stream) : launch_type<false, T>(dev, a, stream);
}

}  // namespace

hipError_t launch_f8_linear(const DeviceInfo& dev, const uint8_t* wq, const float* wd, int64_t n_out, int64_t k,
                            bool silu, const uint8_t* xq, const float* xd, int64_t m, void* y, int type, int64_t ldy,
                            void* gu, int64_t ldgu, hipStream_t stream) {
    F8LinearArgs a{};
    a.w = wq; a.wd = wd; a.x = xq; a.xd = xd;
    a.y = y; a.gu = gu; a.ldy = ldy; a.ldgu = ldgu;
    a.n_out = (int)n_out; a.m = (int)m; a.k = (int)k; a.kb = (int)((k + 127) / 128);
    switch (type) {
        case Q8_F32: return launch_any<float>(dev, silu, a, stream);
        case Q8_F16: return launch_any<_Float16>(dev, silu, a, stream);
        default: return launch_any<__bf16>(dev, silu, a, stream);
    }
}

}  // namespace q8k
