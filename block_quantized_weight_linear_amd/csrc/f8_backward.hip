// Gradients of the block-scaled 8-bit floating-point linears on the bf16 matrix cores of gfx950
// (v_mfma_f32_16x16x32_bf16, float32 accumulation):
//   dx[t][i] = sum_j d[t][j] wd[j/128][i/128] wq[j][i]      dw[j][i] = sum_t d[t][j] x[t][i]
// with d the gradient of the products (the call's own, or behind SiLU(gate) * up its two parts
// beside each other) and x the inputs' values.
//
// An e4m3 code is exact in bf16.  A float operand is a sum of bf16 parts (a gradient one of bf16, two of
// binary16, three of float32; a value of x two, beside float32 gradients three), laid out as planes by a first
// launch; a product runs over the planes (dw: over the pairs of planes that matter) as if they were further terms
// of its sum.  (x's values as one part beside bf16 gradients made dw of 4096 rows of the fused 24576 x 4096 off by
// 2.9e-3 where its own rounding and dg's give 2.3e-3, in 620 us where two take 1234.)
//
// Both sums run over an axis that is not the contiguous one of W (dx), or of both operands (dw).
// Fragments are turned on their way from LDS: ds_read_b64_tr_b16 gives a lane of 16 the four rows of its
// column from four rows of 16 two-byte columns, ds_read_b64_tr_b8 eight rows of 16 one-byte columns (by reads
// of whole words and byte permutes instead, the fused 24576 x 4096 took 909 + 886 us at 4096 rows).
//
// Sums run in steps of 64 terms.  Planes have zeros up to whole steps (d's columns, the values' rows); the
// other operand's rows past its end are its last row again, which adds zeros where it is finite, and where it
// is not changes nothing that is finite without it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "f8_tile.h"
#include "q8_internal.h"
#include "q8_validate.h"

namespace q8k {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f8_f32x4 mfma_bf16(u32x4 a, u32x4 b, f8_f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(f8_bf16x8, a), __builtin_bit_cast(f8_bf16x8, b), c,
                                                   0, 0, 0);
}

// A lane's share of a turned read, from its LDS address.
__device__ __forceinline__ u32x2 read_turned16(const uint8_t* p) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* Lds;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(uint32_t)(uintptr_t)p));
}
__device__ __forceinline__ u32x2 read_turned8(const uint8_t* p) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) i32x2* Lds;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((Lds)(uint32_t)(uintptr_t)p));
}

// The bf16 parts of a gradient of type T, 1 (bf16), 2 (binary16) or 3 (float32), of a value of x beside it, and the
// pairs of them whose products count.
template <class T>
constexpr int kType = sizeof(T) == 4 ? Q8_F32 : __is_same(T, __bf16) ? Q8_BF16 : Q8_F16;
template <class T>
constexpr int kTerms = q8v::f8_terms(kType<T>);
template <class T>
constexpr int kValueTerms = q8v::f8_value_terms(kType<T>);
template <class T>
constexpr int kPairs = q8v::f8_pairs(kType<T>);

// ------------------------------------------------------------------------------ bf16 parts

// v as TERMS bf16 parts, each the rest rounded to nearest even: of 24 bits the first leaves 16, the
// second 7, so that three parts are a float32 and two a binary16 exactly (remainders are exact; a float32 below
// 2^-110 has bits below bf16's least, 2^-133, which are lost).
// What is not finite stays in the first part; the parts of a number that would round to infinity are
// cut off instead, so that no sum of its first parts passes it.
template <int TERMS>
__device__ __forceinline__ void split(float v, uint16_t (&part)[TERMS]) {
    float rest = v;
    bool cut = false;
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        part[i] = __builtin_bit_cast(uint16_t, (__bf16)rest);
        if (i + 1 < TERMS) {
            cut |= (part[i] & 0x7FFF) == 0x7F80 && __builtin_isfinite(rest);
            if (cut) part[i] = (uint16_t)(__float_as_uint(rest) >> 16);
            const float lead = __uint_as_float((uint32_t)part[i] << 16);
            rest = __builtin_isfinite(rest) ? rest - lead : 0.f;
        }
    }
}

constexpr int kPartThreads = 256;

// Eight neighbouring elements of a row of `width`, zeros past it.
template <class T>
__device__ __forceinline__ void load_row8(const T* row, int64_t col, int64_t width, bool vec, float (&v)[8]) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    if (vec && col + 8 <= width) {
        const T8 r = *reinterpret_cast<const T8*>(row + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)r[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < width ? (float)row[col + i] : 0.f;
    }
}
template <int TERMS>
__device__ __forceinline__ void store_parts(uint16_t* at, int64_t plane, const float (&v)[8]) {
    uint16_t p[8][TERMS];
#pragma unroll
    for (int i = 0; i < 8; ++i) split<TERMS>(v[i], p[i]);
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i][t] | (uint32_t)p[2 * i + 1][t] << 16;
        *reinterpret_cast<u32x4*>(at + t * plane) = w;
    }
}

// What the products read, in one launch: the gradient's planes by the first blocks, the inputs' by the others.
// Bound by memory (behind 4096 rows of SiLU(gate) * up, 12288 wide, in bf16: 585 MB in 99 us, 5.9 TB/s).
struct F8PlanesArgs {
    const void* d;    // the call's gradient [m][n]; kind kNoPlanes: it is its own plane
    const void* gu;   // kind kBehindSilu: gate and up products [m][2n]
    const uint8_t* q;  // codes and scales of the inputs
    const float* xd;
    uint16_t *planes, *values;
    int64_t ldd, ldgu, ldo, m, rows;  // rows: of the values, zeros from m on
    int n, k, kb;
    unsigned d_blocks;
    bool vec;
};
enum { kNoPlanes, kSplit, kBehindSilu };

template <class T, int TERMS, int KIND>
__device__ __forceinline__ void f8_gradient_planes(const F8PlanesArgs& a, int64_t first, int64_t step) {
    const int64_t per_row = a.ldo / (KIND == kBehindSilu ? 16 : 8), total = a.m * per_row;
    const T* d = static_cast<const T*>(a.d);
    const T* gu = static_cast<const T*>(a.gu);
    for (int64_t i = first; i < total; i += step) {
        const int64_t row = i / per_row, col = 8 * (i - row * per_row);
        uint16_t* at = a.planes + row * a.ldo + col;
        float h[8];
        load_row8(d + row * a.ldd, col, a.n, a.vec, h);
        if constexpr (KIND == kSplit) {
            store_parts<TERMS>(at, a.m * a.ldo, h);
        } else {
            // the gate's and up's gradients beside each other, in float32: rounded to T, binary16 ones would have its
            // range too, 65504 and 2^-24, which the results may lie within where these do not
            float g[8], u[8], dg[8], du[8];
            load_row8(gu + row * a.ldgu, col, a.n, a.vec, g);
            load_row8(gu + row * a.ldgu + a.n, col, a.n, a.vec && a.n % 8 == 0, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = 1.0f / (1.0f + __expf(-g[e]));
                dg[e] = h[e] * u[e] * (s * (1.0f + g[e] * (1.0f - s)));
                du[e] = h[e] * (g[e] * s);
            }
            store_parts<TERMS>(at, a.m * a.ldo, dg);
            store_parts<TERMS>(at + a.ldo / 2, a.m * a.ldo, du);
        }
    }
}

template <int TERMS>
__device__ __forceinline__ void f8_input_planes(const F8PlanesArgs& a, int64_t first, int64_t step) {
    const int64_t per_row = a.k / 8, total = a.rows * per_row;
    for (int64_t i = first; i < total; i += step) {
        const int64_t row = i / per_row, col = 8 * (i - row * per_row);
        float v[8] = {};
        if (row < a.m) {
            const u32x2 c = *reinterpret_cast<const u32x2*>(a.q + row * a.k + col);
            const float s = a.xd[row * a.kb + col / 128];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 0) * s;
                v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 1) * s;
                v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 2) * s;
                v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 3) * s;
            }
        }
        store_parts<TERMS>(a.values + row * a.k + col, a.rows * a.k, v);
    }
}

template <class T, int TERMS, int KIND>
__global__ __launch_bounds__(kPartThreads) void f8_planes_kernel(F8PlanesArgs a) {
    if constexpr (KIND != kNoPlanes) {
        if (blockIdx.x < a.d_blocks) {
            f8_gradient_planes<T, TERMS, KIND>(a, (int64_t)blockIdx.x * kPartThreads + threadIdx.x,
                                               (int64_t)a.d_blocks * kPartThreads);
            return;
        }
    }
    f8_input_planes<kValueTerms<T>>(a, (int64_t)(blockIdx.x - a.d_blocks) * kPartThreads + threadIdx.x,
                                    (int64_t)(gridDim.x - a.d_blocks) * kPartThreads);
}

template <class T>
__global__ __launch_bounds__(kPartThreads) void f8_zero_rows_kernel(T* __restrict__ out, int64_t rows, int64_t cols,
                                                                   int64_t ld) {
    const int64_t total = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPartThreads)
        out[i / cols * ld + i % cols] = (T)0.f;
}

// Results of ranges [ranges][rows][k] added in their order.  dx's are added by further blocks of the launch of
// dw's small tiles, which leave CUs free (2001 x 1040, 77 rows in float32: a launch of its own for it, the call
// 32.5 us; so, 27.6; fused 1536 x 2048, 130 rows in binary16: 31.6, so 29.0).
struct F8AddRangesArgs {
    const float* sums;
    void* out;
    int64_t rows, ld;
    int ranges, k;
    bool vec;
};
template <class T>
__device__ __forceinline__ void f8_add_ranges(const F8AddRangesArgs& a, int64_t first, int64_t step) {
    const int64_t per_row = a.k / 4, total = a.rows * per_row;
    for (int64_t i = first; i < total; i += step) {
        const int64_t row = i / per_row, col = 4 * (i - row * per_row);
        const float* at = a.sums + row * a.k + col;
        f8_f32x4 v = *reinterpret_cast<const f8_f32x4*>(at);
        for (int r = 1; r < a.ranges; ++r) v += *reinterpret_cast<const f8_f32x4*>(at + r * a.rows * a.k);
        f8_store4(static_cast<T*>(a.out) + row * a.ld + col, v, 4, a.vec);
    }
}
template <class T>
__global__ __launch_bounds__(kPartThreads) void f8_add_ranges_kernel(F8AddRangesArgs a) {
    f8_add_ranges<T>(a, (int64_t)blockIdx.x * kPartThreads + threadIdx.x, (int64_t)gridDim.x * kPartThreads);
}

unsigned part_blocks(int64_t threads) {
    const int64_t b = (threads + kPartThreads - 1) / kPartThreads;
    return (unsigned)(b < 65536 ? (b ? b : 1) : 65536);
}

// -------------------------------------------------------------------------------- dx = d . W

constexpr int kGStep = q8v::kF8Step;  // terms of the sum a step

struct F8InputGradArgs {
    const uint16_t* d;  // planes of bf16 parts
    int64_t plane;      // elements from one to the next
    int64_t ldd;
    int64_t part_cols;  // columns from one part's gradients to the next's
    const uint8_t* w;
    const float* wd;
    void* dx;
    int64_t lddx;
    int n, parts, m, k, kb;
    int m_tiles, k_tiles;
    int ranges, range_steps;  // of the sum; a range's results go range_stride elements behind the one's before
    int64_t range_stride;
    bool vec;
};

// D stages of a tile of eight waves are two, with scale stages of their own (f8_turns).
template <int W, int D>
constexpr int input_grad_scale_stages() {
    return W == 8 ? 4 : D;
}
template <int WK, int WM, int TM, int D>
constexpr size_t input_grad_lds_bytes() {
    return D * ((size_t)WM * TM * 16 * 2 * kGStep + (size_t)WK * 64 * kGStep) + input_grad_scale_stages<WK * WM, D>() * 256;
}

// WK x WM waves, a wave 64 columns of dx (four fragments) x 16 TM rows.  A step is 64 rows of W, all in one
// block of its scales: the step's sums start at zero and join the accumulators times the scale.
// T: the gradients' type, O: the results'.
// The large tile is bound by what a wave issues between its products (a fragment's sum joins by fmas after two of them, and
// codes are widened): fused 24576 x 4096, 4096 rows in bf16, 722 us, 1.14 PFLOP/s, matrix cores busy 45% of the cycles.
template <int WK, int WM, int TM, int D, class T, class O>
__global__ __launch_bounds__(64 * WK * WM) void f8_input_grad_kernel(F8InputGradArgs a) {
    constexpr int W = WK * WM, BK = WK * 64, BM = WM * TM * 16;
    constexpr int PARTS = W == 8 ? 2 : 1, PM = TM / PARTS;
    constexpr int CPR = BK / 16;               // 16-byte chunks of a row of W
    constexpr int WC = kGStep * CPR / 64 / W;  // copies of W of a wave
    constexpr int DC = BM / 8 / W;             // copies of d of a wave: eight rows of 128 bytes each
    constexpr int YC = W == 8 ? DC / 2 : 0, XC = WC + DC - YC;  // pieces of f8_turns: Y is the groups' last rows
    static_assert(BM / 8 % W == 0 && kGStep * CPR / 64 % W == 0, "copies divide evenly");
    static_assert(W != 8 || (D == 2 && WM == 2 && DC % 2 == 0 && PM * 2 % 4 == 0), "pieces divide evenly");
    constexpr int STAGE = BM * 2 * kGStep + BK * kGStep, SCALES = input_grad_scale_stages<W, D>();
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wm = wave / WK;
    const F8Tile tile = f8_tile_of_block((int)blockIdx.x, a.m_tiles, a.k_tiles * a.ranges);
    if (!tile.inside) return;  // block-uniform, before any barrier
    const int range = tile.col / a.k_tiles;
    const int m0 = tile.row * BM, k0 = (tile.col - range * a.k_tiles) * BK;

    // d: copy j is rows r .. r + 7 of the tile, r = d_row(j), chunks as in the forward tiles
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
    auto d_row = [&](int j) __attribute__((always_inline)) {
        const int half = j < DC - YC ? 0 : 1;
        if (W != 8) return 8 * (wave + W * j);
        const int q = wave + W * (half ? j - (DC - YC) : j);  // of 2 PM copies a group and half
        return q / (2 * PM) * (TM * 16) + half * PM * 16 + q % (2 * PM) * 8;
    };
    uint32_t doff[DC];
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        const int row = m0 + d_row(j) + lr;
        doff[j] = (uint32_t)((row < a.m ? row : a.m - 1) - m0) * (uint32_t)(2 * a.ldd) + 16u * lc;
    }
    // W: copy j is chunks 64c .. of the tile, c = wave + W j; chunk i of row r is stored at i ^ turn_of(r), so that
    // the 32 rows of a turned read, 16 bytes of each, fall on all banks
    auto turn_of = [](int r) __attribute__((always_inline)) { return CPR == 16 ? r & 15 : (r >> 1 & 3) | (r >> 3 & 1) << 2; };
    int w_row[WC];
    uint32_t w_col[WC];
#pragma unroll
    for (int j = 0; j < WC; ++j) {
        const int i = 64 * (wave + W * j) + lane;
        w_row[j] = i / CPR;
        const int col = k0 + 16 * (i % CPR ^ turn_of(w_row[j]));  // past the matrix: its last columns, not stored
        w_col[j] = (uint32_t)(col < a.k ? col : a.k - 16);
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const int steps = (a.n + kGStep - 1) / kGStep, row_blocks = (a.n + 127) / 128;
    const int64_t rows = (int64_t)a.parts * a.n;
    const uint32_t scale_col = [&]() {  // word i of the scales: of wave column i's block
        const int b = (k0 + 64 * (lane % WK)) / 128;
        return 4u * (uint32_t)(b < a.kb ? b : a.kb - 1);
    }();
    // Where a step's operands are.  Steps are asked for in order (the last one again past the end), s of `steps`
    // fastest, then the term, then the part; without branches, which between the products cost the large tile
    // its registers.
    constexpr int TERMS = kTerms<T>;
    struct Place {
        int step = 0, s = 0, term = 0, part = 0;
        const uint8_t *d, *w;
        uint32_t woff[WC];
    };
    const int rows_m1 = a.parts * a.n - 1;
    // what a step adds, the first of a term more than that, the first of a part more than both
    const int64_t d_term = 2 * a.plane - (int64_t)steps * 128, d_part = 2 * (a.part_cols - TERMS * a.plane);
    const int64_t w_next = (int64_t)kGStep * a.k, w_term = -(int64_t)steps * w_next, w_part = (int64_t)a.n * a.k;
    auto advance = [&](Place& p, int step) __attribute__((always_inline)) {
        const int on = step != p.step, next = on & (p.s == steps - 1), over = next & (p.term == TERMS - 1);
        p.step = step;
        p.s = (p.s + on) & (next - 1);
        p.term = (p.term + next) & (over - 1);
        p.part += over;
        p.d += (int64_t)128 * on + (d_term & -(int64_t)next) + (d_part & -(int64_t)over);
        p.w += (w_next & -(int64_t)on) + (w_term & -(int64_t)next) + (w_part & -(int64_t)over);
        const int left = rows_m1 - (p.part * a.n + p.s * kGStep);  // rows past the matrix: its last one
#pragma unroll
        for (int j = 0; j < WC; ++j) p.woff[j] = __umul24(min(+w_row[j], +left), a.k) + w_col[j];
    };
    auto copy_d = [&](const Place& p, int j, int to) __attribute__((always_inline)) {
        f8_copy16(p.d, doff[j], lds + (uint32_t)(to * STAGE + d_row(j) * 128));
    };
    auto copy_w = [&](const Place& p, int j, int to) __attribute__((always_inline)) {
        f8_copy16(p.w, p.woff[j], lds + (uint32_t)(to * STAGE + BM * 2 * kGStep + (wave + W * j) * 1024));
    };
    auto copy_scale = [&](const Place& p, int step) __attribute__((always_inline)) {
        f8_copy4(reinterpret_cast<const uint8_t*>(a.wd + __builtin_amdgcn_readfirstlane((p.part * row_blocks + (p.s >> 1)) * a.kb)), scale_col,
                 lds + (uint32_t)(D * STAGE + step % SCALES * 256));
    };

    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t d_at = (uint32_t)(wm * TM * 16 + l16) * 128 + 16u * (uint32_t)(g ^ (l16 & 7));
    // a turned read's source lanes: row 8g + l16 / 2 (and 32 on), 8 bytes l16 % 2 of its 16 columns
    const int t_row = 8 * g + (l16 >> 1);
    const uint32_t w_at = (uint32_t)(BM * 2 * kGStep + t_row * BK + 8 * (l16 & 1)), w_turn = 16u * (uint32_t)turn_of(t_row);
    static_assert(CPR != 16 || kGStep == 64, "rows 32 apart are stored alike");

    f8_f32x4 acc[4][TM];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
    u32x2 raw[4][2];  // codes of a column, rows 8g .. and 32 + 8g ..
    u32x4 av[4][2], bv[PM][2];
    float scale = 0.f, factor = 0.f;
    auto load = [&](int step, int h, int from) __attribute__((always_inline)) {
        const uint8_t* at = f8_smem + from * STAGE;
        if (h == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int o = 0; o < 2; ++o)
                    raw[i][o] = read_turned8(at + w_at + o * 32 * BK + ((uint32_t)(64 * wk + 16 * i) ^ w_turn));
            scale = reinterpret_cast<const float*>(f8_smem + D * STAGE)[step % SCALES * 64 + wk];
        }
#pragma unroll
        for (int j = 0; j < PM; ++j) {
            bv[j][0] = *reinterpret_cast<const u32x4*>(at + d_at + (h * PM + j) * 2048);
            bv[j][1] = *reinterpret_cast<const u32x4*>(at + (d_at ^ 64u) + (h * PM + j) * 2048);
        }
    };
    auto ready = [&](int, int h) __attribute__((always_inline)) {
        if (h) return;
        factor = scale;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o)
                av[i][o] = __builtin_bit_cast(u32x4, f8_widen((int)raw[i][o][0], (int)raw[i][o][1]));
    };
    // The sums of a fragment of columns join the accumulators while the next one's are on their way.
    f8_f32x4 t[PM] = {};
    auto join = [&](int h, int i, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][h * PM + j][e] = __builtin_fmaf(factor, t[j][e], acc[i][h * PM + j][e]);
    };
    auto multiply = [&](int h, auto&& side) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int j = 0; j < PM; ++j) {
                    if (o == 0 && i) join(h, i - 1, j);
                    t[j] = mfma_bf16(av[i][o], bv[j][o], o ? t[j] : f8_f32x4{0.f, 0.f, 0.f, 0.f});
                    if (j % 2 == 1) side((i * 2 + o) * (PM / 2) + j / 2);
                    __builtin_amdgcn_sched_barrier(0);
                }
    };
    auto finish = [&](int h) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PM; ++j) join(h, 3, j);
    };

    const int all = steps * a.parts * TERMS, begin = range * a.range_steps;
    const int total = all - begin < a.range_steps ? all - begin : a.range_steps;  // steps of this range
    Place px;
    px.s = begin % steps;
    px.term = begin / steps % TERMS;
    px.part = begin / steps / TERMS;
    px.d = reinterpret_cast<const uint8_t*>(a.d + (int64_t)m0 * a.ldd + px.part * a.part_cols + px.term * a.plane) + px.s * 128;
    px.w = a.w + px.part * ((int64_t)a.n * a.k) + px.s * w_next;
    Place py = px;
    if constexpr (W == 8) {
        f8_turns<XC + 1, YC>(
            wave >> 2, total,
            [&](int step, int i, int to) __attribute__((always_inline)) {
                if (i < 0) advance(px, step);
                else if (i < WC) copy_w(px, i, to);
                else if (i < XC) copy_d(px, i - WC, to);
                else copy_scale(px, step);
            },
            [&](int step, int i, int to) __attribute__((always_inline)) {
                if (i < 0) advance(py, step);
                else copy_d(py, DC - YC + i, to);
            },
            [&](int step, int h) __attribute__((always_inline)) { load(step, h, step & 1); }, finish, ready, multiply);
    } else {
        f8_ring<D, WC + DC + 1>(
            total,
            [&](int step, int to) __attribute__((always_inline)) {
                advance(px, step);
#pragma unroll
                for (int j = 0; j < WC; ++j) copy_w(px, j, to);
#pragma unroll
                for (int j = 0; j < DC; ++j) copy_d(px, j, to);
                copy_scale(px, step);
            },
            [&](int step, int from) __attribute__((always_inline)) {
                load(step, 0, from);
                ready(step, 0);
                multiply(0, [](int) {});
                finish(0);
            });
    }

    // element e of fragment i: column 16i + 4g + e of the wave's 64
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int row = m0 + (wm * TM + j) * 16 + l16;
        if (row >= a.m) continue;
        O* out = static_cast<O*>(a.dx) + range * a.range_stride + (int64_t)row * a.lddx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = k0 + wk * 64 + 16 * i + 4 * g;
            f8_store4(out + col, acc[i][j], a.k - col, a.vec);
        }
    }
}

template <int WK, int WM, int TM, int D, class T, class O = T>
hipError_t launch_input_grad_tile(F8InputGradArgs a, hipStream_t stream) {
    auto kernel = f8_input_grad_kernel<WK, WM, TM, D, T, O>;
    constexpr size_t lds = input_grad_lds_bytes<WK, WM, TM, D>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    a.m_tiles = (a.m + WM * TM * 16 - 1) / (WM * TM * 16);
    a.k_tiles = (a.k + WK * 64 - 1) / (WK * 64);
    const int64_t tiles = (int64_t)a.m_tiles * a.k_tiles * a.ranges;
    if (f8_grid(tiles) * (64 * WK * WM) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)f8_grid(tiles)), dim3(64 * WK * WM), lds, stream, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------ dw = d^T . x

struct F8WeightGradArgs {
    const uint16_t* d;
    int64_t d_plane, ldd, part_cols;
    const uint16_t* x;  // planes of the inputs' values [m up to a whole step][k]
    int64_t x_plane;
    void* dw;
    int64_t lddw;
    int n, parts, m, k;
    int k_tiles, n_tiles;  // n_tiles: of a part
    int ranges, range_steps;
    int64_t range_stride;
    bool vec;
    F8AddRangesArgs dx;    // small tiles: what dx still has to add, by the blocks from dx_block on
    unsigned dx_block;
};

template <int WK, int WN, int GN, int D>
constexpr size_t weight_grad_lds_bytes() {
    return D * (size_t)(WK + WN * GN) * 64 * 2 * kGStep;
}

// WK x WN waves, a wave 64 columns x 64 GN rows of dw.  A step is 64 activation rows; a tile's operands lie
// in LDS as runs of 64 columns, [64 rows][128 bytes] each.  Its sums stay in the instruction's accumulators: the same
// size 1234 us for its two pairs of planes, 1.34 PFLOP/s, matrix cores busy 60% of the cycles at a clock that they pull down to 1.8 - 2.0 GHz.
template <int WK, int WN, int GN, int D, class T, class O>
__global__ __launch_bounds__(64 * WK * WN) void f8_weight_grad_kernel(F8WeightGradArgs a) {
    constexpr int W = WK * WN, BK = WK * 64, BN = WN * GN * 64;
    constexpr int PARTS = W == 8 ? 2 : 1, PN = GN / PARTS;
    constexpr int XR = WK, DR = WN * GN, RUN = 128 * kGStep;     // runs of x and of d, bytes of one
    constexpr int XC = XR * 8 / W, DC = DR * 8 / W;              // copies of a wave: eight rows of a run each
    constexpr int YC = W == 8 ? DC / 2 : 0, FIRST = XC + DC - YC;  // pieces of f8_turns: Y is the groups' last runs
    static_assert(XR * 8 % W == 0 && DR * 8 % W == 0, "copies divide evenly");
    static_assert(W != 8 || (D == 2 && WN == 2 && GN == 2), "pieces divide evenly");
    constexpr int STAGE = (XR + DR) * RUN;
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK;
    if constexpr (W != 8) {
        if (blockIdx.x >= a.dx_block) {
            f8_add_ranges<T>(a.dx, (int64_t)(blockIdx.x - a.dx_block) * (64 * W) + tid, (int64_t)(gridDim.x - a.dx_block) * (64 * W));
            return;
        }
    }
    const F8Tile tile = f8_tile_of_block((int)blockIdx.x, a.k_tiles, a.n_tiles * a.parts * a.ranges);
    if (!tile.inside) return;  // block-uniform, before any barrier
    const int range = tile.col / (a.n_tiles * a.parts), col = tile.col - range * (a.n_tiles * a.parts);
    const int part = col / a.n_tiles, n0 = (col - part * a.n_tiles) * BN, k0 = tile.row * BK;

    // Copy c of an operand: rows 8(c % 8) .. of run c / 8.  The 32-byte blocks of row r are stored at
    // block ^ turn_of(r), so that the 16 rows of a turned read, 32 bytes of each, fall on all banks.
    auto turn_of = [](int r) __attribute__((always_inline)) { return (r >> 1 & 1) | (r >> 3 & 1) << 1; };
    auto run_of = [&](int j) __attribute__((always_inline)) {  // d's copy j: half 0 first, then half 1 of every group
        const int c = wave + W * (j < DC - YC ? j : j - (DC - YC));
        return W != 8 ? c / 8 : c / 8 * GN + (j < DC - YC ? 0 : 1);
    };
    auto row_of = [&](int j) __attribute__((always_inline)) { return (wave + W * j) % 8 * 8 + (lane >> 3); };
    auto chunk_of = [&](int j) __attribute__((always_inline)) { return (lane & 7) ^ turn_of(row_of(j)) << 1; };
    uint32_t xoff[XC];
    int dcol[DC];
#pragma unroll
    for (int j = 0; j < XC; ++j) {
        const int at = k0 + 64 * ((wave + W * j) / 8) + 8 * chunk_of(j);  // past the matrix: its last columns, not stored
        xoff[j] = 2u * ((uint32_t)row_of(j) * (uint32_t)a.k + (uint32_t)(at < a.k ? at : a.k - 8));
    }
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        const int at = n0 + 64 * run_of(j) + 8 * chunk_of(j), columns = (a.n + 7) / 8 * 8;
        dcol[j] = 2 * (at < columns ? at : columns - 8);
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const int steps = (a.m + kGStep - 1) / kGStep;
    // the pairs of planes (d's, x's) whose products count: (0, 0), then (0, 1), (1, 0), then (0, 2), (1, 1), (2, 0); of
    // one part of d the first two
    auto d_of = [](int pair) { return pair < 2 ? 0 : pair == 2 ? 1 : pair - 3; };
    auto x_of = [](int pair) { return pair < 2 ? pair : pair == 2 ? 0 : 5 - pair; };
    constexpr int PAIRS = kPairs<T>;
    struct Place {
        int step = 0, s = 0, pair = 0;
        const uint8_t *x, *d;
    };
    const uint8_t* x0 = reinterpret_cast<const uint8_t*>(a.x);
    const uint8_t* d0 = reinterpret_cast<const uint8_t*>(a.d + part * a.part_cols);
    const int64_t x_next = (int64_t)2 * kGStep * a.k, d_next = (int64_t)2 * kGStep * a.ldd;
    auto advance = [&](Place& p, int step) __attribute__((always_inline)) {
        const bool on = step != p.step, next = on && p.s == steps - 1;
        p.step = step;
        p.s = next ? 0 : p.s + (on ? 1 : 0);
        p.x += on ? x_next : 0;
        p.d += on ? d_next : 0;
        p.pair += next ? 1 : 0;
        p.x = next ? x0 + 2 * x_of(p.pair) * a.x_plane : p.x;
        p.d = next ? d0 + 2 * d_of(p.pair) * a.d_plane : p.d;
    };
    auto copy_x = [&](const Place& p, int j, int to) __attribute__((always_inline)) {
        f8_copy16(p.x, xoff[j], lds + (uint32_t)(to * STAGE + (wave + W * j) * 1024));
    };
    auto copy_d = [&](const Place& p, int j, int to) __attribute__((always_inline)) {
        const int left = a.m - 1 - p.s * kGStep, row = row_of(j);  // rows past the operand: its last one
        f8_copy16(p.d, 2u * __umul24(min(+row, +left), (int)a.ldd) + (uint32_t)dcol[j],
                  lds + (uint32_t)(to * STAGE + (XR + run_of(j)) * RUN + (wave + W * j) % 8 * 1024));
    };

    const int l16 = lane & 15, g = lane >> 4;
    // a turned read's source lanes: row 8g + l16 / 4 (and 4, 32, 36 on), 8 bytes l16 % 4 of its 16 columns
    const int t_row = 8 * g + (l16 >> 2);
    const uint32_t lane_at = (uint32_t)(t_row * 128 + 8 * (l16 & 3)), lane_turn = 32u * (uint32_t)turn_of(t_row);
    // fragment c (16 columns) of the run at `at`, half h of a step
    auto fragment = [&](const uint8_t* at, int c, int h) __attribute__((always_inline)) {
        const uint8_t* from = at + 32 * h * 128 + lane_at + ((uint32_t)(32 * c) ^ lane_turn);
        const u32x2 lo = read_turned16(from), hi = read_turned16(from + 4 * 128);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };

    f8_f32x4 acc[4][GN][4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < GN; ++j)
#pragma unroll
            for (int o = 0; o < 4; ++o) acc[c][j][o] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 fa[4][2], fb[PN][4][2];
    auto load = [&](int h, int from) __attribute__((always_inline)) {
        const uint8_t* at = f8_smem + from * STAGE;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
#pragma unroll
                for (int j = 0; j < PN; ++j) fb[j][c][o] = fragment(at + (XR + wn * GN + h * PN + j) * RUN, c, o);
                if (h == 0) fa[c][o] = fragment(at + wk * RUN, c, o);
            }
    };
    auto multiply = [&](int h, auto&& side) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PN; ++j)
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        acc[q][h * PN + j][v] = mfma_bf16(fa[q][o], fb[j][v][o], acc[q][h * PN + j][v]);
                        const int p = ((j * 2 + o) * 4 + q) * 4 + v;
                        if (p % 2 == 1) side(p / 2);
                        __builtin_amdgcn_sched_barrier(0);
                    }
    };

    const int all = steps * PAIRS, begin = range * a.range_steps;
    const int total = all - begin < a.range_steps ? all - begin : a.range_steps;  // steps of this range
    Place px;
    px.s = begin % steps;
    px.pair = begin / steps;
    px.x = x0 + 2 * x_of(px.pair) * a.x_plane + px.s * x_next;
    px.d = d0 + 2 * d_of(px.pair) * a.d_plane + px.s * d_next;
    Place py = px;
    if constexpr (W == 8) {
        f8_turns<FIRST, YC>(
            wave >> 2, total,
            [&](int step, int i, int to) __attribute__((always_inline)) {
                if (i < 0) advance(px, step);
                else if (i < XC) copy_x(px, i, to);
                else copy_d(px, i - XC, to);
            },
            [&](int step, int i, int to) __attribute__((always_inline)) {
                if (i < 0) advance(py, step);
                else copy_d(py, DC - YC + i, to);
            },
            [&](int step, int h) __attribute__((always_inline)) { load(h, step & 1); }, [](int) {}, [](int, int) {}, multiply);
    } else {
        f8_ring<D, XC + DC>(
            total,
            [&](int step, int to) __attribute__((always_inline)) {
                advance(px, step);
#pragma unroll
                for (int j = 0; j < XC; ++j) copy_x(px, j, to);
#pragma unroll
                for (int j = 0; j < DC; ++j) copy_d(px, j, to);
            },
            [&](int, int from) __attribute__((always_inline)) {
                load(0, from);
                multiply(0, [](int) {});
            });
    }

    // element e of fragment q: column 16q + 4g + e of the wave's 64; fragment (j, v): row 64j + 16v + l16
#pragma unroll
    for (int j = 0; j < GN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = n0 + (wn * GN + j) * 64 + 16 * v + l16;
            if (row >= a.n) continue;
            O* out = static_cast<O*>(a.dw) + range * a.range_stride + ((int64_t)part * a.n + row) * a.lddw;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = k0 + wk * 64 + 16 * q + 4 * g;
                f8_store4(out + c, acc[q][j][v], a.k - c, a.vec);
            }
        }
}

template <int WK, int WN, int GN, int D, class T, class O = T>
hipError_t launch_weight_grad_tile(F8WeightGradArgs a, hipStream_t stream) {
    auto kernel = f8_weight_grad_kernel<WK, WN, GN, D, T, O>;
    constexpr size_t lds = weight_grad_lds_bytes<WK, WN, GN, D>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    constexpr int BK = WK * 64, BN = WN * GN * 64;
    a.k_tiles = (a.k + BK - 1) / BK;
    a.n_tiles = (a.n + BN - 1) / BN;
    const int64_t tiles = (int64_t)a.k_tiles * a.n_tiles * a.parts * a.ranges;
    a.dx_block = (unsigned)f8_grid(tiles);
    const int64_t blocks = f8_grid(tiles) + (a.dx.sums ? part_blocks(a.dx.rows * (a.dx.k / 4)) : 0);
    if (blocks * (64 * WK * WN) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * WK * WN), lds, stream, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------- the calls

template <class T>
bool rows_aligned(const void* p, int64_t ld, int elements) {
    return ld % elements == 0 && reinterpret_cast<uintptr_t>(p) % (elements * sizeof(T)) == 0;
}

template <class T>
hipError_t zero_rows(void* out, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
    if (!out || rows == 0) return hipSuccess;
    hipLaunchKernelGGL(f8_zero_rows_kernel<T>, dim3(part_blocks(rows * cols)), dim3(kPartThreads), 0, stream,
                       static_cast<T*>(out), rows, cols, ld);
    return hipGetLastError();
}

template <class T>
hipError_t add_ranges(const F8AddRangesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(f8_add_ranges_kernel<T>, dim3(part_blocks(a.rows * (a.k / 4))), dim3(kPartThreads), 0, stream, a);
    return hipGetLastError();
}

template <class T, int TERMS>
hipError_t backward(const uint8_t* wq, const float* wd, int64_t n, int parts, int64_t k,
                    const uint8_t* xq, const float* xd, int64_t m, const void* gu, int64_t ldgu, const void* d,
                    int type, int64_t ldd, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                    hipStream_t stream) {
    if (m == 0) return zero_rows<T>(dw, parts * n, k, lddw, stream);
    if (n == 0) return zero_rows<T>(dx, m, k, lddx, stream);
    const q8v::F8BackwardWorkspace ws = q8v::f8_backward_layout(m, n, parts, k, type);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    uint16_t* planes = reinterpret_cast<uint16_t*>(base + ws.d_off);
    uint16_t* values = reinterpret_cast<uint16_t*>(base + ws.x_off);
    float* dx_sums = reinterpret_cast<float*>(base + ws.sums_off);
    float* dw_sums = reinterpret_cast<float*>(base + ws.dw_sums_off);
    const q8v::F8GradPlan dx_plan = q8v::f8_dx_plan(m, n, parts, k, type), dw_plan = q8v::f8_dw_plan(m, n, parts, k, type);
    F8AddRangesArgs add{};  // what dx still has to add: by the tiles' launch of dw if that is of small tiles, else by one of its own
    const int kb = (int)((k + 127) / 128);
    hipError_t e = hipSuccess;

    F8PlanesArgs p{};
    p.d = d; p.gu = gu; p.q = xq; p.xd = xd; p.planes = planes; p.values = values;
    p.ldd = ldd; p.ldgu = ldgu; p.ldo = ws.ldd; p.m = m; p.rows = (m + kGStep - 1) / kGStep * kGStep;
    p.n = (int)n; p.k = (int)k; p.kb = kb;
    p.vec = rows_aligned<T>(d, ldd, 8) && (parts == 1 || rows_aligned<T>(gu, ldgu, 8));
    const uint16_t* dp = planes;
    int64_t ldp = ws.ldd;
    int kind = parts == 2 ? kBehindSilu : kSplit;
    if (parts == 1 && TERMS == 1 && n % kGStep == 0 && ldd <= (int64_t(1) << 22) && rows_aligned<T>(d, ldd, 8)) {
        dp = static_cast<const uint16_t*>(d);  // bf16 rows are their own plane
        ldp = ldd;
        kind = kNoPlanes;
    }
    p.d_blocks = kind == kNoPlanes ? 0 : part_blocks(m * (ws.ldd / (parts == 2 ? 16 : 8)));
    const unsigned blocks = p.d_blocks + (dw ? part_blocks(p.rows * (k / 8)) : 0);
    if (blocks) {
        auto kernel = kind == kNoPlanes ? f8_planes_kernel<T, TERMS, kNoPlanes>
                      : kind == kSplit  ? f8_planes_kernel<T, TERMS, kSplit>
                                        : f8_planes_kernel<T, TERMS, kBehindSilu>;
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kPartThreads), 0, stream, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }

    if (dx) {
        F8InputGradArgs a{};
        a.d = dp; a.plane = m * ldp; a.ldd = ldp; a.part_cols = ldp / parts;
        a.w = wq; a.wd = wd; a.dx = dx; a.lddx = lddx;
        a.n = (int)n; a.parts = parts; a.m = (int)m; a.k = (int)k; a.kb = kb;
        a.vec = rows_aligned<T>(dx, lddx, 4);
        const q8v::F8GradPlan plan = dx_plan;
        const int64_t steps = parts * TERMS * ((n + kGStep - 1) / kGStep);
        a.range_steps = (int)((steps + plan.ranges - 1) / plan.ranges);
        a.ranges = (int)((steps + a.range_steps - 1) / a.range_steps);
        if (a.ranges > 1) {
            add = {dx_sums, dx, m, lddx, a.ranges, (int)k, a.vec};
            a.dx = dx_sums; a.lddx = k; a.vec = true; a.range_stride = m * k;
            e = launch_input_grad_tile<2, 2, 2, 6, T, float>(a, stream);
            if (e == hipSuccess && (!dw || dw_plan.big)) e = add_ranges<T>(add, stream);
        } else {
            e = plan.big ? launch_input_grad_tile<4, 2, 8, 2, T>(a, stream) : launch_input_grad_tile<2, 2, 2, 6, T>(a, stream);
        }
        if (e != hipSuccess) return e;
    }
    if (dw) {
        F8WeightGradArgs a{};
        a.d = dp; a.d_plane = m * ldp; a.ldd = ldp; a.part_cols = ldp / parts;
        a.x = values; a.x_plane = p.rows * k; a.dw = dw; a.lddw = lddw;
        a.n = (int)n; a.parts = parts; a.m = (int)m; a.k = (int)k;
        a.vec = rows_aligned<T>(dw, lddw, 4);
        const q8v::F8GradPlan plan = dw_plan;
        if (!plan.big) a.dx = add;
        const int64_t steps = kPairs<T> * (p.rows / kGStep);
        a.range_steps = (int)((steps + plan.ranges - 1) / plan.ranges);
        a.ranges = (int)((steps + a.range_steps - 1) / a.range_steps);
        if (a.ranges > 1) {
            const F8AddRangesArgs dw_add{dw_sums, dw, parts * n, lddw, a.ranges, (int)k, a.vec};
            a.dw = dw_sums; a.lddw = k; a.vec = true; a.range_stride = parts * n * k;
            if ((e = launch_weight_grad_tile<2, 2, 1, 4, T, float>(a, stream)) != hipSuccess) return e;
            e = add_ranges<T>(dw_add, stream);
        } else {
            e = plan.big ? launch_weight_grad_tile<4, 2, 2, 2, T>(a, stream) : launch_weight_grad_tile<2, 2, 1, 4, T>(a, stream);
        }
    }
    return e;
}

}  // namespace

hipError_t launch_f8_backward(const uint8_t* wq, const float* wd, int64_t n, int parts,
                              int64_t k, const uint8_t* xq, const float* xd, int64_t m, const void* gu, int64_t ldgu,
                              const void* d, int type, int64_t ldd, void* dx, int64_t lddx, void* dw, int64_t lddw,
                              void* workspace, hipStream_t stream) {
    switch (type) {
        case Q8_F32:
            return backward<float, 3>(wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw, lddw,
                                      workspace, stream);
        case Q8_F16:
            return backward<_Float16, 2>(wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw,
                                         lddw, workspace, stream);
        default:
            return backward<__bf16, 1>(wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw, lddw,
                                       workspace, stream);
    }
}

}  // namespace q8k
