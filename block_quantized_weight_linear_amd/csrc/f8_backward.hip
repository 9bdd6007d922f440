// Gradients of the block-scaled 8-bit floating-point linears on the bf16 matrix cores of gfx950
// (v_mfma_f32_16x16x32_bf16, float32 accumulation):
//   dx[t][i] = sum_j d[t][j] wd[j/128][i/128] wq[j][i]      dw[j][i] = sum_t d[t][j] x[t][i]
// with d the gradient of the products (the call's own, or behind SiLU(gate) * up its two parts
// beside each other) and x the inputs' values.
//
// An e4m3 code is exact in bf16.  A float operand is a sum of bf16 parts (one for bf16 gradients,
// two for binary16, three for float32), laid out as planes by a first launch; a product runs over
// the planes (dw: over the pairs of planes that matter) as if they were further terms of its sum.
//
// Both sums run over an axis that is not the contiguous one of W (dx), or of both operands (dw).
// Fragments are turned in registers: a lane reads eight rows' neighbouring elements of its columns
// from LDS and puts the rows of each column side by side with byte permutes.  A fragment's 16
// columns so are every fourth (eighth) of a run of 64 (128); the lane that holds four neighbouring
// results of each of these fragments has 16 (32) neighbouring columns of one output row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "f8_tile.h"
#include "q8_internal.h"
#include "q8_validate.h"

namespace q8k {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f8_f32x4 mfma_bf16(u32x4 a, u32x4 b, f8_f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(f8_bf16x8, a), __builtin_bit_cast(f8_bf16x8, b), c,
                                                   0, 0, 0);
}

// ------------------------------------------------------------------------------ bf16 parts

// v as TERMS bf16 parts, each the rest rounded to nearest even: of 24 bits the first leaves 16, the
// second 7, so that three parts are a float32 and two a binary16 exactly (remainders are exact).
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

// The planes of a gradient [m][n].
template <class T, int TERMS>
__global__ __launch_bounds__(kPartThreads) void f8_split_kernel(const T* __restrict__ d, int64_t m, int n, int64_t ldd,
                                                               bool vec, uint16_t* __restrict__ out, int64_t ldo) {
    const int64_t per_row = ldo / 8, total = m * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPartThreads) {
        const int64_t row = i / per_row, col = 8 * (i - row * per_row);
        float v[8];
        load_row8(d + row * ldd, col, n, vec, v);
        store_parts<TERMS>(out + row * ldo + col, m * ldo, v);
    }
}

// The planes of the gate's and up's gradients, [m][dg | du]; each a value of type T.
template <class T, int TERMS>
__global__ __launch_bounds__(kPartThreads) void f8_gate_up_gradient_kernel(const T* __restrict__ gu, int64_t ldgu,
                                                                          const T* __restrict__ dh, int64_t lddh,
                                                                          int64_t m, int f, bool vec,
                                                                          uint16_t* __restrict__ out, int64_t ldo) {
    const int64_t per_row = ldo / 16, total = m * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPartThreads) {
        const int64_t row = i / per_row, col = 8 * (i - row * per_row);
        float g[8], u[8], h[8], dg[8], du[8];
        load_row8(gu + row * ldgu, col, f, vec, g);
        load_row8(gu + row * ldgu + f, col, f, vec && f % 8 == 0, u);
        load_row8(dh + row * lddh, col, f, vec, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = 1.0f / (1.0f + __expf(-g[e]));
            dg[e] = (float)f8_round<T>(h[e] * u[e] * (s * (1.0f + g[e] * (1.0f - s))));
            du[e] = (float)f8_round<T>(h[e] * (g[e] * s));
        }
        uint16_t* at = out + row * ldo + col;
        store_parts<TERMS>(at, m * ldo, dg);
        store_parts<TERMS>(at + ldo / 2, m * ldo, du);
    }
}

// The planes of the inputs' values [m][k].
template <int TERMS>
__global__ __launch_bounds__(kPartThreads) void f8_values_kernel(const uint8_t* __restrict__ q,
                                                                const float* __restrict__ d, int64_t m, int k, int kb,
                                                                uint16_t* __restrict__ out) {
    const int64_t per_row = k / 8, total = m * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPartThreads) {
        const int64_t row = i / per_row, col = 8 * (i - row * per_row);
        const u32x2 c = *reinterpret_cast<const u32x2*>(q + row * k + col);
        const float s = d[row * kb + col / 128];
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 0) * s;
            v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 1) * s;
            v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 2) * s;
            v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)c[h], 3) * s;
        }
        store_parts<TERMS>(out + row * k + col, m * k, v);
    }
}

template <class T>
__global__ __launch_bounds__(kPartThreads) void f8_zero_rows_kernel(T* __restrict__ out, int64_t rows, int64_t cols,
                                                                   int64_t ld) {
    const int64_t total = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPartThreads)
        out[i / cols * ld + i % cols] = (T)0.f;
}

unsigned part_blocks(int64_t threads) {
    const int64_t b = (threads + kPartThreads - 1) / kPartThreads;
    return (unsigned)(b < 65536 ? (b ? b : 1) : 65536);
}

// -------------------------------------------------------------------------------- dx = d . W

struct F8InputGradArgs {
    const uint16_t* d;  // planes of bf16 parts
    int64_t plane;      // elements from one to the next
    int64_t ldd;
    int64_t part_cols;  // columns from one part's gradients to the next's
    const uint8_t* w;
    const float* wd;
    void* dx;
    int64_t lddx;
    int n, parts, terms, m, k, kb;
    int m_tiles, k_tiles;
    bool vec;
};

constexpr int kGStep = 64;  // terms of the sum a step

template <int WK, int WM, int TM>
constexpr size_t input_grad_lds_bytes() {
    return 2 * ((size_t)WM * TM * 16 * 2 * kGStep + (size_t)WK * 128 * kGStep);
}

// WK x WM waves, a wave 128 columns of dx (eight fragments) x 16 TM rows.  A step is 64 rows of W,
// all in one block of its scales: the step's sums start at zero and join the accumulators times
// the scale.
template <int WK, int WM, int TM, class T>
__global__ __launch_bounds__(64 * WK * WM) void f8_input_grad_kernel(F8InputGradArgs a) {
    constexpr int W = WK * WM, BK = WK * 128, BM = WM * TM * 16;
    constexpr int DC = BM / 8 / W;             // copies of d of a wave: eight rows of 128 bytes each
    constexpr int CPR = BK / 16;               // 16-byte chunks of a row of W
    constexpr int WC = kGStep * CPR / 64 / W;  // copies of W of a wave
    static_assert(BM / 8 % W == 0 && kGStep * CPR / 64 % W == 0, "copies divide evenly");
    constexpr int STAGE = BM * 2 * kGStep + BK * kGStep;
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wm = wave / WK;
    const F8Tile tile = f8_tile_of_block((int)blockIdx.x, a.m_tiles, a.k_tiles);
    if (!tile.inside) return;  // block-uniform, before any barrier
    const int m0 = tile.row * BM, k0 = tile.col * BK;

    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
    uint32_t doff[DC], woff[WC];
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        const int row = m0 + 8 * (wave + W * j) + lr;
        doff[j] = (uint32_t)((row < a.m ? row : a.m - 1) - m0) * (uint32_t)(2 * a.ldd) + 16u * lc;
    }
#pragma unroll
    for (int j = 0; j < WC; ++j) {
        const int i = 64 * (wave + W * j) + lane;
        const int col = k0 + 16 * (i % CPR);  // past the matrix: its last columns, whose results are not stored
        woff[j] = (uint32_t)(i / CPR) * (uint32_t)a.k + (uint32_t)(col < a.k ? col : a.k - 16);
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const int steps = (a.n + kGStep - 1) / kGStep;
    const uint8_t* d0 = reinterpret_cast<const uint8_t*>(a.d + (int64_t)m0 * a.ldd);
    auto copy = [&](int part, int term, int s, int stage) __attribute__((always_inline)) {
        const uint8_t* db = d0 + 2 * (term * a.plane + part * a.part_cols + (int64_t)s * kGStep);
        const uint8_t* wb = a.w + ((int64_t)part * a.n + (int64_t)s * kGStep) * a.k;
        const uint32_t at = lds + (uint32_t)(stage * STAGE);
        const int left = a.n - s * kGStep;  // rows of W; d has zeros from there to a multiple of eight
        const bool cut = left < kGStep;
#pragma unroll
        for (int j = 0; j < DC; ++j) {
            const uint32_t to = at + (uint32_t)(wave + W * j) * 1024;
            if (!cut) f8_copy16(db, doff[j], to);
            else f8_copy16_or_zeros(db, doff[j], lc * 8 < left, to);
        }
#pragma unroll
        for (int j = 0; j < WC; ++j) {
            const uint32_t to = at + (uint32_t)(BM * 2 * kGStep) + (uint32_t)(wave + W * j) * 1024;
            if (!cut) f8_copy16(wb, woff[j], to);
            else f8_copy16_or_zeros(wb, woff[j], (64 * (wave + W * j) + lane) / CPR < left, to);
        }
    };

    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t d_at = (uint32_t)(wm * TM * 16 + l16) * 128 + 16u * (uint32_t)(g ^ (l16 & 7));
    const uint32_t w_at = (uint32_t)(BM * 2 * kGStep) + (uint32_t)(8 * g) * BK + (uint32_t)(wk * 128 + 8 * l16);
    const int kblock = (k0 + wk * 128) / 128 < a.kb ? (k0 + wk * 128) / 128 : a.kb - 1;
    const int row_blocks = (a.n + 127) / 128;

    f8_f32x4 acc[8][TM];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f8_f32x4{0.f, 0.f, 0.f, 0.f};

    const int total = steps * a.parts * a.terms;
    int part = 0, term = 0, s = 0, npart = 0, nterm = 0, ns = 0;
    auto next = [&]() __attribute__((always_inline)) {  // the step after (npart, nterm, ns)
        if (++ns == steps) {
            ns = 0;
            if (++nterm == a.terms) {
                nterm = 0;
                ++npart;
            }
        }
    };
    copy(0, 0, 0, 0);
    wait_vmcnt_mem<0>();
    __syncthreads();
    for (int c = 0; c < total; ++c) {
        const int stage = c & 1;
        next();
        if (c + 1 < total) copy(npart, nterm, ns, stage ^ 1);
        const uint32_t at = (uint32_t)(stage * STAGE);
        const float scale = f8_uniform(a.wd + (int64_t)(part * row_blocks + s / 2) * a.kb + kblock);
        u32x2 raw[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                raw[h][i] = *reinterpret_cast<const u32x2*>(f8_smem + at + w_at + (32 * h + i) * BK);
        u32x4 b[TM][2];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            b[j][0] = *reinterpret_cast<const u32x4*>(f8_smem + at + d_at + j * 2048);
            b[j][1] = *reinterpret_cast<const u32x4*>(f8_smem + ((at + d_at + j * 2048) ^ 64u));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // columns 2q and 2q + 1 of the lane's eight
            u32x4 av[2][2];            // [column][half of the step]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint32_t v = __builtin_amdgcn_perm(raw[h][2 * p + 1][q >> 1], raw[h][2 * p][q >> 1],
                                                             q & 1 ? 0x07030602u : 0x05010400u);
                    av[0][h][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
                    av[1][h][p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
                }
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    f8_f32x4 t = mfma_bf16(av[o][0], b[j][0], f8_f32x4{0.f, 0.f, 0.f, 0.f});
                    t = mfma_bf16(av[o][1], b[j][1], t);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[2 * q + o][j][e] = __builtin_fmaf(scale, t[e], acc[2 * q + o][j][e]);
                }
        }
        part = npart;
        term = nterm;
        s = ns;
        wait_vmcnt_mem<0>();
        __syncthreads();
    }
    (void)term;

    // element e of fragment i: column 32g + 8e + i of the wave's 128
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int row = m0 + (wm * TM + j) * 16 + l16;
        if (row >= a.m) continue;
        T* out = static_cast<T*>(a.dx) + (int64_t)row * a.lddx;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = k0 + wk * 128 + 32 * g + 8 * e;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                f8_store4(out + col + 4 * h,
                          f8_f32x4{acc[4 * h][j][e], acc[4 * h + 1][j][e], acc[4 * h + 2][j][e], acc[4 * h + 3][j][e]},
                          a.k - col - 4 * h, a.vec);
        }
    }
}

template <int WK, int WM, int TM, class T>
hipError_t launch_input_grad_tile(F8InputGradArgs a, hipStream_t stream) {
    auto kernel = f8_input_grad_kernel<WK, WM, TM, T>;
    constexpr size_t lds = input_grad_lds_bytes<WK, WM, TM>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    a.m_tiles = (a.m + WM * TM * 16 - 1) / (WM * TM * 16);
    a.k_tiles = (a.k + WK * 128 - 1) / (WK * 128);
    const int64_t tiles = (int64_t)a.m_tiles * a.k_tiles;
    if (f8_grid(tiles) * (64 * WK * WM) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)f8_grid(tiles)), dim3(64 * WK * WM), lds, stream, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------ dw = d^T . x

struct F8WeightGradArgs {
    const uint16_t* d;
    int64_t d_plane, ldd, part_cols;
    const uint16_t* x;  // planes of the inputs' values [m][k]
    int64_t x_plane;
    void* dw;
    int64_t lddw;
    int n, parts, pairs, m, k;
    int k_tiles, n_tiles;  // n_tiles: of a part
    bool vec;
};

template <int WK, int WN, int GK, int GN>
constexpr size_t weight_grad_lds_bytes() {
    return 2 * (size_t)(WK * GK + WN * GN) * 64 * 2 * kGStep;
}

// WK x WN waves, a wave 64 GK columns x 64 GN rows of dw.  A step is 64 activation rows.
template <int WK, int WN, int GK, int GN, class T>
__global__ __launch_bounds__(64 * WK * WN) void f8_weight_grad_kernel(F8WeightGradArgs a) {
    constexpr int W = WK * WN, BK = WK * GK * 64, BN = WN * GN * 64;
    constexpr int XR = BK / 8, DR = BN / 8;  // 16-byte chunks of a row of x, of d
    constexpr int XC = kGStep * XR / 64 / W, DC = kGStep * DR / 64 / W;
    static_assert(kGStep * XR / 64 % W == 0 && kGStep * DR / 64 % W == 0, "copies divide evenly");
    constexpr int STAGE = (BK + BN) * 2 * kGStep;
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK;
    const F8Tile tile = f8_tile_of_block((int)blockIdx.x, a.k_tiles, a.n_tiles * a.parts);
    if (!tile.inside) return;  // block-uniform, before any barrier
    const int part = tile.col / a.n_tiles, n0 = (tile.col - part * a.n_tiles) * BN, k0 = tile.row * BK;
    const int n_cols = (a.n + 7) / 8 * 8;  // columns of a part's planes

    uint32_t xoff[XC], doff[DC];
#pragma unroll
    for (int j = 0; j < XC; ++j) {
        const int i = 64 * (wave + W * j) + lane, col = k0 + 8 * (i % XR);
        xoff[j] = (uint32_t)(i / XR) * (uint32_t)(2 * a.k) + 2u * (uint32_t)(col < a.k ? col : a.k - 8);
    }
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        const int i = 64 * (wave + W * j) + lane, col = n0 + 8 * (i % DR);
        doff[j] = (uint32_t)(i / DR) * (uint32_t)(2 * a.ldd) + 2u * (uint32_t)(col < n_cols ? col : n_cols - 8);
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const int steps = (a.m + kGStep - 1) / kGStep;
    // the pairs of planes whose products count: (0, 0), then (0, 1), (1, 0), then (0, 2), (1, 1), (2, 0)
    auto d_of = [](int pair) { return pair < 2 ? 0 : pair == 2 ? 1 : pair - 3; };
    auto x_of = [](int pair) { return pair < 2 ? pair : pair == 2 ? 0 : 5 - pair; };
    auto copy = [&](int pair, int s, int stage) __attribute__((always_inline)) {
        const uint8_t* xb = reinterpret_cast<const uint8_t*>(a.x + x_of(pair) * a.x_plane + (int64_t)s * kGStep * a.k);
        const uint8_t* db = reinterpret_cast<const uint8_t*>(a.d + d_of(pair) * a.d_plane + part * a.part_cols +
                                                             (int64_t)s * kGStep * a.ldd);
        const uint32_t at = lds + (uint32_t)(stage * STAGE);
        const int left = a.m - s * kGStep;
        const bool cut = left < kGStep;
#pragma unroll
        for (int j = 0; j < XC; ++j) {
            const uint32_t to = at + (uint32_t)(wave + W * j) * 1024;
            if (!cut) f8_copy16(xb, xoff[j], to);
            else f8_copy16_or_zeros(xb, xoff[j], (64 * (wave + W * j) + lane) / XR < left, to);
        }
#pragma unroll
        for (int j = 0; j < DC; ++j) {
            const uint32_t to = at + (uint32_t)(BK * 2 * kGStep) + (uint32_t)(wave + W * j) * 1024;
            if (!cut) f8_copy16(db, doff[j], to);
            else f8_copy16_or_zeros(db, doff[j], (64 * (wave + W * j) + lane) / DR < left, to);
        }
    };

    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t x_at = (uint32_t)(8 * g) * (2 * BK) + (uint32_t)(wk * GK * 64 + 4 * l16) * 2;
    const uint32_t d_at = (uint32_t)(BK * 2 * kGStep) + (uint32_t)(8 * g) * (2 * BN) + (uint32_t)(wn * GN * 64 + 4 * l16) * 2;
    // fragments of four neighbouring columns a lane, 32 rows from LDS rows of ROW bytes
    auto turn = [&](auto row_bytes, uint32_t at, u32x4 (&f)[4]) __attribute__((always_inline)) {
        constexpr int ROW = decltype(row_bytes)::value;
        u32x2 raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const u32x2*>(f8_smem + at + i * ROW);
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                f[c][p] = __builtin_amdgcn_perm(raw[2 * p + 1][c >> 1], raw[2 * p][c >> 1],
                                                c & 1 ? 0x07060302u : 0x05040100u);
    };

    f8_f32x4 acc[GK][4][GN][4];
#pragma unroll
    for (int i = 0; i < GK; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < GN; ++j)
#pragma unroll
                for (int o = 0; o < 4; ++o) acc[i][c][j][o] = f8_f32x4{0.f, 0.f, 0.f, 0.f};

    const int total = steps * a.pairs;
    int npair = 0, ns = 0;
    copy(0, 0, 0);
    wait_vmcnt_mem<0>();
    __syncthreads();
    for (int c = 0; c < total; ++c) {
        const int stage = c & 1;
        if (++ns == steps) {
            ns = 0;
            ++npair;
        }
        if (c + 1 < total) copy(npair, ns, stage ^ 1);
        const uint32_t at = (uint32_t)(stage * STAGE);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 fb[GN][4];
#pragma unroll
            for (int j = 0; j < GN; ++j)
                turn(std::integral_constant<int, 2 * BN>{}, at + d_at + 128 * j + 32 * h * 2 * BN, fb[j]);
#pragma unroll
            for (int i = 0; i < GK; ++i) {
                u32x4 fa[4];
                turn(std::integral_constant<int, 2 * BK>{}, at + x_at + 128 * i + 32 * h * 2 * BK, fa);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < GN; ++j)
#pragma unroll
                        for (int o = 0; o < 4; ++o) acc[i][q][j][o] = mfma_bf16(fa[q], fb[j][o], acc[i][q][j][o]);
            }
        }
        wait_vmcnt_mem<0>();
        __syncthreads();
    }

    // element e of fragment (i, q): column 64i + 16g + 4e + q of the wave; fragment (j, o): row 64j + 4 l16 + o
#pragma unroll
    for (int j = 0; j < GN; ++j)
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            const int row = n0 + wn * GN * 64 + 64 * j + 4 * l16 + o;
            if (row >= a.n) continue;
            T* out = static_cast<T*>(a.dw) + ((int64_t)part * a.n + row) * a.lddw;
#pragma unroll
            for (int i = 0; i < GK; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = k0 + wk * GK * 64 + 64 * i + 16 * g + 4 * e;
                    f8_store4(out + col,
                              f8_f32x4{acc[i][0][j][o][e], acc[i][1][j][o][e], acc[i][2][j][o][e], acc[i][3][j][o][e]},
                              a.k - col, a.vec);
                }
        }
}

template <int WK, int WN, int GK, int GN, class T>
hipError_t launch_weight_grad_tile(F8WeightGradArgs a, hipStream_t stream) {
    auto kernel = f8_weight_grad_kernel<WK, WN, GK, GN, T>;
    constexpr size_t lds = weight_grad_lds_bytes<WK, WN, GK, GN>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    constexpr int BK = WK * GK * 64, BN = WN * GN * 64;
    a.k_tiles = (a.k + BK - 1) / BK;
    a.n_tiles = (a.n + BN - 1) / BN;
    const int64_t tiles = (int64_t)a.k_tiles * a.n_tiles * a.parts;
    if (f8_grid(tiles) * (64 * WK * WN) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)f8_grid(tiles)), dim3(64 * WK * WN), lds, stream, a);
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

template <class T, int TERMS>
hipError_t backward(const DeviceInfo& dev, const uint8_t* wq, const float* wd, int64_t n, int parts, int64_t k,
                    const uint8_t* xq, const float* xd, int64_t m, const void* gu, int64_t ldgu, const void* d,
                    int type, int64_t ldd, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                    hipStream_t stream) {
    if (m == 0) return zero_rows<T>(dw, parts * n, k, lddw, stream);
    if (n == 0) return zero_rows<T>(dx, m, k, lddx, stream);
    const q8v::F8BackwardWorkspace ws = q8v::f8_backward_layout(m, n, parts, k, type);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    uint16_t* planes = reinterpret_cast<uint16_t*>(base + ws.d_off);
    uint16_t* values = reinterpret_cast<uint16_t*>(base + ws.x_off);
    const int kb = (int)((k + 127) / 128);
    hipError_t e = hipSuccess;

    const uint16_t* dp = planes;
    int64_t ldp = ws.ldd;
    if (parts == 2) {
        const bool vec = rows_aligned<T>(gu, ldgu, 8) && rows_aligned<T>(d, ldd, 8);
        auto kernel = f8_gate_up_gradient_kernel<T, TERMS>;
        hipLaunchKernelGGL(kernel, dim3(part_blocks(m * (ldp / 16))), dim3(kPartThreads), 0, stream,
                           static_cast<const T*>(gu), ldgu, static_cast<const T*>(d), ldd, m, (int)n, vec, planes, ldp);
        e = hipGetLastError();
    } else if (TERMS == 1 && n % 8 == 0 && ldd <= (int64_t(1) << 22) && rows_aligned<T>(d, ldd, 8)) {
        dp = static_cast<const uint16_t*>(d);  // bf16 rows are their own plane
        ldp = ldd;
    } else {
        auto kernel = f8_split_kernel<T, TERMS>;
        hipLaunchKernelGGL(kernel, dim3(part_blocks(m * (ldp / 8))), dim3(kPartThreads), 0, stream,
                           static_cast<const T*>(d), m, (int)n, ldd, rows_aligned<T>(d, ldd, 8), planes, ldp);
        e = hipGetLastError();
    }
    if (e != hipSuccess) return e;

    if (dx) {
        F8InputGradArgs a{};
        a.d = dp; a.plane = m * ldp; a.ldd = ldp; a.part_cols = ldp / parts;
        a.w = wq; a.wd = wd; a.dx = dx; a.lddx = lddx;
        a.n = (int)n; a.parts = parts; a.terms = TERMS; a.m = (int)m; a.k = (int)k; a.kb = kb;
        a.vec = rows_aligned<T>(dx, lddx, 4);
        const int64_t big = ((m + 255) / 256) * ((k + 255) / 256);
        e = big >= dev.cu_count / 2 ? launch_input_grad_tile<2, 4, 4, T>(a, stream) : launch_input_grad_tile<1, 4, 1, T>(a, stream);
        if (e != hipSuccess) return e;
    }
    if (dw) {
        auto kernel = f8_values_kernel<TERMS>;
        hipLaunchKernelGGL(kernel, dim3(part_blocks(m * (k / 8))), dim3(kPartThreads), 0, stream, xq, xd, m, (int)k, kb,
                           values);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        F8WeightGradArgs a{};
        a.d = dp; a.d_plane = m * ldp; a.ldd = ldp; a.part_cols = ldp / parts;
        a.x = values; a.x_plane = m * k; a.dw = dw; a.lddw = lddw;
        a.n = (int)n; a.parts = parts; a.pairs = TERMS * (TERMS + 1) / 2; a.m = (int)m; a.k = (int)k;
        a.vec = rows_aligned<T>(dw, lddw, 4);
        const int64_t big = parts * ((n + 255) / 256) * ((k + 255) / 256);
        e = big >= dev.cu_count / 2 ? launch_weight_grad_tile<2, 4, 2, 1, T>(a, stream)
                                    : launch_weight_grad_tile<2, 2, 1, 1, T>(a, stream);
    }
    return e;
}

}  // namespace

hipError_t launch_f8_backward(const DeviceInfo& dev, const uint8_t* wq, const float* wd, int64_t n, int parts,
                              int64_t k, const uint8_t* xq, const float* xd, int64_t m, const void* gu, int64_t ldgu,
                              const void* d, int type, int64_t ldd, void* dx, int64_t lddx, void* dw, int64_t lddw,
                              void* workspace, hipStream_t stream) {
    switch (type) {
        case Q8_F32:
            return backward<float, 3>(dev, wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw, lddw,
                                      workspace, stream);
        case Q8_F16:
            return backward<_Float16, 2>(dev, wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw,
                                         lddw, workspace, stream);
        default:
            return backward<__bf16, 1>(dev, wq, wd, n, parts, k, xq, xd, m, gu, ldgu, d, type, ldd, dx, lddx, dw, lddw,
                                       workspace, stream);
    }
}

}  // namespace q8k
