// Block-scaled 8-bit floating-point linears on the matrix cores of gfx950
// (v_mfma_f32_16x16x128_f8f6f4): y[t][j] = sum_b xd[t][b] wd[j/128][b] sum_{i in b} xq[t][i] wq[j][i].
//
// Tile: BN weight rows x BM activation rows, WN x WM waves, TN x TM fragments of 16 x 16 a wave.
// A K step is one block of 128 inputs, 128 bytes a row: weight rows are the instruction's A (so a
// lane ends up with four neighbouring outputs of one row), activation rows its B.  One
// instruction is a whole block of a 16 x 16 fragment; its sum starts at zero and joins the
// accumulators as acc += (xd * wd) * sum, the factor being one number a lane (the lane's
// activation row) since a fragment's weight rows lie in one block of 128.
//
// The instruction aligns the products of eight inputs at the largest of them and cuts them off
// 2^-13 below it before they join its float32 sum (measured with pairs of products; sums of random
// codes are off by 2^-16 of their size).  That is far below a 16-bit result's rounding, and above a
// float32 one's: with float32 results the codes are widened to bf16, which holds them exactly, and
// multiplied by v_mfma_f32_16x16x32_bf16, at half the rate, whose sums of them are off by 2^-26.
//
// Tile rows reach LDS by direct copies of 16 bytes a lane, two stages.  Within a row the eight
// 16-byte chunks are stored at chunk ^ (row % 8), so that the fragments' reads (16 rows, one
// chunk of each) fall on all banks; lane group g reads chunks g and g + 4 of its row, the same
// for both operands, which makes the order of the inputs within a block immaterial.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

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
    int m_tiles, n_tiles, tiles;
    bool vec, vec_gu;  // rows of y (gu) are aligned to four elements
};

// The 32 codes of a row that a lane supplies, and a block's sums of a 16 x 16 fragment.
struct F8Codes {
    f8_i32x8 v;
    __device__ __forceinline__ explicit F8Codes(f8_i32x8 codes) : v(codes) {}
};
struct F8Widened {
    f8_bf16x8 v[4];
    __device__ __forceinline__ explicit F8Widened(f8_i32x8 codes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f8_widen(codes[2 * i], codes[2 * i + 1]);
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

template <int WN, int WM, int TN, int TM>
constexpr size_t f8_linear_lds_bytes() {
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    return 2 * ((size_t)(BN + BM) * 128 + (BM < 64 ? 64 : BM) * 4);
}

template <int WN, int WM, int TN, int TM, bool SILU, class T>
__global__ __launch_bounds__(64 * WN * WM) void f8_linear_kernel(F8LinearArgs a) {
    constexpr int W = WN * WM, BN = WN * TN * 16, BM = WM * TM * 16, ROWS = BN + BM;
    constexpr int COPIES = (ROWS / 8 + W - 1) / W;  // of a wave and step, eight rows each
    constexpr int SX = BM < 64 ? 64 : BM;
    constexpr int OUT = SILU ? TN * 8 : TN * 16;  // outputs of a wave
    using Codes = std::conditional_t<sizeof(T) == 4, F8Widened, F8Codes>;
    static_assert(128 % (TN * 16) == 0 && (!SILU || TN % 2 == 0), "a wave's weight rows lie in one block");
    extern __shared__ __attribute__((aligned(16))) uint8_t f8_smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;

    const int tile = f8_tile_of_block((int)blockIdx.x, a.tiles);
    if (tile >= a.tiles) return;  // block-uniform, before any barrier
    const int mt = tile % a.m_tiles, nt = tile / a.m_tiles;
    const int n0 = nt * (SILU ? BN / 2 : BN), m0 = mt * BM;

    // Copy c of the tile: rows 8c .. 8c + 7 of the stage (weights, then activations), lane l the
    // stage's chunk l % 8 of row l / 8.  Rows past the operand's end are its last row again.
    const uint8_t* base[COPIES];
    uint32_t off[COPIES];
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
        const int c = wave + W * j;
        if (c * 8 < BN) {
            const int wv = c * 8 / (TN * 16), in = c * 8 % (TN * 16);  // the wave whose rows these are
            int first;
            bool up = false;
            if constexpr (SILU) {
                up = in >= TN * 8;
                first = n0 + wv * (TN * 8) + (up ? in - TN * 8 : in);
            } else {
                first = n0 + wv * (TN * 16) + in;
            }
            const int start = first < a.n_out ? first : a.n_out - 1;
            const int row = first + lr < a.n_out ? first + lr - start : a.n_out - 1 - start;
            base[j] = a.w + (int64_t)(start + (up ? a.n_out : 0)) * a.k;
            off[j] = (uint32_t)row * (uint32_t)a.k + 16u * lc;
        } else {
            const int first = m0 + c * 8 - BN;
            const int start = first < a.m ? first : a.m - 1;
            const int row = first + lr < a.m ? first + lr - start : a.m - 1 - start;
            base[j] = a.x + (int64_t)start * a.k;
            off[j] = (uint32_t)row * (uint32_t)a.k + 16u * lc;
        }
    }
    const uint32_t lds = f8_lds_address(f8_smem);
    const uint32_t lds_sx = lds + 2 * ROWS * 128;
    // the scales of 64 rows are one copy of four bytes a lane
    const int sx_row = m0 + 64 * wave + lane;
    const float* sx_base = a.xd + (int64_t)m0 * a.kb;
    const uint32_t sx_off = 4u * (uint32_t)((sx_row < a.m ? sx_row : a.m - 1) - m0) * (uint32_t)a.kb;
    auto copy = [&](int s, int stage) __attribute__((always_inline)) {
        const bool cut = s == a.kb - 1 && (a.k & 127);
#pragma unroll
        for (int j = 0; j < COPIES; ++j) {
            const int c = wave + W * j;
            if (ROWS / 8 % W != 0 && c >= ROWS / 8) break;
            const uint32_t at = lds + (uint32_t)(stage * ROWS * 128 + c * 1024);
            if (!cut) f8_copy16(base[j] + (int64_t)s * 128, off[j], at);
            else f8_copy16_or_zeros(base[j] + (int64_t)s * 128, off[j], lc * 16 < (a.k & 127), at);
        }
        if (64 * wave < BM)
            f8_copy4(reinterpret_cast<const uint8_t*>(sx_base + s), sx_off, lds_sx + (uint32_t)(stage * SX + 64 * wave) * 4);
    };

    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t chunk = 16u * (uint32_t)(g ^ (l16 & 7));
    const uint32_t a_at = (uint32_t)(wn * TN * 16 + l16) * 128 + chunk;
    const uint32_t b_at = (uint32_t)(BN + wm * TM * 16 + l16) * 128 + chunk;
    auto fragment = [&](uint32_t at) __attribute__((always_inline)) {
        const f8_i32x4 lo = *reinterpret_cast<const f8_i32x4*>(f8_smem + at);
        const f8_i32x4 hi = *reinterpret_cast<const f8_i32x4*>(f8_smem + (at ^ 64u));
        return Codes(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };

    // scale rows of the wave's weights (past the matrix: the last one, of rows that are not stored)
    const int out0 = n0 + wn * OUT;
    const int last_block = (a.n_out - 1) / 128;
    const int wb = out0 / 128 < last_block ? out0 / 128 : last_block;
    const float* wd0 = a.wd + (int64_t)wb * a.kb;
    const float* wd1 = SILU ? a.wd + (int64_t)(wb + last_block + 1) * a.kb : wd0;

    f8_f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f8_f32x4{0.f, 0.f, 0.f, 0.f};

    copy(0, 0);
    wait_vmcnt_mem<0>();
    __syncthreads();
    for (int s = 0; s < a.kb; ++s) {
        const int stage = s & 1;
        if (s + 1 < a.kb) copy(s + 1, stage ^ 1);
        const uint32_t at = (uint32_t)(stage * ROWS * 128);
        const float* sx = reinterpret_cast<const float*>(f8_smem + 2 * ROWS * 128) + stage * SX + wm * TM * 16 + l16;
        float c0[TM], c1[TM];
        const float w0 = wd0[s], w1 = wd1[s];
        auto b = f8_each<TM>([&](int j) __attribute__((always_inline)) { return fragment(at + b_at + j * 2048); });
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const float v = sx[16 * j];
            c0[j] = v * w0;
            c1[j] = SILU ? v * w1 : c0[j];
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const Codes av = fragment(at + a_at + i * 2048);
            f8_f32x4 t[TM];
#pragma unroll
            for (int j = 0; j < TM; ++j) t[j] = f8_block_sum(av, b.at[j]);
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const float c = SILU && i >= TN / 2 ? c1[j] : c0[j];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(c, t[j][e], acc[i][j][e]);
            }
        }
        wait_vmcnt_mem<0>();
        __syncthreads();
    }

    // element e of fragment (i, j): output 16i + 4g + e of the wave, row 16j + l16
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int row = m0 + (wm * TM + j) * 16 + l16;
        if (row >= a.m) continue;
        T* y = static_cast<T*>(a.y) + (int64_t)row * a.ldy;
#pragma unroll
        for (int i = 0; i < (SILU ? TN / 2 : TN); ++i) {
            const int n = out0 + 16 * i + 4 * g, inside = a.n_out - n;
            f8_f32x4 v = acc[i][j];
            if constexpr (SILU) {
                const f8_f32x4 u = acc[i + TN / 2][j];
                if (a.gu) {
                    T* gu = static_cast<T*>(a.gu) + (int64_t)row * a.ldgu + n;
                    f8_store4(gu, v, inside, a.vec_gu);
                    f8_store4(gu + a.n_out, u, inside, a.vec_gu && a.n_out % 4 == 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = v[e] / (1.0f + __expf(-v[e])) * u[e];
            }
            f8_store4(y + n, v, inside, a.vec);
        }
    }
}

template <int WN, int WM, int TN, int TM, bool SILU, class T>
hipError_t launch_tile(F8LinearArgs a, hipStream_t stream) {
    constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
    auto kernel = f8_linear_kernel<WN, WM, TN, TM, SILU, T>;
    constexpr size_t lds = f8_linear_lds_bytes<WN, WM, TN, TM>();
    static thread_local uint64_t allowed = 0;
    const hipError_t e = f8_allow_lds(kernel, lds, &allowed);
    if (e != hipSuccess) return e;
    constexpr int COLS = SILU ? BN / 2 : BN;
    a.m_tiles = (a.m + BM - 1) / BM;
    a.n_tiles = (a.n_out + COLS - 1) / COLS;
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    if (f8_grid(tiles) * (64 * WN * WM) >= (int64_t(1) << 32)) return hipErrorInvalidValue;
    a.tiles = (int)tiles;
    hipLaunchKernelGGL(kernel, dim3((unsigned)f8_grid(tiles)), dim3(64 * WN * WM), lds, stream, a);
    return hipGetLastError();
}

template <bool SILU, class T>
hipError_t launch_type(const DeviceInfo& dev, const F8LinearArgs& a, hipStream_t stream) {
    if (a.m <= 16) return launch_tile<4, 1, 2, 1, SILU, T>(a, stream);
    if (a.m <= 128) return launch_tile<4, 1, 2, 4, SILU, T>(a, stream);
    if constexpr (sizeof(T) == 4) return launch_tile<4, 2, 4, 4, SILU, T>(a, stream);
    else return launch_tile<4, 2, 4, 8, SILU, T>(a, stream);
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
