// Low-rank adapters of many requests beside a shared projection (gfx950).
//
// Row t with adapter a adds scale[a] * B[a] (A[a] x[t]) to the shared product.  Two launches:
// the inner products u[t][c] = scale[a] * A[a][c] . x[t] of every row (c over the
// sections' ranks; float32, one wave a product), then each output's dot of u with its row
// of B, added to the shared product (or, for a fused gate_up, the activation behind it).
// In the packed calls the first launch also writes the rows' digits and the second
// computes the shared product (digit_tiles.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "digit_tiles.h"
#include "gemv_core.h"
#include "q8_internal.h"
#include "q8_validate.h"

namespace q8k {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// Element types of A and B: eight values from a 16-byte aligned address, widened exactly.
struct LoraF32 {
    using T = float;
    static __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
struct LoraF16 {
    using T = uint16_t;
    static __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
        const u16x8 a = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)a[i]);
    }
};
struct LoraBF16 {
    using T = uint16_t;
    static __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
        const u16x8 a = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, (uint32_t)a[i] << 16);
    }
};

// What the kernels need of a q8_lora, by value.
struct LoraArgs {
    const void* a;
    const void* b;
    const int32_t* ranks;
    const float* scale;
    const int32_t* adapter;
    int type, n_adapters, rank, n_sections;
    int64_t end[Q8_LORA_MAX_SECTIONS];  // first row past each section

    // the row's adapter, -1 for none
    __device__ __forceinline__ int of_row(int64_t t) const {
        if (n_adapters == 0) return -1;
        const int a = adapter[t];
        return a >= 0 && a < n_adapters ? a : -1;
    }
    __device__ __forceinline__ int rank_of(int a) const {
        if (!ranks) return rank;
        const int r = ranks[a];
        return r < 0 ? 0 : r < rank ? r : rank;
    }
    __device__ __forceinline__ int section(int64_t i) const {
        int s = 0;
#pragma unroll
        for (int q = 0; q < Q8_LORA_MAX_SECTIONS - 1; ++q) s += (q < n_sections - 1 && i >= end[q]) ? 1 : 0;
        return s;
    }
};

// The inner products of blocks block, block + blocks, ... of four (one a wave).
template <class Ty>
__device__ __forceinline__ void lora_shrink(const LoraArgs& lo, const float* __restrict__ x, int m, int k,
                                            int64_t ldx, float* __restrict__ u, int block, int blocks) {
    const int lane = threadIdx.x & 63;
    const int cols = lo.n_sections * lo.rank;
    for (int64_t id = (int64_t)block * 4 + (threadIdx.x >> 6); id < (int64_t)m * cols; id += (int64_t)blocks * 4) {
    const int64_t t = id / cols;
    const int c = (int)(id - t * cols);
    const int a = lo.of_row(t);
    if (a < 0 || c % lo.rank >= lo.rank_of(a)) {
        if (lane == 0) u[id] = 0.0f;
        continue;
    }
    const typename Ty::T* ar = static_cast<const typename Ty::T*>(lo.a) + ((size_t)a * cols + c) * k;
    const float* xr = x + t * ldx;
    float acc = 0.0f;
    for (int i = 8 * lane; i < k; i += 512) {
        float v[8], w[8];
        Ty::load8(ar + i, v);
        LoraF32::load8(xr + i, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc = __builtin_fmaf(v[q], w[q], acc);
    }
    for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
    if (lane == 0) u[id] = acc * (lo.scale ? lo.scale[a] : 1.0f);
    }
}

template <class Ty>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs lo, const float* __restrict__ x, int m, int k,
                                                          int64_t ldx, float* __restrict__ u) {
    lora_shrink<Ty>(lo, x, m, k, ldx, u, blockIdx.x, gridDim.x);
}

// First launch of the packed calls: blocks 0 .. m-1 write the rows' digits, the others the
// inner products.
template <class Ty>
__global__ __launch_bounds__(256) void lora_prepare_kernel(LoraArgs lo, const float* __restrict__ x, int m, int k,
                                                           int64_t ldx, float* __restrict__ u,
                                                           int8_t* __restrict__ dig, int* __restrict__ exps) {
    const int b = blockIdx.x;
    if (b < m)
        write_digits(x + b * ldx, k, dig + (size_t)b * k * 4, exps + b);
    else
        lora_shrink<Ty>(lo, x, m, k, ldx, u, b - m, gridDim.x - m);
}

// sum_j B[a][i][j] u[j] of output row i, u the row's inner products
template <class Ty>
__device__ __forceinline__ float lora_delta(const LoraArgs& lo, int64_t n, int a, int64_t i, const float* u) {
    const typename Ty::T* br = static_cast<const typename Ty::T*>(lo.b) + ((size_t)a * n + i) * lo.rank;
    const float* us = u + lo.section(i) * lo.rank;
    const int r = lo.rank_of(a);
    float acc = 0.0f;
    for (int j = 0; j < r; j += 8) {
        float v[8], w[8];
        Ty::load8(br + j, v);
        LoraF32::load8(us + j, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc = j + q < r ? __builtin_fmaf(v[q], w[q], acc) : acc;
    }
    return acc;
}

__device__ __forceinline__ float lora_delta_any(const LoraArgs& lo, int64_t n, int a, int64_t i, const float* u) {
    if (lo.type == Q8_LORA_BF16) return lora_delta<LoraBF16>(lo, n, a, i, u);
    if (lo.type == Q8_LORA_F16) return lora_delta<LoraF16>(lo, n, a, i, u);
    return lora_delta<LoraF32>(lo, n, a, i, u);
}

template <class Ty, bool SILU>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs lo, const float* __restrict__ u, const float* y,
                                                          int64_t n, int64_t ldy, float* out, int64_t ldo, int m) {
    const int64_t n_out = SILU ? n / 2 : n;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_out) return;
    for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
        const int a = lo.of_row(t);
        const float* ut = u + t * lo.n_sections * lo.rank;
        float g = y[t * ldy + i];
        if (a >= 0) g += lora_delta<Ty>(lo, n, a, i, ut);
        if constexpr (SILU) {
            float v = y[t * ldy + n_out + i];
            if (a >= 0) v += lora_delta<Ty>(lo, n, a, n_out + i, ut);
            g = silu_mul(g, v);
        }
        out[t * ldo + i] = g;
    }
}

// Second launch of the packed calls: the shared product's tiles with the correction (and,
// SILU, the activation) behind each.  A block owns a run of neighbouring tiles and streams
// it once for every 4 * NG rows; a fused tile is 8 gate rows and their 8 up rows.
constexpr int kLoraSumTiles = 64;  // tiles * NG whose sums wait in LDS

template <int NG>
constexpr size_t lora_tiles_lds() {
    return kRingBytes + sizeof(float) * (2 * kTileWaves * NG * 64 + kLoraSumTiles * 64);
}

template <int SP, int NG, bool SILU>
__global__ __launch_bounds__(kTileThreads) void lora_tiles_kernel(const uint8_t* __restrict__ w, int n_out, int k,
                                                                  int log2_wt, const int8_t* __restrict__ dig,
                                                                  const int* __restrict__ exps, LoraArgs lo,
                                                                  const float* __restrict__ u, int m,
                                                                  float* __restrict__ y, int64_t ldy) {
    extern __shared__ float4 smem4[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(smem4);
    float* part = reinterpret_cast<float*>(smem + kRingBytes);
    float* sums = part + 2 * kTileWaves * NG * 64;
    const TileWave W(smem, k >> 8, log2_wt);
    constexpr int kOut = SILU ? kTileRows / 2 : kTileRows;  // outputs of a tile
    const uint32_t rb = (uint32_t)(k >> 5) * 34u;
    const int tiles = (n_out + kOut - 1) / kOut;
    const int t0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
    const int t1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
    // copy offsets of a tile with `rows` outputs: a row past them reads the last one
    auto tile_offsets = [&](int rows, uint32_t (&off)[5]) __attribute__((always_inline)) {
        W.offsets([&](int r) __attribute__((always_inline)) -> uint32_t {
            const int half = SILU ? r / kOut : 0;
            const int i = min(SILU ? r - half * kOut : r, rows - 1);
            return (uint32_t)(i + half * n_out) * rb;
        }, off);
    };
    uint32_t full[5];
    tile_offsets(min(kOut, n_out), full);
    constexpr int kChunk = kLoraSumTiles / NG;
    for (int m0 = 0; m0 < m; m0 += 4 * NG) {
        const int mm = min(4 * NG, m - m0);
        int c0 = t0;
        auto tile_at = [&](int i, const uint8_t*& base, uint32_t (&off)[5]) __attribute__((always_inline)) {
            const int row0 = (c0 + i) * kOut;
            base = w + (size_t)row0 * rb;
            if (row0 + kOut <= n_out) {
#pragma unroll
                for (int c = 0; c < 5; ++c) off[c] = full[c];
            } else {
                tile_offsets(n_out - row0, off);
            }
        };
        TileRun run(W, min(kChunk, t1 - t0), tile_at);
        long a[NG][SP][8];
        load_digits<SP, NG>(W, [&](int s) __attribute__((always_inline)) {
            return s < mm ? dig + (size_t)(m0 + s) * k * 4 : nullptr;
        }, a);
        while (true) {
            const int nt = run.n_tiles;
            multiply_tiles<SP, NG>(run, a, part, sums);
            __syncthreads();
            // outputs of the chunk: (row of the call, tile, output of the tile), outputs fastest
            for (int o = threadIdx.x; o < mm * nt * kOut; o += kTileThreads) {
                const int r = o % kOut, q = o / kOut;
                const int s = q / nt, tile = q - s * nt;
                const int i = (c0 + tile) * kOut + r;
                if (i >= n_out) continue;
                const int t = m0 + s;
                const float* sum = sums + (tile * NG + (s >> 2)) * 64 + 16 * (s & 3) + r;
                const int ex = exps[t];
                const int ad = lo.of_row(t);
                const float* ut = u + (size_t)t * lo.n_sections * lo.rank;
                float v = row_scaled(sum[0], ex);
                if (ad >= 0) v += lora_delta_any(lo, SILU ? 2 * (int64_t)n_out : n_out, ad, i, ut);
                if constexpr (SILU) {
                    float up = row_scaled(sum[kOut], ex);
                    if (ad >= 0) up += lora_delta_any(lo, 2 * (int64_t)n_out, ad, n_out + (int64_t)i, ut);
                    v = silu_mul(v, up);
                }
                y[t * ldy + i] = v;
            }
            __syncthreads();  // the next chunk overwrites the sums
            c0 += nt;
            if (c0 >= t1) break;
            run.restart(min(kChunk, t1 - c0));
        }
    }
}

static LoraArgs lora_args(const q8_lora& lo) {
    LoraArgs a{lo.a, lo.b, lo.ranks, lo.scale, lo.adapter, lo.type, lo.n_adapters, lo.rank, lo.n_sections, {}};
    int64_t end = 0;
    for (int s = 0; s < Q8_LORA_MAX_SECTIONS; ++s) {
        if (s < lo.n_sections) end += lo.section_rows[s];
        a.end[s] = end;
    }
    return a;
}

template <class Ty>
static hipError_t lora_add_typed(const LoraArgs& lo, const float* y, int64_t n, int64_t ldy, bool silu,
                                 const float* x, int64_t m, int64_t k, int64_t ldx, float* out, int64_t ldo,
                                 float* u, hipStream_t stream) {
    const int64_t dots = m * lo.n_sections * lo.rank;
    hipLaunchKernelGGL(lora_shrink_kernel<Ty>, dim3((unsigned)(dots < 262144 ? (dots + 3) / 4 : 65536)), dim3(256), 0, stream, lo, x, (int)m,
                       (int)k, ldx, u);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n_out = silu ? n / 2 : n;
    const dim3 grid((unsigned)((n_out + 255) / 256), (unsigned)(m < 65535 ? m : 65535));
    if (silu)
        hipLaunchKernelGGL((lora_expand_kernel<Ty, true>), grid, dim3(256), 0, stream, lo, u, y, n, ldy, out, ldo,
                           (int)m);
    else
        hipLaunchKernelGGL((lora_expand_kernel<Ty, false>), grid, dim3(256), 0, stream, lo, u, y, n, ldy, out, ldo,
                           (int)m);
    return hipGetLastError();
}

hipError_t launch_lora_add(const DeviceInfo&, const float* y, int64_t n, int64_t ldy, bool silu_pairs,
                           const float* x, int64_t m, int64_t k, int64_t ldx, const q8_lora& lora, float* out,
                           int64_t ldo, void* workspace, hipStream_t stream) {
    const LoraArgs lo = lora_args(lora);
    const q8v::LoraWorkspace L = q8v::lora_workspace_layout(m, lora.n_sections, lora.rank, 0);
    float* u = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.u_off);
    switch (lora.type) {
        case Q8_LORA_F32: return lora_add_typed<LoraF32>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, u, stream);
        case Q8_LORA_F16: return lora_add_typed<LoraF16>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, u, stream);
        default: return lora_add_typed<LoraBF16>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, u, stream);
    }
}

template <int SP, int NG, bool SILU>
static hipError_t launch_lora_tiles(const DeviceInfo& dev, const uint8_t* w, int64_t n_out, int64_t k, int log2_wt,
                                    const int8_t* dig, const int* exps, const LoraArgs& lo, const float* u,
                                    int64_t m, float* y, int64_t ldy, hipStream_t stream) {
    auto kernel = lora_tiles_kernel<SP, NG, SILU>;
    constexpr size_t lds = lora_tiles_lds<NG>();
    static thread_local int attr_dev = -1;
    if (attr_dev != dev.device) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
        attr_dev = dev.device;
    }
    const int64_t per_tile = SILU ? kTileRows / 2 : kTileRows;
    const int64_t tiles = (n_out + per_tile - 1) / per_tile;
    const unsigned grid = (unsigned)(tiles < dev.cu_count ? tiles : dev.cu_count);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kTileThreads), lds, stream, w, (int)n_out, (int)k, log2_wt, dig,
                       exps, lo, u, (int)m, y, ldy);
    return hipGetLastError();
}

// Activation rows a pass takes, in fours: as many as there are, up to 128 registers a lane
// of digits (16 a slice and four rows).
template <int SP, bool SILU, class... Args>
static hipError_t launch_lora_tiles_sp(const DeviceInfo& dev, int64_t m, Args... args) {
    if constexpr (SP <= 2) {
        if (m > 8) return launch_lora_tiles<SP, 4, SILU>(dev, args...);
    }
    if constexpr (SP <= 4) {
        if (m > 4) return launch_lora_tiles<SP, 2, SILU>(dev, args...);
    }
    return launch_lora_tiles<SP, 1, SILU>(dev, args...);
}

template <bool SILU, class... Args>
static hipError_t launch_lora_tiles_m(int sp, const DeviceInfo& dev, int64_t m, Args... args) {
    if (sp <= 1) return launch_lora_tiles_sp<1, SILU>(dev, m, args...);
    if (sp <= 2) return launch_lora_tiles_sp<2, SILU>(dev, m, args...);
    if (sp <= 3) return launch_lora_tiles_sp<3, SILU>(dev, m, args...);
    if (sp <= 4) return launch_lora_tiles_sp<4, SILU>(dev, m, args...);
    if (sp <= 6) return launch_lora_tiles_sp<6, SILU>(dev, m, args...);
    return launch_lora_tiles_sp<8, SILU>(dev, m, args...);
}

hipError_t launch_linear_lora(const DeviceInfo& dev, const uint8_t* w, int64_t n_out, int64_t k, bool silu,
                              const float* x, int64_t m, int64_t ldx, const q8_lora& lora, float* y, int64_t ldy,
                              void* workspace, hipStream_t stream) {
    const int64_t n = silu ? 2 * n_out : n_out;
    const q8v::LoraWorkspace L =
        q8v::lora_workspace_layout(m, lora.n_sections, lora.rank, q8v::lora_base_bytes(m, n, k));
    char* ws = static_cast<char*>(workspace);
    if (!q8v::lora_uses_tiles(m, n, k)) {
        // the shared product, then the correction in place (behind a fused one: its own)
        float* base = silu ? reinterpret_cast<float*>(ws + L.base_off) : y;
        const int64_t ldb = silu ? n : ldy;
        hipError_t e = m >= q8v::kPrefillRows ? launch_gemm_q8_mfma(dev, w, n, k, false, x, m, ldx, base, ldb, stream)
                                              : launch_gemv_q8(dev, w, n, k, false, x, m, ldx, base, ldb, stream);
        if (e != hipSuccess) return e;
        return launch_lora_add(dev, base, n, ldb, silu, x, m, k, ldx, lora, y, ldy, workspace, stream);
    }
    const LoraArgs lo = lora_args(lora);
    float* u = reinterpret_cast<float*>(ws + L.u_off);
    int* exps = reinterpret_cast<int*>(ws + L.base_off);
    int8_t* dig = reinterpret_cast<int8_t*>(exps + q8v::kPrefillRows);
    const int64_t dots = lora.n_adapters ? m * lora.n_sections * lora.rank : 0;
    const dim3 grid((unsigned)(m + (dots + 3) / 4));
    if (lora.type == Q8_LORA_F32)
        hipLaunchKernelGGL(lora_prepare_kernel<LoraF32>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u, dig,
                           exps);
    else if (lora.type == Q8_LORA_F16)
        hipLaunchKernelGGL(lora_prepare_kernel<LoraF16>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u, dig,
                           exps);
    else
        hipLaunchKernelGGL(lora_prepare_kernel<LoraBF16>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u,
                           dig, exps);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const SliceShare sh = slice_share((int)(k >> 8));
    return silu ? launch_lora_tiles_m<true>(sh.sp, dev, m, w, n_out, k, sh.log2_wt, dig, exps, lo, u, m, y, ldy, stream)
                : launch_lora_tiles_m<false>(sh.sp, dev, m, w, n_out, k, sh.log2_wt, dig, exps, lo, u, m, y, ldy,
                                             stream);
}

}  // namespace q8k
