// Low-rank adapters of many requests beside a shared projection (gfx950).
//
// Row t with adapter a adds scale[a] * B[a] (A[a] x[t]) to the shared product.  Two passes:
// the inner products u[t][c] = scale[a] * A[a][c] . x[t] of every row (c over the
// sections' ranks; float32, one wave a product), then each output's dot of u with its row
// of B, added to the shared product (or, for a fused gate_up, the activation behind it).
#include <hip/hip_runtime.h>
#include <stdint.h>

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
    int n_adapters, rank, n_sections;
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

template <class Ty>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs lo, const float* __restrict__ x, int m, int k,
                                                          int64_t ldx, float* __restrict__ u) {
    const int lane = threadIdx.x & 63;
    const int cols = lo.n_sections * lo.rank;
    for (int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); id < (int64_t)m * cols;
         id += (int64_t)gridDim.x * 4) {
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

static LoraArgs lora_args(const q8_lora& lo) {
    LoraArgs a{lo.a, lo.b, lo.ranks, lo.scale, lo.adapter, lo.n_adapters, lo.rank, lo.n_sections, {}};
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

}  // namespace q8k
