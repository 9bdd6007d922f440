// Low-rank adapters: element types, a call's adapters, and an output's correction from its
// row's inner products (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/q8_linear.h"

namespace q8k {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// Element types of A and B: eight values from a 16-byte aligned address, widened exactly.
struct LoraF32 {
    using T = float;
    struct V {
        float4 lo, hi;
    };
    static __device__ __forceinline__ V load8(const T* p) {
        return V{*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
    }
    static __device__ __forceinline__ float at(const V& v, int q) {
        const float4& h = q < 4 ? v.lo : v.hi;
        return (q & 3) == 0 ? h.x : (q & 3) == 1 ? h.y : (q & 3) == 2 ? h.z : h.w;
    }
};
struct LoraF16 {
    using T = uint16_t;
    using V = u16x8;
    static __device__ __forceinline__ V load8(const T* p) { return *reinterpret_cast<const u16x8*>(p); }
    static __device__ __forceinline__ float at(const V& v, int q) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)v[q]);
    }
};
struct LoraBF16 {
    using T = uint16_t;
    using V = u16x8;
    static __device__ __forceinline__ V load8(const T* p) { return *reinterpret_cast<const u16x8*>(p); }
    static __device__ __forceinline__ float at(const V& v, int q) {
        return __builtin_bit_cast(float, (uint32_t)v[q] << 16);
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

// sum_j B[a][i][j] u[j], j < r = rank_of(a), of output i of n, u the row's inner products
template <class Ty, int FLY = 4>
__device__ __forceinline__ float lora_delta(const LoraArgs& lo, int64_t n, int a, int r, int64_t i, const float* u) {
    const typename Ty::T* br = static_cast<const typename Ty::T*>(lo.b) + ((size_t)a * n + i) * lo.rank;
    const float* us = u + lo.section(i) * lo.rank;
    float acc = 0.0f;
    for (int j0 = 0; j0 < r; j0 += 8 * FLY) {  // 8 FLY of B's row in flight
        typename Ty::V v[FLY];
        LoraF32::V w[FLY];
#pragma unroll
        for (int s = 0; s < FLY; ++s) {
            const int j = j0 + 8 * s < r ? j0 + 8 * s : j0;
            v[s] = Ty::load8(br + j);
            w[s] = LoraF32::load8(us + j);
        }
#pragma unroll
        for (int s = 0; s < FLY; ++s)
#pragma unroll
            for (int q = 0; q < 8; ++q)
                acc = j0 + 8 * s + q < r ? __builtin_fmaf(Ty::at(v[s], q), LoraF32::at(w[s], q), acc) : acc;
    }
    return acc;
}

template <int FLY>
__device__ __forceinline__ float lora_delta_any(const LoraArgs& lo, int64_t n, int a, int r, int64_t i, const float* u) {
    if (lo.type == Q8_LORA_BF16) return lora_delta<LoraBF16, FLY>(lo, n, a, r, i, u);
    if (lo.type == Q8_LORA_F16) return lora_delta<LoraF16, FLY>(lo, n, a, r, i, u);
    return lora_delta<LoraF32, FLY>(lo, n, a, r, i, u);
}

inline LoraArgs lora_args(const q8_lora& lo) {
    LoraArgs a{lo.a, lo.b, lo.ranks, lo.scale, lo.adapter, lo.type, lo.n_adapters, lo.rank, lo.n_sections, {}};
    int64_t end = 0;
    for (int s = 0; s < Q8_LORA_MAX_SECTIONS; ++s) {
        if (s < lo.n_sections) end += lo.section_rows[s];
        a.end[s] = end;
    }
    return a;
}

// What the one-row kernel adds to each output of the call's only row; u: its inner products.
struct LoraOneRow {
    static constexpr bool kAdds = true;
    LoraArgs lo;
    const float* u;
    int64_t n;  // rows of the matrix
    struct State {
        int a, r;
    };
    __device__ __forceinline__ State begin() const {
        const int a = lo.of_row(0);
        return State{a, a < 0 ? 0 : lo.rank_of(a)};
    }
    __device__ __forceinline__ float at(const State& s, int64_t i) const {
        return s.a < 0 ? 0.0f : lora_delta_any<2>(lo, n, s.a, s.r, i, u);
    }
};

}  // namespace q8k
