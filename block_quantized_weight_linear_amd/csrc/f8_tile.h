// What the block-scaled 8-bit floating-point kernels share: direct-to-LDS copies of tile rows,
// MFMA operand types, element conversions and the order of tiles on the XCDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "lds_dma.h"

namespace q8k {

typedef float f8_f32x4 __attribute__((ext_vector_type(4)));
typedef int f8_i32x8 __attribute__((ext_vector_type(8)));
typedef int f8_i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 f8_bf16x8 __attribute__((ext_vector_type(8)));

// Sixteen zero bytes: what a lane copies in the place of bytes past an operand's end, so that
// they add exact zeros to a sum.
static __device__ const f8_i32x4 f8_zeros = {0, 0, 0, 0};

// One wave-wide direct-to-LDS copy from a scalar base: lane l copies the 16 (4) bytes at
// base + off to lds + 16*l (lds + 4*l).  base and lds are wave-uniform; M0 is saved and restored,
// and a write of M0 needs one wait state before the copy reads it.  It counts as one
// vector-memory load.
__device__ __forceinline__ void f8_copy16(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(off), "s"(base), "s"(lds)
        : "memory");
}
__device__ __forceinline__ void f8_copy4(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(off), "s"(base), "s"(lds)
        : "memory");
}
// The same where valid, zeros where not (the cut last step of an operand).
__device__ __forceinline__ void f8_copy16_or_zeros(const uint8_t* base, uint32_t off, bool valid, uint32_t lds) {
    asm volatile("" : "+v"(off));  // else the lanes' addresses are kept in registers for this one step
    const uint8_t* src = valid ? base + off : reinterpret_cast<const uint8_t*>(&f8_zeros);
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(src), "s"(lds)
        : "memory");
}

__device__ __forceinline__ uint32_t f8_lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}

// Blocks go to the eight XCDs in turn: give each XCD a run of neighbouring tiles, which share
// their operands in its L2.
constexpr int kF8Xcds = 8;
inline int64_t f8_grid(int64_t tiles) { return (tiles + kF8Xcds - 1) / kF8Xcds * kF8Xcds; }
__device__ __forceinline__ int f8_tile_of_block(int block, int tiles) {
    const int per_xcd = (tiles + kF8Xcds - 1) / kF8Xcds;
    return block % kF8Xcds * per_xcd + block / kF8Xcds;
}

// Eight codes (two words) as bf16, exactly.
__device__ __forceinline__ f8_bf16x8 f8_widen(int lo, int hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return f8_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// An array of f(0) .. f(N - 1), of a type that has no default.
template <class V, int N>
struct F8Array {
    V at[N];
};
template <class F, int... I>
__device__ __forceinline__ auto f8_each_of(F&& f, std::integer_sequence<int, I...>) {
    return F8Array<decltype(f(0)), sizeof...(I)>{{f(I)...}};
}
template <int N, class F>
__device__ __forceinline__ auto f8_each(F&& f) {
    return f8_each_of(f, std::make_integer_sequence<int, N>{});
}

// Float results: one rounding to the element type (to nearest even).
template <class T>
__device__ __forceinline__ T f8_round(float v) {
    return (T)v;
}

// Four neighbouring results of a row, n of them inside the matrix (vec: rows are aligned to four
// elements).
template <class T>
__device__ __forceinline__ void f8_store4(T* p, f8_f32x4 v, int n, bool vec) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    if (vec && n >= 4) {
        *reinterpret_cast<T4*>(p) = __builtin_convertvector(v, T4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = f8_round<T>(v[i]);
    }
}

// Raises a kernel's limit of dynamic LDS above the default, once per device and thread.
template <class Kernel>
inline hipError_t f8_allow_lds(Kernel kernel, size_t bytes, uint64_t* allowed) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev >= 64 || !((*allowed >> dev) & 1)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)bytes);
        if (e != hipSuccess) return e;
        if (dev < 64) *allowed |= uint64_t(1) << dev;
    }
    return hipSuccess;
}

}  // namespace q8k
