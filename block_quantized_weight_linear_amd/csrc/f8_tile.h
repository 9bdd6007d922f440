// What the block-scaled 8-bit floating-point kernels share: direct-to-LDS copies of tile rows,
// MFMA operand types, element conversions and the order of tiles on the XCDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
// base + off to lds + 16*l (lds + 4*l).  base and lds are wave-uniform; a write of M0 needs one
// wait state before the copy reads it.  M0 is left written and declared so, which makes the compiler write it
// anew before an instruction of its own that reads it (saved around each copy instead, the copies between a
// wave's products took two instructions more).  clang warns that a reserved register is not saved for the
// caller, which is what is wanted here.  It counts as one vector-memory load.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void f8_copy16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, %1"
        :
        : "v"(off), "s"(base), "s"(lds)
        : "m0", "memory");
}
__device__ __forceinline__ void f8_copy4(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %0, %1"
        :
        : "v"(off), "s"(base), "s"(lds)
        : "m0", "memory");
}
// Four bytes a lane from addresses of their own.
__device__ __forceinline__ void f8_copy4_from(const float* src, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %0, off"
        :
        : "v"(src), "s"(lds)
        : "m0", "memory");
}
// The same where valid, zeros where not (the cut last step of an operand).
__device__ __forceinline__ void f8_copy16_or_zeros(const uint8_t* base, uint32_t off, bool valid, uint32_t lds) {
    asm volatile("" : "+v"(off));  // else the lanes' addresses are kept in registers for this one step
    const uint8_t* src = valid ? base + off : reinterpret_cast<const uint8_t*>(&f8_zeros);
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off"
        :
        : "v"(src), "s"(lds)
        : "m0", "memory");
}
#pragma clang diagnostic pop

__device__ __forceinline__ uint32_t f8_lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}

// Blocks go to the eight XCDs in turn: give each XCD a run of neighbouring tiles, which share
// their operands in its L2; the run goes through bands of eight rows of tiles, column by column,
// so that the 32 tiles that an XCD works at once read 8 + 4 pieces of the operands, not 32 + 1.
constexpr int kF8Xcds = 8, kF8Band = 8;
inline int64_t f8_grid(int64_t tiles) { return (tiles + kF8Xcds - 1) / kF8Xcds * kF8Xcds; }
struct F8Tile {
    int row, col;
    bool inside;
};
__device__ __forceinline__ F8Tile f8_tile_of_block(int block, int rows, int cols) {
    const int tiles = rows * cols, per_xcd = (tiles + kF8Xcds - 1) / kF8Xcds;
    const int t = block % kF8Xcds * per_xcd + block / kF8Xcds;
    const int band = t / (kF8Band * cols), in = t - band * kF8Band * cols;
    const int left = rows - band * kF8Band, height = left < kF8Band ? left : kF8Band;
    // (t past the last tile: height may not be positive)
    const int h = height > 0 ? height : 1;
    return {band * kF8Band + in % h, in / h, t < tiles && block / kF8Xcds < per_xcd};
}

// Waits until at most MOST stages of COPIES copies each, or `younger` if those are fewer, are on their way.
template <int MOST, int COPIES>
__device__ __forceinline__ void f8_wait_stages(int younger) {
    static_assert(MOST * COPIES < 64, "copies are counted");
    if constexpr (MOST == 0) {
        wait_vmcnt_mem<0>();
    } else {
        if (younger >= MOST) wait_vmcnt_mem<MOST * COPIES>();
        else f8_wait_stages<MOST - 1, COPIES>(younger);
    }
}

// The steps of a tile whose waves work alike, on D stages of LDS: step s + D - 1 is asked for when every wave
// has read step s - 1, whose stage it takes.  copies(s, to): kCopies of a wave; work(s, from).  At the end
// every copy has landed and no wave reads LDS any more.
template <int D, int kCopies, class Copies, class Work>
__device__ __forceinline__ void f8_ring(int steps, Copies&& copies, Work&& work) {
#pragma unroll
    for (int d = 0; d + 1 < D; ++d)
        if (d < steps) copies(d, d);
    int stage = 0, free = D - 1;
    for (int s = 0; s < steps; ++s) {
        f8_wait_stages<D - 2, kCopies>(steps - 1 - s);
        __syncthreads();
        if (s + D - 1 < steps) copies(s + D - 1, free);
        work(s, stage);
        free = stage;
        stage = stage + 1 < D ? stage + 1 : 0;
    }
    __syncthreads();
}

// The steps of a tile of eight waves, two on a SIMD, in turns: while the waves 0 .. 3 (group 0) read
// fragments from LDS, the waves 4 .. 7 (group 1) multiply, and the other way round, so that the matrix
// cores of a SIMD always have one wave's products.  A turn ends with a barrier of all eight.  A step is
// two pairs of turns: group 0 reads its first fragments of step s in turn 4s, multiplies in 4s + 1, reads the
// rest in 4s + 2 and multiplies in 4s + 3; group 1 is one turn behind.
//
// LDS has two stages.  The piece X of step s, what both groups read first, is done with after turn
// 4s + 1, the piece Y, what they read last, after 4s + 3: each is asked for again, for step s + 2, as soon
// as that, between products (X by group 1 in 4s + 2 and by group 0 in 4s + 3, Y in 4s + 4 and 4s + 5), and
// waited for in the turn before it is read, 4s + 7 and 4s + 9, by a count of the copies that are younger, so
// that a copy has at least four turns.  (4096 rows of 8192 x 8192 in e4m3: whole stages copied again, 260 us;
// so, 237 us; asked for in the reading turns instead, 247 us; of which the products are about 150.)
//   x(s, i, to), i < kX, y(s, i, to), i < kY: copies of step s, into stage `to`; past the end the last
//                        step is copied again, unread.  i = -1 comes first, in the reading turn: what
//                        the copies need to know (a wave's instructions between its products bound a turn)
//   load(s, h)         : asks for the fragments of part h
//   finish(h)          : adds up what multiply(h) left, while the other group multiplies and the
//                        fragments of the next part are on their way
//   ready(s, h)        : what has to be done with the fragments of part h before they are multiplied
//   multiply(h, side)  : the products; side(p) is called between them, p = 0, 1, .. (at least kX times)
// At the end every copy has landed and no wave reads LDS any more.
__device__ __forceinline__ void f8_end_turn() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
template <int kX, int kY, class X, class Y, class Load, class Finish, class Ready, class Multiply>
__device__ __forceinline__ void f8_turns(int group, int steps, X&& x, Y&& y, Load&& load, Finish&& finish,
                                         Ready&& ready, Multiply&& multiply) {
    const int last = steps - 1;
    auto x_copy = [&](int s, int i) __attribute__((always_inline)) {
        if (i < kX) x(s < last ? s : last, i, s & 1);
    };
    auto y_copy = [&](int s, int i) __attribute__((always_inline)) {
        if (i < kY) y(s < last ? s : last, i, s & 1);
    };
    auto turns = [&](int s, auto hc, auto gc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, of = decltype(gc)::value;
        load(s, h);
        __builtin_amdgcn_sched_barrier(0);
        finish(h ^ 1);
        if (of == h) y_copy(s + 1 + of, -1);
        else x_copy(s + 2, -1);
        __builtin_amdgcn_sched_barrier(0);
        wait_lgkmcnt_mem<0>();
        ready(s, h);
        if (of == 1) wait_vmcnt_mem<kX + kY>();  // h = 0: Y of step s, 1: X of step s + 1
        f8_end_turn();
        __builtin_amdgcn_s_setprio(1);
        multiply(h, [&](int p) __attribute__((always_inline)) {
            if (of == h) y_copy(s + 1 + of, p);
            else x_copy(s + 2, p);
        });
        __builtin_amdgcn_s_setprio(0);
        if (of == 0) wait_vmcnt_mem<kX + kY>();
        f8_end_turn();
    };
#pragma unroll
    for (int i = -1; i < kX; ++i) x_copy(0, i);
#pragma unroll
    for (int i = -1; i < kY; ++i) y_copy(0, i);
#pragma unroll
    for (int i = -1; i < kX; ++i) x_copy(1, i);
    wait_vmcnt_mem<kX + kY>();
    f8_end_turn();
    // a loop for each group: with the waits under a branch in one loop the registers do not suffice
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};
    if (group == 0) {
#pragma clang loop unroll(disable)
        for (int s = 0; s < steps; ++s) {
            turns(s, zero, zero);
            turns(s, one, zero);
        }
        f8_end_turn();
    } else {
#pragma unroll
        for (int i = -1; i < kY; ++i) y_copy(1, i);
        f8_end_turn();
#pragma clang loop unroll(disable)
        for (int s = 0; s < steps; ++s) {
            turns(s, zero, one);
            turns(s, one, one);
        }
    }
    finish(1);
    wait_vmcnt_mem<0>();
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
