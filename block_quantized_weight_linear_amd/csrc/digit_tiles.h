// Q8_0 weight tiles against a few activation rows on the int8 matrix cores, at float32
// accuracy (gfx950), shared by the adapter linears and the whole MoE layer.
//
// Arithmetic.  A Q8_0 quant is an int8, so v_mfma_i32_16x16x32_i8 multiplies one block (32
// quants) of 16 weight rows with no conversion if the activations are int8 too.  Each
// activation row is therefore written once as a 32-bit fixed-point number with a
// power-of-two row scale 2^(e-29), 2^e <= max |x| < 2^(e+1), in four balanced base-256
// digits: q = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3, |q| <= 2^30, off by at most half a step,
// 2^(e-30) (a row's largest magnitude times 2^-30 at most, a float32 rounding of the
// largest element being 2^-24 of it).  The 16 rows of the instruction's A operand are 4
// activation rows x 4 digits; a block's four digit sums come back exact (|sum| <= 2^19) in
// the four registers of one lane:
//     t = (256 s3 + s2) 2^16 + (256 s1 + s0)   (one fma of the halves, exact integers below
//                                               2^27 that float32 takes with one rounding)
//     acc = fma(d, t, acc)                      (d: the block's scale)
// so a weight costs a lane 6 VALU operations per 512 weights and 4 activation rows instead
// of a conversion and 4 fmas each.  Per output: the chain over the blocks of a 256-wide
// slice, over the wave's slices, then the waves' sums in order: it depends on k (and, for the
// packed calls' k > 4096, on the ranges that k is cut into, which the matrix's rows and the
// device choose), never on the other rows of the call.
//
// Streaming.  A tile is 16 weight rows; its 256-wide slices (16 x 272 bytes) are copied by
// the wave that owns the slice straight into the wave's own LDS ring (coalesced
// direct-to-LDS loads, kRing items ahead).  WT waves share a tile, wave w taking the slices
// w, w + WT, ...: their digits stay in its registers for every tile.  The 8 / WT tiles in
// work together end in one barrier; their sums are added by one wave each into `sums`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemv_core.h"
#include "lds_dma.h"

namespace q8k {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 16;
constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kSliceBytes = 272;  // 8 blocks: 256 weights of a row
constexpr int kRing = 3;          // items in flight per wave
constexpr int kRingBytes = kTileWaves * kRing * kLdsItemBytes;
static_assert(kTileRows * kSliceBytes == kLdsItemBytes, "an item is one slice of a tile");

// How a tile's S = k / 256 slices are shared: WT waves (1, 2, 4 or 8) with at most SP
// slices each, for S <= 24 at most three.  The fewest idle wave slices win, ties go to more
// waves (fewer registers).
struct SliceShare {
    int log2_wt, sp;
};
__host__ __device__ inline SliceShare slice_share(int S) {
    SliceShare best{-1, 0};
    for (int l = 3; l >= 0; --l) {
        const int sp = (S + (1 << l) - 1) >> l;
        if ((1 << l) > S || (sp > 3 && l < 3)) continue;
        if (best.log2_wt < 0 || (sp << l) < (best.sp << best.log2_wt)) best = SliceShare{l, sp};
    }
    return best;
}

// One item into lds .. lds + 4351: four copies of 16 bytes a lane and one of 4 from base +
// off[c] (base wave-uniform), five vmcnt events, with the non-temporal hint (weights are
// read once).  The compiler counts these loads, so the digits loaded before them are waited
// for without waiting for the copies; nothing it can see reads LDS until the run's end
// (read_item, read_sums and write_sum are inline assembly), or it would drain the copies.
typedef __attribute__((address_space(1))) const uint8_t GlobalBytes;
typedef __attribute__((address_space(3))) uint8_t LdsBytes;
__device__ __forceinline__ void copy_item(const uint8_t* base, const uint32_t (&off)[5], uint32_t lds) {
    constexpr int kNonTemporal = 2;
    GlobalBytes* g = (GlobalBytes*)base;
    LdsBytes* l = (LdsBytes*)lds;
    __builtin_amdgcn_global_load_lds(g + off[0], l, 16, 0, kNonTemporal);
    __builtin_amdgcn_global_load_lds(g + off[1], l + 1 * 1024, 16, 0, kNonTemporal);
    __builtin_amdgcn_global_load_lds(g + off[2], l + 2 * 1024, 16, 0, kNonTemporal);
    __builtin_amdgcn_global_load_lds(g + off[3], l + 3 * 1024, 16, 0, kNonTemporal);
    __builtin_amdgcn_global_load_lds(g + off[4], l + 4 * 1024, 4, 0, kNonTemporal);
}

// A lane's share of an item: of each block pair q the dwords holding the lane's quants of its
// first block (e, f: 12 bytes, shifted by two), of its second (o) and both scales (s: low half
// of the first dword, high half of the second).  row: the lane's weight row, mine: row + 8 *
// (lane >> 4).  Done when it returns.
struct ItemWords {
    uint64_t e[4], o[4], s[4], f[2];
};
__device__ __forceinline__ void read_item(uint32_t row, uint32_t mine, ItemWords& v) {
    asm volatile(
        "ds_read2_b32 %0, %14 offset0:0 offset1:1\n\t"
        "ds_read2_b32 %1, %14 offset0:17 offset1:18\n\t"
        "ds_read2_b32 %2, %14 offset0:34 offset1:35\n\t"
        "ds_read2_b32 %3, %14 offset0:51 offset1:52\n\t"
        "ds_read2_b32 %4, %14 offset0:9 offset1:10\n\t"
        "ds_read2_b32 %5, %14 offset0:26 offset1:27\n\t"
        "ds_read2_b32 %6, %14 offset0:43 offset1:44\n\t"
        "ds_read2_b32 %7, %14 offset0:60 offset1:61\n\t"
        "ds_read2_b32 %8, %15 offset0:0 offset1:8\n\t"
        "ds_read2_b32 %9, %15 offset0:17 offset1:25\n\t"
        "ds_read2_b32 %10, %15 offset0:34 offset1:42\n\t"
        "ds_read2_b32 %11, %15 offset0:51 offset1:59\n\t"
        "ds_read2_b32 %12, %14 offset0:2 offset1:19\n\t"
        "ds_read2_b32 %13, %14 offset0:36 offset1:53\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v.e[0]), "=&v"(v.e[1]), "=&v"(v.e[2]), "=&v"(v.e[3]), "=&v"(v.o[0]), "=&v"(v.o[1]), "=&v"(v.o[2]),
          "=&v"(v.o[3]), "=&v"(v.s[0]), "=&v"(v.s[1]), "=&v"(v.s[2]), "=&v"(v.s[3]), "=&v"(v.f[0]), "=&v"(v.f[1])
        : "v"(mine), "v"(row)
        : "memory");
}
__device__ __forceinline__ void write_sum(uint32_t lds, float v) {
    asm volatile("ds_write_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" ::"v"(lds), "v"(v) : "memory");
}
// The sum of n floats at lds, lds + stride, ... in order.
__device__ __forceinline__ float read_sums(uint32_t lds, int n, uint32_t stride) {
    float s = 0.0f;
    for (int w = 0; w < n; w += 2, lds += 2 * stride) {  // n: 2, 4 or 8
        float a, b;
        asm volatile("ds_read_b32 %0, %2\n\tds_read_b32 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(a), "=&v"(b)
                     : "v"(lds), "v"(lds + stride)
                     : "memory");
        s += a;
        s += b;
    }
    return s;
}

template <class F, int... I>
__device__ __forceinline__ void unroll_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F&& f) {
    unroll_impl(f, std::make_integer_sequence<int, N>{});
}

// Where digit d of element i lies in a row's digits: [block pair][digit][8 elements' place
// in their block][block of the pair][8], so that a lane's bytes of two blocks are 16
// consecutive ones.
__host__ __device__ constexpr size_t digit_at(int i, int d) {
    return (size_t)(i >> 6) * 256 + 64 * d + 16 * ((i >> 3) & 3) + 8 * ((i >> 5) & 1) + (i & 7);
}

// Digits of one activation row, by a block of 256 threads: dig is the row's 4 k bytes,
// *exp_out the exponent e - 29 of its scale.  A row that holds a NaN or an infinity gets
// kNotFinite and zero digits: all its outputs are NaN.
constexpr int kNotFinite = 1 << 20;
__device__ __forceinline__ float row_scaled(float sum, int exp) {
    return exp == kNotFinite ? __builtin_nanf("") : __builtin_ldexpf(sum, exp);
}
__device__ __forceinline__ int row_exponent(uint32_t max_bits) { return max((int)(max_bits >> 23) - 127, -126); }
__device__ __forceinline__ void write_digits(const float* __restrict__ xr, int k, int8_t* __restrict__ dig,
                                             int* __restrict__ exp_out) {
    __shared__ uint32_t wave_max_bits[4];
    constexpr int kKeep = 4;  // the first 4096 elements stay in registers, the rest is read twice
    const int tid = threadIdx.x;
    float4 keep[kKeep];
    uint32_t mx = 0;  // magnitudes as bits: ordered like the values, NaN above infinity
    auto larger = [&](const float4& v) __attribute__((always_inline)) {
        const uint32_t a = __builtin_bit_cast(uint32_t, v.x) & 0x7fffffffu;
        const uint32_t b = __builtin_bit_cast(uint32_t, v.y) & 0x7fffffffu;
        const uint32_t c = __builtin_bit_cast(uint32_t, v.z) & 0x7fffffffu;
        const uint32_t d = __builtin_bit_cast(uint32_t, v.w) & 0x7fffffffu;
        mx = max(max(max(mx, a), b), max(c, d));
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = 4 * tid + 1024 * j;
        keep[j] = i < k ? *reinterpret_cast<const float4*>(xr + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kKeep; ++j) larger(keep[j]);
    for (int i = 4 * tid + 1024 * kKeep; i < k; i += 1024) larger(*reinterpret_cast<const float4*>(xr + i));
    for (int off = 32; off >= 1; off >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, off, 64));
    if ((tid & 63) == 0) wave_max_bits[tid >> 6] = mx;
    __syncthreads();
    mx = max(max(wave_max_bits[0], wave_max_bits[1]), max(wave_max_bits[2], wave_max_bits[3]));
    const bool finite = mx < 0x7f800000u;
    const int e = row_exponent(mx);
    if (tid == 0) *exp_out = finite ? e - 29 : kNotFinite;
    auto write = [&](const float4& v, int i) __attribute__((always_inline)) {
        const float f[4] = {v.x, v.y, v.z, v.w};
        uint32_t out[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            int q = finite ? (int)__builtin_rintf(__builtin_ldexpf(f[c], 29 - e)) : 0;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int lo = (int8_t)q;
                out[d] |= (uint32_t)(lo & 255) << (8 * c);
                q = (q - lo) >> 8;
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
            *reinterpret_cast<uint32_t*>(dig + digit_at(i, d)) = out[d];
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = 4 * tid + 1024 * j;
        if (i < k) write(keep[j], i);
    }
    for (int i = 4 * tid + 1024 * kKeep; i < k; i += 1024) write(*reinterpret_cast<const float4*>(xr + i), i);
}

// What a wave knows about its place: its slices of the S from `first` on, its tiles of a step.
struct TileWave {
    int lane, wv, wt, tg, log2_wt, n_sl, row, grp, first;  // row, grp: lane & 15, lane >> 4
    uint32_t ring_lds;
    const uint8_t* ring;
    __device__ __forceinline__ TileWave(uint8_t* smem_ring, int S, int log2_wt_, int first_ = 0)
        : log2_wt(log2_wt_), first(first_) {
        lane = threadIdx.x & 63;
        wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wt = wv & ((1 << log2_wt) - 1);
        tg = wv >> log2_wt;
        n_sl = (S - wt + (1 << log2_wt) - 1) >> log2_wt;
        row = lane & 15;
        grp = lane >> 4;
        ring = smem_ring + (size_t)wv * (kRing * kLdsItemBytes);
        ring_lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring);
    }
    // the wave's copy offsets within a tile slice whose row r lies at row_off(r) bytes
    template <class RowOff>
    __device__ __forceinline__ void offsets(RowOff&& row_off, uint32_t (&off)[5]) const {
#pragma unroll
        for (int c = 0; c < 5; ++c) {
            const int i = c < 4 ? 1024 * c + 16 * lane : 4096 + 4 * lane;
            const int r = i / kSliceBytes;
            off[c] = row_off(r) + (uint32_t)(i - r * kSliceBytes);
        }
    }
};

// A operands of the wave's slices for 4 * NG activation rows, a[g][slice][block pair][block];
// digits_of(slot) gives the digits of the row in a slot (for a slot without one: of any row,
// its sums are not used).
typedef long i64x2 __attribute__((ext_vector_type(2)));
template <int SP, int NG, class DigitsOf>
__device__ __forceinline__ void load_digits(const TileWave& W, DigitsOf&& digits_of, i64x2 (&a)[NG][SP][4]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int8_t* d = digits_of(4 * g + (W.row >> 2)) + 64 * (W.row & 3) + 16 * W.grp;
#pragma unroll
        for (int sl = 0; sl < SP; ++sl) {
            // a wave without a slice (it multiplies nothing): any
            const int s = W.first + (W.n_sl > 0 ? W.wt + (min(sl, W.n_sl - 1) << W.log2_wt) : 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) a[g][sl][q] = *reinterpret_cast<const i64x2*>(d + (size_t)(4 * s + q) * 256);
        }
    }
}

// A run of n_tiles >= 1 tiles: tile_at(i) gives tile i's first byte of slice 0 (wave-uniform),
// off the lanes' copy offsets from there.  Constructing it issues the first copies: a
// wait for a load issued afterwards waits for them too, so the digits are loaded before.
template <class TileAt>
struct TileRun {
    const TileWave& W;
    const uint32_t (&off)[5];
    TileAt tile_at;
    int n_tiles, tps, n_items, next_tile, next_sl;
    __device__ __forceinline__ TileRun(const TileWave& W_, const uint32_t (&off_)[5], int n, TileAt t)
        : W(W_), off(off_), tile_at(t) {
        restart(n);
    }
    __device__ __forceinline__ void restart(int n) {
        start(n);
        if (n_items > 0)
            wait_vmcnt<5 * kRing>();
        else
            wait_vmcnt<0>();
    }
    // The first copies alone: the caller waits, with wait_vmcnt, for digits loaded before.
    __device__ __forceinline__ void start(int n) {
        n_tiles = n;
        tps = kTileWaves >> W.log2_wt;
        next_tile = W.tg;
        next_sl = 0;
        n_items = (W.tg < n_tiles ? (n_tiles - W.tg + tps - 1) / tps : 0) * W.n_sl;
        // kRing items (past the last one: it again) or none, so that the compiler knows how
        // many copies are younger than the digits
        if (n_items > 0) unroll<kRing>([&](auto sc) __attribute__((always_inline)) { issue(decltype(sc)::value); });
    }
    __device__ __forceinline__ void issue(int slot) {
        const uint8_t* tile = tile_at(min(next_tile, n_tiles - 1));
        copy_item(tile + (size_t)(W.first + W.wt + (next_sl << W.log2_wt)) * kSliceBytes, off, W.ring_lds + slot * kLdsItemBytes);
        if (++next_sl == W.n_sl) {
            next_sl = 0;
            next_tile += tps;
        }
    }
};

// Multiplies a run.  sums[(i * NG + g) * 64 + lane] gets, for weight row lane & 15 of tile i
// and activation row 4 g + (lane >> 4), the tile's sum without the row scale.  part:
// 2 * kTileWaves * NG * 64 floats.  Every wave of the block calls it; after a barrier by
// the caller the sums are there.
template <int SP, int NG, class Run>
__device__ __forceinline__ void multiply_tiles(Run& R, const i64x2 (&a)[NG][SP][4], float* part, float* sums) {
    const TileWave& W = R.W;
    const int n_tiles = R.n_tiles, tps = R.tps, n_items = R.n_items;
    const int steps = (n_tiles + tps - 1) / tps;
    const uint32_t part_lds = (uint32_t)(uintptr_t)part + 4 * W.lane;
    const uint32_t sums_lds = (uint32_t)(uintptr_t)sums + 4 * W.lane;
    int it = 0, slot = 0;
    for (int step = 0; step < steps; ++step) {
        float acc[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[g] = 0.0f;
        const int tile = W.tg + step * tps;
        if (tile < n_tiles) {
            unroll<SP>([&](auto slc) __attribute__((always_inline)) {
                constexpr int sl = decltype(slc)::value;
                if (sl < W.n_sl) {
                    // the item is the oldest of min(kRing, items issued and not read) in flight
                    const int rem = max(n_items, kRing) - 1 - it;
                    if (rem >= kRing - 1) {
                        wait_vmcnt_mem<(kRing - 1) * 5>();
                    } else {
                        unroll<kRing - 1>([&](auto kc) __attribute__((always_inline)) {
                            constexpr int k = decltype(kc)::value;
                            if (rem == k) wait_vmcnt_mem<k * 5>();
                        });
                    }
                    ItemWords v;
                    const uint32_t row = W.ring_lds + slot * kLdsItemBytes + kSliceBytes * W.row;
                    read_item(row, row + 8 * W.grp, v);
                    if (it + kRing < n_items) R.issue(slot);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t e1 = (uint32_t)(v.e[q] >> 32);
                        const uint32_t e2 = (uint32_t)(q & 1 ? v.f[q / 2] >> 32 : v.f[q / 2]);
                        const uint32_t b00 = __builtin_amdgcn_alignbyte(e1, (uint32_t)v.e[q], 2);
                        const uint32_t b01 = __builtin_amdgcn_alignbyte(e2, e1, 2);
                        const long b0 = (long)(((uint64_t)b01 << 32) | b00);
                        const long b1 = (long)v.o[q];
                        const float d0 = half_lo((uint32_t)v.s[q]), d1 = half_hi((uint32_t)(v.s[q] >> 32));
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const i32x4 z = {0, 0, 0, 0};
                            const i32x4 s0 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[g][sl][q][0], b0, z, 0, 0, 0);
                            const i32x4 s1 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[g][sl][q][1], b1, z, 0, 0, 0);
                            const float t0 = __builtin_fmaf((float)(s0[3] * 256 + s0[2]), 65536.0f,
                                                            (float)(s0[1] * 256 + s0[0]));
                            acc[g] = __builtin_fmaf(d0, t0, acc[g]);
                            const float t1 = __builtin_fmaf((float)(s1[3] * 256 + s1[2]), 65536.0f,
                                                            (float)(s1[1] * 256 + s1[0]));
                            acc[g] = __builtin_fmaf(d1, t1, acc[g]);
                        }
                        // products of all four block pairs in flight together only where
                        // their results (8 registers a pair and four rows) leave room
                        if constexpr (NG * SP > 4) __builtin_amdgcn_sched_barrier(0);
                    }
                    ++it;
                    slot = slot == kRing - 1 ? 0 : slot + 1;
                }
            });
        }
        if (W.log2_wt == 0) {  // one wave a tile: nothing to add
            if (tile < n_tiles) {
#pragma unroll
                for (int g = 0; g < NG; ++g) write_sum(sums_lds + 256 * (tile * NG + g), acc[g]);
            }
            continue;
        }
        const uint32_t buf = part_lds + (step & 1) * (kTileWaves * NG * 256);
#pragma unroll
        for (int g = 0; g < NG; ++g) write_sum(buf + 256 * (W.wv * NG + g), acc[g]);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // tile step * tps + q is added up by wave (step * tps + q) mod 8
        const int q = (W.wv - step * tps) & (kTileWaves - 1);
        if (q < tps && step * tps + q < n_tiles) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
                write_sum(sums_lds + 256 * ((step * tps + q) * NG + g),
                          read_sums(buf + 256 * ((q << W.log2_wt) * NG + g), 1 << W.log2_wt, 256 * NG));
        }
    }
    wait_vmcnt_mem<0>();  // copies past the last item
}

}  // namespace q8k
