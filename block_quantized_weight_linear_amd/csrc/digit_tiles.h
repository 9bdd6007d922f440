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
//     t = (256 s3 + s2) 2^16 + (256 s1 + s0)   (the halves exact integers, one fma)
//     acc = fma(d, t, acc)                      (d: the block's scale)
// so a weight costs a lane 6 VALU operations per 512 weights and 4 activation rows instead
// of a conversion and 4 fmas each.  Per output: the chain over the blocks of a 256-wide
// slice, over the wave's slices, then the waves' sums in order: it depends on k alone,
// never on the other rows of the call.
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
// slices each.  The fewest idle wave slices win, ties go to more waves (fewer registers),
// and SP stays at 3 or below while S <= 24.
struct SliceShare {
    int log2_wt, sp;
};
__host__ __device__ inline SliceShare slice_share(int S) {
    SliceShare best{3, (S + 7) / 8};
    for (int l = 2; l >= 0; --l) {
        const int sp = (S + (1 << l) - 1) >> l;
        if (sp <= 3 && (sp << l) < (best.sp << best.log2_wt) && (1 << l) <= S) best = SliceShare{l, sp};
    }
    while (best.log2_wt > 0 && (1 << best.log2_wt) > S) best = SliceShare{best.log2_wt - 1, 1};
    return best;
}

// One item into lds .. lds + 4351: four copies of 16 bytes a lane and one of 4 from base (an
// SGPR pair) + off[c], five vmcnt events, with the non-temporal hint (weights are read once).
__device__ __forceinline__ void copy_item(const uint8_t* base, const uint32_t (&off)[5], uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %7\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %6 nt\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %2, %6 nt\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %3, %6 nt\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %4, %6 nt\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %5, %6 nt\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "v"(off[4]), "s"(base), "s"(lds)
        : "memory", "scc");
}

template <class F, int... I>
__device__ __forceinline__ void unroll_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F&& f) {
    unroll_impl(f, std::make_integer_sequence<int, N>{});
}

// Digits of one activation row, by a block of 256 threads: dig is the row's
// [k / 32][4 digits][32] bytes, *exp_out the exponent e - 29 of its scale.  A row that holds
// a NaN or an infinity gets kNotFinite and zero digits: all its outputs are NaN.
constexpr int kNotFinite = 1 << 20;
__device__ __forceinline__ float row_scaled(float sum, int exp) {
    return exp == kNotFinite ? __builtin_nanf("") : __builtin_ldexpf(sum, exp);
}
__device__ __forceinline__ int row_exponent(uint32_t max_bits) { return max((int)(max_bits >> 23) - 127, -126); }
__device__ __forceinline__ void write_digits(const float* __restrict__ xr, int k, int8_t* __restrict__ dig,
                                             int* __restrict__ exp_out) {
    __shared__ uint32_t wave_max_bits[4];
    const int tid = threadIdx.x;
    uint32_t mx = 0;  // magnitudes as bits: ordered like the values, NaN above infinity
    for (int i = 4 * tid; i < k; i += 1024) {
        const float4 v = *reinterpret_cast<const float4*>(xr + i);
        const uint32_t a = __builtin_bit_cast(uint32_t, v.x) & 0x7fffffffu;
        const uint32_t b = __builtin_bit_cast(uint32_t, v.y) & 0x7fffffffu;
        const uint32_t c = __builtin_bit_cast(uint32_t, v.z) & 0x7fffffffu;
        const uint32_t d = __builtin_bit_cast(uint32_t, v.w) & 0x7fffffffu;
        mx = max(max(max(mx, a), b), max(c, d));
    }
    for (int off = 32; off >= 1; off >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, off, 64));
    if ((tid & 63) == 0) wave_max_bits[tid >> 6] = mx;
    __syncthreads();
    mx = max(max(wave_max_bits[0], wave_max_bits[1]), max(wave_max_bits[2], wave_max_bits[3]));
    const bool finite = mx < 0x7f800000u;
    const int e = row_exponent(mx);
    if (tid == 0) *exp_out = finite ? e - 29 : kNotFinite;
    for (int i = 4 * tid; i < k; i += 1024) {
        const float4 v = *reinterpret_cast<const float4*>(xr + i);
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
            *reinterpret_cast<uint32_t*>(dig + (size_t)(i >> 5) * 128 + 32 * d + (i & 31)) = out[d];
    }
}

// What a wave knows about its place: its slices of a row of S, its tiles of a step.
struct TileWave {
    int lane, wv, wt, tg, log2_wt, n_sl, row, grp;  // row, grp: lane & 15, lane >> 4
    uint32_t ring_lds;
    const uint8_t* ring;
    __device__ __forceinline__ TileWave(uint8_t* smem_ring, int S, int log2_wt_) : log2_wt(log2_wt_) {
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

// A operands of the wave's slices for 4 * NG activation rows; digits_of(slot) gives the
// row's digits (nullptr: no such row, zeros).
template <int SP, int NG, class DigitsOf>
__device__ __forceinline__ void load_digits(const TileWave& W, DigitsOf&& digits_of, long (&a)[NG][SP][8]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int8_t* d = digits_of(4 * g + (W.row >> 2));
#pragma unroll
        for (int sl = 0; sl < SP; ++sl) {
            const int s = W.wt + (sl << W.log2_wt);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[g][sl][j] = 0;
                if (d && sl < W.n_sl)
                    a[g][sl][j] = *reinterpret_cast<const long*>(d + (size_t)(8 * s + j) * 128 + 32 * (W.row & 3) +
                                                                 8 * W.grp);
            }
        }
    }
}

// A run of n_tiles tiles: tile_at(i, base, off) gives tile i's first byte of slice 0
// (wave-uniform) and the lanes' copy offsets.  Constructing it issues the first copies; a
// load issued afterwards waits for them too.
template <class TileAt>
struct TileRun {
    const TileWave& W;
    TileAt tile_at;
    int n_tiles, tps, n_items, next_tile, next_sl;
    __device__ __forceinline__ TileRun(const TileWave& W_, int n, TileAt t) : W(W_), tile_at(t) { restart(n); }
    __device__ __forceinline__ void restart(int n) {
        n_tiles = n;
        tps = kTileWaves >> W.log2_wt;
        next_tile = W.tg;
        next_sl = 0;
        n_items = (W.tg < n_tiles ? (n_tiles - W.tg + tps - 1) / tps : 0) * W.n_sl;
        unroll<kRing>([&](auto sc) __attribute__((always_inline)) {
            constexpr int s = decltype(sc)::value;
            if (s < n_items) issue(s);
        });
    }
    __device__ __forceinline__ void issue(int slot) {
        const uint8_t* base;
        uint32_t off[5];
        tile_at(next_tile, base, off);
        base += (size_t)(W.wt + (next_sl << W.log2_wt)) * kSliceBytes;
        copy_item(base, off, W.ring_lds + slot * kLdsItemBytes);
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
__device__ __forceinline__ void multiply_tiles(Run& R, const long (&a)[NG][SP][8], float* part, float* sums) {
    const TileWave& W = R.W;
    const int n_tiles = R.n_tiles, tps = R.tps, n_items = R.n_items;
    const int steps = (n_tiles + tps - 1) / tps;
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
                    const int rem = n_items - 1 - it;
                    if (rem >= kRing - 1) {
                        wait_vmcnt_mem<(kRing - 1) * 5>();
                    } else {
                        unroll<kRing - 1>([&](auto kc) __attribute__((always_inline)) {
                            constexpr int k = decltype(kc)::value;
                            if (rem == k) wait_vmcnt_mem<k * 5>();
                        });
                    }
                    const uint32_t* p =
                        reinterpret_cast<const uint32_t*>(W.ring + slot * kLdsItemBytes) + 68 * W.row + 2 * W.grp;
                    const uint32_t* ps = p - 2 * W.grp;
                    uint32_t v[4][7];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[q][0] = p[17 * q];
                        v[q][1] = p[17 * q + 1];
                        v[q][2] = p[17 * q + 2];
                        v[q][3] = p[17 * q + 9];
                        v[q][4] = p[17 * q + 10];
                        v[q][5] = ps[17 * q];
                        v[q][6] = ps[17 * q + 8];
                    }
                    wait_lgkmcnt_mem<0>();
                    if (rem >= kRing) R.issue(slot);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t b00 = __builtin_amdgcn_alignbyte(v[q][1], v[q][0], 2);
                        const uint32_t b01 = __builtin_amdgcn_alignbyte(v[q][2], v[q][1], 2);
                        const long b0 = (long)(((uint64_t)b01 << 32) | b00);
                        const long b1 = (long)(((uint64_t)v[q][4] << 32) | v[q][3]);
                        const float d0 = half_lo(v[q][5]), d1 = half_hi(v[q][6]);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const i32x4 z = {0, 0, 0, 0};
                            const i32x4 s0 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[g][sl][2 * q], b0, z, 0, 0, 0);
                            const i32x4 s1 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[g][sl][2 * q + 1], b1, z, 0, 0, 0);
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
                for (int g = 0; g < NG; ++g) sums[(tile * NG + g) * 64 + W.lane] = acc[g];
            }
            continue;
        }
        float* mine = part + ((step & 1) * kTileWaves + W.wv) * (NG * 64) + W.lane;
#pragma unroll
        for (int g = 0; g < NG; ++g) mine[64 * g] = acc[g];
        wait_lgkmcnt_mem<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // tile step * tps + q is added up by wave (step * tps + q) mod 8
        const int q = (W.wv - step * tps) & (kTileWaves - 1);
        if (q < tps && step * tps + q < n_tiles) {
            const float* from = part + ((step & 1) * kTileWaves + (q << W.log2_wt)) * (NG * 64) + W.lane;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float s = from[64 * g];
                for (int w = 1; w < (1 << W.log2_wt); ++w) s += from[(w * NG + g) * 64];
                sums[((step * tps + q) * NG + g) * 64 + W.lane] = s;
            }
        }
    }
}

}  // namespace q8k
