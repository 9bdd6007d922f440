// Low-rank adapters of many requests beside a shared projection (gfx950).
//
// Row t with adapter a adds scale[a] * B[a] (A[a] x[t]) to the shared product.  Two launches:
// the inner products u[t][c] = scale[a] * A[a][c] . x[t] of every row (c over the
// sections' ranks; float32, a block of four waves four products), then each output's dot of u
// with its row of B, added to the shared product (or, for a fused gate_up, the activation behind it).
// In the packed calls the second launch computes the shared product too: one row on the
// one-row kernel of gemv_q8.hip, more on the digit tiles (digit_tiles.h), whose digits the
// first launch writes.  Bound by the weights' bytes and, in small matrices, by the two
// launches' starts: 6144 x 4096 (27 MB, rank 16, weights from memory) takes 12.8 us at 1 row (4
// to 5 of them the first launch) and 22.3 at 16, the fused 24576 x 4096 (107 MB) 33.9 at 8 and
// 41.3 at 16.  More rows (38, 63 and 116 us at 64, 128 and 255 rows of 6144 x 4096; 105, 195 and
// 379 fused) add passes over the tiles: of the tile launch's cycles the lanes issue 26 % and the
// matrix cores work 9 % at 16 rows, 48 % and 21 % at 255 (counters); the rest is the chain of
// copies, LDS reads, products and sums that two waves a SIMD leave open.  With many rows the
// correction has a form of its own.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "digit_tiles.h"
#include "gemv_core.h"
#include "lora_core.h"
#include "q8_internal.h"
#include "q8_validate.h"
#include "shared_mem.h"
#include "wave_dpp.h"

namespace q8k {

// gemv_q8.hip: q8_linear of one row (k <= 16384) with a correction behind its sums
hipError_t launch_gemv_q8_lora_row(const DeviceInfo& dev, const uint8_t* w, int64_t n_out, int64_t k, bool silu_pairs,
                                   const float* x, const LoraOneRow& lora, float* y, hipStream_t stream);

// Four inner products u[t][c0 .. c0+3] by a block of 256 threads, every load of up to 8192
// elements of the row and the four rows of A issued before the first product.
constexpr int kShrinkCols = 4;
template <class Ty>
__device__ __forceinline__ void lora_shrink(const LoraArgs& lo, const float* __restrict__ x, int k, int64_t ldx,
                                            float* __restrict__ u, int64_t unit) {
    __shared__ float wave_sums[4][kShrinkCols];
    const int tid = threadIdx.x;
    const int cols = lo.n_sections * lo.rank;
    const int groups = cols / kShrinkCols;
    const int64_t t = unit / groups;
    const int c0 = (int)(unit - t * groups) * kShrinkCols;
    const int a = lo.of_row(t);
    const int left = a < 0 ? 0 : lo.rank_of(a) - c0 % lo.rank;  // products the adapter has here
    if (left <= 0) {
        if (tid < kShrinkCols) u[t * cols + c0 + tid] = 0.0f;
        return;
    }
    const typename Ty::T* ar = static_cast<const typename Ty::T*>(lo.a) + ((size_t)a * cols + c0) * k;
    const float* xr = x + t * ldx;
    float acc[kShrinkCols] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = 8 * tid; i0 < k; i0 += 8192) {
        typename Ty::V v[4][kShrinkCols];
        LoraF32::V w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int i = i0 + 2048 * s < k ? i0 + 2048 * s : 8 * tid;  // past the end: not multiplied
            w[s] = LoraF32::load8(xr + i);
#pragma unroll
            for (int c = 0; c < kShrinkCols; ++c) v[s][c] = Ty::load8(ar + (size_t)c * k + i);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (i0 + 2048 * s < k) {
#pragma unroll
                for (int c = 0; c < kShrinkCols; ++c)
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[c] = __builtin_fmaf(Ty::at(v[s][c], q), LoraF32::at(w[s], q), acc[c]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kShrinkCols; ++c)
        for (int off = 32; off >= 1; off >>= 1) acc[c] += __shfl_xor(acc[c], off, 64);
    if ((tid & 63) == 0)
#pragma unroll
        for (int c = 0; c < kShrinkCols; ++c) wave_sums[tid >> 6][c] = acc[c];
    __syncthreads();
    if (tid < kShrinkCols) {
        const float sum = (wave_sums[0][tid] + wave_sums[1][tid]) + (wave_sums[2][tid] + wave_sums[3][tid]);
        u[t * cols + c0 + tid] = tid < left ? sum * (lo.scale ? lo.scale[a] : 1.0f) : 0.0f;
    }
}

template <class Ty>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs lo, const float* __restrict__ x, int m, int k,
                                                          int64_t ldx, float* __restrict__ u) {
    const int64_t units = (int64_t)m * (lo.n_sections * lo.rank / kShrinkCols);
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        lora_shrink<Ty>(lo, x, k, ldx, u, unit);
        __syncthreads();  // the next unit overwrites the waves' sums
    }
}

// What the second launch needs of a row beside its digits, in one load: an output's loads of
// its exponent, adapter and rank one after the other were a good part of a tile's end.
struct alignas(16) TileRow {
    int exp, adapter, rank, unused;
};

// First launch of the packed calls: blocks 0 .. m-1 write the rows' digits, the others the
// inner products.
template <class Ty>
__global__ __launch_bounds__(256) void lora_prepare_kernel(LoraArgs lo, const float* __restrict__ x, int m, int k,
                                                           int64_t ldx, float* __restrict__ u,
                                                           int8_t* __restrict__ dig, TileRow* __restrict__ rows,
                                                           uint32_t* __restrict__ arrived, int counters) {
    const int b = blockIdx.x;
    for (int i = b * 256 + threadIdx.x; i < counters; i += gridDim.x * 256) arrived[i] = 0;
    if (b < m) {
        write_digits(x + b * ldx, k, dig + (size_t)b * k * 4, &rows[b].exp);
        if (threadIdx.x == 0) {
            const int a = lo.of_row(b);
            rows[b].adapter = a;
            rows[b].rank = a < 0 ? 0 : lo.rank_of(a);
        }
    } else {
        lora_shrink<Ty>(lo, x, k, ldx, u, b - m);
    }
}

template <class Ty, bool SILU>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs lo, const float* __restrict__ u, const float* y,
                                                          int64_t n, int64_t ldy, float* out, int64_t ldo, int m) {
    const int64_t n_out = SILU ? n / 2 : n;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_out) return;
    for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
        const int a = lo.of_row(t), r = a < 0 ? 0 : lo.rank_of(a);
        const float* ut = u + t * lo.n_sections * lo.rank;
        float g = y[t * ldy + i];
        if (a >= 0) g += lora_delta<Ty>(lo, n, a, r, i, ut);
        if constexpr (SILU) {
            float v = y[t * ldy + n_out + i];
            if (a >= 0) v += lora_delta<Ty>(lo, n, a, r, n_out + i, ut);
            g = silu_mul(g, v);
        }
        out[t * ldo + i] = g;
    }
}

// Second launch of the packed calls: the shared product's tiles with the correction (and,
// SILU, the activation) behind each.  A block owns a run of neighbouring tiles and streams
// them once for every 4 * NG rows (every gy-th group of those); a fused tile is
// 8 gate rows and their 8 up rows.  A row of more than 16 slices (k > 4096) is cut into ks
// ranges, each with blocks of its own for the same tiles: the digits of a range fit
// the registers for as many tiles as the block has.  The ranges' sums then go through
// memory, and the last block of a tile adds them up, in their order, and finishes it.
struct TileSplit {
    int ks, log2_wt;    // ranges; waves a tile within a range
    int runs, gy;       // runs of tiles; groups of rows at a time
    float* partial;     // [row group][range][tile][NG * 64]
    uint32_t* arrived;  // [row group][tile]: ranges there, zero before the launch
};
constexpr int kLoraSumTiles = 64;  // tiles * NG whose sums wait in LDS

template <int NG>
constexpr size_t lora_tiles_lds() {
    return kRingBytes + sizeof(float) * (2 * kTileWaves * NG * 64 + kLoraSumTiles * 64);
}

template <int SP, int NG, bool SILU>
__global__ __launch_bounds__(kTileThreads) void lora_tiles_kernel(const uint8_t* __restrict__ w, int n_out, int k,
                                                                  TileSplit split,
                                                                  const int8_t* __restrict__ dig,
                                                                  const TileRow* __restrict__ rows, LoraArgs lo,
                                                                  const float* __restrict__ u, int m,
                                                                  float* __restrict__ y, int64_t ldy) {
    extern __shared__ float4 smem4[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(smem4);
    float* part = reinterpret_cast<float*>(smem + kRingBytes);
    float* sums = part + 2 * kTileWaves * NG * 64;
    __shared__ uint32_t before;
    // blocks that stream the same weights for other rows lie on the same XCD (workgroups go to
    // the 8 XCDs in turn), whose L2 reads them once
    const int place = blockIdx.x / 8, unit = blockIdx.x % 8 + 8 * (place / split.gy), gy = split.gy, runs = split.runs;
    if (unit >= runs * split.ks) return;
    const int kz = unit % split.ks, run_id = unit / split.ks;
    const int s0 = (k >> 8) * kz / split.ks, s1 = (k >> 8) * (kz + 1) / split.ks;
    const TileWave W(smem, s1 - s0, split.log2_wt, s0);
    constexpr int kOut = SILU ? kTileRows / 2 : kTileRows;  // outputs of a tile
    const uint32_t rb = (uint32_t)(k >> 5) * 34u;
    const int tiles_all = (n_out + kOut - 1) / kOut;
    const int first = (int)((int64_t)tiles_all * run_id / runs);
    const int tiles = (int)((int64_t)tiles_all * (run_id + 1) / runs) - first;
    // the last tile starts early enough to be whole; a matrix smaller than a tile repeats its
    // last row
    const int last_row0 = max(0, n_out - kOut);
    auto row0_of = [&](int i) __attribute__((always_inline)) { return min((first + i) * kOut, last_row0); };
    uint32_t off[5];
    W.offsets([&](int r) __attribute__((always_inline)) -> uint32_t {
        const int half = SILU ? r / kOut : 0;
        return (uint32_t)(min(r - half * kOut, n_out - 1) + half * n_out) * rb;
    }, off);
    constexpr int kChunk = kLoraSumTiles / NG;
    constexpr int kFly = SP * NG >= 6 ? 1 : SP * NG >= 4 ? 2 : 4;  // what the digits' registers leave
    int m0 = 4 * NG * (place % gy), c0 = 0;  // the rows and the block's tile the run starts at
    auto tile_at = [&](int i) __attribute__((always_inline)) { return w + (size_t)row0_of(c0 + i) * rb; };
    i64x2 a[NG][SP][4];
    auto load = [&] __attribute__((always_inline)) {
        const int last = min(4 * NG, m - m0) - 1;
        load_digits<SP, NG>(W, [&](int s) __attribute__((always_inline)) {
            return dig + (size_t)(m0 + min(s, last)) * k * 4;
        }, a);
    };
    load();
    TileRun run(W, off, min(kChunk, tiles), tile_at);
    while (true) {
        const int nt = run.n_tiles, t0 = m0, tile0 = c0, mm = min(4 * NG, m - m0);
        multiply_tiles<SP, NG>(run, a, part, sums);
        __syncthreads();
        // the next run's digits and first weights come while this one's outputs are finished
        // (24576 x 4096 fused, 64 rows, one group of rows at a time: 134 us without, 128 with)
        c0 += nt;
        if (c0 >= tiles) {
            c0 = 0;
            m0 += 4 * NG * gy;
            if (m0 < m) load();
        }
        const bool more = m0 < m;
        if (more) run.start(min(kChunk, tiles - c0));
        bool finish = true;
        if (split.ks > 1) {
            const int64_t group = t0 / (4 * NG);
            float* mine = split.partial + ((group * split.ks + kz) * tiles_all + first + tile0) * (NG * 64);
            const int64_t range = (int64_t)tiles_all * (NG * 64);
            for (int i = threadIdx.x; i < nt * NG * 64; i += kTileThreads) store_shared(mine + i, sums[i]);
            wait_vmcnt_mem<0>();
            __syncthreads();
            if (threadIdx.x == 0)
                before = __hip_atomic_fetch_add(split.arrived + group * tiles_all + first + tile0, 1u, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            finish = (int)before == split.ks - 1;
            if (finish)
                for (int i = 2 * threadIdx.x; i < nt * NG * 64; i += 2 * kTileThreads) {
                    float2 v = load_shared(mine + i - kz * range);
                    for (int z = 1; z < split.ks; ++z) {
                        const float2 t = load_shared(mine + i + (z - kz) * range);
                        v.x += t.x;
                        v.y += t.y;
                    }
                    sums[i] = v.x;
                    sums[i + 1] = v.y;
                }
            __syncthreads();
        }
        // outputs of the chunk: (row of the call, tile, output of the tile), outputs fastest
        for (int o = threadIdx.x; finish && o < mm * nt * kOut; o += kTileThreads) {
            const int r = o % kOut, q = o / kOut;
            const int s = q / nt, tile = q - s * nt;
            const int i = row0_of(tile0 + tile) + r;
            if (i >= n_out) continue;
            const int t = t0 + s;
            const float* sum = sums + (tile * NG + (s >> 2)) * 64 + 16 * (s & 3) + r;
            const int4 row = *reinterpret_cast<const int4*>(rows + t);
            const int ex = row.x, ad = row.y, rank = row.z;
            const float* ut = u + (size_t)t * lo.n_sections * lo.rank;
            float v = row_scaled(sum[0], ex);
            if (ad >= 0) v += lora_delta_any<kFly>(lo, SILU ? 2 * (int64_t)n_out : n_out, ad, rank, i, ut);
            if constexpr (SILU) {
                float up = row_scaled(sum[kOut], ex);
                if (ad >= 0) up += lora_delta_any<kFly>(lo, 2 * (int64_t)n_out, ad, rank, n_out + (int64_t)i, ut);
                v = silu_mul(v, up);
            }
            y[t * ldy + i] = v;
        }
        __syncthreads();  // the next run overwrites the sums
        if (!more) break;
        wait_vmcnt<0>();
    }
}

// ------------------------------------------------------------------- many rows
//
// For many rows (q8v::lora_uses_matrix_cores) the correction runs on the bf16 matrix cores at
// float32 accuracy.  A float32 value is the exact sum of three bf16 values (its leading 8 bits, the
// next 8, the last 8, each cut off, not rounded); a bf16 element of A or B is itself, a
// binary16 one the sum of two.  A product takes the partial products of parts i + j <= 2: 3, 5
// or 6 instructions for bf16, binary16 and float32 elements, with float32 accumulation.  The
// products with a bf16 element are exact.  For the others the pairs of parts 1 and 2 are left
// out, each below 2^-22 of the product (a part 1 is below 2^-7 of its value, a part 2 below
// 2^-15) and of its sign: a product falls short by up to 2^-22 of itself for binary16 elements,
// 2^-21 for float32 ones, 2^-24.5 on average, the size of a float32 rounding.  The pairs left out
// would be up to a third more instructions.
//
//   1. plan:   the rows sorted by adapter (those without one last), in tiles of 64 rows.
//   2. inner:  block (tile half of 32 rows, part of k): u of all sections' ranks; its four
//              waves take 64-wide steps of k in turn and add up through LDS.  The parts of k
//              give the few tiles enough blocks.
//   3. sum:    the parts added up, scaled and split, laid out as the next launch's operand.
//   4. outer:  block (tile, 128 outputs), 64 rows x 32 outputs a wave: u and B start out,
//              then the product's values, and no barrier lies between.
// Bound by the memory: x once, the product in and out.  6144 x 4096, three sections of rank
// 32 and 2048 rows: 59.8 us (plan 4.7, inner 19.2, sum 6.3, outer 29.6: 100 MB of product in
// and out at 3.4 TB/s).  Measured and not kept: u staged through LDS in the outer launch (37 us), the
// parts added by the last block of the inner one (33 us against 19 + 6), its next step's
// loads ahead (25 us).

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowTile = 64;

// Eight values as PARTS bf16 vectors that add up to them.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&v)[8], bf16x8 (&p)[PARTS]) {
    uint32_t r[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) r[q] = __builtin_bit_cast(uint32_t, v[q]);
#pragma unroll
    for (int s = 0; s < PARTS; ++s) {
        u32x4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __builtin_amdgcn_perm(r[2 * q + 1], r[2 * q], 0x07060302u);
        p[s] = __builtin_bit_cast(bf16x8, w);
        if (s + 1 < PARTS) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                r[q] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, r[q]) -
                                                        __builtin_bit_cast(float, r[q] & 0xffff0000u));
        }
    }
}

// Eight elements of A or B as bf16 parts; from the n-th on zero.
template <class Ty>
struct LoraParts;
template <>
struct LoraParts<LoraBF16> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void get(LoraBF16::V v, int n, bf16x8 (&p)[N]) {
        if (n < 8)
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q >= n) v[q] = 0;
        p[0] = __builtin_bit_cast(bf16x8, v);
    }
};
template <class Ty, int PARTS>
struct LoraFloatParts {
    static constexpr int N = PARTS;
    static __device__ __forceinline__ void get(const typename Ty::V& v, int n, bf16x8 (&p)[N]) {
        float f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = q < n ? Ty::at(v, q) : 0.0f;
        split8<PARTS>(f, p);
    }
};
template <>
struct LoraParts<LoraF16> : LoraFloatParts<LoraF16, 2> {};
template <>
struct LoraParts<LoraF32> : LoraFloatParts<LoraF32, 3> {};

template <int N>
__device__ __forceinline__ f32x16 mfma_parts(const bf16x8 (&a)[3], const bf16x8 (&b)[N], f32x16 c) {
#pragma unroll
    for (int i = 2; i >= 0; --i)
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
            if (i + j <= 2) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], c, 0, 0, 0);
    return c;
}

// Rows by adapter: sorted [m], and the tiles: adapter (n_adapters: none), first place, rows.
struct LoraPlan {
    bf16x8* split;         // [tile][3 parts][cols / 8][64 rows]
    int32_t* sorted;
    int4* tiles;
    int32_t* n_tiles;
};

__global__ __launch_bounds__(1024) void lora_plan_kernel(LoraArgs lo, int m, LoraPlan P) {
    constexpr int kBins = q8v::kLoraMaxAdapters + 64;  // five a lane of one wave
    __shared__ int count[kBins], at[kBins], tile_at[kBins];
    const int tid = threadIdx.x;
    auto bin = [&](int t) __attribute__((always_inline)) {
        const int a = lo.of_row(t);
        return a < 0 ? lo.n_adapters : a;
    };
    for (int b = tid; b < kBins; b += 1024) count[b] = 0;
    __syncthreads();
    for (int t = tid; t < m; t += 1024) atomicAdd(&count[bin(t)], 1);
    __syncthreads();
    if (tid < 64) {
        int rows = 0, tiles = 0;
        for (int q = 0; q < 5; ++q) {
            rows += count[5 * tid + q];
            tiles += (count[5 * tid + q] + kRowTile - 1) / kRowTile;
        }
        int r = wave_scan(rows) - rows;
        const int incl = wave_scan(tiles);
        int tl = incl - tiles;
        for (int q = 0; q < 5; ++q) {
            at[5 * tid + q] = r;
            tile_at[5 * tid + q] = tl;
            r += count[5 * tid + q];
            tl += (count[5 * tid + q] + kRowTile - 1) / kRowTile;
        }
        if (tid == 63) *P.n_tiles = incl;
    }
    __syncthreads();
    if (tid <= lo.n_adapters)
        for (int i = 0; i < count[tid]; i += kRowTile) {
            const int t = tile_at[tid] + i / kRowTile;
            P.tiles[t] = make_int4(tid, at[tid] + i, min(kRowTile, count[tid] - i), 0);
        }
    __syncthreads();
    // the order within an adapter is free: a row's result does not depend on its tile
    for (int t = tid; t < m; t += 1024) P.sorted[atomicAdd(&at[bin(t)], 1)] = t;
}

template <class Ty>
__global__ __launch_bounds__(256) void lora_inner_kernel(LoraArgs lo, LoraPlan P, const float* __restrict__ x, int m,
                                                         int k, int64_t ldx, float* __restrict__ u) {
    constexpr int kChunks = 4;  // of 32 columns a pass
    __shared__ float sums[4][kChunks * 16][64];
    if ((int)(blockIdx.x >> 1) >= *P.n_tiles) return;
    const int4 tile = P.tiles[blockIdx.x >> 1];
    const int a = tile.x, rows = min(32, tile.z - 32 * (int)(blockIdx.x & 1));
    if (a >= lo.n_adapters || rows <= 0) return;  // all parts alike
    const int32_t* ids = P.sorted + tile.y + 32 * (blockIdx.x & 1);
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
    const int cols = lo.n_sections * lo.rank;
    // a lane's k of instruction q within a step of 64: 16 q + 8 half, so that a load
    // instruction takes neighbouring bytes of every row
    const float* xr = x + (int64_t)ids[min(col, rows - 1)] * ldx + 8 * half;
    const typename Ty::T* ab = static_cast<const typename Ty::T*>(lo.a) + (size_t)a * cols * k + 8 * half;
    const int steps = k >> 6;
    const int s0 = (int)((int64_t)steps * blockIdx.y / gridDim.y), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / gridDim.y);
    for (int c0 = 0; c0 < cols; c0 += 32 * kChunks) {
        const int chunks = min(kChunks, (cols - c0 + 31) >> 5);
        f32x16 acc[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c][i] = 0.0f;
        for (int st = s0 + wv; st < s1; st += 4) {
            LoraF32::V xv[4];
            typename Ty::V av[kChunks][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) xv[q] = LoraF32::load8(xr + 64 * st + 16 * q);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (c < chunks) {
                    // a column past the last one repeats it
                    const typename Ty::T* p = ab + (size_t)min(c0 + 32 * c + col, cols - 1) * k + 64 * st;
#pragma unroll
                    for (int q = 0; q < 4; ++q) av[c][q] = Ty::load8(p + 16 * q);
                }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = LoraF32::at(xv[q], i);
                bf16x8 xs[3];
                split8<3>(f, xs);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c < chunks) {
                        bf16x8 as[LoraParts<Ty>::N];
                        LoraParts<Ty>::get(av[c][q], 8, as);
                        acc[c] = mfma_parts(xs, as, acc[c]);
                    }
            }
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if (c < chunks)
#pragma unroll
                for (int i = 0; i < 16; ++i) sums[wv][16 * c + i][lane] = acc[c][i];
        __syncthreads();
        for (int e = wv; e < 16 * chunks; e += 4) {
            const int i = e & 15, c = c0 + 32 * (e >> 4) + col;
            const int row = 8 * (i >> 2) + 4 * half + (i & 3);
            const float v = (sums[0][e][lane] + sums[1][e][lane]) + (sums[2][e][lane] + sums[3][e][lane]);
            if (c < cols && row < rows) u[((int64_t)blockIdx.y * m + ids[row]) * cols + c] = v;
        }
        __syncthreads();
    }
}

// u of a tile, its parts of k added up in their order, scaled and split.
__global__ __launch_bounds__(256) void lora_sum_kernel(LoraArgs lo, LoraPlan P, const float* __restrict__ u, int parts,
                                                       int m) {
    if ((int)blockIdx.x >= *P.n_tiles) return;
    const int4 tile = P.tiles[blockIdx.x];
    if (tile.x >= lo.n_adapters) return;
    const int cols = lo.n_sections * lo.rank, groups = cols >> 3, r = lo.rank_of(tile.x);
    const float sc = lo.scale ? lo.scale[tile.x] : 1.0f;
    const int row = threadIdx.x & (kRowTile - 1);
    const float* ur = u + (int64_t)P.sorted[tile.y + min(row, tile.z - 1)] * cols;
    const int64_t part = (int64_t)m * cols;
    for (int g = (threadIdx.x >> 6) + 4 * blockIdx.y; g < groups; g += 4 * gridDim.y) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int p0 = 0; p0 < parts; p0 += 4) {
            LoraF32::V v[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) v[p] = LoraF32::load8(ur + 8 * g + min(p0 + p, parts - 1) * part);
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (p0 + p < parts)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += LoraF32::at(v[p], e);
        }
        // products past the adapter's own rank (whatever A holds there) are 0
        const int j = 8 * g % lo.rank;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = j + e < r ? f[e] * sc : 0.0f;
        bf16x8 sv[3];
        split8<3>(f, sv);
#pragma unroll
        for (int p = 0; p < 3; ++p) P.split[(((int64_t)blockIdx.x * 3 + p) * groups + g) * kRowTile + row] = sv[p];
    }
}

constexpr int kOuterColumns = q8v::kLoraOuterColumns;  // outputs of a block, 32 a wave

// Outputs whose rows of B belong to one section (SILU: gate rows to one, up rows to one), in
// blocks of kOuterColumns.
struct LoraSpans {
    int n;
    int64_t begin[2 * Q8_LORA_MAX_SECTIONS + 1];
    int block[2 * Q8_LORA_MAX_SECTIONS + 1];  // first block; [n]: their number
};

template <class Ty, bool SILU>
__global__ __launch_bounds__(256) void lora_outer_kernel(LoraArgs lo, LoraPlan P, const float* y, int64_t n, int64_t ldy,
                                                         float* out, int64_t ldo, LoraSpans S) {
    constexpr int kSides = SILU ? 2 : 1;
    constexpr int kN = LoraParts<Ty>::N;
    // neighbouring blocks take neighbouring outputs of the same rows: the memory sees whole rows
    const int row_tile = blockIdx.x / S.block[S.n], part = blockIdx.x - row_tile * S.block[S.n];
    if (row_tile >= *P.n_tiles) return;
    const int4 tile = P.tiles[row_tile];
    const int a = tile.x, rows = tile.z;
    const int32_t* ids = P.sorted + tile.y;
    int sp = 0;
    while (sp + 1 < S.n && part >= S.block[sp + 1]) ++sp;
    const int64_t n_out = SILU ? n / 2 : n;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
    const int64_t j1 = S.begin[sp + 1];
    const int64_t j = S.begin[sp] + kOuterColumns * (int64_t)(part - S.block[sp]) + 32 * wv + col;
    const int64_t jc = min(j, j1 - 1);  // a lane past the span repeats its last output, not stored
    const bool with = a < lo.n_adapters;
    const int r = with ? lo.rank_of(a) : 0, pairs = (r + 15) >> 4;

    // operands of k pair g: u of both row halves, B's row (entries past the adapter's rank as 0)
    const int groups = lo.n_sections * lo.rank >> 3;
    const bf16x8* ua[kSides];
    const typename Ty::T* bp[kSides];
#pragma unroll
    for (int s = 0; s < kSides; ++s) {
        const int sec = lo.section(s * n_out + S.begin[sp]);
        ua[s] = P.split + ((int64_t)row_tile * 3 * groups + sec * (lo.rank >> 3)) * kRowTile + col;
        bp[s] = static_cast<const typename Ty::T*>(lo.b) + ((size_t)(with ? a : 0) * n + s * n_out + jc) * lo.rank;
    }
    bf16x8 av[kSides][2][3];
    typename Ty::V bv[kSides];
    auto load = [&](int g) __attribute__((always_inline)) {
        const int q = min(2 * g + half, (lo.rank >> 3) - 1);
#pragma unroll
        for (int s = 0; s < kSides; ++s) {
            bv[s] = Ty::load8(bp[s] + 8 * q);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < 3; ++p) av[s][h][p] = ua[s][((int64_t)p * groups + q) * kRowTile + 32 * h];
        }
    };
    if (pairs) load(0);
    // then the product's values; the lane's rows of the tile: 32 h + 8 (e / 4) + 4 half + e % 4
    float py[kSides][2][16];
    int id[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e) id[h][e] = ids[min(32 * h + 8 * (e >> 2) + 4 * half + (e & 3), rows - 1)];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int s = 0; s < kSides; ++s) py[s][h][e] = y[(int64_t)id[h][e] * ldy + s * n_out + jc];
    f32x16 acc[kSides][2];
#pragma unroll
    for (int s = 0; s < kSides; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[s][h][e] = 0.0f;
    for (int g = 0; g < pairs; ++g) {
#pragma unroll
        for (int s = 0; s < kSides; ++s) {
            bf16x8 b[kN];
            LoraParts<Ty>::get(bv[s], r - 16 * g - 8 * half, b);
#pragma unroll
            for (int h = 0; h < 2; ++h) acc[s][h] = mfma_parts(av[s][h], b, acc[s][h]);
        }
        if (g + 1 < pairs) load(g + 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int row = 32 * h + 8 * (e >> 2) + 4 * half + (e & 3);
            float v = py[0][h][e] + acc[0][h][e];
            if constexpr (SILU) v = silu_mul(v, py[1][h][e] + acc[1][h][e]);
            if (row < rows && j < j1) out[(int64_t)id[h][e] * ldo + j] = v;
        }
}

static hipError_t launch_lora_shrink(const LoraArgs& lo, const float* x, int64_t m, int64_t k, int64_t ldx, float* u,
                                     hipStream_t stream) {
    const int64_t units = m * (lo.n_sections * lo.rank / kShrinkCols);
    auto kernel = lo.type == Q8_LORA_F32   ? lora_shrink_kernel<LoraF32>
                  : lo.type == Q8_LORA_F16 ? lora_shrink_kernel<LoraF16>
                                           : lora_shrink_kernel<LoraBF16>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(units < 65536 ? units : 65536)), dim3(256), 0, stream, lo, x, (int)m, (int)k,
                       ldx, u);
    return hipGetLastError();
}

template <class Ty>
static hipError_t lora_add_typed(const LoraArgs& lo, const float* y, int64_t n, int64_t ldy, bool silu,
                                 const float* x, int64_t m, int64_t k, int64_t ldx, float* out, int64_t ldo,
                                 float* u, hipStream_t stream) {
    hipError_t e = launch_lora_shrink(lo, x, m, k, ldx, u, stream);
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

template <class Ty>
static hipError_t lora_add_tiled(const LoraArgs& lo, const float* y, int64_t n, int64_t ldy, bool silu, const float* x,
                                 int64_t m, int64_t k, int64_t ldx, float* out, int64_t ldo, char* ws,
                                 const q8v::LoraWorkspace& L, hipStream_t stream) {
    float* u = reinterpret_cast<float*>(ws + L.u_off);
    const LoraPlan P{reinterpret_cast<bf16x8*>(ws + L.split_off),
                     reinterpret_cast<int32_t*>(ws + L.sorted_off), reinterpret_cast<int4*>(ws + L.tiles_off),
                     reinterpret_cast<int32_t*>(ws + L.count_off)};
    hipLaunchKernelGGL(lora_plan_kernel, dim3(1), dim3(1024), 0, stream, lo, (int)m, P);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned tiles = (unsigned)q8v::lora_max_tiles(m, lo.n_adapters);
    const int64_t steps = k / 64;
    const int parts = (int)(q8v::lora_parts(m) * 4 <= steps ? q8v::lora_parts(m) : (steps + 3) / 4);  // a step a wave at least
    hipLaunchKernelGGL(lora_inner_kernel<Ty>, dim3(2 * tiles, (unsigned)parts), dim3(256), 0, stream, lo, P, x, (int)m,
                       (int)k, ldx, u);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int groups = lo.n_sections * lo.rank / 8;
    hipLaunchKernelGGL(lora_sum_kernel, dim3(tiles, (unsigned)((groups + 3) / 4)), dim3(256), 0, stream, lo, P, u,
                       parts, (int)m);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    // the outputs' spans: cut at every section's end, and (SILU) at those of the up rows
    const int64_t n_out = silu ? n / 2 : n;
    int64_t cuts[2 * Q8_LORA_MAX_SECTIONS + 2];
    int nc = 0;
    cuts[nc++] = 0;
    cuts[nc++] = n_out;
    for (int s = 0; s < lo.n_sections; ++s)
        for (int64_t c : {lo.end[s], lo.end[s] - n_out})
            if (c > 0 && c < n_out) cuts[nc++] = c;
    std::sort(cuts, cuts + nc);
    nc = (int)(std::unique(cuts, cuts + nc) - cuts);
    LoraSpans S{};
    S.n = nc - 1;
    int blocks = 0;
    for (int i = 0; i < nc; ++i) {
        S.begin[i] = cuts[i];
        S.block[i] = blocks;
        if (i + 1 < nc) blocks += (int)((cuts[i + 1] - cuts[i] + kOuterColumns - 1) / kOuterColumns);
    }
    const dim3 grid(tiles * (unsigned)blocks);
    if (silu)
        hipLaunchKernelGGL((lora_outer_kernel<Ty, true>), grid, dim3(256), 0, stream, lo, P, y, n, ldy, out, ldo, S);
    else
        hipLaunchKernelGGL((lora_outer_kernel<Ty, false>), grid, dim3(256), 0, stream, lo, P, y, n, ldy, out, ldo, S);
    return hipGetLastError();
}

template <class Ty>
static hipError_t lora_add_any(const LoraArgs& lo, const float* y, int64_t n, int64_t ldy, bool silu, const float* x,
                               int64_t m, int64_t k, int64_t ldx, float* out, int64_t ldo, bool with_matrix_cores,
                               char* ws, const q8v::LoraWorkspace& L, hipStream_t stream) {
    if (with_matrix_cores)
        return lora_add_tiled<Ty>(lo, y, n, ldy, silu, x, m, k, ldx, out, ldo, ws, L, stream);
    return lora_add_typed<Ty>(lo, y, n, ldy, silu, x, m, k, ldx, out, ldo, reinterpret_cast<float*>(ws + L.u_off), stream);
}

hipError_t launch_lora_add(const DeviceInfo&, const float* y, int64_t n, int64_t ldy, bool silu_pairs,
                           const float* x, int64_t m, int64_t k, int64_t ldx, const q8_lora& lora, float* out,
                           int64_t ldo, void* workspace, hipStream_t stream) {
    const LoraArgs lo = lora_args(lora);
    const q8v::LoraWorkspace L = q8v::lora_workspace_layout(m, lora.n_sections, lora.rank, 0);
    char* ws = static_cast<char*>(workspace);
    const bool mc = q8v::lora_uses_matrix_cores(lora, m, n, k);
    switch (lora.type) {
        case Q8_LORA_F32: return lora_add_any<LoraF32>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, mc, ws, L, stream);
        case Q8_LORA_F16: return lora_add_any<LoraF16>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, mc, ws, L, stream);
        default: return lora_add_any<LoraBF16>(lo, y, n, ldy, silu_pairs, x, m, k, ldx, out, ldo, mc, ws, L, stream);
    }
}

// How the packed calls cut a matrix: ranges of k (a function of the sizes and the device
// alone, never of m), waves a tile and slices a wave within a range, runs of tiles.
struct TileCut {
    int ks, log2_wt, sp, runs;
};
static TileCut tile_cut(const DeviceInfo& dev, int64_t tiles, int64_t k) {
    const int S = (int)(k >> 8);
    const int least = (S + 15) / 16;
    TileCut best{};
    int64_t cost = 0;
    // beyond 16 slices, of the fewest ranges and the next two the one whose busiest block has
    // the fewest items a wave
    for (int ks = least; ks <= (least == 1 ? 1 : least + 2); ++ks) {
        const SliceShare sh = slice_share((S + ks - 1) / ks);
        const int64_t runs = std::min<int64_t>(tiles, std::max(1, dev.cu_count / ks));
        const int64_t most = (tiles + runs - 1) / runs, at_once = kTileWaves >> sh.log2_wt;
        const int64_t items = (most + at_once - 1) / at_once * sh.sp;
        if (!best.ks || items < cost) {
            cost = items;
            best = TileCut{ks, sh.log2_wt, sh.sp, (int)runs};
        }
    }
    return best;
}

template <int SP, int NG, bool SILU>
static hipError_t launch_lora_tiles(const DeviceInfo& dev, const TileCut& cut, int64_t m, const uint8_t* w,
                                    int64_t n_out, int64_t k, TileSplit split, const int8_t* dig,
                                    const TileRow* rows, const LoraArgs& lo, const float* u, float* y, int64_t ldy,
                                    hipStream_t stream) {
    auto kernel = lora_tiles_kernel<SP, NG, SILU>;
    constexpr size_t lds = lora_tiles_lds<NG>();
    static thread_local int attr_dev = -1;
    if (attr_dev != dev.device) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
        attr_dev = dev.device;
    }
    // one block per CU, shared between runs of tiles and groups of rows: gy groups at a time,
    // the gy with the cheapest block.  Costs in items (a wave's 16 x 256 weights): a pass over
    // the rows about 6, finishing the tiles whose sums fit LDS about 10.  One group at a time,
    // which streams the weights anew for each, against this: 6144 x 4096 at 64 rows 68 | 37 us, 255
    // rows 252 | 116 us; 83 rows of 2001 x 1024 24.5 | 16.7 us.
    const int64_t groups = (m + 4 * NG - 1) / (4 * NG), tiles = (n_out + (SILU ? 8 : 16) - 1) / (SILU ? 8 : 16);
    const int64_t at_once = kTileWaves >> cut.log2_wt, chunk = kLoraSumTiles / NG;
    int64_t gy = 1, runs = cut.runs, cost = 0;
    for (int64_t g = 1; g <= groups; ++g) {
        // (g > 1: every XCD's blocks have CUs of their own)
        const int64_t r = std::min<int64_t>(tiles, g == 1 ? cut.runs : dev.cu_count / (8 * g) * 8 / cut.ks);
        if (r < 1) break;
        const int64_t most = (tiles + r - 1) / r;
        const int64_t c = (groups + g - 1) / g *
                          (6 + 10 * ((most + chunk - 1) / chunk) + (most + at_once - 1) / at_once * cut.sp);
        if (cost == 0 || c < cost) {
            cost = c;
            gy = g;
            runs = r;
        }
    }
    split.runs = (int)runs;
    split.gy = (int)gy;
    const dim3 grid((unsigned)(8 * gy * ((runs * cut.ks + 7) / 8)));
    hipLaunchKernelGGL(kernel, grid, dim3(kTileThreads), lds, stream, w, (int)n_out, (int)k, split, dig, rows, lo, u,
                       (int)m, y, ldy);
    return hipGetLastError();
}

// Activation rows a pass takes, in fours: as many as there are, up to 128 registers a lane
// of digits (16 a slice and four rows).
template <bool SILU, class... Args>
static hipError_t launch_lora_tiles_m(const DeviceInfo& dev, const TileCut& cut, int64_t m, Args... args) {
    if (cut.sp == 1) {
        if (m > 8) return launch_lora_tiles<1, 4, SILU>(dev, cut, m, args...);
        if (m > 4) return launch_lora_tiles<1, 2, SILU>(dev, cut, m, args...);
        return launch_lora_tiles<1, 1, SILU>(dev, cut, m, args...);
    }
    if (cut.sp == 2) {
        if (m > 8) return launch_lora_tiles<2, 4, SILU>(dev, cut, m, args...);
        if (m > 4) return launch_lora_tiles<2, 2, SILU>(dev, cut, m, args...);
        return launch_lora_tiles<2, 1, SILU>(dev, cut, m, args...);
    }
    if (m > 4) return launch_lora_tiles<3, 2, SILU>(dev, cut, m, args...);
    return launch_lora_tiles<3, 1, SILU>(dev, cut, m, args...);
}

hipError_t launch_linear_lora(const DeviceInfo& dev, const uint8_t* w, int64_t n_out, int64_t k, bool silu,
                              const float* x, int64_t m, int64_t ldx, const q8_lora& lora, float* y, int64_t ldy,
                              void* workspace, hipStream_t stream) {
    const int64_t n = silu ? 2 * n_out : n_out;
    const q8v::LoraWorkspace L =
        q8v::lora_workspace_layout(m, lora.n_sections, lora.rank, q8v::lora_base_bytes(m, n, k));
    char* ws = static_cast<char*>(workspace);
    if (q8v::lora_uses_one_row(m, k)) {
        // the inner products, then the one-row kernel with the correction behind its sums
        const LoraArgs lo = lora_args(lora);
        float* u = reinterpret_cast<float*>(ws + L.u_off);
        hipError_t e = lora.n_adapters ? launch_lora_shrink(lo, x, m, k, ldx, u, stream) : hipSuccess;
        if (e != hipSuccess) return e;
        return launch_gemv_q8_lora_row(dev, w, n_out, k, silu, x, LoraOneRow{lo, u, n}, y, stream);
    }
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
    const int64_t per_tile = silu ? kTileRows / 2 : kTileRows;
    const int64_t tiles = (n_out + per_tile - 1) / per_tile;
    const TileCut cut = tile_cut(dev, tiles, k);
    const q8v::LoraTilesWorkspace T = q8v::lora_tiles_workspace_layout(m, n, k);
    TileRow* rows = reinterpret_cast<TileRow*>(ws + L.base_off + T.rows_off);
    int8_t* dig = reinterpret_cast<int8_t*>(ws + L.base_off + T.dig_off);
    TileSplit split{cut.ks, cut.log2_wt, 0, 0, reinterpret_cast<float*>(ws + L.base_off + T.partial_off),
                    reinterpret_cast<uint32_t*>(ws + L.base_off + T.arrived_off)};
    const int counters = cut.ks > 1 ? (int)(q8v::lora_row_groups(m) * tiles) : 0;
    const int units = lora.n_adapters ? (int)m * (lora.n_sections * lora.rank / kShrinkCols) : 0;
    const dim3 grid((unsigned)((int)m + units));
    if (lora.type == Q8_LORA_F32)
        hipLaunchKernelGGL(lora_prepare_kernel<LoraF32>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u, dig,
                           rows, split.arrived, counters);
    else if (lora.type == Q8_LORA_F16)
        hipLaunchKernelGGL(lora_prepare_kernel<LoraF16>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u, dig,
                           rows, split.arrived, counters);
    else
        hipLaunchKernelGGL(lora_prepare_kernel<LoraBF16>, grid, dim3(256), 0, stream, lo, x, (int)m, (int)k, ldx, u, dig,
                           rows, split.arrived, counters);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return silu ? launch_lora_tiles_m<true>(dev, cut, m, w, n_out, k, split, dig, rows, lo, u, y, ldy, stream)
                : launch_lora_tiles_m<false>(dev, cut, m, w, n_out, k, split, dig, rows, lo, u, y, ldy, stream);
}

}  // namespace q8k
