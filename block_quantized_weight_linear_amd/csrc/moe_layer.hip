// The whole mixture-of-experts layer (gfx950): softmax top-k routing and the router-weighted
// SwiGLU mixture of the chosen experts, for a few tokens in two launches.
//
//   1. prepare: the router's logits (summed in the order of the routers of route_topk.hip),
//      every token's digits (digit_tiles.h), the counters of the second launch cleared.
//   2. layer: one block per CU.  Every block selects all tokens' experts by itself (the
//      routers' choice, to the bit) and so knows the whole work list: the gate_up
//      tiles of the chosen experts (8 gate rows and their 8 up rows), their down tiles, then
//      the tokens' weighted sums.  An expert's tokens, eight at most, are one job; the jobs'
//      tiles are cut into one chunk of neighbouring tiles for each block.  A down chunk
//      waits until its jobs' hidden rows are there, the sums until all down tiles are.
//
// No block needs another one to start: every chunk is claimed by a flag before it is worked
// on, and a block that has waited for a while takes over chunks nobody has claimed (those
// of blocks that other work keeps off the device).  A chunk waits for gate_up chunks
// alone, which wait for nothing, so every wait ends.  A claim costs one uncontended atomic,
// a counter is shared by few blocks: 256 blocks taking turns at one address measured
// 25 ns each.
//
// Arithmetic: gate, up and down as in digit_tiles.h (the hidden row of a pair is written as
// digits with its own scale when the down tiles take it), y[t] = sum_j w_j out_j in slot
// order.  A token's result depends on its own row alone.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "digit_tiles.h"
#include "gemv_core.h"
#include "q8_internal.h"
#include "q8_validate.h"
#include "shared_mem.h"
#include "wave_dpp.h"

namespace q8k {

// A token whose router probabilities are not finite gets NaN outputs (its expert ids are
// invalid, so the mixture gave zeros).
__global__ __launch_bounds__(256) void moe_poison_kernel(const float* __restrict__ wts, int k, int h,
                                                         float* __restrict__ y, int ldy) {
    const int t = blockIdx.x;
    bool bad = false;
    for (int j = 0; j < k; ++j) bad |= wts[(size_t)t * k + j] != wts[(size_t)t * k + j];
    if (!bad) return;
    for (int c = threadIdx.x; c < h; c += 256) y[(size_t)t * ldy + c] = __builtin_nanf("");
}

// Flags and counters of the second launch, cleared by the first.
constexpr int kMaxChunks = q8v::kLayerMaxChunks;
constexpr int kMaxJobs = q8v::kLayerMaxJobs;  // an expert's tokens in eights
constexpr int kDoneParts = 16;                // the down tiles' count
// Each in a cache line of its own: a line that several blocks raise and poll is taken in
// turns (256 blocks on counters of the same line measured 6 us from the last raise to the
// last block that saw it).
struct alignas(128) LayerWord {
    uint32_t v;
};
struct LayerCounters {
    LayerWord down_done[kDoneParts];
    LayerWord claim_up[kMaxChunks], claim_down[kMaxChunks];
    LayerWord up_done[kMaxJobs];  // gate_up tiles
};
static_assert(sizeof(LayerCounters) == q8v::kLayerCounterBytes, "workspace layout");

// What the second launch works on.
struct LayerArgs {
    const float* logits;            // [m][n_exp]
    const int8_t* dig;              // [m] digits of h elements
    const int* exps;                // [m]
    float* hidden;                  // [m * k][f]  SiLU(gate) * up
    uint32_t* hid_max;              // [m * k] largest |hidden| as bits
    float* out;                     // [m * k][h]
    LayerCounters* cnt;
    const uint8_t* wgu;
    const uint8_t* wdn;
    float* y;
    int ldy, m, k, n_exp, f, h, normalize;
    float top_p;
    int log2_wt_h, log2_wt_f;
};

constexpr int kPrepareTokens = 4;

__global__ __launch_bounds__(256) void moe_layer_prepare_kernel(const float* __restrict__ x, int m, int h, int ldx,
                                                                const float* __restrict__ wr, int n_exp, int k,
                                                                float* __restrict__ logits, int8_t* __restrict__ dig,
                                                                int* __restrict__ exps,
                                                                uint32_t* __restrict__ hid_max,
                                                                LayerWord* __restrict__ counters, int n_counters) {
    const int b = blockIdx.x;
    for (int i = b * 256 + threadIdx.x; i < n_counters; i += gridDim.x * 256) counters[i].v = 0;
    if (b < m) {
        for (int i = threadIdx.x; i < k; i += 256) hid_max[b * k + i] = 0;
        write_digits(x + (size_t)b * ldx, h, dig + (size_t)b * h * 4, exps + b);
        return;
    }
    // logits of four experts (one a wave) and four tokens: the lane slices, fma order and
    // butterfly of route_logits_kernel
    const int groups = (n_exp + 3) >> 2;
    const int t0 = (b - m) / groups * kPrepareTokens;
    const int e = (b - m) % groups * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (e >= n_exp) return;
    const float* we = wr + (size_t)e * h;
    float acc[kPrepareTokens] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c0 = 0; c0 < h; c0 += 1024) {
        float4 v[4], a[kPrepareTokens][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 256 * i < h ? c0 + 256 * i : c0;  // past h: not multiplied
            v[i] = *reinterpret_cast<const float4*>(we + c + 4 * lane);
#pragma unroll
            for (int t = 0; t < kPrepareTokens; ++t)
                if (t0 + t < m) a[t][i] = *reinterpret_cast<const float4*>(x + (size_t)(t0 + t) * ldx + c + 4 * lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 + 256 * i < h) {
#pragma unroll
                for (int t = 0; t < kPrepareTokens; ++t) {
                    if (t0 + t < m) {
                        acc[t] = __builtin_fmaf(a[t][i].x, v[i].x, acc[t]);
                        acc[t] = __builtin_fmaf(a[t][i].y, v[i].y, acc[t]);
                        acc[t] = __builtin_fmaf(a[t][i].z, v[i].z, acc[t]);
                        acc[t] = __builtin_fmaf(a[t][i].w, v[i].w, acc[t]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kPrepareTokens; ++t) {
        if (t0 + t < m) {
            for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
            if (lane == 0) logits[(size_t)(t0 + t) * n_exp + e] = acc[t];
        }
    }
}

constexpr int kLayerMaxPairs = 2048;  // m * k < 8 * n_exp <= 2048
constexpr int kLayerSums = 64;        // tiles * NG whose sums wait in LDS
constexpr int kJobRows = 8;

struct LayerLds {
    float part[2 * kTileWaves * 2 * 64];
    union {  // a barrier lies between their uses
        float sums[kLayerSums * 64];
        uint8_t stage[16384];  // digits of 4 rows x 4 slices
    };
    float w[kLayerMaxPairs];                // the pairs' weights
    int16_t idx[kLayerMaxPairs];            // their experts, -1: none
    uint16_t list[kLayerMaxPairs];          // pairs by expert
    uint8_t list_token[kLayerMaxPairs];     // and their tokens
    int token_exp[q8v::kMoeLayerMaxTokens];
    alignas(16) int fill[q8v::kMaxExperts];
    uint16_t job_expert[kMaxJobs], job_first[kMaxJobs], job_rows[kMaxJobs];  // first: in list
    uint32_t max_bits[kJobRows];
    int row_exp[kJobRows];                  // of the job in work: its rows' exponents
    uint32_t row_pair[kJobRows];            // and pairs
    int n_jobs, word;
};
constexpr size_t kLayerLdsBytes = kRingBytes + sizeof(LayerLds);
static_assert(kLayerLdsBytes <= 160 * 1024, "one block per CU");

constexpr uint64_t kPatience = 3000;  // of the 100 MHz clock

// Wave 0 waits until the counts at p, p + stride, ... (n of them, n <= 64) sum up to
// target, for about 30 us at most; then load_shared sees what was stored before they did.
// False (in every thread): not yet.
__device__ __forceinline__ bool wait_counts(const uint32_t* p, int n, int stride, uint32_t target, int* word) {
    if (threadIdx.x < 64) {
        const uint64_t began = wall_clock64();
        bool there = false;
        while (true) {
            uint32_t v = (int)threadIdx.x < n
                             ? __hip_atomic_load(p + threadIdx.x * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                             : 0u;
            for (int o = 32; o >= 1; o >>= 1) v += (uint32_t)__shfl_xor((int)v, o, 64);
            there = v >= target;
            if (there || wall_clock64() - began > kPatience) break;
            __builtin_amdgcn_s_sleep(1);
        }
        if (threadIdx.x == 0) *word = there;
    }
    __syncthreads();
    const bool there = __builtin_amdgcn_readfirstlane(*word) != 0;
    __syncthreads();
    return there;
}

// Wave 0 claims the first chunk nobody has; -1 (in every thread): all are claimed.
__device__ __forceinline__ int take_over(LayerWord* claim, int chunks, int* word) {
    if (threadIdx.x < 64) {
        int got = -1;
        for (int c0 = 0; c0 < chunks && got < 0; c0 += 64) {
            const int c = c0 + (int)threadIdx.x;
            const bool open =
                c < chunks && __hip_atomic_load(&claim[c].v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0;
            uint64_t who = __ballot(open);
            while (who && got < 0) {
                const int l = (int)__builtin_ctzll(who);
                who &= who - 1;
                uint32_t old = 1;
                if ((int)threadIdx.x == l)
                    old = __hip_atomic_exchange(&claim[c].v, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (__builtin_amdgcn_readlane((int)old, l) == 0) got = c0 + l;
            }
        }
        if (threadIdx.x == 0) *word = got;
    }
    __syncthreads();
    const int got = __builtin_amdgcn_readfirstlane(*word);
    __syncthreads();
    return got;
}

// The whole block: every wave's stores are done, then one thread counts.
__device__ __forceinline__ void raise_count(uint32_t* p, uint32_t n) {
    wait_vmcnt_mem<0>();
    __syncthreads();
    if (threadIdx.x == 0 && n) __hip_atomic_fetch_add(p, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Tiles [tile0, tile0 + nt) of an expert's gate_up matrix for the pairs list[0 .. n), n <= 4 NG.
template <int SP, int NG>
__device__ __forceinline__ void layer_gate_up(const LayerArgs& A, LayerLds& L, const TileWave& W,
                                              const uint32_t (&off)[5], const uint8_t* w, int tile0, int nt,
                                              const uint16_t* list, const uint8_t* tokens, int n) {
    const uint32_t rb = (uint32_t)(A.h >> 5) * 34u;
    if ((int)threadIdx.x < n) {
        const int pair = list[threadIdx.x];
        L.row_pair[threadIdx.x] = pair;
        L.row_exp[threadIdx.x] = L.token_exp[tokens[threadIdx.x]];
        L.max_bits[threadIdx.x] = 0;
    }
    i64x2 a[NG][SP][4];
    load_digits<SP, NG>(W, [&](int s) __attribute__((always_inline)) {
        return A.dig + (size_t)tokens[min(s, n - 1)] * A.h * 4;
    }, a);
    int c0 = 0;
    auto tile_at = [&](int i) __attribute__((always_inline)) { return w + (size_t)((tile0 + c0 + i) * 8) * rb; };
    constexpr int kChunk = kLayerSums / NG;
    TileRun run(W, off, min(kChunk, nt), tile_at);
    while (true) {
        const int ct = run.n_tiles;
        multiply_tiles<SP, NG>(run, a, L.part, L.sums);
        __syncthreads();
        // a wave takes a tile: 8 rows of up to 8 pairs
        const int r = threadIdx.x & 7, s = (threadIdx.x >> 3) & 7;
        if (s < n) {
            const int ex = L.row_exp[s];
            float* row = A.hidden + (size_t)L.row_pair[s] * A.f + (tile0 + c0) * 8 + r;
            uint32_t mx = 0;
            for (int tile = threadIdx.x >> 6; tile < ct; tile += kTileWaves) {
                const float* sum = L.sums + (tile * NG + (s >> 2)) * 64 + 16 * (s & 3) + r;
                const float v = silu_mul(row_scaled(sum[0], ex), row_scaled(sum[8], ex));
                store_shared(row + 8 * tile, v);
                mx = max(mx, __builtin_bit_cast(uint32_t, v) & 0x7fffffffu);
            }
            for (int o = 4; o >= 1; o >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o, 64));
            if (r == 0 && mx) atomicMax(&L.max_bits[s], mx);
        }
        __syncthreads();
        c0 += ct;
        if (c0 >= nt) break;
        run.restart(min(kChunk, nt - c0));
    }
    if ((int)threadIdx.x < n)
        __hip_atomic_fetch_max(A.hid_max + L.row_pair[threadIdx.x], L.max_bits[threadIdx.x], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
}

// A wave's 16 bytes of the staged digits.
__device__ __forceinline__ i64x2 read_stage(uint32_t lds) {
    i64x2 v;
    asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(lds) : "memory");
    return v;
}

// Tiles [tile0, tile0 + nt) of an expert's down matrix for the pairs list[0 .. n), whose
// hidden rows are ready once *ready reaches target; false: they are not, nothing done.
template <int SP, int NG>
__device__ __forceinline__ bool layer_down(const LayerArgs& A, LayerLds& L, const TileWave& W,
                                           const uint32_t (&off)[5], const uint8_t* w, int tile0, int nt,
                                           const uint16_t* list, int n, const uint32_t* ready, uint32_t target) {
    const uint32_t rb = (uint32_t)(A.f >> 5) * 34u;
    int c0 = 0;
    auto tile_at = [&](int i) __attribute__((always_inline)) { return w + (size_t)((tile0 + c0 + i) * 16) * rb; };
    constexpr int kChunk = kLayerSums / NG;
    TileRun run(W, off, min(kChunk, nt), tile_at);  // the first weights come while the block waits
    if (!wait_counts(ready, 1, 0, target, &L.word)) {
        wait_vmcnt_mem<0>();  // the copies in flight
        return false;
    }
    // the hidden rows' digits: four rows and four slices (1024 elements) staged at a time,
    // 8 elements a thread, then every wave takes its slices of them
    i64x2 a[NG][SP][4];
    const int S = A.f >> 8;
    const uint32_t stage = (uint32_t)(uintptr_t)L.stage;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int slot = threadIdx.x >> 7;
        const int pair = list[min(4 * g + slot, n - 1)];
        const uint32_t bits = load_shared(A.hid_max + pair);
        const bool finite = bits < 0x7f800000u;
        const int e = row_exponent(bits);
        if ((threadIdx.x & 127) == 0) {
            L.row_pair[4 * g + slot] = pair;
            L.row_exp[4 * g + slot] = finite ? e - 29 : kNotFinite;
        }
        for (int s0 = 0; s0 < S; s0 += 4) {
            const int i = 8 * (threadIdx.x & 127);  // element within the four slices
            if (s0 * 256 + i < A.f) {
                float v[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 t = load_shared(A.hidden + (size_t)pair * A.f + s0 * 256 + i + 2 * c);
                    v[2 * c] = t.x;
                    v[2 * c + 1] = t.y;
                }
                uint64_t d[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    int q = finite ? (int)__builtin_rintf(__builtin_ldexpf(v[c], 29 - e)) : 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int b = (int8_t)q;
                        d[x] |= (uint64_t)(uint32_t)(b & 255) << (8 * c);
                        q = (q - b) >> 8;
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    *reinterpret_cast<uint64_t*>(L.stage + (i >> 6) * 1024 + (4 * slot + x) * 64 +
                                                 16 * ((i >> 3) & 3) + 8 * ((i >> 5) & 1)) = d[x];
            }
            __syncthreads();
#pragma unroll
            for (int sl = 0; sl < SP; ++sl) {
                const int s = W.wt + (sl << W.log2_wt);
                if (s >= s0 && s < s0 + 4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        a[g][sl][q] = read_stage(stage + (4 * (s - s0) + q) * 1024 + W.row * 64 + W.grp * 16);
                }
            }
            __syncthreads();
        }
    }
    while (true) {
        const int ct = run.n_tiles;
        multiply_tiles<SP, NG>(run, a, L.part, L.sums);
        __syncthreads();
        // two waves take a tile: 16 rows of up to 8 pairs
        const int r = threadIdx.x & 15, s = (threadIdx.x >> 4) & 7;
        if (s < n) {
            const int ex = L.row_exp[s];
            float* row = A.out + (size_t)L.row_pair[s] * A.h + (tile0 + c0) * 16 + r;
            for (int tile = threadIdx.x >> 7; tile < ct; tile += kTileWaves / 2)
                store_shared(row + 16 * tile, row_scaled(L.sums[(tile * NG + (s >> 2)) * 64 + 16 * (s & 3) + r], ex));
        }
        __syncthreads();
        c0 += ct;
        if (c0 >= nt) return true;
        run.restart(min(kChunk, nt - c0));
    }
}

// Order-preserving integers and the wave's largest of them: six DPP steps, then lane 63.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 counts as 0
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, (k >> 31) ? k & 0x7fffffffu : ~k);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_largest(uint32_t v) {
    v = dpp_max<0x111>(v);  // row_shr 1, 2, 4, 8: lane 15 of each row has its row's largest
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142>(v);  // row_bcast 15, 31: lane 63 has the wave's
    v = dpp_max<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Softmax, top-k choice (k <= 64) and top-p cut of one token on one wave, n_exp <= 64 NP: what
// route_topk.hip's select_topk chooses, to the bit, with the choice made on integer keys
// (about a quarter of its time) and the chosen experts' probabilities
// formed together, lane j holding slot j.  put(expert, weight) is called on lanes j < k; a
// token whose probabilities are not finite gets NaN weights.
template <int NP, class Put>
__device__ __forceinline__ void choose_experts(const float (&l)[NP], int lane, int n_exp, int k, int normalize,
                                               float top_p, Put&& put) {
    uint32_t key[NP];
#pragma unroll
    for (int c = 0; c < NP; ++c) key[c] = lane + 64 * c < n_exp ? order_key(l[c]) : 0u;
    float mx = l[0];
#pragma unroll
    for (int c = 1; c < NP; ++c) mx = fmaxf(mx, l[c]);
    mx = wave_max(mx);
    float part = 0.0f;
#pragma unroll
    for (int c = 0; c < NP; ++c) part += lane + 64 * c < n_exp ? expf(l[c] - mx) : 0.0f;
    const float inv_sum = 1.0f / wave_sum(part);

    uint32_t my_key = 0;
    int my_expert = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t v = key[0];
#pragma unroll
        for (int c = 1; c < NP; ++c) v = max(v, key[c]);
        const uint32_t best = wave_largest(v);
        // its lowest holder: the lowest plane of 64 experts, then the lowest lane
        uint64_t who = 0;
        int plane = 0;
#pragma unroll
        for (int c = NP - 1; c >= 0; --c) {
            const uint64_t w = __ballot(key[c] == best);
            plane = w ? c : plane;
            who = w ? w : who;
        }
        const int at = (int)__builtin_ctzll(who);
#pragma unroll
        for (int c = 0; c < NP; ++c) key[c] = lane == at && c == plane ? 0u : key[c];
        if (lane == j) {
            my_key = best;
            my_expert = 64 * plane + at;
        }
    }
    const float ex = lane < k ? expf(key_value(my_key) - mx) : 0.0f;
    const float p = ex * inv_sum;
    // running sums in selection order, each step one fma of the unscaled exponential, as the
    // routers form them: adding the rounded p instead gives other last bits in a quarter of
    // the normalized weights, and another cut next to the top-p share
    float psum = 0.0f, before = 0.0f, through = 0.0f;
    for (int j = 0; j < k; ++j) {
        if (lane == j) before = psum;
        psum = __builtin_fmaf(lane_f(ex, j), inv_sum, psum);
        if (lane == j) through = psum;
    }
    const bool all = !(top_p < 1.0f);
    const bool kept = lane < k && (all || lane == 0 || before < top_p * psum);
    const float ksum = all ? psum : wave_max(kept ? through : 0.0f);
    if (lane < k) put(kept ? my_expert : -1, kept ? (normalize ? p / ksum : p) : 0.0f);
}

// How a list of jobs x `per` tiles is cut into the blocks' chunks, ranges of neighbouring
// tiles: where a job has at least one block to itself, q = blocks / jobs equal parts of every
// job (a chunk then starts one job only), unless equal parts of the whole list leave the
// busiest block less to do although it starts two; a start (the first copies, the digits)
// counts as `start` tiles.  It takes about as long as kStartSlices slices of a tile (16 x 256
// weights), whatever the width.  Measured, in us, against a count fixed in tiles (6 gate_up and
// 16 down tiles, right for 2048 and 768 inputs alone), m tokens, k of E experts of f x h: h = f
// = 6144, 16, 2 of 32 438.0 | 435.7; 4096 x 4096, 16, 2 of 64 248.2 | 246.7; f = 1536, h = 4096, 40, 2 of 64
// 185.5 | 183.8; f = 6144, h = 256, 30, 2 of 64 62.0 | 62.2; 256 x 256, 60, 8 of 160 50.1 | 50.0.
constexpr int kStartSlices = 48;
struct Cut {
    int q, per, all, blocks;
    __device__ __forceinline__ Cut(int jobs, int per_, int blocks_, int start)
        : per(per_), all(jobs * per_), blocks(blocks_) {
        q = jobs > 0 ? min((int)((uint32_t)blocks / (uint32_t)jobs), per) : 0;
        if (q > 0 && (int)((uint32_t)(per + q - 1) / (uint32_t)q) > (int)((uint32_t)(all + blocks - 1) / (uint32_t)blocks) + start) q = 0;
    }
    __device__ __forceinline__ int begin(int chunk) const {
        // all <= 512 jobs x 768 tiles and chunk <= 512: 32 bits hold the products
        if (q == 0) return (int)((uint32_t)(all * chunk) / (uint32_t)blocks);
        const int job = (int)((uint32_t)chunk / (uint32_t)q), part = chunk - job * q;
        return min(job * per + (int)((uint32_t)(per * part) / (uint32_t)q), all);
    }
    __device__ __forceinline__ int end(int chunk) const { return begin(chunk + 1); }
};

template <int SP_H, int SP_F>
__global__ __launch_bounds__(kTileThreads) void moe_layer_kernel(LayerArgs A) {
    extern __shared__ float4 smem4[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(smem4);
    LayerLds& L = *reinterpret_cast<LayerLds*>(smem + kRingBytes);
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int pairs = A.m * A.k;
    const int blocks = gridDim.x, me = blockIdx.x;

    // selection and the jobs
    uint32_t taken_up = 0, taken_down = 0;
    if (tid == 0) {
        taken_up = __hip_atomic_exchange(&A.cnt->claim_up[me].v, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        taken_down = __hip_atomic_exchange(&A.cnt->claim_down[me].v, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int e = tid; e < q8v::kMaxExperts; e += kTileThreads) L.fill[e] = 0;
    for (int t = tid; t < A.m; t += kTileThreads) L.token_exp[t] = A.exps[t];
    __syncthreads();
    auto choose_all = [&](auto np) __attribute__((always_inline)) {
        constexpr int NP = decltype(np)::value;
        float l[NP], next[NP];
        auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
            for (int c = 0; c < NP; ++c) {
                const int e = lane + 64 * c;
                next[c] = e < A.n_exp ? A.logits[(size_t)min(t, A.m - 1) * A.n_exp + e] : -INFINITY;
            }
        };
        load(wv);
        for (int t = wv; t < A.m; t += kTileWaves) {
#pragma unroll
            for (int c = 0; c < NP; ++c) l[c] = next[c];
            load(t + kTileWaves);
            choose_experts<NP>(l, lane, A.n_exp, A.k, A.normalize, A.top_p, [&](int e, float p) __attribute__((always_inline)) {
                const int keep = p == p ? e : -1;  // weights NaN: no expert
                L.idx[t * A.k + lane] = (int16_t)keep;
                L.w[t * A.k + lane] = p;
                if (keep >= 0) atomicAdd(&L.fill[keep], 1);
            });
        }
    };
    if (A.n_exp <= 128)
        choose_all(std::integral_constant<int, 2>{});
    else
        choose_all(std::integral_constant<int, 4>{});
    if (tid == 0) L.word = (int)(taken_up | taken_down << 1);
    __syncthreads();
    if (wv == 0) {  // lane l: experts 4l .. 4l + 3
        const int4 counts = *reinterpret_cast<const int4*>(&L.fill[4 * lane]);
        const int c[4] = {counts.x, counts.y, counts.z, counts.w};
        int sum = 0, jobs = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sum += c[q];
            jobs += (c[q] + kJobRows - 1) / kJobRows;
        }
        const int incl = wave_scan(sum), jincl = wave_scan(jobs);
        int at = incl - sum, jat = jincl - jobs;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            L.fill[4 * lane + q] = at;
            for (int r = 0; r < c[q]; r += kJobRows, ++jat) {
                L.job_expert[jat] = (uint16_t)(4 * lane + q);
                L.job_first[jat] = (uint16_t)(at + r);
                L.job_rows[jat] = (uint16_t)min(kJobRows, c[q] - r);
            }
            at += c[q];
        }
        if (lane == 63) L.n_jobs = jincl;
        wait_lgkmcnt_mem<0>();
        // the pairs in ascending order within their expert (every block lists them alike): a
        // pair's place is its expert's running position plus the number of earlier lanes of
        // the step with the same expert, found with a ballot a bit of the id
        for (int i0 = 0; i0 < pairs; i0 += 64) {
            const int e = i0 + lane < pairs ? L.idx[i0 + lane] : -1;
            uint64_t same = __ballot(e >= 0);
#pragma unroll
            for (int bit = 0; bit < 8; ++bit) {
                const uint64_t set = __ballot(e >= 0 && ((e >> bit) & 1));
                same &= ((e >> bit) & 1) ? set : ~set;
            }
            if (e >= 0) {
                const int pos = L.fill[e] + __popcll(same & ((1ull << lane) - 1));
                L.list[pos] = (uint16_t)(i0 + lane);
                L.list_token[pos] = (uint8_t)((uint32_t)(i0 + lane) / (uint32_t)A.k);
                wait_lgkmcnt_mem<0>();                        // every lane has read its position
                if ((same >> lane) == 1ull) L.fill[e] = pos + 1;  // the highest lane of its expert
            }
            wait_lgkmcnt_mem<0>();
        }
    }
    const int taken = __builtin_amdgcn_readfirstlane(L.word);
    __syncthreads();
    const int jobs = __builtin_amdgcn_readfirstlane(L.n_jobs);
    const int up_tiles = A.f / 8, down_tiles = A.h / 16;
    const Cut cut_up(jobs, up_tiles, blocks, kStartSlices / (A.h >> 8)),
        cut_down(jobs, down_tiles, blocks, kStartSlices / (A.f >> 8));
    const uint32_t rb_h = (uint32_t)(A.h >> 5) * 34u, rb_f = (uint32_t)(A.f >> 5) * 34u;
    // the tiles [t, end) as far as they belong to one job
    struct Piece {
        int job, expert, rows, tile0, tiles;
        const uint16_t* list;
        const uint8_t* tokens;
    };
    auto piece_at = [&](int t, int end, int per) __attribute__((always_inline)) {
        Piece r;
        r.job = (int)((uint32_t)t / (uint32_t)per);
        r.tile0 = t - r.job * per;
        r.tiles = min(per - r.tile0, end - t);
        r.expert = __builtin_amdgcn_readfirstlane((int)L.job_expert[r.job]);
        r.rows = __builtin_amdgcn_readfirstlane((int)L.job_rows[r.job]);
        const int first = __builtin_amdgcn_readfirstlane((int)L.job_first[r.job]);
        r.list = L.list + first;
        r.tokens = L.list_token + first;
        return r;
    };
    const TileWave Wh(smem, A.h >> 8, A.log2_wt_h), Wf(smem, A.f >> 8, A.log2_wt_f);

    int up = taken & 1 ? -1 : me;    // the gate_up chunk to work on
    int down = taken & 2 ? -1 : me;  // the down chunk, its next tile
    int down_at = cut_down.begin(me);
    while (true) {
        if (up >= 0) {
            uint32_t off[5];
            Wh.offsets([&](int r) __attribute__((always_inline)) -> uint32_t {
                return (uint32_t)(r < 8 ? r : A.f + r - 8) * rb_h;
            }, off);
            const int end = cut_up.end(up);
            for (int t = cut_up.begin(up); t < end;) {
                const Piece pc = piece_at(t, end, up_tiles);
                const uint8_t* w = A.wgu + (size_t)pc.expert * (2 * A.f) * rb_h;
                if (pc.rows > 4)
                    layer_gate_up<SP_H, 2>(A, L, Wh, off, w, pc.tile0, pc.tiles, pc.list, pc.tokens, pc.rows);
                else
                    layer_gate_up<SP_H, 1>(A, L, Wh, off, w, pc.tile0, pc.tiles, pc.list, pc.tokens, pc.rows);
                raise_count(&A.cnt->up_done[pc.job].v, (uint32_t)pc.tiles);
                t += pc.tiles;
            }
            up = -1;
        }
        if (down >= 0) {
            uint32_t off[5];
            Wf.offsets([&](int r) __attribute__((always_inline)) -> uint32_t { return (uint32_t)r * rb_f; }, off);
            const int end = cut_down.end(down);
            uint32_t done = 0;
            bool ready = true;
            while (down_at < end) {
                const Piece pc = piece_at(down_at, end, down_tiles);
                const uint8_t* w = A.wdn + (size_t)pc.expert * A.h * rb_f;
                const uint32_t* count = &A.cnt->up_done[pc.job].v;
                if (pc.rows > 4)
                    ready = layer_down<SP_F, 2>(A, L, Wf, off, w, pc.tile0, pc.tiles, pc.list, pc.rows, count, up_tiles);
                else
                    ready = layer_down<SP_F, 1>(A, L, Wf, off, w, pc.tile0, pc.tiles, pc.list, pc.rows, count, up_tiles);
                if (!ready) break;
                done += pc.tiles;
                down_at += pc.tiles;
            }
            raise_count(&A.cnt->down_done[me % kDoneParts].v, done);
            if (!ready) {
                up = take_over(A.cnt->claim_up, blocks, &L.word);
                continue;
            }
            down = -1;
        }
        if (wait_counts(&A.cnt->down_done[0].v, kDoneParts, sizeof(LayerWord) / 4, (uint32_t)cut_down.all, &L.word)) break;
        up = take_over(A.cnt->claim_up, blocks, &L.word);
        if (up < 0) {
            down = take_over(A.cnt->claim_down, blocks, &L.word);
            if (down >= 0) down_at = cut_down.begin(down);
        }
    }

    // the tokens' sums, in slot order, two columns a thread, eight slots' loads together
    const int half_h = A.h / 2;
    const int64_t all = (int64_t)A.m * half_h;
    const int64_t i1 = all * (me + 1) / blocks;
    for (int64_t i = all * me / blocks + tid; i < i1; i += kTileThreads) {
        const int t = (int)(i / half_h), col = 2 * (int)(i - (int64_t)t * half_h);
        const float* o = A.out + (size_t)t * A.k * A.h + col;
        float2 s = make_float2(0.f, 0.f);
        for (int j0 = 0; j0 < A.k; j0 += 8) {
            float2 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = load_shared(o + (size_t)min(j0 + j, A.k - 1) * A.h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= A.k) continue;
                const float p = L.w[t * A.k + j0 + j];
                if (p != p) s = make_float2(p, p);
                if (L.idx[t * A.k + j0 + j] < 0) continue;  // a dropped slot's row was never written
                s.x = __builtin_fmaf(p, v[j].x, s.x);
                s.y = __builtin_fmaf(p, v[j].y, s.y);
            }
        }
        float* yo = A.y + (size_t)t * A.ldy + col;
        yo[0] = s.x;
        yo[1] = s.y;
    }
}

template <int SP_H, int SP_F>
static hipError_t launch_layer_kernel(const DeviceInfo& dev, const LayerArgs& A, hipStream_t stream) {
    auto kernel = moe_layer_kernel<SP_H, SP_F>;
    static thread_local int attr_dev = -1;
    if (attr_dev != dev.device) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLayerLdsBytes);
        if (e != hipSuccess) return e;
        attr_dev = dev.device;
    }
    const int blocks = dev.cu_count < kMaxChunks ? dev.cu_count : kMaxChunks;  // one per CU
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kTileThreads), kLayerLdsBytes, stream, A);
    return hipGetLastError();
}

template <int SP_H>
static hipError_t launch_layer_f(const DeviceInfo& dev, int sp_f, const LayerArgs& A, hipStream_t stream) {
    if (sp_f <= 1) return launch_layer_kernel<SP_H, 1>(dev, A, stream);
    if (sp_f <= 2) return launch_layer_kernel<SP_H, 2>(dev, A, stream);
    return launch_layer_kernel<SP_H, 3>(dev, A, stream);
}

hipError_t launch_moe_layer(const DeviceInfo& dev, const float* w_router, const uint8_t* wgu, const uint8_t* wdn,
                            int64_t n_exp, int64_t f, int64_t h, const float* x, int64_t m, int64_t ldx, int k,
                            bool normalize, float top_p, float* y, int64_t ldy, void* workspace, hipStream_t stream) {
    const q8v::MoeLayerWorkspace L = q8v::moe_layer_workspace_layout(m, k, n_exp, f, h);
    char* ws = static_cast<char*>(workspace);
    if (q8v::moe_layer_uses_tiles(m, k, n_exp, f, h)) {
        LayerArgs A{};
        A.logits = reinterpret_cast<float*>(ws + L.logits_off);
        A.dig = reinterpret_cast<int8_t*>(ws + L.dig_off);
        A.exps = reinterpret_cast<int*>(ws + L.exps_off);
        A.hidden = reinterpret_cast<float*>(ws + L.hidden_off);
        A.hid_max = reinterpret_cast<uint32_t*>(ws + L.max_off);
        A.out = reinterpret_cast<float*>(ws + L.out_off);
        A.cnt = reinterpret_cast<LayerCounters*>(ws + L.count_off);
        A.wgu = wgu;
        A.wdn = wdn;
        A.y = y;
        A.ldy = (int)ldy;
        A.m = (int)m;
        A.k = k;
        A.n_exp = (int)n_exp;
        A.f = (int)f;
        A.h = (int)h;
        A.normalize = normalize ? 1 : 0;
        A.top_p = top_p;
        const SliceShare sh = slice_share((int)(h >> 8)), sf = slice_share((int)(f >> 8));
        A.log2_wt_h = sh.log2_wt;
        A.log2_wt_f = sf.log2_wt;
        const int64_t blocks = m + (n_exp + 3) / 4 * ((m + kPrepareTokens - 1) / kPrepareTokens);
        // the counters in use: of the jobs (one for an expert's first eight tokens, and for every
        // eight more), the last ones
        const int jobs = (int)(m * k < n_exp ? m * k : n_exp) + (int)(m * k / kJobRows);
        const int counters = (int)(offsetof(LayerCounters, up_done) / sizeof(LayerWord)) + (jobs < kMaxJobs ? jobs : kMaxJobs);
        hipLaunchKernelGGL(moe_layer_prepare_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, x, (int)m, (int)h,
                           (int)ldx, w_router, (int)n_exp, k, const_cast<float*>(A.logits),
                           const_cast<int8_t*>(A.dig), const_cast<int*>(A.exps), A.hid_max,
                           reinterpret_cast<LayerWord*>(A.cnt), counters);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (sh.sp <= 1) return launch_layer_f<1>(dev, sf.sp, A, stream);
        if (sh.sp <= 2) return launch_layer_f<2>(dev, sf.sp, A, stream);
        return launch_layer_f<3>(dev, sf.sp, A, stream);
    }
    int32_t* idx = reinterpret_cast<int32_t*>(ws + L.idx_off);
    float* wts = reinterpret_cast<float*>(ws + L.w_off);
    hipError_t e = launch_route_topk(dev, x, m, h, ldx, w_router, n_exp, k, normalize, top_p, idx, wts,
                                     reinterpret_cast<float*>(ws + L.logits_off), stream);
    if (e != hipSuccess) return e;
    e = launch_moe_grouped(dev, wgu, wdn, n_exp, f, h, x, m, ldx, idx, wts, k, y, ldy, ws + L.moe_off, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_poison_kernel, dim3((unsigned)m), dim3(256), 0, stream, wts, k, (int)h, y, (int)ldy);
    return hipGetLastError();
}

}  // namespace q8k
