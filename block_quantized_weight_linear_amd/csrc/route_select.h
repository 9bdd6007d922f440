// Softmax, top-k selection and the top-p cut of one token on one wave (gfx950), shared by the
// routers and the whole mixture-of-experts layer so that both choose the same experts with
// the same weights.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

namespace q8k {

__device__ __forceinline__ bool better(float v, int i, float bv, int bi) {
    return v > bv || (v == bv && i < bi);
}

// Cross-lane steps on the DPP network (no LDS round trip): within each row of 16 lanes,
// xor 1 and xor 2 (quad permutes), then the half-row and row mirrors; the four rows are
// then combined from lanes 0, 16, 32, 48 with readlane, in row order.
constexpr int kDppXor1 = 0xB1;        // quad_perm(1, 0, 3, 2)
constexpr int kDppXor2 = 0x4E;        // quad_perm(2, 3, 0, 1)
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ float lane_f(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// Every lane gets the wave's best (value, index) under better().
__device__ __forceinline__ void wave_best(float& v, int& i) {
    auto step = [&](auto c) __attribute__((always_inline)) {
        constexpr int C = decltype(c)::value;
        const float ov = dpp_f<C>(v);
        const int oi = dpp_i<C>(i);
        if (better(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    };
    step(std::integral_constant<int, kDppXor1>{});
    step(std::integral_constant<int, kDppXor2>{});
    step(std::integral_constant<int, kDppHalfMirror>{});
    step(std::integral_constant<int, kDppMirror>{});
    float bv = lane_f(v, 0);
    int bi = __builtin_amdgcn_readlane(i, 0);
#pragma unroll
    for (int r = 1; r < 4; ++r) {
        const float rv = lane_f(v, 16 * r);
        const int ri = __builtin_amdgcn_readlane(i, 16 * r);
        if (better(rv, ri, bv, bi)) {
            bv = rv;
            bi = ri;
        }
    }
    v = bv;
    i = bi;
}

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_f<kDppXor1>(v));
    v = fmaxf(v, dpp_f<kDppXor2>(v));
    v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
    v = fmaxf(v, dpp_f<kDppMirror>(v));
    return fmaxf(fmaxf(lane_f(v, 0), lane_f(v, 16)), fmaxf(lane_f(v, 32), lane_f(v, 48)));
}

// Fixed order: the DPP tree within each row, then ((row0 + row1) + row2) + row3.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f<kDppXor1>(v);
    v += dpp_f<kDppXor2>(v);
    v += dpp_f<kDppHalfMirror>(v);
    v += dpp_f<kDppMirror>(v);
    return ((lane_f(v, 0) + lane_f(v, 16)) + lane_f(v, 32)) + lane_f(v, 48);
}

// The wave's best untaken expert by comparing (logit, index) pairs across the lanes.
struct PickPairs {
    int taken = 0;  // bit c: expert lane + 64c already selected
    __device__ __forceinline__ PickPairs(const float (&)[4], int lane, int n_exp) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (lane + 64 * c >= n_exp) taken |= 1 << c;
    }
    __device__ __forceinline__ int next(const float (&l)[4], int lane) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int e = lane + 64 * c;
            if (!(taken & (1 << c)) && better(l[c], e, bv, bi)) {
                bv = l[c];
                bi = e;
            }
        }
        wave_best(bv, bi);
        if (lane == (bi & 63)) taken |= 1 << (bi >> 6);
        return bi;
    }
};

// The same choice from order-preserving integer keys: the largest key by six DPP steps, then
// its lowest holder from the lanes' ballots (finite logits; -0 counts as 0).
struct PickKeys {
    uint32_t key[4];
    __device__ __forceinline__ PickKeys(const float (&l)[4], int lane, int n_exp) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t b = __builtin_bit_cast(uint32_t, l[c] + 0.0f);
            key[c] = lane + 64 * c < n_exp ? ((b >> 31) ? ~b : b | 0x80000000u) : 0u;
        }
    }
    template <int CTRL>
    static __device__ __forceinline__ uint32_t step(uint32_t v) {
        return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
    }
    __device__ __forceinline__ int next(const float (&)[4], int lane) {
        uint32_t v = max(max(key[0], key[1]), max(key[2], key[3]));
        v = step<0x111>(v);  // row_shr 1, 2, 4, 8: lane 15 of each row has its row's largest
        v = step<0x112>(v);
        v = step<0x114>(v);
        v = step<0x118>(v);
        v = step<0x142>(v);  // row_bcast 15, 31: lane 63 has the wave's
        v = step<0x143>(v);
        const uint32_t best = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
        int bi = 0;
#pragma unroll
        for (int c = 3; c >= 0; --c) {
            const uint64_t who = __ballot(key[c] == best);
            if (who) bi = 64 * c + (int)__builtin_ctzll(who);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (lane + 64 * c == bi) key[c] = 0;
        return bi;
    }
};

// Softmax, top-k selection and the top-p cut for one token on one wave; logit_of(e)
// returns expert e's float32 logit (e < n_exp).  Lane l owns experts l, l+64, l+128, l+192.
// put(j, expert, weight) is called for every slot j (a dropped one: expert -1, weight 0), on
// the lane that holds it.
template <class Pick, class LogitOf, class Put>
__device__ __forceinline__ void select_topk(LogitOf&& logit_of, int lane, int n_exp, int k, int normalize,
                                            float top_p, Put&& put) {
    float l[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int e = lane + 64 * c;
        l[c] = e < n_exp ? logit_of(e) : -INFINITY;
    }
    Pick pick(l, lane, n_exp);
    const float mx = wave_max(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
    float ex[4];
    float part = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        ex[c] = (lane + 64 * c < n_exp) ? expf(l[c] - mx) : 0.0f;
        part += ex[c];
    }
    const float inv_sum = 1.0f / wave_sum(part);

    // k rounds; each picks the wave's best untaken expert (every lane learns it) and the
    // owner lane's probability by readlane.  Lane (j % 64) keeps round j's result in its
    // register slot j / 64; the chosen probabilities are summed in selection order,
    // identically on all lanes.
    int keep_i[4] = {0, 0, 0, 0};
    float keep_p[4] = {0.f, 0.f, 0.f, 0.f};
    float keep_cb[4] = {0.f, 0.f, 0.f, 0.f};  // running sum before the slot
    float keep_ca[4] = {0.f, 0.f, 0.f, 0.f};  // running sum through the slot
    float psum = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int bi = pick.next(l, lane);
        const int wl = bi & 63, wc = bi >> 6;
        const float mine = wc == 0 ? ex[0] : wc == 1 ? ex[1] : wc == 2 ? ex[2] : ex[3];
        const float bp = lane_f(mine, wl);
        const float p = bp * inv_sum;
        const float before = psum;
        psum += p;
        if ((j & 63) == lane) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if ((j >> 6) == c) {
                    keep_i[c] = bi;
                    keep_p[c] = p;
                    keep_cb[c] = before;
                    keep_ca[c] = psum;
                }
            }
        }
    }
    // top-p cut: every lane holds the same running sums for its slots, so the kept sum is
    // the largest running sum through a kept slot (the sums only grow)
    const bool all = !(top_p < 1.0f);
    const float thr = top_p * psum;
    bool kept[4];
    float ksum = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = lane + 64 * c;
        kept[c] = j < k && (all || j == 0 || keep_cb[c] < thr);
        if (kept[c]) ksum = fmaxf(ksum, keep_ca[c]);
    }
    ksum = wave_max(ksum);
    if (all) ksum = psum;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = lane + 64 * c;
        if (j < k) put(j, kept[c] ? keep_i[c] : -1, kept[c] ? (normalize ? keep_p[c] / ksum : keep_p[c]) : 0.0f);
    }
}

}  // namespace q8k
