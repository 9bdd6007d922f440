// Codes (e4m3) and scales of float rows in blocks of 128 inputs, and of matrices in blocks of
// 128 x 128.
//
// A block with largest magnitude a gets scale a/448 (448: e4m3's largest value) and codes
// e4m3(x * (448/a)), or the least power of two at least a/448 and codes e4m3(x / scale); every
// quotient and product is one float32 rounding, the code one more (v_cvt_pk_fp8_f32 rounds to
// nearest even), so the result is bit-exact.  Both kernels read an element once, hold it in
// registers across the block's maximum, and are bound by memory (12288 x 4096 in float32: 252 MB in 44 us, 5.7 TB/s;
// 16 rows of 4096: 2.1 us, a launch).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8_tile.h"
#include "q8_internal.h"
#include "wave_dpp.h"

namespace q8k {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight neighbouring elements as float32.
template <class T>
__device__ __forceinline__ f32x8 load8(const T* p) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    if constexpr (sizeof(T) == 4) {
        const f8_f32x4 a = reinterpret_cast<const f8_f32x4*>(p)[0], b = reinterpret_cast<const f8_f32x4*>(p)[1];
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        return __builtin_convertvector(*reinterpret_cast<const T8*>(p), f32x8);
    }
}

// Magnitudes as integers: ordered like the numbers, infinities and NaN above all of them.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t top8(f32x8 v) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, magnitude(v[i]));
    return t;
}

constexpr uint32_t kInfinity = 0x7F800000u, kTiny = (127u - 116u) << 23;  // 2^-116

// A block's scale and the factor that its elements are multiplied with.
struct Scale {
    float scale, by;
};
__device__ __forceinline__ Scale block_scale(uint32_t top, bool pow2) {
    const float a = __uint_as_float(top);
    if (top >= kInfinity) return {__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u)};
    if (top < kTiny) return {0.f, 0.f};
    if (pow2) {
        // a = f 2^e with 1 <= f < 2 and 448 = 1.75 2^8: 2^(e-8), doubled where f > 1.75
        const uint32_t e = (top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        return {__uint_as_float(e << 23), __uint_as_float((254u - e) << 23)};
    }
    return {a / 448.f, 448.f / a};
}

// Codes of eight elements; a NaN factor gives NaN codes.
__device__ __forceinline__ uint2 codes8(f32x8 v, float by) {
    if (__builtin_isnan(by)) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(v[i] * by, -448.f), 448.f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The largest of a row of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, (uint32_t)dpp_i<kDppXor1>((int)v));
    v = max(v, (uint32_t)dpp_i<kDppXor2>((int)v));
    v = max(v, (uint32_t)dpp_i<kDppHalfMirror>((int)v));
    return max(v, (uint32_t)dpp_i<kDppMirror>((int)v));
}

constexpr int kQThreads = 256;

// Activation rows: 16 lanes a block, eight elements a lane.
template <class T>
__global__ __launch_bounds__(kQThreads) void f8_quantize_act_kernel(const T* __restrict__ x, int64_t rows, int k,
                                                                   int64_t ldx, int kb, bool pow2,
                                                                   uint8_t* __restrict__ q, float* __restrict__ d) {
    const int sub = threadIdx.x & 15;
    const int64_t total = rows * kb;
    for (int64_t b = (int64_t)blockIdx.x * (kQThreads / 16) + (threadIdx.x >> 4); b < total;
         b += (int64_t)gridDim.x * (kQThreads / 16)) {
        const int64_t row = b / kb;
        const int col = (int)(b - row * kb) * 128 + 8 * sub;
        f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (col < k) v = load8(x + row * ldx + col);
        const Scale s = block_scale(row_max(top8(v)), pow2);
        if (col < k) *reinterpret_cast<uint2*>(q + row * k + col) = codes8(v, s.by);
        if (sub == 0) d[b] = s.scale;
    }
}

// A matrix: one workgroup a block, rows 16p + t/16 and columns 8(t%16) .. of it in thread t.
template <class T>
__global__ __launch_bounds__(kQThreads) void f8_quantize_weight_kernel(const T* __restrict__ w, int n, int k,
                                                                       int64_t ldw, int kb, int blocks, bool pow2,
                                                                       uint8_t* __restrict__ q,
                                                                       float* __restrict__ d) {
    __shared__ uint32_t tops[2][kQThreads / 64];
    const int sub = threadIdx.x & 15, lane = threadIdx.x & 63;
    int turn = 0;
    for (int b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const int rb = b / kb;
        const int row0 = rb * 128 + (threadIdx.x >> 4), col = (b - rb * kb) * 128 + 8 * sub;
        f32x8 v[8];
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            v[p] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (row0 + 16 * p < n && col < k) v[p] = load8(w + (int64_t)(row0 + 16 * p) * ldw + col);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) top = max(top, top8(v[p]));
        top = row_max(top);
        top = max(max((uint32_t)__builtin_amdgcn_readlane((int)top, 0), (uint32_t)__builtin_amdgcn_readlane((int)top, 16)),
                  max((uint32_t)__builtin_amdgcn_readlane((int)top, 32), (uint32_t)__builtin_amdgcn_readlane((int)top, 48)));
        if (lane == 0) tops[turn][threadIdx.x >> 6] = top;
        __syncthreads();  // the other turn's words may still be read by a wave that has not come here
        top = max(max(tops[turn][0], tops[turn][1]), max(tops[turn][2], tops[turn][3]));
        const Scale s = block_scale(top, pow2);
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (row0 + 16 * p < n && col < k)
                *reinterpret_cast<uint2*>(q + (int64_t)(row0 + 16 * p) * k + col) = codes8(v[p], s.by);
        if (threadIdx.x == 0) d[b] = s.scale;
    }
}

constexpr int64_t kQMaxBlocks = 1 << 20;  // more work than that goes round

template <class T>
hipError_t act(const void* x, int64_t m, int64_t k, int64_t ldx, bool pow2, uint8_t* q, float* d, hipStream_t stream) {
    const int64_t kb = (k + 127) / 128;
    const int64_t blocks = (m * kb + kQThreads / 16 - 1) / (kQThreads / 16);
    hipLaunchKernelGGL(f8_quantize_act_kernel<T>, dim3((unsigned)(blocks < kQMaxBlocks ? blocks : kQMaxBlocks)),
                       dim3(kQThreads), 0, stream, static_cast<const T*>(x), m, (int)k, ldx, (int)kb, pow2, q, d);
    return hipGetLastError();
}
template <class T>
hipError_t weight(const void* w, int64_t n, int64_t k, int64_t ldw, bool pow2, uint8_t* q, float* d,
                  hipStream_t stream) {
    const int64_t kb = (k + 127) / 128, blocks = kb * ((n + 127) / 128);
    hipLaunchKernelGGL(f8_quantize_weight_kernel<T>, dim3((unsigned)(blocks < kQMaxBlocks ? blocks : kQMaxBlocks)),
                       dim3(kQThreads), 0, stream, static_cast<const T*>(w), (int)n, (int)k, ldw, (int)kb,
                       (int)blocks, pow2, q, d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize_act(const void* x, int type, int64_t m, int64_t k, int64_t ldx, bool pow2, uint8_t* q,
                                  float* d, hipStream_t stream) {
    switch (type) {
        case Q8_F32: return act<float>(x, m, k, ldx, pow2, q, d, stream);
        case Q8_F16: return act<_Float16>(x, m, k, ldx, pow2, q, d, stream);
        default: return act<__bf16>(x, m, k, ldx, pow2, q, d, stream);
    }
}

hipError_t launch_f8_quantize_weight(const void* w, int type, int64_t n, int64_t k, int64_t ldw, bool pow2,
                                     uint8_t* q, float* d, hipStream_t stream) {
    switch (type) {
        case Q8_F32: return weight<float>(w, n, k, ldw, pow2, q, d, stream);
        case Q8_F16: return weight<_Float16>(w, n, k, ldw, pow2, q, d, stream);
        default: return weight<__bf16>(w, n, k, ldw, pow2, q, d, stream);
    }
}

}  // namespace q8k
