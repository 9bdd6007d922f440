// The whole mixture-of-experts layer (gfx950): softmax top-k routing and the router-weighted
// SwiGLU mixture of the chosen experts in one call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q8_internal.h"
#include "q8_validate.h"

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

hipError_t launch_moe_layer(const DeviceInfo& dev, const float* w_router, const uint8_t* wgu, const uint8_t* wdn,
                            int64_t n_exp, int64_t f, int64_t h, const float* x, int64_t m, int64_t ldx, int k,
                            bool normalize, float top_p, float* y, int64_t ldy, void* workspace, hipStream_t stream) {
    const q8v::MoeLayerWorkspace L = q8v::moe_layer_workspace_layout(m, k, n_exp, f, h);
    char* ws = static_cast<char*>(workspace);
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
