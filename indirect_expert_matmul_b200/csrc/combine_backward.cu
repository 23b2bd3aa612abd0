// Gradient of the weighted combine y[t] = sum_s w[t][s] * dst[t][s] (+ shared[t]):
//   dw[t][s]      = sum_j dy[t][j] * dst[t][s][j]
//   ddst[t][s][j] = w[t][s] * dy[t][j]          (the shared term's gradient is dy)
// One CTA per (token, slot) pair, handed out grid-stride.
#include "common.cuh"

namespace moe {

namespace {

constexpr int kCbThreads = 256;

__global__ void __launch_bounds__(kCbThreads)
combine_backward_kernel(const float* __restrict__ dy, const float* __restrict__ dst, const float* __restrict__ w,
                        int64_t n_slots, int k, int64_t n, float* __restrict__ dw, float* __restrict__ ddst) {
    __shared__ float s_part[kCbThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t s = blockIdx.x; s < n_slots; s += gridDim.x) {
        const float* g = dy + s / k * n;
        const float* d = dst + s * n;
        const float ws = __ldg(w + s);
        float acc = 0.f;
        for (int64_t j = threadIdx.x; j < n; j += kCbThreads) {
            const float v = __ldg(g + j);
            acc = __fmaf_rn(v, __ldcs(d + j), acc);
            if (ddst) __stcs(ddst + s * n + j, __fmul_rn(ws, v));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
        if (lane == 0) s_part[warp] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
            float r = 0.f;
            for (int i = 0; i < kCbThreads / 32; ++i) r = __fadd_rn(r, s_part[i]);
            dw[s] = r;
        }
        __syncthreads();
    }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_combine_backward(const float* dy, const float* dst, const float* weights, int64_t n_tokens,
                                           int k, int64_t n, float* dweights, float* ddst, moe_stream stream) {
    if (n_tokens < 0 || k < 1 || n < 1) return MOE_ERR_INVALID;
    if (n_tokens >= kMaxTokens || k >= kMaxK || n >= ((int64_t)1 << 31)) return MOE_ERR_RANGE;
    if (n_tokens == 0) return MOE_OK;
    if (!dy || !dst || !weights || !dweights) return MOE_ERR_INVALID;
    if (((uintptr_t)dy | (uintptr_t)dst | (uintptr_t)weights | (uintptr_t)dweights | (uintptr_t)ddst) & 3u)
        return MOE_ERR_INVALID;
    const int64_t slots = n_tokens * k;
    const unsigned grid = (unsigned)(slots < 148 * 8 ? slots : 148 * 8);
    combine_backward_kernel<<<grid, kCbThreads, 0, (cudaStream_t)stream>>>(dy, dst, weights, slots, k, n, dweights,
                                                                           ddst);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
