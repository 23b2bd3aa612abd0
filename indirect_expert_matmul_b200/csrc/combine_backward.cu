// Gradient of the weighted combine y[t] = sum_s w[t][s] * dst[t][s] (+ shared[t]):
//   dw[t][s]      = sum_j dy[t][j] * dst[t][s][j]
//   ddst[t][s][j] = w[t][s] * dy[t][j]          (the shared term's gradient is dy)
//
// One pass over dst, bound by HBM: a CTA takes up to KB slots of a token and
// walks the row once, reading dy once and each slot's vector once, writing the
// slot's gradient where it has just read it (so ddst may be dst), with KB
// independent loads in flight a thread.  Per slot a thread sums its n / 256
// products in ascending order, then the CTA adds the threads in a fixed tree:
// bit-identical reruns, whatever KB is.
//
// KB is the largest of 8, 4, 2, 1 that still gives about four CTAs an SM: with
// fewer slots a CTA the 512-token case (k = 6, n = 2048) has 1024 CTAs to share
// out instead of 512.
#include <atomic>

#include "common.cuh"

namespace moe {

namespace {

constexpr int kCbThreads = 256;

template <int KB, bool VEC>
__global__ void __launch_bounds__(kCbThreads)
combine_backward_kernel(const float* __restrict__ dy, const float* dst, const float* __restrict__ w, int k, int64_t n,
                        int groups, float* __restrict__ dw, float* ddst) {
    __shared__ float s_part[KB][kCbThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x / groups;
    const int s0 = (int)(blockIdx.x - t * groups) * KB, ns = min(KB, k - s0);
    const int64_t slot = t * k + s0;
    float ws[KB], acc[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
        ws[i] = i < ns ? __ldg(w + slot + i) : 0.f;
        acc[i] = 0.f;
    }
    if (VEC) {
        const float4* g = (const float4*)(dy + t * n);
        const int nv = (int)(n / 4);
        for (int j = threadIdx.x; j < nv; j += kCbThreads) {
            const float4 v = __ldcs(g + j);
            float4 d[KB];
#pragma unroll
            for (int i = 0; i < KB; ++i)
                if (i < ns) d[i] = __ldcs((const float4*)(dst + (slot + i) * n) + j);
#pragma unroll
            for (int i = 0; i < KB; ++i)
                if (i < ns) {
                    acc[i] = __fmaf_rn(v.x, d[i].x, acc[i]);
                    acc[i] = __fmaf_rn(v.y, d[i].y, acc[i]);
                    acc[i] = __fmaf_rn(v.z, d[i].z, acc[i]);
                    acc[i] = __fmaf_rn(v.w, d[i].w, acc[i]);
                    if (ddst)
                        __stcs((float4*)(ddst + (slot + i) * n) + j,
                               make_float4(__fmul_rn(ws[i], v.x), __fmul_rn(ws[i], v.y), __fmul_rn(ws[i], v.z),
                                           __fmul_rn(ws[i], v.w)));
                }
        }
    } else {
        for (int64_t j = threadIdx.x; j < n; j += kCbThreads) {
            const float v = __ldg(dy + t * n + j);
            float d[KB];
#pragma unroll
            for (int i = 0; i < KB; ++i)
                if (i < ns) d[i] = __ldcs(dst + (slot + i) * n + j);
#pragma unroll
            for (int i = 0; i < KB; ++i)
                if (i < ns) {
                    acc[i] = __fmaf_rn(v, d[i], acc[i]);
                    if (ddst) __stcs(ddst + (slot + i) * n + j, __fmul_rn(ws[i], v));
                }
        }
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[i] = __fadd_rn(acc[i], __shfl_xor_sync(0xffffffffu, acc[i], o));
        if (lane == 0) s_part[i][warp] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x < ns) {
        float r = 0.f;
#pragma unroll
        for (int i = 0; i < kCbThreads / 32; ++i) r = __fadd_rn(r, s_part[threadIdx.x][i]);
        dw[slot + threadIdx.x] = r;
    }
}

template <int KB>
void launch(bool vec, unsigned grid, const float* dy, const float* dst, const float* w, int k, int64_t n, int groups,
            float* dw, float* ddst, cudaStream_t s) {
    if (vec) combine_backward_kernel<KB, true><<<grid, kCbThreads, 0, s>>>(dy, dst, w, k, n, groups, dw, ddst);
    else combine_backward_kernel<KB, false><<<grid, kCbThreads, 0, s>>>(dy, dst, w, k, n, groups, dw, ddst);
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
    const bool vec = n % 4 == 0 && (((uintptr_t)dy | (uintptr_t)dst | (uintptr_t)ddst) & 15u) == 0;
    int kb = 8;
    while (kb > 1 && (kb >= 2 * k || n_tokens * ((k + kb - 1) / kb) < 4 * 148)) kb >>= 1;
    const int groups = (k + kb - 1) / kb;
    if (n_tokens * groups >= ((int64_t)1 << 31)) return MOE_ERR_RANGE;
    const unsigned grid = (unsigned)(n_tokens * groups);
    cudaStream_t s = (cudaStream_t)stream;
    if (kb == 8) launch<8>(vec, grid, dy, dst, weights, k, n, groups, dweights, ddst, s);
    else if (kb == 4) launch<4>(vec, grid, dy, dst, weights, k, n, groups, dweights, ddst, s);
    else if (kb == 2) launch<2>(vec, grid, dy, dst, weights, k, n, groups, dweights, ddst, s);
    else launch<1>(vec, grid, dy, dst, weights, k, n, groups, dweights, ddst, s);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
