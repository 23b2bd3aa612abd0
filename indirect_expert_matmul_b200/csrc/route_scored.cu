// Scored router and its gradient: the step before the indirect matmul in layers
// whose router scores the experts by a sigmoid or a softmax, adds a balance
// bias to the scores for the choice only, and may restrict the choice to the
// best groups of experts.  For token t with logits l and scores
//   s[e] = 1 / (1 + exp(-l[e]))   or   exp(l[e]) / sum_j exp(l[j]) :
//
//   key[e]  = s[e] + bias[e]
//   G[g]    = the largest key of group g, or the sum of its two largest
//   open    = the topk_groups groups of largest G (equal G: lower group)
//   ids[t]  = the k largest keys inside open groups, descending (equal: lower e)
//   w[t][i] = scale * s[ids[i]]            (/ sum over the k chosen s)
//
// The choice is that of the rule over real numbers: keys are evaluated in
// double precision, because a float key cannot tell apart two scores that
// differ by less than 2^-24 and the choice would depend on the evaluation
// (without a bias the logits themselves are compared).
#include <math.h>

#include "common.cuh"

namespace moe {

namespace {

constexpr int kRsWarps = 4;
constexpr int kRsMaxPerLane = 32;  // n_experts <= 1024
constexpr int kRsMaxGroups = 32;

__device__ __forceinline__ float load_logit(const void* p, int type, int64_t i) {
    if (type == MOE_F32) return __ldg((const float*)p + i);
    const uint16_t h = __ldg((const uint16_t*)p + i);
    return type == MOE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// sigmoid(l) * exp(-c) for c <= 0, c >= min(l, 0): no overflow, and no underflow for l near c.
__device__ __forceinline__ float sigmoid_over(float l, float c) {
    return __fdiv_rn(expf(__fsub_rn(fminf(l, 0.f), c)), __fadd_rn(1.f, expf(-fabsf(l))));
}

struct RouteScoredArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int64_t n_tokens;
    int type, n_experts, k, softmax, n_groups, topk_groups, group_top, normalize;
    float scale;
    int32_t* ids;
    float* weights;
};

// One warp per token; expert j*32 + lane in slot j of the lane.
template <int NPL>
__global__ void __launch_bounds__(kRsWarps * 32) route_scored_kernel(const RouteScoredArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRsWarps + (threadIdx.x >> 5);
    if (t >= p.n_tokens) return;
    const int E = p.n_experts;
    float l[NPL];
    double key[NPL];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * 32 + lane;
        l[j] = e < E ? load_logit(p.logits, p.type, t * p.ld + e) : -INFINITY;
        mx = fmaxf(mx, l[j]);
    }
    mx = warp_max(mx);
    double z = 1.0;
    if (p.softmax) {
        z = 0.0;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (j * 32 + lane < E) z += exp((double)l[j] - (double)mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * 32 + lane;
        double s = p.softmax ? exp((double)l[j] - (double)mx) / z : 1.0 / (1.0 + exp(-(double)l[j]));
        if (l[j] == -INFINITY) s = 0.0;  // also a row of -inf only
        if (p.bias && e < E) s += (double)__ldg(p.bias + e);
        key[j] = e < E && s == s ? s : -INFINITY;  // a NaN key sorts below every number, ids stay in range
    }
    uint32_t shut = 0u;  // bit j: expert j*32 + lane lies in a closed group (or was chosen)
    if (p.topk_groups < p.n_groups) {
        const int size = E / p.n_groups;
        double mine = -INFINITY;  // lane g: the score of group g
        for (int g = 0; g < p.n_groups; ++g) {
            double a = -INFINITY, b = -INFINITY;  // the two largest keys of the group
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const int e = j * 32 + lane;
                if (e >= g * size && e < (g + 1) * size) {
                    b = fmax(b, fmin(a, key[j]));
                    a = fmax(a, key[j]);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
                b = fmax(fmax(b, ob), fmin(a, oa));
                a = fmax(a, oa);
            }
            if (lane == g) mine = p.group_top == 2 ? a + b : a;
        }
        int rank = 0;  // groups ahead of this lane's
        for (int g = 0; g < p.n_groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const uint32_t open = __ballot_sync(0xffffffffu, lane < p.n_groups && rank < p.topk_groups);
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const int e = j * 32 + lane;
            if (e < E && !(open >> (e / size) & 1u)) shut |= 1u << j;
        }
    }
    if (!p.bias) {  // the order of the scores is that of the logits, also where scores round to one value
#pragma unroll
        for (int j = 0; j < NPL; ++j) key[j] = l[j] != l[j] ? -INFINITY : fmax((double)l[j], -1e300);
    }
    int32_t* it = p.ids + t * p.k;
    float* wt = p.weights + t * p.k;
    for (int i = 0; i < p.k; ++i) {
        double bk = -INFINITY;
        float bl = 0.f;
        int be = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (j * 32 + lane < E && !(shut >> j & 1u) && (be == 0x7fffffff || key[j] > bk)) {
                bk = key[j];
                bl = l[j];
                be = j * 32 + lane;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ok = __shfl_xor_sync(0xffffffffu, bk, o);
            const float ol = __shfl_xor_sync(0xffffffffu, bl, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (ok > bk || (ok == bk && oe < be)) {
                bk = ok;
                bl = ol;
                be = oe;
            }
        }
        if ((be & 31) == lane) shut |= 1u << (be >> 5);
        if (lane == 0) {
            it[i] = be;
            wt[i] = bl;
        }
    }
    __syncwarp();
    // weights from the chosen logits, in choice order
    float top = -INFINITY;
    for (int i = lane; i < p.k; i += 32) top = fmaxf(top, wt[i]);
    top = warp_max(top);
    float zf = 1.f, c = 0.f;
    if (p.softmax) {
        c = p.normalize ? top : mx;
        zf = (float)z;
    } else if (p.normalize) {
        c = fminf(top, 0.f);
    }
    const bool dead = c == -INFINITY;  // no chosen expert (or no expert at all) has a score: weights 0
    float sum = 0.f;
    for (int i = lane; i < p.k; i += 32) {
        const float v = wt[i];
        float s = p.softmax ? expf(__fsub_rn(v, c)) : sigmoid_over(v, c);
        if (dead) s = 0.f;
        wt[i] = s;
        sum = __fadd_rn(sum, s);
    }
    if (p.normalize) zf = warp_sum(sum);
    for (int i = lane; i < p.k; i += 32) wt[i] = dead ? 0.f : __fmul_rn(__fdiv_rn(wt[i], zf), p.scale);
}

struct RouteScoredBwdArgs {
    const void* logits;
    int64_t ld;
    const int32_t* ids;
    const float* dw;
    int64_t n_tokens;
    int type, n_experts, k, softmax, normalize;
    float scale;
    void* out;
};

__device__ __forceinline__ void store_logit(void* p, int type, int64_t i, float v) {
    if (type == MOE_F32) ((float*)p)[i] = v;
    else if (type == MOE_BF16) ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
    else ((__half*)p)[i] = __float2half_rn(v);
}

// Gradient of the scored router's weights with respect to the logits (the
// choice itself has none).  With g = scale * dweights and, normalised,
// p_i = s_i / sum of the chosen s:
//   sigmoid, normalised:  dl[ids_i] += p_i (g_i - sum_j g_j p_j) (1 - s_i)
//   sigmoid:              dl[ids_i] += g_i s_i (1 - s_i)
//   softmax, normalised:  dl[ids_i] += p_i (g_i - sum_j g_j p_j)
//   softmax:              dl[e]      = s_e (sum of g_i with ids_i = e  -  sum_j g_j s_{ids_j})
// One warp per token; the row of gradients is put together in shared memory.
// A slot whose id is outside [0, n_experts) is left out.
__global__ void __launch_bounds__(kRsWarps * 32) route_scored_bwd_kernel(const RouteScoredBwdArgs p) {
    extern __shared__ float s_rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRsWarps + warp;
    if (t >= p.n_tokens) return;
    const int E = p.n_experts;
    const int32_t* it = p.ids + t * p.k;
    const float* gt = p.dw + t * p.k;
    float* row = s_rows + (size_t)warp * E;
    for (int e = lane; e < E; e += 32) row[e] = 0.f;
    auto slot_logit = [&](int i) {
        const int e = it[i];
        return (unsigned)e < (unsigned)E ? load_logit(p.logits, p.type, t * p.ld + e) : -INFINITY;
    };
    const bool dense = p.softmax && !p.normalize;
    float top = -INFINITY;
    if (dense)
        for (int e = lane; e < E; e += 32) top = fmaxf(top, load_logit(p.logits, p.type, t * p.ld + e));
    else
        for (int i = lane; i < p.k; i += 32) top = fmaxf(top, slot_logit(i));
    top = warp_max(top);
    const float c = p.softmax ? top : p.normalize ? fminf(top, 0.f) : 0.f;
    const bool dead = c == -INFINITY;
    float z = 0.f, dot = 0.f;
    if (dense)
        for (int e = lane; e < E; e += 32)
            z = __fadd_rn(z, expf(__fsub_rn(load_logit(p.logits, p.type, t * p.ld + e), c)));
    for (int i = lane; i < p.k; i += 32) {
        const float v = slot_logit(i);
        const float r = v == -INFINITY ? 0.f : p.softmax ? expf(__fsub_rn(v, c)) : sigmoid_over(v, c);
        if (!dense) z = __fadd_rn(z, r);
        dot = __fmaf_rn(gt[i], r, dot);
    }
    z = warp_sum(z);
    dot = warp_sum(dot);
    if (!p.normalize && !p.softmax) {
        z = 1.f;
        dot = 0.f;
    }
    dot = dead ? 0.f : __fdiv_rn(dot, z);
    __syncwarp();
    for (int i0 = 0; i0 < p.k; i0 += 32) {
        const int i = i0 + lane;
        int e = -1;
        float v = 0.f;
        if (i < p.k) {
            e = it[i];
            const float lg = slot_logit(i);
            if ((unsigned)e >= (unsigned)E) e = -1;
            if (dense) v = gt[i];
            else if (lg != -INFINITY) {
                const float r = p.softmax ? expf(__fsub_rn(lg, c)) : sigmoid_over(lg, c);
                v = __fmul_rn(__fdiv_rn(r, z), __fsub_rn(gt[i], dot));
                if (!p.softmax) v = __fmul_rn(v, sigmoid_over(-lg, 0.f));
            }
        }
        for (int q = 0; q < 32; ++q) {  // in slot order, so that a repeated id adds up the same way each time
            if (lane == q && e >= 0) row[e] = __fadd_rn(row[e], v);
            __syncwarp();
        }
    }
    for (int e = lane; e < E; e += 32) {
        float v = row[e];
        if (dense) {
            const float lg = load_logit(p.logits, p.type, t * p.ld + e);
            v = lg == -INFINITY ? 0.f
                                : __fmul_rn(__fdiv_rn(expf(__fsub_rn(lg, c)), z), __fsub_rn(v, dot));
        }
        store_logit(p.out, p.type, t * E + e, __fmul_rn(v, p.scale));
    }
}

bool valid_dtype(int t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; }
uintptr_t type_mask(int t) { return t == MOE_F32 ? 3u : 1u; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_route_scored(const void* logits, moe_dtype l_type, int64_t row_stride, const float* bias,
                                       int64_t n_tokens, int n_experts, int k, moe_score score, int n_groups,
                                       int topk_groups, int group_top, int normalize, float scale, int32_t* ids,
                                       float* weights, moe_stream stream) {
    if (!valid_dtype(l_type) || (score != MOE_SOFTMAX && score != MOE_SIGMOID)) return MOE_ERR_INVALID;
    if (n_tokens < 0 || n_experts < 1 || k < 1 || k > n_experts || row_stride < n_experts) return MOE_ERR_INVALID;
    if (n_groups < 1 || topk_groups < 1 || topk_groups > n_groups || group_top < 1 || group_top > 2)
        return MOE_ERR_INVALID;
    if (n_tokens >= kMaxTokens || n_experts > kRsMaxPerLane * 32 || k >= kMaxK || n_groups > kRsMaxGroups ||
        row_stride >= ((int64_t)1 << 40))
        return MOE_ERR_RANGE;
    if (n_experts % n_groups || group_top > n_experts / n_groups || k > topk_groups * (n_experts / n_groups))
        return MOE_ERR_INVALID;
    if (n_tokens == 0) return MOE_OK;
    if (!logits || !ids || !weights) return MOE_ERR_INVALID;
    if (((uintptr_t)logits & type_mask(l_type)) || (((uintptr_t)bias | (uintptr_t)ids | (uintptr_t)weights) & 3u))
        return MOE_ERR_INVALID;
    RouteScoredArgs a = {logits, row_stride, bias, n_tokens, (int)l_type, n_experts, k, score == MOE_SOFTMAX,
                         n_groups, topk_groups, group_top, normalize != 0, scale, ids, weights};
    const unsigned blocks = (unsigned)((n_tokens + kRsWarps - 1) / kRsWarps);
    const dim3 block(kRsWarps * 32);
    cudaStream_t s = (cudaStream_t)stream;
    if (n_experts <= 64) route_scored_kernel<2><<<blocks, block, 0, s>>>(a);
    else if (n_experts <= 128) route_scored_kernel<4><<<blocks, block, 0, s>>>(a);
    else if (n_experts <= 256) route_scored_kernel<8><<<blocks, block, 0, s>>>(a);
    else if (n_experts <= 512) route_scored_kernel<16><<<blocks, block, 0, s>>>(a);
    else route_scored_kernel<32><<<blocks, block, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_route_scored_backward(const void* logits, moe_dtype l_type, int64_t row_stride,
                                                const int32_t* ids, const float* dweights, int64_t n_tokens,
                                                int n_experts, int k, moe_score score, int normalize, float scale,
                                                void* dlogits, moe_stream stream) {
    if (!valid_dtype(l_type) || (score != MOE_SOFTMAX && score != MOE_SIGMOID)) return MOE_ERR_INVALID;
    if (n_tokens < 0 || n_experts < 1 || k < 1 || k > n_experts || row_stride < n_experts) return MOE_ERR_INVALID;
    if (n_tokens >= kMaxTokens || n_experts > kRsMaxPerLane * 32 || k >= kMaxK || row_stride >= ((int64_t)1 << 40))
        return MOE_ERR_RANGE;
    if (n_tokens == 0) return MOE_OK;
    if (!logits || !ids || !dweights || !dlogits) return MOE_ERR_INVALID;
    if ((((uintptr_t)logits | (uintptr_t)dlogits) & type_mask(l_type)) || (((uintptr_t)ids | (uintptr_t)dweights) & 3u))
        return MOE_ERR_INVALID;
    RouteScoredBwdArgs a = {logits, row_stride, ids, dweights, n_tokens, (int)l_type, n_experts, k,
                            score == MOE_SOFTMAX, normalize != 0, scale, dlogits};
    const unsigned blocks = (unsigned)((n_tokens + kRsWarps - 1) / kRsWarps);
    route_scored_bwd_kernel<<<blocks, kRsWarps * 32, (size_t)kRsWarps * n_experts * 4, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
