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
// The choice is that of the rule over real numbers.  Float keys carry a bound on
// their error; wherever two of them are closer than that, the candidates (or
// the groups) are compared again in double, so that the choice does not depend
// on how a float was rounded, nor on a score that rounds to 0, 1/2 or 1.  Without
// a bias the order of the scores is that of the logits, which are compared as
// they are.
//
// One warp per token, NPL consecutive experts a lane (E <= 32 NPL), read once
// with 16-byte loads.  A round of the choice is one warp-wide maximum of the
// lanes' best keys (as integers that order like the floats) and one ballot;
// the winner's lane looks for its next best.  Such a call is bound by latency,
// not by its bytes: one load, the scores, k rounds, one store.
#include <math.h>

#include "common.cuh"

namespace moe {

namespace {

constexpr int kRsWarps = 4;
template <int NPL, bool BIAS>
constexpr int kRsCtaWarps = BIAS && NPL == 32 ? 2 : kRsWarps;  // (16 bytes an expert and warp of shared memory)
constexpr int kRsMaxPerLane = 32;  // n_experts <= 1024
constexpr int kRsMaxGroups = 32;
constexpr int64_t kRsHalfTokens = 148 * 32;  // above: a scheduler has more than 8 tokens

__device__ __forceinline__ float load_logit(const void* p, int type, int64_t i) {
    if (type == MOE_F32) return __ldg((const float*)p + i);
    const uint16_t h = __ldg((const uint16_t*)p + i);
    return type == MOE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// Over the LANES lanes of `mask` (a token's), in a fixed order.
template <int LANES>
__device__ __forceinline__ float group_max(float v, uint32_t mask) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
    return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(mask, v, o));
    return v;
}
__device__ __forceinline__ float warp_max(float v) { return group_max<32>(v, 0xffffffffu); }
__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v, 0xffffffffu); }

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
    int vec;  // bit 0: rows of logits start on 16 bytes, bit 1: bias does
};

// Elements lane * NPL .. + NPL - 1 of a row of E (fill past its end).
template <int NPL>
__device__ __forceinline__ void load_row(const void* base, int type, int64_t first, int E, int lane, bool vec,
                                         float fill, float (&v)[NPL]) {
    const int e0 = lane * NPL;
    if (vec && e0 + NPL <= E) {
        if (type == MOE_F32) {
            const float* f = (const float*)base + first + e0;
            if constexpr (NPL % 4 == 0) {
#pragma unroll
                for (int j = 0; j < NPL; j += 4) {
                    const float4 q = __ldg((const float4*)(f + j));
                    v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < NPL; ++j) v[j] = __ldg(f + j);
            }
        } else {
            const uint16_t* h = (const uint16_t*)base + first + e0;
            uint32_t w[(NPL + 1) / 2];
            if constexpr (NPL % 8 == 0) {
#pragma unroll
                for (int j = 0; j < NPL; j += 8) {
                    const uint4 q = __ldg((const uint4*)(h + j));
                    w[j / 2] = q.x; w[j / 2 + 1] = q.y; w[j / 2 + 2] = q.z; w[j / 2 + 3] = q.w;
                }
            } else if constexpr (NPL == 4) {
                const uint2 q = __ldg((const uint2*)h);
                w[0] = q.x; w[1] = q.y;
            } else {
                w[0] = NPL == 2 ? __ldg((const uint32_t*)h) : (uint32_t)__ldg(h);
            }
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const uint32_t b = w[j / 2] >> (16 * (j & 1)) & 0xffffu;
                v[j] = type == MOE_BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) v[j] = e0 + j < E ? load_logit(base, type, first + e0 + j) : fill;
}

// Integers that order like floats (-0 as 0); 0 is left for "not available", NaN is 1.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.f));
    return f != f ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
// The lowest ordered key that may still equal or beat key u, both within err
// plus one rounding of the true ones.
__device__ __forceinline__ uint32_t rival(uint32_t u, float err) {
    const float f = from_ordered(u);
    const float t = f - 2.f * (err + fabsf(f) * 1.2e-7f);
    return u <= 1u || !(fabsf(f) < INFINITY) ? u : min(u, ordered(t));
}

// NPL (a power of two) keys with their indexes into descending order by an
// odd-even merge sort; TIES: equal keys by ascending index.
template <int NPL, bool TIES>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NPL], int (&idx)[NPL]) {
#pragma unroll
    for (int p = 1; p < NPL; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < NPL; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    const int a = i + j, b = i + j + q;
                    if (b < NPL && a / (2 * p) == b / (2 * p)) {
                        const bool swap = key[a] < key[b] || (TIES && key[a] == key[b] && idx[a] > idx[b]);
                        const uint32_t ka = key[a];
                        const int ia = idx[a];
                        key[a] = swap ? key[b] : ka;
                        idx[a] = swap ? idx[b] : ia;
                        key[b] = swap ? ka : key[b];
                        idx[b] = swap ? ia : idx[b];
                    }
                }
}

// A key in two doubles, hi + lo exactly what their sum says and hi the sum rounded.
struct Key {
    double hi, lo;
    // hi and lo of a + b (exact) + c
    static __device__ Key sum(double a, double b, double c) {
        const double h = __dadd_rn(a, b), bb = __dsub_rn(h, a);
        const double r = __dadd_rn(__dadd_rn(__dsub_rn(a, __dsub_rn(h, bb)), __dsub_rn(b, bb)), c);
        const double hi = __dadd_rn(h, r), rr = __dsub_rn(hi, h);
        const double lo = __dadd_rn(__dsub_rn(h, __dsub_rn(hi, rr)), __dsub_rn(r, rr));
        if (fabs(hi) < INFINITY) return {hi, lo};
        return {fabs(h) == INFINITY && c == c ? h : -INFINITY, 0.0};  // an infinite bias; NaN counts as the lowest
    }
    __device__ bool operator>(const Key& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
    __device__ bool operator==(const Key& o) const { return hi == o.hi && lo == o.lo; }
};

// The double-precision side of a token, for close keys only, one expert at a
// time: kept in registers and unrolled over the lane's experts it took so many
// that the 4096-token prompt of 256 experts ran in 29 us.  A score is worked out
// as its distance from 0, 1/2 or 1 (softmax: from 0 or the largest score), so
// that scores which round to one double, a sigmoid's above 37 to 1, keep their
// order: keys are a double and what it lacks, both in shared memory (worked out
// again where two doubles are equal, it took 7 us more in a cold instruction cache).
// Without a bias keys order like logits, which stand for the rests.
template <bool BIAS>
struct Exact {
    const RouteScoredArgs& p;
    int64_t row;
    float mx;      // softmax: the largest logit
    double* key;   // [n_experts]: the keys' hi
    double* rest;  // [n_experts]: their lo (with a bias)
    double z;      // softmax: the denominator

    __device__ void denominator(int lane) {
        if (!p.softmax || z != 0.0) return;
#pragma unroll 1
        for (int e = lane; e < p.n_experts; e += 32) {
            const float l = load_logit(p.logits, p.type, row + e);
            if (l != -INFINITY) z += exp((double)l - (double)mx);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    __device__ Key key_of(int e) const {
        const float l = load_logit(p.logits, p.type, row + e);
        const double b = BIAS ? (double)__ldg(p.bias + e) : 0.0;
        double base = 0.0, far = 0.0;
        if (l != -INFINITY) {
            // r = exp of -|l| or of l - mx, m = r - 1 without its cancellation
            const double x = p.softmax ? (double)l - (double)mx : -fabs((double)l), r = exp(x);
            const double m = x > -0x1p-10 ? x * (1.0 + x * (0.5 + x * (1.0 / 6 + x * (1.0 / 24)))) : r - 1.0;
            const double big = 1.0 / (p.softmax ? z : 1.0 + r);
            if (p.softmax) {
                base = x > -0.5 ? big : 0.0;
                far = big * (x > -0.5 ? m : r);
            } else if (x > -1.0) {  // 1 / (1 + exp(-l)) - 1/2 = (1 - exp(-|l|)) / (1 + exp(-|l|)) / 2, signed
                base = 0.5;
                far = copysign(0.5 * m * big, (double)l);
            } else {
                base = l > 0.f ? 1.0 : 0.0;
                far = r * big;
                if (l > 0.f) far = -far;
            }
        }
        return Key::sum(base, b, far);
    }
    __device__ void fill(int lane) {
        denominator(lane);
#pragma unroll 1
        for (int e = lane; e < p.n_experts; e += 32) {
            const Key k = key_of(e);
            key[e] = k.hi;
            if (BIAS) rest[e] = k.lo;
        }
        __syncwarp();
    }
    // Whether expert e with the high part v comes before f with w (kNone: no
    // expert): the larger key, equal keys by the lower index.
    static constexpr int kNone = 0x7fffffff;
    __device__ bool before(double v, int e, double w, int f) const {
        if (v != w || e == kNone || f == kNone) return e != kNone && (f == kNone || v > w);
        const double a = BIAS ? rest[e] : load_logit(p.logits, p.type, row + e);
        const double b = BIAS ? rest[f] : load_logit(p.logits, p.type, row + f);
        return a > b || (a == b && e < f);
    }
    // Lane g: the score of group g, each group scanned by as many lanes as there are for it
    // (one group after the other by the whole warp took 2 us a token).
    __device__ Key group_score(int lane, int size) const {
        int P = 1;
        while (2 * P * p.n_groups <= 32) P *= 2;
        const int g = lane / P, end = g < p.n_groups ? (g + 1) * size : 0;
        double a = -INFINITY, b = -INFINITY;  // the group's two first, ea and eb
        int ea = kNone, eb = kNone;
        auto take = [&](double v, int e) {
            if (before(v, e, a, ea)) {
                b = a; eb = ea;
                a = v; ea = e;
            } else if (before(v, e, b, eb)) {
                b = v; eb = e;
            }
        };
#pragma unroll 1
        for (int e = g * size + lane % P; e < end; e += P) take(key[e], e);
        __syncwarp();
#pragma unroll 1
        for (int o = 1; o < P; o <<= 1) {
            const double oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
            const int oea = __shfl_xor_sync(0xffffffffu, ea, o), oeb = __shfl_xor_sync(0xffffffffu, eb, o);
            take(oa, oea);
            take(ob, oeb);
            __syncwarp();
        }
        double lo = 0.0;
#pragma unroll 1
        for (int j = 0; j < p.group_top; ++j) {
            const int e = j ? eb : ea;
            if (e != kNone) lo += BIAS ? rest[e] : key_of(e).lo;
        }
        __syncwarp();
        const Key k = Key::sum(a, p.group_top == 2 ? b : 0.0, lo);
        const int from = lane < p.n_groups ? lane * P : 0;
        const Key mine = {__shfl_sync(0xffffffffu, k.hi, from), __shfl_sync(0xffffffffu, k.lo, from)};
        return lane < p.n_groups ? mine : Key{-INFINITY, 0.0};
    }
    // The k largest keys of open groups (equal: lower expert) to ids.
    __device__ void choose(int lane, int size, uint32_t open, int32_t* ids) const {
        uint32_t taken = 0u;
#pragma unroll 1
        for (int i = 0; i < p.k; ++i) {
            double best = -INFINITY;
            int be = kNone, q = 0;
#pragma unroll 1
            for (int e = lane; e < p.n_experts; e += 32, ++q) {
                const double v = key[e];
                if ((taken >> q & 1u) || !(open >> (e / size) & 1u)) continue;
                if (before(v, e, best, be)) {
                    best = v;
                    be = e;
                }
            }
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) {
                const double ov = __shfl_xor_sync(0xffffffffu, best, o);
                const int oe = __shfl_xor_sync(0xffffffffu, be, o);
                if (before(ov, oe, best, be)) {
                    best = ov;
                    be = oe;
                }
            }
            if ((be & 31) == lane) taken |= 1u << (be >> 5);
            if (lane == 0) ids[i] = be;
        }
        __syncwarp();
    }
};

// The two largest values (a >= b) of the experts of group g; value(j) is that of
// the lane's j-th expert, NaN counts as the lowest.
template <int NPL, typename F>
__device__ __forceinline__ void group_top2(const F& value, int lane, int E, int size, int g, float& a, float& b) {
    a = b = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = lane * NPL + j;
        if (e < E && e >= g * size && e < (g + 1) * size) {
            float v = value(j);
            v = v == v ? v : -INFINITY;
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
        a = fmaxf(a, oa);
    }
}

// (registers held to what the float side needs: where the double-precision side set
// them, 8191 x 128 softmax without a bias took 7.4 us for 7.0)
template <int NPL, bool BIAS>
__global__ void __launch_bounds__(kRsCtaWarps<NPL, BIAS> * 32, NPL <= 2 ? 12 : NPL == 4 ? 9 : NPL == 8 ? 8 : 1)
route_scored_kernel(const RouteScoredArgs p) {
    constexpr int kWarps = kRsCtaWarps<NPL, BIAS>;
    __shared__ double s_key[kWarps][32 * NPL], s_rest[BIAS ? kWarps : 1][BIAS ? 32 * NPL : 1];
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.n_tokens) return;
    const int E = p.n_experts, e0 = lane * NPL;
    const bool softmax = p.softmax, grouped = p.topk_groups < p.n_groups;
    const bool score_keys = BIAS || (grouped && p.group_top == 2);
    float l[NPL], b[NPL];
    load_row<NPL>(p.logits, p.type, t * p.ld, E, lane, p.vec & 1, -INFINITY, l);
    if (BIAS) load_row<NPL>(p.bias, MOE_F32, 0, E, lane, p.vec & 2, 0.f, b);
    float mx = -INFINITY, z = 1.f;
    if (softmax && (score_keys || !p.normalize)) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) mx = fmaxf(mx, l[j]);
        mx = warp_max(mx);
    }
    // Float scores for the choice; each within 2^-21 of the true one (sigmoid: the
    // fast exponential's 2 + 1.2 |l| ulp come in times s (1 - s), the division's 2
    // ulp and the sum's half), or within 2^-18 (softmax: the exponential's argument
    // is rounded, p |l - mx| <= 1/e, and a sum of NPL + 5 levels).
    float s[NPL];
    const float err = softmax ? 3.8e-6f : 4.8e-7f;
    if (softmax) {
        if (score_keys || !p.normalize) {
            z = 0.f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                s[j] = l[j] == -INFINITY ? 0.f : expf(__fsub_rn(l[j], mx));
                z = __fadd_rn(z, s[j]);
            }
            z = warp_sum(z);
            const float rz = z > 0.f ? __fdiv_rn(1.f, z) : 0.f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) s[j] *= rz;
        }
    } else if (score_keys) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) s[j] = __fdividef(1.f, 1.f + __expf(-l[j]));
    }
    Exact<BIAS> exact64 = {p, t * p.ld, mx, s_key[threadIdx.x >> 5], s_rest[BIAS ? threadIdx.x >> 5 : 0], 0.0};
    const int size = E / p.n_groups;
    uint32_t open = 0xffffffffu;  // bit g: group g
    // keys; 0: not available (past the row's end, later: chosen or in a closed group)
    uint32_t key[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) key[j] = e0 + j < E ? ordered(BIAS ? __fadd_rn(s[j], b[j]) : l[j]) : 0u;

    if (grouped) {
        const int G = p.n_groups;
        const bool exact = !BIAS && p.group_top == 1;  // the groups' best logits, compared as they are
        auto group_key = [&](int j) { return BIAS ? __fadd_rn(s[j], b[j]) : exact ? l[j] : s[j]; };
        float mine = -INFINITY, mag = 0.f;  // lane g: the score of group g, what its terms' roundings scale with
        const int P = size / NPL;
        const bool lanes = P * NPL == size && (P & (P - 1)) == 0;
        if (lanes) {
            // a group is P lanes: its two largest by log2 P exchanges (the loop over
            // the groups below takes that many times G)
            float a = -INFINITY, c = -INFINITY;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const float k0 = group_key(j), v = k0 == k0 ? k0 : -INFINITY;
                c = fmaxf(c, fminf(a, v));
                a = fmaxf(a, v);
            }
            for (int o = 1; o < P; o <<= 1) {
                const float oa = __shfl_xor_sync(0xffffffffu, a, o), oc = __shfl_xor_sync(0xffffffffu, c, o);
                c = fmaxf(fmaxf(c, oc), fminf(a, oa));
                a = fmaxf(a, oa);
            }
            const float sc = p.group_top == 2 ? __fadd_rn(a, c) : a;
            mine = __shfl_sync(0xffffffffu, sc, lane < G ? lane * P : 0);
            if (lane >= G) mine = -INFINITY;
            if (BIAS && p.group_top == 2) mag = fabsf(a) + fabsf(c);
        } else {
            for (int g = 0; g < G; ++g) {
                float a, c;
                group_top2<NPL>(group_key, lane, E, size, g, a, c);
                if (lane == g) mine = p.group_top == 2 ? __fadd_rn(a, c) : a;
                // (a group without two finite keys takes no part: its sum is -inf whatever its roundings)
                const float terms = fabsf(a) + fabsf(c);
                if (BIAS && p.group_top == 2 && terms < INFINITY) mag = fmaxf(mag, terms);
            }
        }
        int rank = 0;  // groups ahead of this lane's
        for (int g = 0; g < G; ++g) {
            const float o = __shfl_sync(0xffffffffu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        bool in = lane < G && rank < p.topk_groups;
        if (!exact) {
            // the open groups' lowest score against the closed groups' highest
            const uint32_t u = ordered(mine);
            const uint32_t lo = __reduce_min_sync(0xffffffffu, in ? u : 0xffffffffu);
            const uint32_t hi = __reduce_max_sync(0xffffffffu, lane < G && !in ? u : 0u);
            // (a sum of two keys of opposite sign: each rounded as large as it is)
            const float own = mag < INFINITY ? mag : 0.f;
            const float terms = 1.2e-7f * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(own)));
            if (hi >= rival(lo, 2.f * err + terms) && lo > ordered(-INFINITY)) {
                exact64.fill(lane);
                const Key best = exact64.group_score(lane, size);
                rank = 0;
                for (int g = 0; g < G; ++g) {
                    const Key o = {__shfl_sync(0xffffffffu, best.hi, g), __shfl_sync(0xffffffffu, best.lo, g)};
                    rank += o > best || (o == best && g < lane);
                }
                in = lane < G && rank < p.topk_groups;
            }
        }
        open = __ballot_sync(0xffffffffu, in);
        if (lanes) {
            const bool shut = !(open >> (lane / P) & 1u);
#pragma unroll
            for (int j = 0; j < NPL; ++j) key[j] = shut ? 0u : key[j];
        } else {
            int g = e0 / size, r = e0 - g * size;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                if (!(open >> (g & 31) & 1u)) key[j] = 0u;
                if (++r == size) {
                    r = 0;
                    ++g;
                }
            }
        }
    }

    int32_t* it = p.ids + t * p.k;
    float* wt = p.weights + t * p.k;
    // The lane's keys in descending order: what a round needs is at the front.
    // Equal float keys with a bias count as close, below.
    int idx[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) idx[j] = j;
    sort_keys<NPL, !BIAS>(key, idx);
    int my_id = 0;
    uint32_t my_key = 0u, before = 0xffffffffu;  // lane i: choice i of the current 32 and its key; the last choice's key
    bool close = false;
    for (int i = 0; i < p.k; ++i) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
        const int win = __ffs(__ballot_sync(0xffffffffu, key[0] == m)) - 1;
        const int wj = __shfl_sync(0xffffffffu, idx[0], win);
        if (lane == win) {
#pragma unroll
            for (int j = 0; j + 1 < NPL; ++j) {
                key[j] = key[j + 1];
                idx[j] = idx[j + 1];
            }
            key[NPL - 1] = 0u;
        }
        if (lane == (i & 31)) {
            my_id = win * NPL + wj;
            my_key = m;
        }
        if ((i & 31) == 31 || i == p.k - 1) {
            const int at = (i & ~31) + lane;
            if (at <= i) it[at] = my_id;
            if (BIAS) {  // each choice against the one before it
                uint32_t up = __shfl_up_sync(0xffffffffu, my_key, 1);
                if (lane == 0) up = before;
                close = close || (at <= i && up != 0xffffffffu && my_key >= rival(up, err));
                before = m;
            }
        }
    }
    if (BIAS) {  // and the last against the best of the rest
        uint32_t rest = __reduce_max_sync(0xffffffffu, key[0]);
        if (__any_sync(0xffffffffu, close || (rest != 0u && rest >= rival(before, err)))) {
            __syncwarp();  // other lanes write the entries of it[] again
            // Draw on until a gap, so that the list holds every expert that may belong to
            // the k; order it by double keys, one lane an entry (~0.5 us for the token).
            int n = p.k;
            while (n < 32 && rest != 0u && rest >= rival(before, err)) {
                const int win = __ffs(__ballot_sync(0xffffffffu, key[0] == rest)) - 1;
                const int wj = __shfl_sync(0xffffffffu, idx[0], win);
                if (lane == win) {
#pragma unroll
                    for (int j = 0; j + 1 < NPL; ++j) {
                        key[j] = key[j + 1];
                        idx[j] = idx[j + 1];
                    }
                    key[NPL - 1] = 0u;
                }
                if (lane == n) my_id = win * NPL + wj;
                ++n;
                before = rest;
                rest = __reduce_max_sync(0xffffffffu, key[0]);
            }
            if (n <= 32 && (rest == 0u || rest < rival(before, err))) {
                exact64.denominator(lane);
                const Key v = lane < n ? exact64.key_of(my_id) : Key{0.0, 0.0};
                int place = 0;
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const Key o = {__shfl_sync(0xffffffffu, v.hi, j), __shfl_sync(0xffffffffu, v.lo, j)};
                    const int oe = __shfl_sync(0xffffffffu, my_id, j);
                    place += o > v || (o == v && oe < my_id);
                }
                if (lane < n && place < p.k) it[place] = my_id;
                __syncwarp();
            } else {  // more than 32 in one run of close keys
                exact64.fill(lane);
                exact64.choose(lane, size, open, it);
            }
            if (p.k <= 32 && lane < p.k) my_id = it[lane];
        }
    }
    __syncwarp();
    float my_l = 0.f;
    for (int i = lane; i < p.k; i += 32) {
        my_l = load_logit(p.logits, p.type, t * p.ld + (p.k <= 32 ? my_id : it[i]));
        if (p.k > 32) wt[i] = my_l;  // turned into weights below
    }
    // weights from the chosen logits, in choice order
    auto chosen = [&](int i) { return p.k > 32 ? wt[i] : my_l; };
    __syncwarp();
    float top = -INFINITY;
    for (int i = lane; i < p.k; i += 32) top = fmaxf(top, chosen(i));
    top = warp_max(top);
    const float c = softmax ? (p.normalize ? top : mx) : p.normalize ? fminf(top, 0.f) : 0.f;
    const bool dead = c == -INFINITY;  // no chosen expert (or no expert at all) has a score: weights 0
    float sum = 0.f, w0 = 0.f;
    for (int i = lane; i < p.k; i += 32) {
        const float v = chosen(i);
        w0 = dead || v == -INFINITY ? 0.f : softmax ? expf(__fsub_rn(v, c)) : sigmoid_over(v, c);
        if (p.k > 32) wt[i] = w0;
        sum = __fadd_rn(sum, w0);
    }
    const float zf = p.normalize ? warp_sum(sum) : softmax ? z : 1.f;
    for (int i = lane; i < p.k; i += 32)
        wt[i] = dead ? 0.f : __fmul_rn(__fdiv_rn(p.k > 32 ? wt[i] : w0, zf), p.scale);
}

template <int NPL>
void launch_fwd(const RouteScoredArgs& a, cudaStream_t s) {
    auto grid = [&](int warps) { return (unsigned)((a.n_tokens + warps - 1) / warps); };
    constexpr int kBiased = kRsCtaWarps<NPL, true>, kPlain = kRsCtaWarps<NPL, false>;
    if (a.bias) route_scored_kernel<NPL, true><<<grid(kBiased), kBiased * 32, 0, s>>>(a);
    else route_scored_kernel<NPL, false><<<grid(kPlain), kPlain * 32, 0, s>>>(a);
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
    int vec;  // bit 0: rows of logits start on 16 bytes, bit 1: rows of the gradient do
};

__device__ __forceinline__ void store_logit(void* p, int type, int64_t i, float v) {
    if (type == MOE_F32) ((float*)p)[i] = v;
    else if (type == MOE_BF16) ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
    else ((__half*)p)[i] = __float2half_rn(v);
}

// Elements lane * NPL .. of a row of E, rounded to the type.
template <int NPL>
__device__ __forceinline__ void store_row(void* base, int type, int64_t first, int E, int lane, bool vec,
                                          const float (&v)[NPL]) {
    const int e0 = lane * NPL;
    if (vec && e0 + NPL <= E) {
        if (type == MOE_F32) {
            if constexpr (NPL % 4 == 0) {
                float* f = (float*)base + first + e0;
#pragma unroll
                for (int j = 0; j < NPL; j += 4) *(float4*)(f + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                return;
            }
        } else if constexpr (NPL % 4 == 0) {
            uint32_t w[NPL / 2];
#pragma unroll
            for (int j = 0; j < NPL; j += 2) {
                if (type == MOE_BF16) {
                    const __nv_bfloat162 q = __floats2bfloat162_rn(v[j], v[j + 1]);
                    w[j / 2] = *(const uint32_t*)&q;
                } else {
                    const __half2 q = __floats2half2_rn(v[j], v[j + 1]);
                    w[j / 2] = *(const uint32_t*)&q;
                }
            }
            uint16_t* h = (uint16_t*)base + first + e0;
            if constexpr (NPL == 4) {
                *(uint2*)h = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int j = 0; j < NPL / 2; j += 4) *(uint4*)(h + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        if (e0 + j < E) store_logit(base, type, first + e0 + j, v[j]);
}

// Gradient of the scored router's weights with respect to the logits (the
// choice itself has none).  With g = scale * dweights and, normalised,
// p_i = s_i / sum of the chosen s:
//   sigmoid, normalised:  dl[ids_i] += p_i (g_i - sum_j g_j p_j) (1 - s_i)
//   sigmoid:              dl[ids_i] += g_i s_i (1 - s_i)
//   softmax, normalised:  dl[ids_i] += p_i (g_i - sum_j g_j p_j)
//   softmax:              dl[e]      = s_e (sum of g_i with ids_i = e  -  sum_j g_j s_{ids_j})
// LANES lanes a token.  The slots' terms go to the row's place in shared memory
// and come back NPL consecutive experts a lane, so that the row is written with
// wide stores; only the last form reads the whole row of logits.  A slot whose
// id is outside [0, n_experts) is left out.
template <int NPL, int LANES>
__global__ void __launch_bounds__(kRsWarps * 32) route_scored_bwd_kernel(const RouteScoredBwdArgs p) {
    constexpr int kRows = kRsWarps * 32 / LANES;
    __shared__ __align__(16) float s_rows[kRows][LANES * NPL];
    const int lane = threadIdx.x % LANES, place = threadIdx.x / LANES;
    const uint32_t mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
    const int64_t t = (int64_t)blockIdx.x * kRows + place;
    if (t >= p.n_tokens) return;
    const int E = p.n_experts, e0 = lane * NPL;
    const int32_t* it = p.ids + t * p.k;
    const float* gt = p.dw + t * p.k;
    float* row = s_rows[place];
    const bool dense = p.softmax && !p.normalize;
    float l[NPL];
    if (dense) load_row<NPL>(p.logits, p.type, t * p.ld, E, lane, p.vec & 1, -INFINITY, l);
    // the first LANES slots stay in registers
    auto slot_id = [&](int i) {
        const int e = it[i];
        return (unsigned)e < (unsigned)E ? e : -1;
    };
    auto slot_logit = [&](int e) { return e >= 0 ? load_logit(p.logits, p.type, t * p.ld + e) : -INFINITY; };
    const int id0 = lane < p.k ? slot_id(lane) : -1;
    const float g0 = lane < p.k ? __ldg(gt + lane) : 0.f;
    const float l0 = slot_logit(id0);
#pragma unroll
    for (int j = 0; j < NPL; ++j) row[j * LANES + lane] = 0.f;
    float top = l0;
    if (dense) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) top = fmaxf(top, l[j]);
    } else {
        for (int i = LANES + lane; i < p.k; i += LANES) top = fmaxf(top, slot_logit(slot_id(i)));
    }
    top = group_max<LANES>(top, mask);
    const float c = p.softmax ? top : p.normalize ? fminf(top, 0.f) : 0.f;
    const bool dead = c == -INFINITY;
    auto raw = [&](float v) {  // the score over the common factor
        return v == -INFINITY ? 0.f : p.softmax ? expf(__fsub_rn(v, c)) : sigmoid_over(v, c);
    };
    float z = 0.f, dot = 0.f;
    if (dense) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            l[j] = raw(l[j]);
            z = __fadd_rn(z, l[j]);
        }
    }
    const float r0 = raw(l0);
    for (int i = lane; i < p.k; i += LANES) {
        const float r = i < LANES ? r0 : raw(slot_logit(slot_id(i)));
        if (!dense) z = __fadd_rn(z, r);
        dot = __fmaf_rn(i < LANES ? g0 : gt[i], r, dot);
    }
    if (!p.normalize && !p.softmax) {
        z = 1.f;
        dot = 0.f;
    } else {
        z = group_sum<LANES>(z, mask);
        dot = group_sum<LANES>(dot, mask);
        dot = dead ? 0.f : __fdiv_rn(dot, z);
    }
    __syncwarp(mask);
    for (int i0 = 0; i0 < p.k; i0 += LANES) {
        const int i = i0 + lane;
        int e = id0;
        float v = 0.f;
        if (i < p.k) {
            float g = g0, r = r0, lg = l0;
            if (i0) {
                e = slot_id(i);
                g = gt[i];
                lg = slot_logit(e);
                r = raw(lg);
            }
            if (dense) {
                v = g;
            } else if (lg != -INFINITY) {
                v = __fmul_rn(__fdiv_rn(r, z), __fsub_rn(g, dot));
                if (!p.softmax) v = __fmul_rn(v, sigmoid_over(-lg, 0.f));
            }
        } else {
            e = -1;
        }
        const uint32_t same = __match_any_sync(mask, e);
        if (__all_sync(mask, e < 0 || (same & (same - 1)) == 0u)) {
            if (e >= 0) row[e] = __fadd_rn(row[e], v);
        } else {
            for (int q = 0; q < LANES; ++q) {  // an id occurs twice: in slot order, the same way each time
                if (lane == q && e >= 0) row[e] = __fadd_rn(row[e], v);
                __syncwarp(mask);
            }
        }
        __syncwarp(mask);
    }
    float v[NPL];
    if constexpr (NPL % 4 == 0) {
#pragma unroll
        for (int j = 0; j < NPL; j += 4) {
            const float4 q = *(const float4*)(row + e0 + j);
            v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j) v[j] = row[e0 + j];
    }
    const float rz = dense && !dead ? __fdiv_rn(1.f, z) : 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        if (dense) v[j] = __fmul_rn(__fmul_rn(l[j], rz), __fsub_rn(v[j], dot));
        v[j] = __fmul_rn(v[j], p.scale);
    }
    store_row<NPL>(p.out, p.type, t * E, E, lane, p.vec & 2, v);
}

template <int NPL, int LANES>
void launch_bwd(const RouteScoredBwdArgs& a, cudaStream_t s) {
    constexpr int kRows = kRsWarps * 32 / LANES;
    const unsigned blocks = (unsigned)((a.n_tokens + kRows - 1) / kRows);
    route_scored_bwd_kernel<NPL, LANES><<<blocks, kRsWarps * 32, 0, s>>>(a);
}

bool valid_dtype(int t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; }
uintptr_t type_mask(int t) { return t == MOE_F32 ? 3u : 1u; }
bool rows_aligned(const void* p, int type, int64_t ld) {
    return ((uintptr_t)p & 15u) == 0 && ld * (type == MOE_F32 ? 4 : 2) % 16 == 0;
}

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
                         n_groups, topk_groups, group_top, normalize != 0, scale, ids, weights,
                         (rows_aligned(logits, l_type, row_stride) ? 1 : 0) | (((uintptr_t)bias & 15u) ? 0 : 2)};
    cudaStream_t s = (cudaStream_t)stream;
    if (n_experts <= 32) launch_fwd<1>(a, s);
    else if (n_experts <= 64) launch_fwd<2>(a, s);
    else if (n_experts <= 128) launch_fwd<4>(a, s);
    else if (n_experts <= 256) launch_fwd<8>(a, s);
    else if (n_experts <= 512) launch_fwd<16>(a, s);
    else launch_fwd<32>(a, s);
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
                            score == MOE_SOFTMAX, normalize != 0, scale, dlogits,
                            (rows_aligned(logits, l_type, row_stride) ? 1 : 0) |
                                (rows_aligned(dlogits, l_type, n_experts) ? 2 : 0)};
    cudaStream_t s = (cudaStream_t)stream;
    // Half a warp a token where that leaves fewer instructions and there are enough
    // tokens to hide its longer chain: 128 experts, softmax, 16 / 32 lanes, us:
    // 3.5 / 3.2 at 4096 tokens, 3.8 / 4.1 at 6000, 4.5 / 5.4 at 8192, 6.8 / 8.1 at
    // 16384 (256 experts, 4096 tokens: 4.5 / 3.8).
    if (n_experts <= 128 && n_tokens > kRsHalfTokens) {
        if (n_experts <= 32) launch_bwd<2, 16>(a, s);
        else if (n_experts <= 64) launch_bwd<4, 16>(a, s);
        else launch_bwd<8, 16>(a, s);
    } else if (n_experts <= 32) launch_bwd<1, 32>(a, s);
    else if (n_experts <= 64) launch_bwd<2, 32>(a, s);
    else if (n_experts <= 128) launch_bwd<4, 32>(a, s);
    else if (n_experts <= 256) launch_bwd<8, 32>(a, s);
    else if (n_experts <= 512) launch_bwd<16, 32>(a, s);
    else launch_bwd<32, 32>(a, s);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
