// The indirect expert product with both operands in MXFP4:
//   dst[t][s] = W[ids[t][s]] . Q(x[t] or x[t][s]),
// Q rounding every 32 consecutive values to one E8M0 scale and E2M1 codes.
// The gather rounds each row while it moves it to its expert's tile rows; the
// rounded values are exact in bf16, so the grouped GEMM of bf16 operands gives
// the product of the rounded operands.
#include "gemm_api.cuh"
#include "mxfp4.cuh"

namespace moe {

moe_status launch_row_ids(const int32_t* ids, int64_t S, int k, int E, int mode, int32_t* ids_src1,
                          int32_t* ids_dst, int32_t* bounds, int32_t* active, int32_t* ntile_prefix,
                          int32_t* pad_start, int32_t* slot_prow, int bn, int* hdr, int32_t* rid_scratch,
                          cudaStream_t stream, int* launches = nullptr);

namespace {

// One warp per slot: eight values per lane, four lanes per block of 32.
__global__ void __launch_bounds__(256)
mx4_gather_kernel(const void* __restrict__ x, int type, int n_in, int KT, const int32_t* __restrict__ slot_prow,
                  int k, int per_slot, int64_t S, int64_t rows_pad, uint8_t* __restrict__ xt, const int* hdr) {
    if (read_status(hdr + kHdrStatus) != 0) return;
    const int lane = threadIdx.x & 31;
    const int esz = type == MOE_F32 ? 4 : 2;
    const int64_t nw = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t p = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); p < S; p += nw) {
        const int64_t row = per_slot ? p : p / k;
        const int prow = __ldg(slot_prow + p);
        for (int s0 = 0; s0 < KT * 8; s0 += 32) {
            const int seg = s0 + lane, col = seg * 8;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (col < n_in) mx_load8<true>((const char*)x + (row * n_in + col) * esz, type, v);
            const uint32_t X = mx_scale_byte(mx_block_bits(v, 0xffffffffu));
            const uint32_t w = X == 255u ? 0u : mx_codes8(v, mx_inv_scale(X));
            mx_values8(w, mx_scale(X), v);
            if (seg < KT * 8) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    h[i] = *(const uint32_t*)&b;
                }
                *(uint4*)(xt + ((size_t)(seg >> 3) * rows_pad + prow) * 128u + (((seg & 7) ^ (prow & 7)) << 4)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mul_mat_id_mx4(const void* W_prepared, int n_experts, int n_out, int n_in, const void* x,
                                         moe_dtype x_type, const int32_t* ids, int64_t n_tokens, int k, moe_mode mode,
                                         float* dst, void* workspace, moe_stream stream) {
    if (n_tokens < 0 || k < 1 || n_experts < 1) return MOE_ERR_INVALID;
    if (n_tokens >= kMaxTokens || k >= kMaxK || k > n_experts) return MOE_ERR_RANGE;
    if (n_tokens * (int64_t)k >= ((int64_t)1 << 31) || n_experts > kMaxExperts) return MOE_ERR_RANGE;
    if (mode != MOE_BROADCAST && mode != MOE_PER_SLOT) return MOE_ERR_INVALID;
    if (x_type != MOE_BF16 && x_type != MOE_F16 && x_type != MOE_F32) return MOE_ERR_INVALID;
    if (n_out <= 0 || n_in <= 0 || n_in % 32) return MOE_ERR_INVALID;
    if (!workspace || ((uintptr_t)workspace & 255u)) return MOE_ERR_INVALID;
    if (n_tokens == 0) return MOE_OK;
    if (!W_prepared || !x || !ids || !dst || ((uintptr_t)W_prepared & 255u)) return MOE_ERR_INVALID;
    if (((uintptr_t)x | (uintptr_t)dst) & 15u) return MOE_ERR_INVALID;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t S = n_tokens * k;
    WsLayout W(n_tokens, k, n_experts, n_in, 0, 0, x_type);
    char* ws = (char*)workspace;
    int* hdr = (int*)(ws + W.hdr);
    prof_begin(s);
    int n_rid = 1;
    moe_status st = launch_row_ids(ids, S, k, n_experts, mode, (int32_t*)(ws + W.src1), (int32_t*)(ws + W.dst),
                                   (int32_t*)(ws + W.bounds), (int32_t*)(ws + W.active), (int32_t*)(ws + W.tiles),
                                   (int32_t*)(ws + W.pad), (int32_t*)(ws + W.sprow), kGemmBN, hdr,
                                   n_experts <= kRidMaxE ? (int32_t*)(ws + W.rid) : nullptr, s, &n_rid);
    if (st) return st;
    prof_mark(s, "row_ids", n_rid);
    const int KT = (n_in + kTileK - 1) / kTileK;
    const int64_t blocks = (S + 7) / 8;
    mx4_gather_kernel<<<(unsigned)(blocks < 148 * 8 ? blocks : 148 * 8), 256, 0, s>>>(
        x, x_type, n_in, KT, (const int32_t*)(ws + W.sprow), k, mode == MOE_PER_SLOT, S, W.rows_pad,
        (uint8_t*)(ws + W.xt), hdr);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    prof_mark(s, "gather");
    GemmMulMatId g = {};
    g.wtype = MOE_MXFP4;
    g.W = (const uint8_t*)W_prepared;
    g.E = n_experts;
    g.n_out = n_out;
    g.n_in = n_in;
    g.xt = ws + W.xt;
    g.xs = (float*)(ws + W.xs);
    g.rows_pad = W.rows_pad;
    g.pad_start = (const int32_t*)(ws + W.pad);
    g.S = S;
    g.dst = dst;
    g.bounds = (const int32_t*)(ws + W.bounds);
    g.ntile_prefix = (const int32_t*)(ws + W.tiles);
    g.ids_src1 = (const int32_t*)(ws + W.src1);
    g.ids_dst = (const int32_t*)(ws + W.dst);
    g.slot_prow = (const int32_t*)(ws + W.sprow);
    g.k = k;
    g.hdr = hdr;
    g.xt_ready = 1;
    return launch_gemm_mul_mat_id(g, s);
}
