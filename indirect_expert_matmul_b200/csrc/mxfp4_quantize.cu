// Quantisation of rows to MXFP4 blocks (17 bytes per 32 values, the layout
// that weights_prepare reads): scale byte X = floor(log2 max|v|) - 2 + 127, then
// 16 bytes holding element i in the low nibble of byte i and element 16 + i in
// its high nibble.  Every step is exact but the rounding to E2M1, so the
// result is a pure function of the values.
//
// Four lanes per block, eight values each; a thread takes its place in kQzUnroll
// blocks, all loads first, and a CTA's blocks are put together in shared memory
// and leave as one contiguous run of bytes.
#include "mxfp4.cuh"

namespace moe {

namespace {

constexpr int kQzThreads = 256;
constexpr int kQzUnroll = 4;
constexpr int kQzBlocks = kQzUnroll * (kQzThreads / 4);  // blocks of a CTA
constexpr int kQzBytes = kQzBlocks * 17;

// nibbles 0..3 of w, one to a byte
__device__ __forceinline__ uint32_t spread4(uint32_t w) {
    w &= 0xffffu;
    w = (w | w << 8) & 0x00ff00ffu;
    return (w | w << 4) & 0x0f0f0f0fu;
}

// CONTIG: the rows have no gaps, block b's values start at 32 b (a division by
// the blocks of a row for each place otherwise).
template <bool VEC, bool CONTIG>
__global__ void __launch_bounds__(kQzThreads)
mxfp4_quantize_kernel(const void* __restrict__ x, int type, int64_t ld, int64_t n_blocks, int nb,
                      uint8_t* __restrict__ out, void* __restrict__ values) {
    __shared__ __align__(16) uint8_t s_out[kQzBytes];
    const int q = threadIdx.x & 3, lb = threadIdx.x >> 2;
    const int64_t b0 = (int64_t)blockIdx.x * kQzBlocks;
    const int esz = type == MOE_F32 ? 4 : 2;
    float v[kQzUnroll][8];
#pragma unroll
    for (int i = 0; i < kQzUnroll; ++i) {
        const int64_t b = b0 + i * (kQzThreads / 4) + lb;
        if (b < n_blocks) {
            int64_t at = b * 32 + q * 8;
            if (!CONTIG) {
                const int64_t row = b / nb;
                at = row * ld + (b - row * nb) * 32 + q * 8;
            }
            mx_load8<VEC>((const char*)x + at * esz, type, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < kQzUnroll; ++i) {
        const int64_t b = b0 + i * (kQzThreads / 4) + lb;
        const uint32_t X = mx_scale_byte(mx_block_bits(v[i], 0xffffffffu));
        const uint32_t w = X == 255u ? 0u : mx_codes8(v[i], mx_inv_scale(X));
        // lanes 0 / 1 hold elements 0-15 (low nibbles), lanes 2 / 3 elements 16-31:
        // lane q writes bytes 8 * (q & 1) + 4 * (q >> 1) .. + 3
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 2);
        const uint32_t lo = q < 2 ? w : o >> 16, hi = q < 2 ? o : w >> 16;
        const uint32_t bytes = spread4(lo) | spread4(hi) << 4;
        uint8_t* dst = s_out + (i * (kQzThreads / 4) + lb) * 17;
        if (q == 0) dst[0] = (uint8_t)X;
        dst += 1 + 8 * (q & 1) + 4 * (q >> 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = (uint8_t)(bytes >> (8 * j));
        if (values && b < n_blocks) {
            float u[8];
            mx_values8(w, mx_scale(X), u);
            char* vp = (char*)values + (b * 32 + q * 8) * esz;  // contiguous rows
            if (type == MOE_F32) {
                __stcs((float4*)vp, make_float4(u[0], u[1], u[2], u[3]));
                __stcs((float4*)vp + 1, make_float4(u[4], u[5], u[6], u[7]));
            } else {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (type == MOE_BF16) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(u[2 * j], u[2 * j + 1]);
                        h[j] = *(const uint32_t*)&p;
                    } else {
                        const __half2 p = __floats2half2_rn(u[2 * j], u[2 * j + 1]);
                        h[j] = *(const uint32_t*)&p;
                    }
                }
                __stcs((uint4*)vp, make_uint4(h[0], h[1], h[2], h[3]));
            }
        }
    }
    __syncthreads();
    const int64_t left = n_blocks - b0;
    const int nbytes = (int)(left < kQzBlocks ? left * 17 : kQzBytes);
    uint8_t* base = out + b0 * 17;
    if (((uintptr_t)base & 15u) == 0) {
        for (int i = threadIdx.x; i < nbytes / 16; i += kQzThreads) ((uint4*)base)[i] = ((const uint4*)s_out)[i];
        for (int i = nbytes / 16 * 16 + threadIdx.x; i < nbytes; i += kQzThreads) base[i] = s_out[i];
    } else {
        for (int i = threadIdx.x; i < nbytes; i += kQzThreads) base[i] = s_out[i];
    }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mxfp4_quantize(const void* x, moe_dtype x_type, int64_t row_stride, int64_t n_rows, int n,
                                         void* blocks, void* values, moe_stream stream) {
    if (x_type != MOE_BF16 && x_type != MOE_F16 && x_type != MOE_F32) return MOE_ERR_INVALID;
    if (n_rows < 0 || n < 1 || n % 32 || row_stride < n) return MOE_ERR_INVALID;
    if (n_rows >= ((int64_t)1 << 31) || row_stride >= ((int64_t)1 << 40)) return MOE_ERR_RANGE;
    const int64_t n_blocks = n_rows * (n / 32);
    if (n_blocks / kQzBlocks >= ((int64_t)1 << 31) - 1) return MOE_ERR_RANGE;
    if (n_rows == 0) return MOE_OK;
    if (!x || !blocks) return MOE_ERR_INVALID;
    const int esz = x_type == MOE_F32 ? 4 : 2;
    if ((uintptr_t)x % esz || ((uintptr_t)values & 15u)) return MOE_ERR_INVALID;
    const bool vec = ((uintptr_t)x & 15u) == 0 && row_stride * esz % 16 == 0;
    const unsigned grid = (unsigned)((n_blocks + kQzBlocks - 1) / kQzBlocks);
    cudaStream_t s = (cudaStream_t)stream;
    const int nb = n / 32;
    uint8_t* out = (uint8_t*)blocks;
    if (!vec) mxfp4_quantize_kernel<false, false><<<grid, kQzThreads, 0, s>>>(x, x_type, row_stride, n_blocks, nb, out, values);
    else if (row_stride == n) mxfp4_quantize_kernel<true, true><<<grid, kQzThreads, 0, s>>>(x, x_type, row_stride, n_blocks, nb, out, values);
    else mxfp4_quantize_kernel<true, false><<<grid, kQzThreads, 0, s>>>(x, x_type, row_stride, n_blocks, nb, out, values);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
