// Quantisation of rows to MXFP4 blocks (17 bytes per 32 values, the layout
// that weights_prepare reads): scale byte X = floor(log2 max|v|) - 2 + 127, then
// 16 bytes holding element i in the low nibble of byte i and element 16 + i in
// its high nibble.  Every step is exact but the rounding to E2M1, so the
// result is a pure function of the values.
//
// Four lanes per block; lane q takes elements 4q .. 4q+3 and 16+4q .. 16+4q+3, so
// that a conversion of the pair (i, 16 + i) gives byte i whole.  A thread takes
// its place in kQzUnroll blocks, all loads first; a CTA's blocks are put
// together in shared memory and leave as one contiguous run of bytes.
//
// Bytes are the bound, but instructions come close (with eight consecutive
// elements a lane, nibbles spread and exchanged, and values taken through
// float, 64 x 1408 x 2048 bf16 with values took 178 us): 16-bit types find
// their maximum packed, and bf16 values come from a byte table.
#include "mxfp4.cuh"

namespace moe {

namespace {

constexpr int kQzThreads = 256;
constexpr int kQzUnroll = 4;
constexpr int kQzBlocks = kQzUnroll * (kQzThreads / 4);  // blocks of a CTA
constexpr int kQzBytes = kQzBlocks * 17;

// A lane's eight elements: words as they lie in memory.
template <int TYPE>
struct Eight {
    static constexpr int kHalf = TYPE == MOE_F32 ? 4 : 2;  // words of four elements
    uint32_t w[2 * kHalf];

    template <bool VEC>
    __device__ __forceinline__ void load(const void* x, int64_t at) {
        const char* p = (const char*)x + at * (TYPE == MOE_F32 ? 4 : 2);
#pragma unroll
        for (int h = 0; h < 2; ++h, p += 16 * (TYPE == MOE_F32 ? 4 : 2)) {
            if constexpr (TYPE == MOE_F32) {
                if (VEC) {
                    const uint4 v = __ldcs((const uint4*)p);
                    w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[4 * h + i] = __ldg((const uint32_t*)p + i);
                }
            } else {
                if (VEC) {
                    const uint2 v = __ldcs((const uint2*)p);
                    w[2 * h] = v.x; w[2 * h + 1] = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[2 * h + i] = __ldg((const uint16_t*)p + 2 * i) |
                                       (uint32_t)__ldg((const uint16_t*)p + 2 * i + 1) << 16;
                }
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 2 * kHalf; ++i) w[i] = 0u;
    }
    // element i of half h as float
    __device__ __forceinline__ float get(int h, int i) const {
        if constexpr (TYPE == MOE_F32) {
            return __uint_as_float(w[4 * h + i]);
        } else {
            const uint32_t v = w[2 * h + i / 2];
            return TYPE == MOE_BF16 ? __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16)
                                    : __half2float(__ushort_as_half((unsigned short)(i & 1 ? v >> 16 : v & 0xffffu)));
        }
    }
    // the largest magnitude's bits as a float's
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0u;
        if constexpr (TYPE == MOE_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            m = max(m >> 16, m & 0xffffu);
            return TYPE == MOE_BF16 ? m << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
        }
    }
};

// CONTIG: the rows have no gaps, block b's values start at 32 b (a division by
// the blocks of a row for each place otherwise).
template <int TYPE, bool VEC, bool CONTIG>
__global__ void __launch_bounds__(kQzThreads)
mxfp4_quantize_kernel(const void* __restrict__ x, int64_t ld, int64_t n_blocks, int nb, uint8_t* __restrict__ out,
                      void* __restrict__ values) {
    __shared__ __align__(16) uint8_t s_out[kQzBytes];
    const int q = threadIdx.x & 3, lb = threadIdx.x >> 2;
    const int64_t b0 = (int64_t)blockIdx.x * kQzBlocks;
    Eight<TYPE> v[kQzUnroll];
#pragma unroll
    for (int i = 0; i < kQzUnroll; ++i) {
        const int64_t b = b0 + i * (kQzThreads / 4) + lb;
        if (b < n_blocks) {
            int64_t at = b * 32 + q * 4;
            if (!CONTIG) {
                const int64_t row = b / nb;
                at = row * ld + (b - row * nb) * 32 + q * 4;
            }
            v[i].template load<VEC>(x, at);
        } else {
            v[i].zero();
        }
    }
#pragma unroll
    for (int i = 0; i < kQzUnroll; ++i) {
        const int64_t b = b0 + i * (kQzThreads / 4) + lb;
        uint32_t m = v[i].amax_bits();
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t X = mx_scale_byte(m);
        const float inv = mx_inv_scale(X);
        float e[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[2 * j] = v[i].get(0, j);
            e[2 * j + 1] = v[i].get(1, j);
        }
        const uint32_t w = X == 255u ? 0u : mx_codes8(e, inv);  // byte j: elements j (low) and 16 + j
        uint8_t* dst = s_out + (i * (kQzThreads / 4) + lb) * 17;
        if (q == 0) dst[0] = (uint8_t)X;
        dst += 1 + 4 * q;
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = (uint8_t)(w >> (8 * j));
        if (values && b < n_blocks) {
            const int64_t at = b * 32 + q * 4;  // contiguous rows
            if constexpr (TYPE == MOE_BF16) {
                // magnitudes 0 .. 6 as bf16, by byte; the scale is a bf16 power of two and
                // the product has two significant bits: exact.  Signs are the elements' own.
                const uint32_t c0 = w & 0x7777u, c1 = w >> 16 & 0x7777u;
                const uint32_t l0 = __byte_perm(0xc0800000u, 0xc0804000u, c0), l1 = __byte_perm(0xc0800000u, 0xc0804000u, c1);
                const uint32_t h0 = __byte_perm(0x3f3f3f00u, 0x40404040u, c0), h1 = __byte_perm(0x3f3f3f00u, 0x40404040u, c1);
                uint32_t p[4] = {__byte_perm(l0, h0, 0x6240), __byte_perm(l1, h1, 0x6240), __byte_perm(l0, h0, 0x7351),
                                 __byte_perm(l1, h1, 0x7351)};
                const uint32_t sc = X == 0u ? 0x0040u : X == 255u ? 0x7fc0u : X << 7;
                const uint32_t s2 = sc | sc << 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[j] |= v[i].w[j] & 0x80008000u;
                    const __nv_bfloat162 r = __hmul2(*(const __nv_bfloat162*)&p[j], *(const __nv_bfloat162*)&s2);
                    p[j] = *(const uint32_t*)&r;
                }
                char* vp = (char*)values + at * 2;
                __stcs((uint2*)vp, make_uint2(p[0], p[1]));
                __stcs((uint2*)(vp + 32), make_uint2(p[2], p[3]));
            } else {
                float u[8];
                mx_values8(w, mx_scale(X), u);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (TYPE == MOE_F32) {
                        __stcs((float4*)((float*)values + at + 16 * h), make_float4(u[h], u[2 + h], u[4 + h], u[6 + h]));
                    } else {
                        const __half2 a = __floats2half2_rn(u[h], u[2 + h]), c = __floats2half2_rn(u[4 + h], u[6 + h]);
                        __stcs((uint2*)((uint16_t*)values + at + 16 * h),
                               make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&c));
                    }
                }
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

template <int TYPE>
void launch(bool vec, const void* x, int64_t ld, int64_t n_blocks, int nb, uint8_t* out, void* values, cudaStream_t s) {
    const unsigned grid = (unsigned)((n_blocks + kQzBlocks - 1) / kQzBlocks);
    if (!vec) mxfp4_quantize_kernel<TYPE, false, false><<<grid, kQzThreads, 0, s>>>(x, ld, n_blocks, nb, out, values);
    else if (ld == (int64_t)nb * 32)
        mxfp4_quantize_kernel<TYPE, true, true><<<grid, kQzThreads, 0, s>>>(x, ld, n_blocks, nb, out, values);
    else mxfp4_quantize_kernel<TYPE, true, false><<<grid, kQzThreads, 0, s>>>(x, ld, n_blocks, nb, out, values);
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
    cudaStream_t s = (cudaStream_t)stream;
    if (x_type == MOE_BF16) launch<MOE_BF16>(vec, x, row_stride, n_blocks, n / 32, (uint8_t*)blocks, values, s);
    else if (x_type == MOE_F16) launch<MOE_F16>(vec, x, row_stride, n_blocks, n / 32, (uint8_t*)blocks, values, s);
    else launch<MOE_F32>(vec, x, row_stride, n_blocks, n / 32, (uint8_t*)blocks, values, s);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
