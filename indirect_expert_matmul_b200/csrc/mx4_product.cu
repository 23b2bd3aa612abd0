// The indirect expert product with both operands in MXFP4:
//   dst[t][s] = W[ids[t][s]] . Q(x[t] or x[t][s]),
// Q rounding every 32 consecutive values to one E8M0 scale and E2M1 codes.
//
// Quantising gather: each row is rounded once and its codes go to the tile rows
// of every slot that reads it: [K plane of 256 values][row][128 bytes], 16-byte
// chunk c at c ^ (row % 8) (the 128-byte swizzle); the scales of 128 values of
// a row are one word of [K / 128][row].
//
// Grouped GEMM (tcgen05 kind::mxf4, block scales): a CTA takes units of (up to
// 192 sorted rows of one expert) x (one or two 128-row weight tiles) and streams
// K in stages of 256 values.  The 4-bit weights go from their repacked form
// straight to the tensor cores, no thread touches them.  The codes of a 32-row
// sub-block are 32 rows of 32 bytes, which the MMA reads in the 32-byte swizzle
// (address bit 4 ^= bit 7).  Copied as such, in boxes 32 bytes wide, they kept
// the copy engine busy for ~3.5 cycles a row (567 us for the 4096-token gate
// product); copied as lines of 128 bytes in the 128-byte swizzle (bits 4-6 ^=
// bits 7-9) bit 4 comes out the same and bits 5-6 only permute rows: row r of
// the sub-block lands in row r ^ (r >> 3).  The scales and the epilogue follow
// that order (perm_row).  Four warps move the scales (1/17 of the
// bytes) from shared to tensor memory, one thread issues the copies, one the
// MMAs, and eight warps scatter the accumulators to dst.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "bounded_wait.cuh"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace moe {

moe_status launch_row_ids(const int32_t* ids, int64_t S, int k, int E, int mode, int32_t* ids_src1,
                          int32_t* ids_dst, int32_t* bounds, int32_t* active, int32_t* ntile_prefix,
                          int32_t* pad_start, int32_t* slot_prow, int bn, int* hdr, int32_t* rid_scratch,
                          cudaStream_t stream, int* launches = nullptr);
bool testing_stall_state(int* cta, int* stage, long long* limit_cycles);

namespace {

// ----------------------------------------------------------------- geometry
constexpr int kMxThreads = 512;
constexpr int kMxBN = kGemmBN;    // sorted rows (columns of the accumulator) of a unit
constexpr int kMxStageKt = 4;     // 64-value k-steps of a stage
constexpr int kMxStages = 3;
constexpr uint32_t kMxCodes = kTileM * 32;                 // codes of a tile's k-step
constexpr uint32_t kMxACodes = kMxStageKt * kMxCodes;      // 16384
constexpr uint32_t kMxAScales = kMxStageKt * kTileM * 2;   // 1024
constexpr uint32_t kMxB = kMxBN * 128;                     // 24576
constexpr uint32_t kMxBScales = 2 * kMxBN * 4;             // 1536
constexpr uint32_t kMxStageBytes = 2 * kMxACodes + kMxB + 2 * kMxAScales + kMxBScales;
static_assert(kMxStageBytes % 1024 == 512, "stages are padded to the swizzle's 1024 bytes below");
constexpr uint32_t kMxStagePitch = (kMxStageBytes + 1023) / 1024 * 1024;
constexpr uint32_t kMxOffB = 2 * kMxACodes, kMxOffAS = kMxOffB + kMxB, kMxOffBS = kMxOffAS + 2 * kMxAScales;
constexpr uint32_t kMxBarOff = kMxStages * kMxStagePitch;
constexpr uint32_t kMxSmem = kMxBarOff + 256 + 1024;
// tensor memory: two accumulators, then per stage 16 columns of A scales
// (two tiles x two 128-value halves x four) and 16 of B scales (two halves x eight)
constexpr uint32_t kMxScaleCol0 = 2 * kMxBN;
static_assert(kMxScaleCol0 + kMxStages * 32 <= 512, "accumulators and scales fill tensor memory");
constexpr int kMxSmemGroups = 256;

struct Mx4Params {
    CUtensorMap codes, scales;      // full 128-row tiles
    CUtensorMap t_codes, r_codes;   // last tile: its 32-row sub-blocks, its 16-row sub-block
    const uint8_t* W;
    WLayout L;
    int full_tiles;                 // tiles of 128 rows
    int tail_subs, tail_r;          // last tile: number of 32-row sub-blocks, of 16-row ones (0 or 1)
    int tiles_per_unit;             // 1 or 2
    int n_groups;
    const int32_t *bounds, *ntile_prefix, *pad_start;
    const uint8_t* B;               // codes [plane][rows_pad][128]
    const uint32_t* BS;             // scales [K / 128][scale_ld]
    int64_t rows_pad, scale_ld;
    const int32_t* dst_rows;
    float* out;
    int out_ld;
    int* hdr;
    long long wait_limit;
    int stall_cta, stall_stage;     // test only: that CTA's activation copy of that stage is never issued (-1: off)
};

// The sub-block row that the 128-byte swizzle puts in place r (and back).
__device__ __forceinline__ int perm_row(int r) { return r ^ (r >> 3); }

struct MxTile {
    int e, mu, p0, n, p0pad;
};

__global__ void __launch_bounds__(kMxThreads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4Params p) {
    extern __shared__ uint8_t smem_dyn[];
    __shared__ int s_prefix[kMxSmemGroups + 1];
    __shared__ int s_bounds[kMxSmemGroups + 1];
    __shared__ int s_pad[kMxSmemGroups + 1];
    __shared__ __align__(16) int s_rows[8][kMxBN];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    if (read_status(p.hdr + kHdrStatus) != 0) return;

    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_dyn + 1023) & ~(uintptr_t)1023);
    uint64_t* full = (uint64_t*)(smem + kMxBarOff);  // a stage's copies have landed
    uint64_t* sf_full = full + kMxStages;            // its scales are in tensor memory
    uint64_t* empty = sf_full + kMxStages;           // its MMAs have completed
    uint64_t* acc_full = empty + kMxStages;
    uint64_t* acc_empty = acc_full + 1;
    uint64_t* drained = acc_empty + 1;
    volatile int* abort_flag = &s_abort;
    int* status = p.hdr + kHdrStatus;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WLayout L = p.L;
    const int MT = L.mt_count, KT = L.kt_count, KS = (KT + kMxStageKt - 1) / kMxStageKt;
    const int TPU = p.tiles_per_unit, MU = (MT + TPU - 1) / TPU;
    const bool in_smem = p.n_groups <= kMxSmemGroups;

    if (tid == 0) {
        for (int i = 0; i < kMxStages; ++i) {
            ptx::mbar_init(&full[i], 3);
            ptx::mbar_init(&sf_full[i], 4);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(acc_full, 1);
        ptx::mbar_init(acc_empty, 8);
        ptx::mbar_init(drained, 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, 512);
        ptx::tmem_relinquish();
    }
    if (in_smem)
        for (int i = tid; i <= p.n_groups; i += kMxThreads) {
            s_prefix[i] = p.ntile_prefix[i];
            s_bounds[i] = p.bounds[i];
            s_pad[i] = p.pad_start[i];
        }
    const int total = p.hdr[kHdrTiles] * MU;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_tmem;

    auto unit = [&](int t) {
        MxTile r;
        const int q = t / MU;
        r.mu = t - q * MU;
        const int* pre = in_smem ? s_prefix : p.ntile_prefix;
        const int* bnd = in_smem ? s_bounds : p.bounds;
        const int* pad = in_smem ? s_pad : p.pad_start;
        int lo = 0, hi = p.n_groups;  // pre[lo] <= q < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= q) lo = mid; else hi = mid;
        }
        r.e = lo;
        const int j = q - pre[lo];
        r.p0 = bnd[lo] + j * kMxBN;
        r.p0pad = pad[lo] + j * kMxBN;
        r.n = min(kMxBN, bnd[lo + 1] - r.p0);
        return r;
    };

    // One k-step of the last, partial tile: its 32-row sub-blocks' codes in one
    // tensor copy, its 16-row sub-block's in another, the scales by sub-block
    // (a tensor copy's destination would need 128-byte alignment).
    auto load_tail = [&](uint8_t* codes, uint8_t* scales, int e, int kt, uint64_t* bar) {
        const uint8_t* src = p.W + L.block(e, MT - 1, kt);
        if (p.tail_subs) ptx::tma_load_5d(codes, &p.t_codes, 0, 0, 0, kt, e, bar);
        if (p.tail_r) ptx::tma_load_5d(codes + p.tail_subs * 1024, &p.r_codes, 0, 0, 0, kt, e, bar);
        for (int sb = 0; sb < p.tail_subs; ++sb)
            ptx::bulk_g2s(scales + sb * 64, src + sb * (kSubRows * kRowBytesMx) + kSubRows * 32, kSubRows * 2, bar);
        if (p.tail_r)
            ptx::bulk_g2s(scales + p.tail_subs * 64, src + p.tail_subs * (kSubRows * kRowBytesMx) + 16 * 32, 16 * 2,
                          bar);
    };

    if (warp == 0 || warp == 2 || warp == 3) {
        // ------------------------------------------------------------ copies
        // Warps 0 and 2: the codes and scales of the unit's first and second
        // weight tile; warp 3: the rows' codes and scales.  One thread issuing all
        // of a stage's copies needed ~1300 cycles for it, twice the MMAs' time.
        const uint32_t issue = ptx::elect_one();
        const int i = warp >> 1;  // weight tile of warps 0 and 2
        int s = 0, q = 0;
        uint32_t ph = 0, used = 0, par = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const MxTile u = unit(t);
            const uint32_t n16 = (uint32_t)(u.n + 15) & ~15u;
            const int mt = u.mu * TPU + i;
            const uint8_t* bsrc = p.B + (size_t)u.p0pad * 128u;
            const uint32_t* ssrc = p.BS + u.p0pad;
            for (int ks = 0; ks < KS; ++ks, ++q) {
                ok = warp_wait(&empty[s], ph ^ 1, abort_flag, status, p.wait_limit);
                if (!ok) break;
                uint8_t* st = smem + s * kMxStagePitch;
                const int kts = min(kMxStageKt, KT - ks * kMxStageKt), halves = (kts + 1) / 2;
                if (warp == 3) {
                    const bool stalled = (int)blockIdx.x == p.stall_cta && q == p.stall_stage;
                    if (issue && !stalled) {
                        ptx::mbar_arrive_expect_tx(&full[s], n16 * 128u + halves * n16 * 4u);
                        ptx::bulk_g2s(st + kMxOffB, bsrc, n16 * 128u, &full[s]);
                        ptx::bulk_g2s(st + kMxOffBS, ssrc, n16 * 4u, &full[s]);
                        if (halves == 2)
                            ptx::bulk_g2s(st + kMxOffBS + kMxBN * 4, ssrc + p.scale_ld, n16 * 4u, &full[s]);
                    }
                    bsrc += (size_t)p.rows_pad * 128u;
                    ssrc += 2 * p.scale_ld;
                    if (!stalled) {
                        used |= 1u << s;
                        par = (par & ~(1u << s)) | (ph << s);
                    }
                } else if (issue) {
                    uint8_t* ac = st + i * kMxACodes;
                    uint8_t* as = st + kMxOffAS + i * kMxAScales;
                    if (i < TPU && mt < p.full_tiles) {
                        ptx::mbar_arrive_expect_tx(&full[s], kMxACodes + kMxAScales);
                        ptx::tma_load_5d(ac, &p.codes, 0, 0, ks * kMxStageKt * 4, mt, u.e, &full[s]);
                        ptx::tma_load_4d(as, &p.scales, 0, ks * kMxStageKt * 4, mt, u.e, &full[s]);
                    } else if (i < TPU && mt < MT) {
                        ptx::mbar_arrive_expect_tx(&full[s], (uint32_t)(kts * L.rows(mt) * kRowBytesMx));
                        for (int j = 0; j < kts; ++j)
                            load_tail(ac + j * kMxCodes, as + j * 256, u.e, ks * kMxStageKt + j, &full[s]);
                    } else {
                        ptx::mbar_arrive(&full[s]);
                    }
                }
                if (++s == kMxStages) { s = 0; ph ^= 1; }
            }
        }
        // let every copy issued land before the CTA can exit (bounded): a stage
        // completes when all three warps' copies have
        if (warp == 3) {
            volatile int never = 0;
            for (int j = 0; j < kMxStages; ++j)
                if (used >> j & 1) warp_wait(&full[j], (par >> j) & 1, &never, status, p.wait_limit);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMAs
        const uint32_t issue = ptx::elect_one(), smem_a = ptx::smem_u32(smem);
        int s = 0;
        uint32_t ph = 0, use = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const MxTile u = unit(t);
            const int n16 = (u.n + 15) & ~15;
            const uint32_t id0 = ptx::idesc_mxf4(n16, 0), id1 = ptx::idesc_mxf4(n16, 1);
            const bool two = TPU == 2 && u.mu * 2 + 1 < MT;
            ok = warp_wait(acc_empty, (use & 1) ^ 1, abort_flag, status, p.wait_limit);
            if (!ok) break;
            use += 1;
            for (int ks = 0; ks < KS; ++ks) {
                ok = warp_wait(&full[s], ph, abort_flag, status, p.wait_limit) &&
                     warp_wait(&sf_full[s], ph, abort_flag, status, p.wait_limit);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t st = smem_a + (uint32_t)s * kMxStagePitch;
                const uint32_t sf = tmem + kMxScaleCol0 + (uint32_t)s * 32u;
                const uint64_t ad = ptx::desc_k_sw32(st), bd = ptx::desc_k_sw128(st + kMxOffB);
                const int kts = KT - ks * kMxStageKt;
#pragma unroll
                for (int j = 0; j < kMxStageKt; ++j) {
                    if (j < kts) {  // address fields count 16 bytes; sums stay inside their 14 bits
                        const uint32_t id = j & 1 ? id1 : id0;
                        ptx::mma_mxf4_ss(tmem, ad + (j * kMxCodes >> 4), bd + j * 2, id, sf + (j >> 1) * 4,
                                         sf + 16 + (j >> 1) * 8, (ks | j) != 0, issue);
                        if (two)
                            ptx::mma_mxf4_ss(tmem + kMxBN, ad + ((kMxACodes + j * kMxCodes) >> 4), bd + j * 2, id,
                                             sf + 8 + (j >> 1) * 4, sf + 16 + (j >> 1) * 8, (ks | j) != 0, issue);
                    }
                }
                if (issue) ptx::mma_commit(&empty[s]);
                __syncwarp();
                if (++s == kMxStages) { s = 0; ph ^= 1; }
            }
            if (!ok) break;
            if (issue) ptx::mma_commit(acc_full);
            __syncwarp();
        }
        // every MMA issued has completed before the CTA can release tensor memory
        if (issue) {
            ptx::mma_commit(drained);
            volatile int never = 0;
            wait_bar(drained, 0, &never, status, p.wait_limit);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------- scales, per stage
        // Every warp writes its quarter of the lanes with the same words: lane r
        // holds rows r, 32 + r, ... of a tile (or of the sorted rows), one column each.
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        const uint32_t dst = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + kMxScaleCol0;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            for (int ks = 0; ks < KS; ++ks) {
                ok = warp_wait(&full[s], ph, abort_flag, status, p.wait_limit);
                if (!ok) break;
                const uint32_t as = ptx::smem_u32(smem + s * kMxStagePitch + kMxOffAS) + perm_row(lane) * 2;
                const uint32_t bs = ptx::smem_u32(smem + s * kMxStagePitch + kMxOffBS) + lane * 4;
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int sb = 0; sb < 4; ++sb) {
                            const uint32_t a = as + i * kMxAScales + h * 512 + sb * 64;
                            v[i * 8 + h * 4 + sb] = ptx::lds16(a) | ptx::lds16(a + 256) << 16;
                        }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        v[16 + h * 8 + c] = c < kMxBN / 32 ? ptx::lds32(bs + h * (kMxBN * 4) + c * 128) : 0u;
                ptx::tc_fence_after();
                ptx::tmem_st_32x32b_x32(dst + (uint32_t)s * 32u, v);
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sf_full[s]);
                if (++s == kMxStages) { s = 0; ph ^= 1; }
            }
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------- epilogue
        // Warps 8-11 drain the first tile's accumulator, 12-15 the second's.
        const int wq = warp & 3, i = (warp - 8) >> 2;
        int* rows = s_rows[warp - 8];  // the warp's copy of the unit's output rows
        uint32_t use = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            const MxTile u = unit(t);
            const int mt = u.mu * TPU + i;
            const bool live = i < TPU && mt < MT;
            __syncwarp();
            for (int c = lane; c < u.n; c += 32) rows[c] = __ldg(p.dst_rows + u.p0 + c);
            __syncwarp();
            if (!warp_wait(acc_full, use & 1, abort_flag, status, p.wait_limit)) break;
            use += 1;
            ptx::tc_fence_after();
            if (live) {
                const int m = mt * kTileM + 32 * wq + perm_row(lane);
                const bool m_ok = m < L.n_out;
                float* out = p.out + m;
                // A column is a sorted row: its 32 lanes are 128 consecutive bytes of one
                // row of dst.  The rows' numbers come from shared memory, four to a load: by
                // shuffles under a test a column cost 105 cycles (20000 a unit) against ~25.
                for (int c0 = 0; c0 < u.n; c0 += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * wq) << 16) + i * kMxBN + c0, v);
                    ptx::tmem_ld_wait();
                    if (!m_ok) continue;
                    if (c0 + 32 <= u.n) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const int4 r = *(const int4*)(rows + c0 + j);
                            out[(int64_t)r.x * p.out_ld] = __uint_as_float(v[j]);
                            out[(int64_t)r.y * p.out_ld] = __uint_as_float(v[j + 1]);
                            out[(int64_t)r.z * p.out_ld] = __uint_as_float(v[j + 2]);
                            out[(int64_t)r.w * p.out_ld] = __uint_as_float(v[j + 3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < u.n) out[(int64_t)rows[c0 + j] * p.out_ld] = __uint_as_float(v[j]);
                    }
                }
                __syncwarp();
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(acc_empty);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------- quantising gather
// One warp per source row (broadcast: a token, whose codes go to the tile rows
// of its k slots; per slot: one slot): eight values a lane, four lanes a block.
__global__ void __launch_bounds__(256)
mx4_gather_kernel(const void* __restrict__ x, int type, int n_in, const int32_t* __restrict__ slot_prow, int copies,
                  int64_t n_rows, int64_t rows_pad, int64_t scale_ld, uint8_t* __restrict__ codes,
                  uint32_t* __restrict__ scales, const int* hdr) {
    if (read_status(hdr + kHdrStatus) != 0) return;
    const int lane = threadIdx.x & 31;
    const int esz = type == MOE_F32 ? 4 : 2;
    const int planes = (n_in + 255) / 256;
    const int64_t nw = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); r < n_rows; r += nw) {
        const int32_t* pr = slot_prow + r * copies;
        for (int kp = 0; kp < planes; ++kp) {
            const int col = kp * 256 + lane * 8;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (col < n_in) mx_load8<true>((const char*)x + (r * n_in + col) * esz, type, v);
            const uint32_t X = mx_scale_byte(mx_block_bits(v, 0xffffffffu));
            const uint32_t w = X == 255u ? 0u : mx_codes8(v, mx_inv_scale(X));
            uint32_t sw = X << (8 * ((lane >> 2) & 3));  // the scales of this half's four blocks in one word
            sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
            sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
            const bool sc = (lane & 15) == 0 && col < n_in;
            uint8_t* plane = codes + (size_t)kp * rows_pad * 128u + (lane & 3) * 4;
            uint32_t* sp = scales + (size_t)(2 * kp + (lane >> 4)) * scale_ld;
            for (int j = 0; j < copies; ++j) {
                const int prow = __ldg(pr + j);
                *(uint32_t*)(plane + (size_t)prow * 128u + (((lane >> 2) ^ (prow & 7)) << 4)) = w;
                if (sc) sp[prow] = sw;
            }
        }
    }
}

// ------------------------------------------------------------------- host
int mx_sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && (n = cached[dev].load()) > 0) return n;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
    if (dev >= 0 && dev < 64) cached[dev].store(n);
    return n;
}

PFN_cuTensorMapEncodeTiled_v12000 mx_encoder() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load();
    if (fn) return fn;
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    cached.store(fn);
    return fn;
}

bool encode(CUtensorMap* m, const uint8_t* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    auto enc = mx_encoder();
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<uint8_t*>(base), dims, strides,
                      box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The repacked MXFP4 form as tensors of bytes.  A 32-row sub-block of a k-step
// is 1088 bytes: 32 rows of 32 code bytes (eight lines of 128), then 64 scale
// bytes; a full tile's k-steps and sub-blocks follow one another, so they are
// one dimension.
bool plan_weights(Mx4Params& p, int n_experts) {
    const WLayout& L = p.L;
    const cuuint64_t sub = kSubRows * kRowBytesMx, ex = (cuuint64_t)L.expert_bytes, KT = (cuuint64_t)L.kt_count;
    p.full_tiles = L.n_out_pad / kTileM;
    const int tail = L.n_out_pad % kTileM;
    p.tail_subs = tail / kSubRows;
    p.tail_r = tail % kSubRows != 0;
    if (p.full_tiles) {
        const cuuint64_t tile = kTileM * KT * kRowBytesMx;
        const cuuint64_t cd[5] = {128, 8, KT * 4, (cuuint64_t)p.full_tiles, (cuuint64_t)n_experts};
        const cuuint64_t cs[4] = {128, sub, tile, ex};
        const cuuint32_t cb[5] = {128, 8, kMxStageKt * 4, 1, 1};
        const cuuint64_t sd[4] = {64, KT * 4, (cuuint64_t)p.full_tiles, (cuuint64_t)n_experts};
        const cuuint64_t ss[3] = {sub, tile, ex};
        const cuuint32_t sb[4] = {64, kMxStageKt * 4, 1, 1};
        if (!encode(&p.codes, p.W, 5, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode(&p.scales, p.W + kSubRows * 32, 4, sd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE))
            return false;
    }
    const uint8_t* last = p.W + L.block(0, L.mt_count - 1, 0);
    const cuuint64_t step = (cuuint64_t)tail * kRowBytesMx;
    if (p.tail_subs) {
        const cuuint64_t d[5] = {128, 8, (cuuint64_t)p.tail_subs, KT, (cuuint64_t)n_experts};
        const cuuint64_t s[4] = {128, sub, step, ex};
        const cuuint32_t b[5] = {128, 8, (cuuint32_t)p.tail_subs, 1, 1};
        if (!encode(&p.t_codes, last, 5, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    }
    if (p.tail_r) {
        const cuuint64_t d[5] = {128, 4, 1, KT, (cuuint64_t)n_experts};
        const cuuint64_t s[4] = {128, step, step, ex};
        const cuuint32_t b[5] = {128, 4, 1, 1, 1};
        if (!encode(&p.r_codes, last + p.tail_subs * sub, 5, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    }
    return true;
}

moe_status launch_mx4_gemm(Mx4Params& p, int64_t max_coltiles, cudaStream_t stream) {
    p.wait_limit = kWaitLimitCycles;
    p.stall_cta = -1;
    p.stall_stage = 0;
    long long limit = 0;
    if (testing_stall_state(&p.stall_cta, &p.stall_stage, &limit)) p.wait_limit = limit;
    if (cudaFuncSetAttribute(mx4_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMxSmem) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    const int64_t units = max_coltiles * ((p.L.mt_count + p.tiles_per_unit - 1) / p.tiles_per_unit);
    const int sms = mx_sm_count();
    const unsigned grid = (unsigned)(units < sms ? units : sms);
    mx4_gemm_kernel<<<grid, kMxThreads, kMxSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    Mx4Params p = {};
    p.W = (const uint8_t*)W_prepared;
    p.L = WLayout(n_out, n_in, MOE_MXFP4);
    if (!plan_weights(p, n_experts)) return MOE_ERR_CUDA;
    prof_begin(s);
    int n_rid = 1;
    moe_status st = launch_row_ids(ids, S, k, n_experts, mode, (int32_t*)(ws + W.src1), (int32_t*)(ws + W.dst),
                                   (int32_t*)(ws + W.bounds), (int32_t*)(ws + W.active), (int32_t*)(ws + W.tiles),
                                   (int32_t*)(ws + W.pad), (int32_t*)(ws + W.sprow), kMxBN, hdr,
                                   n_experts <= kRidMaxE ? (int32_t*)(ws + W.rid) : nullptr, s, &n_rid);
    if (st) return st;
    prof_mark(s, "row_ids", n_rid);
    // The rounded rows take the workspace of the 16-bit ones: 128 bytes per 256
    // values and 4 per 128 where those take 128 per 64.  Only up to 64 values do
    // the scales not fit behind the codes; there they take the rows' factors.
    uint8_t* codes = (uint8_t*)(ws + W.xt);
    uint32_t* scales = n_in <= kTileK ? (uint32_t*)(ws + W.xs)
                                      : (uint32_t*)(codes + (size_t)((n_in + 255) / 256) * W.rows_pad * 128u);
    const int64_t scale_ld = (W.rows_pad + 3) / 4 * 4;  // bulk copies start on 16 bytes
    const int64_t rows = mode == MOE_BROADCAST ? n_tokens : S, blocks = (rows + 7) / 8;
    const int64_t cap = (int64_t)mx_sm_count() * 8;
    mx4_gather_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(
        x, x_type, n_in, (const int32_t*)(ws + W.sprow), mode == MOE_BROADCAST ? k : 1, rows, W.rows_pad, scale_ld,
        codes, scales, hdr);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    prof_mark(s, "gather");
    p.tiles_per_unit = 2;
    p.n_groups = n_experts;
    p.bounds = (const int32_t*)(ws + W.bounds);
    p.ntile_prefix = (const int32_t*)(ws + W.tiles);
    p.pad_start = (const int32_t*)(ws + W.pad);
    p.B = codes;
    p.BS = scales;
    p.rows_pad = W.rows_pad;
    p.scale_ld = scale_ld;
    p.dst_rows = (const int32_t*)(ws + W.dst);
    p.out = dst;
    p.out_ld = n_out;
    p.hdr = hdr;
    st = launch_mx4_gemm(p, (S + kMxBN - 1) / kMxBN + (S < n_experts ? S : n_experts), s);
    prof_mark(s, "gemm");
    return st;
}
