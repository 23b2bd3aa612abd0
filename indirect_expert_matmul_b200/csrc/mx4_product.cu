// The indirect expert product with both operands in MXFP4:
//   dst[t][s] = W[ids[t][s]] . Q(x[t] or x[t][s]),
// Q rounding every 32 consecutive values to one E8M0 scale and E2M1 codes.
//
// Rounding: each row is rounded once and its codes go to the tile rows of every
// slot that reads it: [plane of 256 values][row][128 bytes], the 16-byte chunk
// of block c at c ^ (row % 8) (the 128-byte swizzle); its scales are two words a
// plane, [plane][row].
//
// Grouped GEMM (tcgen05 kind::mxf4, block scales): a pair of CTAs takes units of
// (up to 192 sorted rows of one expert) x (two 128-row weight tiles, one a CTA)
// and streams K in stages of 256 values.  A pair MMA reads both CTAs' tiles and
// half of the rows from each, so that an SM fetches a tile and half the rows for
// 128 x 192 results - as little as a 256 x 192 unit of one CTA would - and its
// tensor memory has room for two accumulators: one is drained while the next
// fills.  (One CTA a unit stopped for the drain, 6000 of 20000 cycles; the GEMM
// of the 4096-token gate product took 410 us, against 382.)
//
// The 4-bit weights go from their repacked form to the tensor cores without
// passing through threads.  The codes of a 32-row sub-block are 32 rows of 32
// bytes, which the MMA reads in the 32-byte swizzle (address bit 4 ^= bit 7).
// Copied as lines of 128 bytes in the 128-byte swizzle (bits 4-6 ^= bits 7-9)
// bit 4 comes out the same and bits 5-6 only permute rows: row r of the
// sub-block lands in row r ^ (r >> 3), and the scales and the drain follow that
// order (perm_row).  (Copied in boxes 32 bytes wide the first kernel took 567 us
// for that product, in lines 528.)  Four warps move the weights' and the rows'
// scales from shared to tensor memory, two issue the copies, one thread the
// MMAs, one warp finds the units, four scatter the accumulators to dst.
//
// What bounds it: the gate product (256 experts, 4096 tokens top-8, 7168 -> 2048:
// 2.0 GB of weights, 0.27 of results, 0.12 of rounded rows) takes 377 us, 6.4 TB/s
// where a copy reaches 6.46, and 419 to 440 where the power limit holds the SM clock at
// 1.3 GHz.  A product whose experts' weights are read again from L2 (128 experts,
// 8192 tokens top-4, 2880 -> 2880: 229 us, 259 in long runs) is bound by the way of a
// stage through copies, scales and MMAs, 7 in flight: ~770 cycles a stage, of which ~260 are
// MMAs; DRAM is at half its rate.  Weights asked into L2 ahead (by bulk prefetches
// or by a warp's) made both slower: 274 and 426 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "bounded_wait.cuh"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "warp_match.cuh"

namespace moe {

moe_status launch_row_ids(const int32_t* ids, int64_t S, int k, int E, int mode, int32_t* ids_src1,
                          int32_t* ids_dst, int32_t* bounds, int32_t* active, int32_t* ntile_prefix,
                          int32_t* pad_start, int32_t* slot_prow, int bn, int* hdr, int32_t* rid_scratch,
                          cudaStream_t stream, int* launches = nullptr);
bool testing_stall_state(int* cta, int* stage, long long* limit_cycles);

namespace {

// ----------------------------------------------------------------- geometry
constexpr int kMxThreads = 384;
constexpr int kMxBN = kGemmBN;    // sorted rows (columns of the accumulator) of a unit
constexpr int kMxStageKt = 4;     // 64-value k-steps of a stage
constexpr int kMxDrains = 4;      // warps that drain the accumulators
constexpr int kMxStages = 7;
constexpr int kMxScaleSlots = 5;  // stages whose scales have a place in tensor memory
constexpr uint32_t kMxCodes = kTileM * 32;                 // codes of a tile's k-step
constexpr uint32_t kMxACodes = kMxStageKt * kMxCodes;      // 16384
constexpr uint32_t kMxAScales = kMxStageKt * kTileM * 2;   // 1024
constexpr uint32_t kMxB = kMxBN / 2 * 128;                 // 12288: half the rows
constexpr uint32_t kMxBScales = kMxBN * 8;                 // 1536: every row's two words
constexpr uint32_t kMxOffB = kMxACodes, kMxOffAS = kMxOffB + kMxB, kMxOffBS = kMxOffAS + kMxAScales;
constexpr uint32_t kMxStagePitch = (kMxOffBS + kMxBScales + 1023) / 1024 * 1024;
constexpr int kMxUnits = 2;       // units known ahead
constexpr uint32_t kMxBarOff = kMxStages * kMxStagePitch;
constexpr uint32_t kMxBars = 3 * kMxStages + 4 + 4 * kMxUnits + 1;
constexpr uint32_t kMxSmem = kMxBarOff + kMxBars * 8 + 1024;
// tensor memory: two accumulators, then per slot 8 columns of A scales (two
// 128-value halves x four) and 16 of B scales (two halves x eight)
constexpr uint32_t kMxScaleCol0 = 2 * kMxBN, kMxScaleCols = 24;
static_assert(kMxScaleCol0 + kMxScaleSlots * kMxScaleCols <= 512, "accumulators and scales fill tensor memory");
constexpr int kMxSmemGroups = 256;

struct Mx4Params {
    CUtensorMap codes, scales;      // full 128-row tiles
    CUtensorMap t_codes, r_codes;   // last tile: its 32-row sub-blocks, its 16-row sub-block
    const uint8_t* W;
    WLayout L;
    int full_tiles;                 // tiles of 128 rows
    int tail_subs, tail_r;          // last tile: number of 32-row sub-blocks, of 16-row ones (0 or 1)
    int n_groups;
    const int32_t *bounds, *ntile_prefix, *pad_start;
    const uint8_t* B;               // codes [plane][rows_pad][128]
    const uint2* BS;                // scales [plane][scale_ld]
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

// One thread: the copies of a 128-row tile's stage (codes to `codes`, 4096 bytes
// a k-step; scales to `scales`, 256 bytes a k-step) and their arrival on `bar`.
// Of the last, partial tile a k-step is one copy of its 32-row sub-blocks'
// codes, one of its 16-row sub-block's, and the scales by sub-block (a tensor
// copy's destination would need 128-byte alignment).
template <int STAGE_KT>
__device__ __forceinline__ void load_weights(const Mx4Params& p, const WLayout& L, uint8_t* codes, uint8_t* scales, int e,
                                             int mt, int ks, uint64_t* bar) {
    if (mt < p.full_tiles) {
        ptx::mbar_arrive_expect_tx(bar, STAGE_KT * (kMxCodes + 256));
        ptx::tma_load_5d(codes, &p.codes, 0, 0, ks * STAGE_KT * 4, mt, e, bar);
        ptx::tma_load_4d(scales, &p.scales, 0, ks * STAGE_KT * 4, mt, e, bar);
        return;
    }
    const int kts = min(STAGE_KT, L.kt_count - ks * STAGE_KT);
    ptx::mbar_arrive_expect_tx(bar, (uint32_t)(kts * L.rows(mt) * kRowBytesMx));
    for (int j = 0; j < kts; ++j, codes += kMxCodes, scales += 256) {
        const int kt = ks * STAGE_KT + j;
        const uint8_t* src = p.W + L.block(e, mt, kt);
        if (p.tail_subs) ptx::tma_load_5d(codes, &p.t_codes, 0, 0, 0, kt, e, bar);
        if (p.tail_r) ptx::tma_load_5d(codes + p.tail_subs * 1024, &p.r_codes, 0, 0, 0, kt, e, bar);
        for (int sb = 0; sb < p.tail_subs; ++sb)
            ptx::bulk_g2s(scales + sb * 64, src + sb * (kSubRows * kRowBytesMx) + kSubRows * 32, kSubRows * 2, bar);
        if (p.tail_r)
            ptx::bulk_g2s(scales + p.tail_subs * 64, src + p.tail_subs * (kSubRows * kRowBytesMx) + 16 * 32, 16 * 2, bar);
    }
}

// The scales of a 128-row tile's stage at `as` as this lane's eight words of
// tensor memory (two 128-value halves x four rows 32 apart).
__device__ __forceinline__ void weight_scales(uint32_t as, int lane, uint32_t* v) {
    as += perm_row(lane) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int sb = 0; sb < 4; ++sb) {
            const uint32_t a = as + h * 512 + sb * 64;
            v[h * 4 + sb] = ptx::lds16(a) | ptx::lds16(a + 256) << 16;
        }
}

// A value that is the same in all lanes, so that the compiler knows it.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

struct MxTile {
    int e, mu, p0, n, p0pad;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4Params p) {
    extern __shared__ uint8_t smem_dyn[];
    __shared__ int s_prefix[kMxSmemGroups + 1];
    __shared__ int s_bounds[kMxSmemGroups + 1];
    __shared__ int s_pad[kMxSmemGroups + 1];
    __shared__ __align__(16) int s_rows[kMxDrains][kMxBN * 4 / kMxDrains];
    __shared__ MxTile s_unit[kMxUnits];  // n == 0: no more
    __shared__ int s_next[2 * kMxUnits];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_total;
    __shared__ int s_issued[2];  // stages whose weights, whose rows have been asked for

    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_dyn + 1023) & ~(uintptr_t)1023);
    uint64_t* full = (uint64_t*)(smem + kMxBarOff);  // a stage's copies have landed
    uint64_t* sf_full = full + kMxStages;            // its scales are in tensor memory
    uint64_t* empty = sf_full + kMxStages;           // its MMAs have completed
    uint64_t* acc_full = empty + kMxStages;          // [2]
    uint64_t* acc_empty = acc_full + 2;              // [2]
    uint64_t* unit_full = acc_empty + 2;             // [kMxUnits]
    uint64_t* unit_empty = unit_full + kMxUnits;     // [kMxUnits]
    uint64_t* next_full = unit_empty + kMxUnits;     // [2 * kMxUnits], of CTA 1
    uint64_t* drained = next_full + 2 * kMxUnits;
    volatile int* abort_flag = &s_abort;
    int* status = p.hdr + kHdrStatus;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = ptx::cluster_rank();  // of the pair; CTA 0 issues the MMAs
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const WLayout L = p.L;
    const int MT = L.mt_count, KT = L.kt_count, KS = (KT + kMxStageKt - 1) / kMxStageKt, MU = (MT + 1) / 2;
    const bool in_smem = p.n_groups <= kMxSmemGroups;

    if (tid == 0) {
        for (int i = 0; i < kMxStages; ++i) {
            ptx::mbar_init(&full[i], 2);
            ptx::mbar_init(&sf_full[i], 8);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], 2 * kMxDrains);
        }
        for (int i = 0; i < kMxUnits; ++i) {
            ptx::mbar_init(&unit_full[i], 1);
            ptx::mbar_init(&unit_empty[i], 4 + kMxDrains + (rank == 0 ? 3 : 2));  // scales, drains, two copy warps, the MMAs'
        }
        for (int i = 0; i < 2 * kMxUnits; ++i) ptx::mbar_init(&next_full[i], 1);
        ptx::mbar_init(drained, 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    // The pair allocates tensor memory together, once both CTAs run: an SM has room
    // for one CTA of this library's tensor-memory users (145 KB of shared memory and
    // more each), so what it waits for here is given back by a CTA that has ended.
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tmem_alloc_pair(&s_tmem, 512);
        ptx::tmem_relinquish_pair();
    }
    // (by one thread's reading: another CTA may set the status meanwhile; CTA 1 goes by CTA 0's units)
    if (tid == 0) s_total = read_status(status) != 0 ? 0 : p.hdr[kHdrTiles] * MU;
    if (in_smem)
        for (int i = tid; i <= p.n_groups; i += kMxThreads) {
            s_prefix[i] = p.ntile_prefix[i];
            s_bounds[i] = p.bounds[i];
            s_pad[i] = p.pad_start[i];
        }
    ptx::tc_fence_before();
    ptx::cluster_sync();  // both CTAs' barriers, tensor memory and tables are set up
    ptx::tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    const int total = uniform(s_total);

    // Unit t, by a whole warp: the largest group whose first column tile is at most
    // q, 32 candidates a step (by bisection a unit's start cost ~1000 cycles).
    auto unit = [&](int t) {
        MxTile r;
        const int q = t / MU;
        r.mu = t - q * MU;
        int lo = 0, hi = p.n_groups;  // pre[lo] <= q < pre[hi]
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
            const bool below = at < hi && (in_smem ? s_prefix[at] : __ldg(p.ntile_prefix + at)) <= q;
            lo += (__popc(__ballot_sync(0xffffffffu, below)) - 1) * step;
            hi = min(hi, lo + step);
        }
        r.e = lo;
        const int j = q - (in_smem ? s_prefix[lo] : __ldg(p.ntile_prefix + lo));
        const int first = in_smem ? s_bounds[lo] : __ldg(p.bounds + lo);
        r.p0 = first + j * kMxBN;
        r.p0pad = (in_smem ? s_pad[lo] : __ldg(p.pad_start + lo)) + j * kMxBN;
        r.n = min(kMxBN, (in_smem ? s_bounds[lo + 1] : __ldg(p.bounds + lo + 1)) - r.p0);
        return r;
    };

    // Units are found by warp 3, ahead; the others take them from shared memory
    // (found by each role itself, a unit's start was a gap of 2500 cycles in the
    // MMAs).  False behind the last, or where a wait has expired.
    auto take_unit = [&](int k, MxTile& u) {
        const int slot = k % kMxUnits;
        if (!warp_wait(&unit_full[slot], (uint32_t)(k / kMxUnits) & 1u, abort_flag, status, p.wait_limit)) return false;
        u = s_unit[slot];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&unit_empty[slot]);
        return u.n > 0;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ weights
        const uint32_t issue = ptx::elect_one();
        int s = 0, q = 0;
        uint32_t ph = 0;
        bool ok = true;
        MxTile u;
        for (int k = 0; ok && take_unit(k, u); ++k) {
            const int mt = u.mu * 2 + (int)rank;
            for (int ks = 0; ks < KS; ++ks, ++q) {
                ok = warp_wait(&empty[s], ph ^ 1, abort_flag, status, p.wait_limit);
                if (!ok) break;
                uint8_t* st = smem + s * kMxStagePitch;
                if (issue) {
                    if (mt < MT) load_weights<kMxStageKt>(p, L, st, st + kMxOffAS, u.e, mt, ks, &full[s]);
                    else ptx::mbar_arrive(&full[s]);
                }
                if (++s == kMxStages) { s = 0; ph ^= 1; }
            }
        }
        if (lane == 0) s_issued[0] = q;
    } else if (warp == 2) {
        // --------------------------------------------------------------- rows
        // This CTA's half of the unit's rows (contiguous and swizzled) and every
        // row's scales.
        const uint32_t issue = ptx::elect_one();
        int s = 0, q = 0;
        uint32_t ph = 0;
        bool ok = true;
        MxTile u;
        for (int k = 0; ok && take_unit(k, u); ++k) {
            const uint32_t nh = (uint32_t)(u.n + 31) / 32u * 16u;
            const uint8_t* bsrc = p.B + (size_t)(u.p0pad + (int)(rank * nh)) * 128u;
            const uint2* ssrc = p.BS + u.p0pad;
            for (int ks = 0; ks < KS; ++ks, ++q) {
                ok = warp_wait(&empty[s], ph ^ 1, abort_flag, status, p.wait_limit);
                if (!ok) break;
                if (issue && !((int)blockIdx.x == p.stall_cta && q == p.stall_stage)) {
                    uint8_t* st = smem + s * kMxStagePitch;
                    ptx::mbar_arrive_expect_tx(&full[s], nh * 144u);
                    ptx::bulk_g2s(st + kMxOffB, bsrc, nh * 128u, &full[s]);
                    ptx::bulk_g2s(st + kMxOffBS, ssrc, nh * 16u, &full[s]);
                }
                __syncwarp();
                bsrc += (size_t)p.rows_pad * 128u;
                ssrc += p.scale_ld;
                if (++s == kMxStages) { s = 0; ph ^= 1; }
            }
        }
        if (lane == 0) s_issued[1] = q;
    } else if (warp == 3) {
        // -------------------------------------------------------------- units
        // A pair's first unit goes by its number, every further one is the next that no
        // pair has (units differ in their rows; by number alone the pairs of the skewed
        // 8192-token product idled for 10 % of the launch).  CTA 0 asks and tells CTA 1,
        // in a ring that needs no answer: that a slot of s_unit is free again says that
        // the MMAs of unit k - kMxUnits have begun, so those of the unit before it were
        // all issued, for which CTA 1 had read that unit's number, and k - 2 * kMxUnits
        // is no later.
        static_assert(kMxUnits >= 1, "the ring of numbers is read in time");
        bool ok = true;
        int ahead = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k % kMxUnits, n = k % (2 * kMxUnits);
            int t = pair;
            if (rank == 0) {
                if (k > 0) t = ahead;
                if (t >= total) t = -1;
                if (t >= 0) {
                    if (lane == 0) ahead = pairs + atomicAdd(p.hdr + kHdrUnits, 1);
                    ahead = uniform(ahead);
                }
            }
            ok = warp_wait(&unit_empty[slot], ((uint32_t)(k / kMxUnits) & 1u) ^ 1u, abort_flag, status, p.wait_limit);
            if (!ok) break;
            if (rank == 0) {
                if (lane == 0) {
                    ptx::st_cluster(&s_next[n], 1, (uint32_t)t);
                    ptx::mbar_arrive_cluster<true>(&next_full[n], 1);
                }
                __syncwarp();
            } else {
                ok = warp_wait<true>(&next_full[n], (uint32_t)(k / (2 * kMxUnits)) & 1u, abort_flag, status, p.wait_limit);
                if (!ok) break;
                t = *(volatile int*)&s_next[n];
            }
            MxTile u = {};
            if (t >= 0) u = unit(t);
            if (lane == 0) {
                s_unit[slot] = u;
                ptx::mbar_arrive(&unit_full[slot]);
            }
            __syncwarp();
            if (t < 0) break;
        }
    } else if (warp == 1 && rank == 0) {
        // -------------------------------------------------------------- MMAs
        // One thread's loop (a predicate on each MMA cost ~80 cycles an MMA).
        if (ptx::elect_one()) {
            const uint32_t smem_a = ptx::smem_u32(smem);
            int s = 0, slot = 0;
            uint32_t ph = 0, use = 0;
            bool ok = true;
            for (; ok; ++use) {
                const int k = (int)use % kMxUnits;
                ok = wait_bar(&unit_full[k], (use / kMxUnits) & 1u, abort_flag, status, p.wait_limit);
                if (!ok) break;
                const int n32 = (s_unit[k].n + 31) & ~31;
                ptx::mbar_arrive(&unit_empty[k]);
                if (n32 == 0) break;
                const uint32_t id0 = ptx::idesc_mxf4(n32, 0, 256), id1 = ptx::idesc_mxf4(n32, 1, 256), buf = use & 1;
                const uint32_t d = tmem + buf * kMxBN;
                ok = wait_bar<true>(&acc_empty[buf], ((use >> 1) & 1) ^ 1, abort_flag, status, p.wait_limit);
                if (!ok) break;
                for (int ks = 0; ks < KS; ++ks) {
                    // (the scale warps of both CTAs arrive after they have seen the stage's copies land)
                    ok = wait_bar<true>(&sf_full[s], ph, abort_flag, status, p.wait_limit);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t st = smem_a + (uint32_t)s * kMxStagePitch;
                    const uint32_t sf = tmem + kMxScaleCol0 + (uint32_t)slot * kMxScaleCols;
                    const uint64_t ad = ptx::desc_k_sw32(st), bd = ptx::desc_k_sw128(st + kMxOffB);
                    const int kts = KT - ks * kMxStageKt;
                    auto step = [&](int j) {  // address fields count 16 bytes; sums stay inside their 14 bits
                        ptx::mma_mxf4_pair(d, ad + (j * kMxCodes >> 4), bd + j * 2, j & 1 ? id1 : id0, sf + (j >> 1) * 4,
                                           sf + 8 + (j >> 1) * 8, (ks | j) != 0);
                    };
                    if (kts >= kMxStageKt) {
#pragma unroll
                        for (int j = 0; j < kMxStageKt; ++j) step(j);
                    } else {
                        for (int j = 0; j < kts; ++j) step(j);
                    }
                    ptx::mma_commit_pair(&empty[s]);
                    if (++s == kMxStages) { s = 0; ph ^= 1; }
                    if (++slot == kMxScaleSlots) slot = 0;
                }
                if (!ok) break;
                ptx::mma_commit_pair(&acc_full[buf]);
            }
            // every MMA issued has completed before the CTAs can release tensor memory
            ptx::mma_commit_pair(drained);
            volatile int never = 0;
            wait_bar(drained, 0, &never, status, kWaitLimitCycles);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------- scales, per stage
        // Every warp writes its quarter of the lanes with the same words: lane r
        // holds rows r, 32 + r, ... of the tile (or of the sorted rows), one column each.
        int s = 0, slot = 0;
        int old = -kMxScaleSlots;  // the stage that had the slot before, counted on (negative: none)
        uint32_t ph = 0, old_ph = 0;
        bool ok = true;
        const uint32_t dst = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + kMxScaleCol0;
        MxTile u;
        for (int k = 0; ok && take_unit(k, u); ++k) {
            for (int ks = 0; ks < KS; ++ks) {
                ok = warp_wait(&full[s], ph, abort_flag, status, p.wait_limit) &&
                     (old < 0 || warp_wait(&empty[old], old_ph, abort_flag, status, p.wait_limit));
                if (!ok) break;
                if (++old == kMxStages) { old = 0; old_ph ^= 1; }
                const uint32_t as = ptx::smem_u32(smem + s * kMxStagePitch + kMxOffAS);
                const uint32_t bs = ptx::smem_u32(smem + s * kMxStagePitch + kMxOffBS) + lane * 8;
                uint32_t v[8], w[16];
                weight_scales(as, lane, v);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint2 q = c < kMxBN / 32 ? ptx::lds64(bs + c * 256) : make_uint2(0u, 0u);
                    w[c] = q.x;
                    w[8 + c] = q.y;
                }
                ptx::tc_fence_after();
                ptx::tmem_st_32x32b_x8(dst + (uint32_t)slot * kMxScaleCols, v);
                ptx::tmem_st_32x32b_x16(dst + (uint32_t)slot * kMxScaleCols + 8u, w);
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster<false>(&sf_full[s], 0);
                if (++s == kMxStages) { s = 0; ph ^= 1; }
                if (++slot == kMxScaleSlots) slot = 0;
            }
        }
    } else if (warp >= 8 && warp < 8 + kMxDrains) {
        // ---------------------------------------------------------- epilogue
        // kMxDrains warps, a lane quarter and a part of the columns each.
        constexpr int kCols = kMxBN * 4 / kMxDrains;
        const int wq = warp & 3, part = (warp - 8) >> 2;
        int* rows = s_rows[warp - 8];  // the output rows of the warp's columns
        uint32_t use = 0;
        MxTile u;
        for (; take_unit((int)use, u); ++use) {
            const int mt = u.mu * 2 + (int)rank, c_lo = part * kCols, n = min(kCols, u.n - c_lo);
            const uint32_t buf = use & 1;
            __syncwarp();
            for (int c = lane; c < n; c += 32) rows[c] = __ldg(p.dst_rows + u.p0 + c_lo + c);
            __syncwarp();
            if (!warp_wait(&acc_full[buf], (use >> 1) & 1, abort_flag, status, p.wait_limit)) break;
            ptx::tc_fence_after();
            const int m = mt * kTileM + 32 * wq + perm_row(lane);
            const bool m_ok = mt < MT && m < L.n_out;
            float* out = p.out + m;
            // A column is a sorted row: its 32 lanes are 128 consecutive bytes of one
            // row of dst.  The rows' numbers come from shared memory, four to a load: by
            // shuffles under a test a column cost 105 cycles.
            // (Tensor memory is read by the whole warp: the lanes meet again after their stores.)
            for (int c0 = 0; c0 < n; c0 += 32) {
                uint32_t v[32];
                __syncwarp();
                ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * wq) << 16) + buf * kMxBN + c_lo + c0, v);
                ptx::tmem_ld_wait();
                if (m_ok && c0 + 32 <= n) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const int4 r = *(const int4*)(rows + c0 + j);
                        out[(int64_t)r.x * p.out_ld] = __uint_as_float(v[j]);
                        out[(int64_t)r.y * p.out_ld] = __uint_as_float(v[j + 1]);
                        out[(int64_t)r.z * p.out_ld] = __uint_as_float(v[j + 2]);
                        out[(int64_t)r.w * p.out_ld] = __uint_as_float(v[j + 3]);
                    }
                } else if (m_ok) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c0 + j < n) out[(int64_t)rows[c0 + j] * p.out_ld] = __uint_as_float(v[j]);
                }
            }
            __syncwarp();
            ptx::tc_fence_before();
            if (lane == 0) ptx::mbar_arrive_cluster<false>(&acc_empty[buf], 0);
        }
    }

    // (the other CTA's MMAs read this one's memory, its warps arrive on this one's barriers)
    ptx::tc_fence_before();
    __syncthreads();
    volatile int never = 0;
    if (warp == 1 && rank == 1)  // the last arrival of the pair's MMAs on this CTA
        warp_wait<true>(drained, 0, &never, status, kWaitLimitCycles);
    if (tid == 0) {
        // Every copy issued lands before the CTA can exit (bounded).  A stage's barrier
        // counts its weights and its rows; where waits have expired one of the two warps
        // may have asked for stages that the other has not, whose arrival is made here
        // (as is that of the rows that the test-only stall left out).
        const int lo = min(s_issued[0], s_issued[1]), hi = max(s_issued[0], s_issued[1]);
        for (int j = lo; j < hi; ++j) ptx::mbar_arrive(&full[j % kMxStages]);
        if ((int)blockIdx.x == p.stall_cta && p.stall_stage < s_issued[1])
            ptx::mbar_arrive(&full[p.stall_stage % kMxStages]);
        for (int j = max(0, hi - kMxStages); j < hi; ++j)
            wait_bar(&full[j % kMxStages], (uint32_t)(j / kMxStages) & 1u, &never, status, kWaitLimitCycles);
    }
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 512);
    }
    // Tensor memory is given back by both CTAs together: neither leaves before the
    // other has done its part, or the next CTA on its SM (another stream's) could ask
    // for the memory in between.
    __syncwarp();
    ptx::cluster_sync();
}

// ------------------------------------------------------------ rounding rows
// Where the rounded rows go: codes [plane of 256 values][row][128 bytes], the
// 16-byte chunk of block c at c ^ (row % 8); scales [plane][row], two words of
// four scale bytes.
struct MxRows {
    uint8_t* codes;
    uint2* scales;
    int64_t rows_pad, scale_ld;
};

// Eight consecutive values as they lie in memory: maximum and codes.
template <int TYPE>
struct MxEight {
    uint32_t w[TYPE == MOE_F32 ? 8 : 4];

    __device__ __forceinline__ void load(const void* p) {
        const uint4 a = __ldg((const uint4*)p);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        if constexpr (TYPE == MOE_F32) {
            const uint4 b = __ldg((const uint4*)p + 1);
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (TYPE == MOE_F32 ? 8 : 4); ++i) w[i] = 0u;
    }
    // the largest magnitude's bits as a float's (16-bit types: two at a time)
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
    __device__ __forceinline__ uint32_t codes(float inv) const {
        float v[8];
        if constexpr (TYPE == MOE_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (TYPE == MOE_BF16) {
                    // scaled as bf16 pairs: a power of two, exact where the result rounds to a
                    // code other than 0
                    const uint32_t p = (__float_as_uint(inv) >> 16) * 0x10001u;
                    const __nv_bfloat162 q = __hmul2(*(const __nv_bfloat162*)&w[i], *(const __nv_bfloat162*)&p);
                    const uint32_t u = *(const uint32_t*)&q;
                    v[2 * i] = __uint_as_float(u << 16);
                    v[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*(const __half2*)&w[i]);
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        }
        return mx_codes8(v, TYPE == MOE_BF16 ? 1.f : inv);
    }
};

constexpr int kMxPlanes = 4;  // planes of a row a warp has in flight

// Planes kp0 .. kp0 + 3 (256 values each) of source row r by one warp, two
// planes at a time, sixteen values a lane and two lanes a block, to the tile
// rows prow[0 .. copies).  (Instructions are the bound next to the bytes: eight
// values a lane took half as many again.)
template <int TYPE>
__device__ __forceinline__ void round_planes(const void* __restrict__ x, int64_t r, int n_in, int kp0, int planes,
                                             const int32_t* prow, int copies, const MxRows& o, int lane) {
    constexpr int esz = TYPE == MOE_F32 ? 4 : 2, kPairs = kMxPlanes / 2;
    const int col = kp0 * 256 + lane * 16;
    const char* src = (const char*)x + (r * n_in + col) * esz;
    MxEight<TYPE> v[kPairs][2];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (col + i * 512 < n_in) v[i][h].load(src + (i * 512 + h * 8) * esz);
            else v[i][h].zero();
        }
    uint2 w[kPairs], sw[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        uint32_t m = max(v[i][0].amax_bits(), v[i][1].amax_bits());
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t X = mx_scale_byte(m);
        const float inv = mx_inv_scale(X);
        w[i] = X == 255u ? make_uint2(0u, 0u) : make_uint2(v[i][0].codes(inv), v[i][1].codes(inv));
        uint32_t half = X << (8 * ((lane >> 1) & 3));  // the scales of 128 values' four blocks in one word
        half |= __shfl_xor_sync(0xffffffffu, half, 2);
        half |= __shfl_xor_sync(0xffffffffu, half, 4);
        sw[i] = make_uint2(half, __shfl_xor_sync(0xffffffffu, half, 8));  // (lanes 0 and 16: the plane's two)
    }
    const int kp = kp0 + (lane >> 4);
    const size_t pitch = (size_t)o.rows_pad * 128u;
    uint8_t* plane = o.codes + (size_t)kp * pitch + (lane & 1) * 8;
    uint2* sp = o.scales + (size_t)kp * o.scale_ld;
    for (int j = 0; j < copies; ++j) {
        const uint32_t pr = (uint32_t)prow[j];
        uint8_t* c = plane + ((size_t)pr * 128u + ((((uint32_t)(lane >> 1) ^ pr) & 7u) << 4));
        uint2* q = sp + pr;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            if (kp + 2 * i < planes) {
                *(uint2*)(c + 2 * i * pitch) = w[i];
                if ((lane & 15) == 0) q[2 * i * o.scale_ld] = sw[i];
            }
        }
    }
}

// After the general row-id pass: one warp per source row (broadcast: a token,
// whose codes go to the tile rows of its k slots; per slot: one slot).
template <int TYPE>
__global__ void __launch_bounds__(256)
mx4_gather_kernel(const void* __restrict__ x, int n_in, const int32_t* __restrict__ slot_prow, int copies,
                  int64_t n_rows, MxRows o, int* hdr) {
    if (read_status(hdr + kHdrStatus) != 0) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) hdr[kHdrUnits] = 0;
    const int lane = threadIdx.x & 31;
    const int planes = (n_in + 255) / 256;
    const int64_t nw = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); r < n_rows; r += nw)
        for (int kp = 0; kp < planes; kp += kMxPlanes)
            round_planes<TYPE>(x, r, n_in, kp, planes, slot_prow + r * copies, copies, o, lane);
}

// ------------------------------------------- tables and rounded rows in one launch
// For up to kRidMaxE experts one launch of up to 148 CTAs makes the tables and
// rounds the rows, 54 us of the gate product above and 58 of the skewed one (the
// row-id pass and a launch for the rows: 35 + 60 and 32 + 98).  The bytes bound it:
// 58 MB read and 125 written, 189 and 50.  Each CTA counts the
// slots by expert before its own and in all (the place of its first slot of
// every expert, the tables' prefixes), ranks its slots in slot order - the same
// stable counting sort - and rounds its rows straight into their tile rows.
// Up to kMpSelfSlots slots every CTA reads all the ids.  Beyond, a launch before
// counts the chunk of kMpParts CTAs and a CTA sums the chunks' counts and counts
// its chunk's slots before its own.  The whole call for 256 experts, top-8, 512 ->
// 128, by itself / with the launch before, us: 20.8 / 25.8 at 8192 slots, 27.8 / 30.5
// at 32768, 42.3 / 41.9 at 65536, 69.8 / 61.8 at 131072; 25.8 / 28.4 and 37.6 / 36.8
// where one expert takes all 32768 or 65536 (8 experts, top-2: 29.3 / 30.3 and 44.0 / 42.6).
constexpr int kMpThreads = 1024;
constexpr int kMpMaxCtas = 148, kMpParts = 4;
constexpr int64_t kMpSelfSlots = 32768;
static_assert((kMpMaxCtas + kMpParts - 1) / kMpParts <= 2 * kRidMaxCtas, "counts take the row-id pass's scratch");

__device__ __forceinline__ int64_t mp_token(int64_t T, int g, int G) { return T * g / G; }

// Count slots [s0, s1) by expert into cnt (shared; integers: the order does not
// matter).  An id outside [0, E) is left out; true where one was met.
__device__ __forceinline__ bool count_slots(const int32_t* __restrict__ ids, int s0, int s1, int E, int* cnt) {
    bool bad = false;
    for (int i0 = s0 + threadIdx.x; i0 < s1; i0 += 8 * kMpThreads) {  // eight loads in flight
        int e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = s1 - i0 > j * kMpThreads ? __ldg(ids + i0 + j * kMpThreads) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (s1 - i0 <= j * kMpThreads) break;
            if ((unsigned)e[j] < (unsigned)E) atomicAdd(&cnt[e[j]], 1);
            else bad = true;
        }
    }
    return bad;
}

// CTA c: the chunk of tokens of place CTAs [c * kMpParts, (c + 1) * kMpParts) of G.
__global__ void __launch_bounds__(kMpThreads)
mx4_count_kernel(const int32_t* __restrict__ ids, int64_t T, int k, int E, int G, int32_t* __restrict__ counts, int* hdr) {
    extern __shared__ int s_cnt[];
    if (__syncthreads_or(threadIdx.x == 0 && read_status(hdr + kHdrStatus) != 0)) return;
    for (int e = threadIdx.x; e < E; e += kMpThreads) s_cnt[e] = 0;
    __syncthreads();
    const int g0 = blockIdx.x * kMpParts;
    if (count_slots(ids, (int)(mp_token(T, g0, G) * k), (int)(mp_token(T, min(g0 + kMpParts, G), G) * k), E, s_cnt))
        set_status(hdr + kHdrStatus, MOE_ERR_BAD_ID);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kMpThreads) counts[(size_t)blockIdx.x * E + e] = s_cnt[e];
}

struct MxPlaceArgs {
    const int32_t* ids;
    const void* x;
    int n_in;
    int64_t T;
    int k, E, per_slot;
    const int32_t* counts;
    int32_t *bounds, *ntile_prefix, *pad_start, *ids_dst, *slot_prow;
    int* hdr;
    MxRows rows;
};

// Exclusive prefix over the CTA's 1024 threads (and the total), in thread order.
__device__ __forceinline__ int cta_prefix(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    const int w = warp_sums[lane];
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    *total = __reduce_add_sync(0xffffffffu, w);
    __syncthreads();  // warp_sums reusable afterwards
    return before + incl - v;
}

template <int TYPE>
__global__ void __launch_bounds__(kMpThreads) mx4_place_kernel(const MxPlaceArgs p) {
    extern __shared__ int s_dyn[];
    const int E = p.E, G = gridDim.x, g = blockIdx.x, k = p.k;
    int* s_base = s_dyn;        // [E] slots of the chunk before the CTA's, then the position of its next slot
    int* s_delta = s_base + E;  // [E] tile row minus sorted position
    int* s_row = s_delta + E;   // [32][E] a warp's counts, then its first positions
    __shared__ int s_sums[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t0 = mp_token(p.T, g, G), t1 = mp_token(p.T, g + 1, G);
    const int64_t r0 = p.per_slot ? t0 * k : t0, r1 = p.per_slot ? t1 * k : t1;
    // counts before this CTA's slots (or, here, those of its chunk) and in all
    int before = 0, all = 0;
    for (int e = tid; e < E; e += kMpThreads) s_base[e] = s_row[e] = 0;
    __syncthreads();
    if (!p.counts) {
        const bool stop = tid == 0 && read_status(p.hdr + kHdrStatus) != 0;
        bool bad = count_slots(p.ids, 0, (int)(t0 * k), E, s_base);
        bad |= count_slots(p.ids, (int)(t0 * k), (int)(p.T * k), E, s_row);
        if (bad) set_status(p.hdr + kHdrStatus, MOE_ERR_BAD_ID);
        if (__syncthreads_or(bad || stop)) return;
        if (tid < E) all = s_base[tid] + s_row[tid];
        __syncthreads();
    } else {
        const int chunk = g / kMpParts, C = (G + kMpParts - 1) / kMpParts;
        count_slots(p.ids, (int)(mp_token(p.T, chunk * kMpParts, G) * k), (int)(t0 * k), E, s_base);
        if (__syncthreads_or(tid == 0 && read_status(p.hdr + kHdrStatus) != 0)) return;
        // 1024 / E threads an expert, each some of the chunks
        const int Ep = (E + 31) & ~31, parts = kMpThreads / Ep;
        const int e = tid % Ep, part = tid / Ep;
        if (part < parts && e < E) {
#pragma unroll 8
            for (int c = part; c < C; c += parts) {
                const int v = __ldcg(p.counts + (size_t)c * E + e);
                all += v;
                before += c < chunk ? v : 0;
            }
        }
        // s_row has room for parts * 2 <= 64 rows of Ep <= 1024 / parts words
        if (part < parts) {
            s_row[part * 2 * Ep + e] = before;
            s_row[(part * 2 + 1) * Ep + e] = all;
        }
        __syncthreads();
        before = all = 0;
        if (tid < E)
            for (int i = 0; i < parts; ++i) {
                before += s_row[i * 2 * Ep + tid];
                all += s_row[(i * 2 + 1) * Ep + tid];
            }
    }
    {
        int S, tiles, padded;
        const int b = cta_prefix(all, s_sums, &S);
        const int q = cta_prefix((all + kMxBN - 1) / kMxBN, s_sums, &tiles);
        const int pad = cta_prefix((all + 7) & ~7, s_sums, &padded);
        if (tid < E) {
            s_base[tid] += b + before;
            s_delta[tid] = pad - b;
            if (g == 0) {
                p.bounds[tid] = b;
                p.ntile_prefix[tid] = q;
                p.pad_start[tid] = pad;
            }
        }
        if (g == 0 && tid == 0) {
            p.bounds[E] = S;
            p.ntile_prefix[E] = tiles;
            p.pad_start[E] = padded;
            p.hdr[kHdrTiles] = tiles;
            p.hdr[kHdrUnits] = 0;
        }
    }
    __syncthreads();
    // rank the CTA's slots, 1024 at a time: within a warp by ballots, across the
    // warps by a prefix of their counts
    const int nb = E > 1 ? 32 - __clz(E - 1) : 1;
    const int s0 = (int)(t0 * k), s1 = (int)(t1 * k);
    for (int i0 = s0; i0 < s1; i0 += kMpThreads) {
        const int nw = min(32, (s1 - i0 + 31) / 32);  // warps with slots
        for (int i = tid; i < nw * E; i += kMpThreads) s_row[i] = 0;
        __syncthreads();
        const int i = i0 + tid;
        const int e = i < s1 ? __ldg(p.ids + i) : -1;
        int rank = 0;
        if (warp < nw) {
            const unsigned m = match_by_ballots(e, nb);
            rank = __popc(m & ((1u << lane) - 1u));
            if (e >= 0 && rank == 0) s_row[warp * E + e] = __popc(m);
        }
        __syncthreads();
        if (tid < E) {
            int run = s_base[tid];
            for (int w = 0; w < nw; ++w) {
                const int c = s_row[w * E + tid];
                s_row[w * E + tid] = run;
                run += c;
            }
            s_base[tid] = run;
        }
        __syncthreads();
        if (e >= 0) {
            const int pos = s_row[warp * E + e] + rank;
            p.ids_dst[pos] = i;
            p.slot_prow[i] = pos + s_delta[e];
        }
        __syncthreads();
    }
    // round the CTA's rows, four planes of a row to a warp at a time
    const int planes = (p.n_in + 255) / 256, chunks = (planes + kMxPlanes - 1) / kMxPlanes, copies = p.per_slot ? 1 : k;
    const int dr = 32 / chunks, dc = 32 % chunks;
    int64_t r = r0 + warp / chunks;
    for (int c = warp % chunks; r < r1; r += dr) {
        round_planes<TYPE>(p.x, r, p.n_in, c * kMxPlanes, planes, p.slot_prow + r * copies, copies, p.rows, lane);
        c += dc;
        if (c >= chunks) {
            c -= chunks;
            ++r;
        }
    }
}

// ------------------------------------------------- few slots: one launch
// For up to kMdMaxSlots slots the call is bound by launches and latency, and then
// by the touched experts' bytes, so one launch does it all: every CTA finds the
// experts and their slots from the ids itself (up to kMdN slots of an expert
// are a group), takes a contiguous range of (group, 128-row tile) items, rounds
// its group's rows into shared memory - all of K, they are few - while the
// weights already stream into a ring, and runs the MMAs 16 columns wide.
// Roles: warp 0 copies weights, warp 1 issues the MMAs, warps 4-7 move the
// weights' scales as the stages land, so that by the time warps 2, 3 and 8-19
// have rounded the rows the ring is ready for the MMAs; warps 8-11 drain the
// accumulator.  (With six rounding warps instead of fourteen: 31.5 us for 26.1, 64
// slots on 8 experts, 4096 -> 4096; the same where a group has few rows.)
constexpr int kMdThreads = 640;
constexpr int kMdRounders = kMdThreads / 32 - 6;  // warps 2, 3 and from 8 on
constexpr int kMdMaxSlots = 256;
constexpr int kMdN = 16;            // columns of an accumulator
static_assert(kMdMaxSlots <= kMdThreads, "a thread a slot");
constexpr int kMdMaxPlanes = 36;    // K up to 9216
constexpr int kMdKt = 8;            // k-steps of a stage: half the copies to issue, ~450 cycles a stage
constexpr int kMdMaxStages = 5;
constexpr uint32_t kMdCodes = kMdKt * kMxCodes, kMdScales = kMdKt * 256, kMdStage = kMdCodes + kMdScales;
constexpr uint32_t kMdPlane = kMdN * 128, kMdPlaneScales = 2 * kMdN * 4;
constexpr uint32_t kMdSmem = 211 * 1024;
// Tensor memory: two accumulators, the stages' A scales (16 columns each), the B
// scales of all of K (4 columns per 128 values, of which 16 rows take the first).
constexpr uint32_t kMdColA = 2 * kMdN, kMdColB = kMdColA + 2 * kMdKt * kMdMaxStages;
static_assert(kMdColA % 4 == 0 && kMdColB % 4 == 0 && kMdColB + 8 * kMdMaxPlanes <= 512, "tensor memory");
constexpr int kMdBarRed = 1;  // named barrier of the workers

struct MxDecodeArgs {
    Mx4Params w;  // weights, output, status
    const int32_t* ids;
    const void* x;
    int n_in, S, k, E, per_slot, stages;
};

template <int TYPE>
__global__ void __launch_bounds__(kMdThreads, 1) mx4_decode_kernel(const __grid_constant__ MxDecodeArgs a) {
    extern __shared__ uint8_t smem_dyn[];
    __shared__ __align__(16) int s_ids[kMdMaxSlots];
    __shared__ __align__(16) int s_pass[kMdMaxSlots];  // of an expert's first slot: its groups; 0 elsewhere
    __shared__ int s_base[kMdMaxSlots];                // of an expert's first slot: its first group
    __shared__ int s_expert[kMdMaxSlots];              // of a group
    __shared__ short s_count[kMdMaxSlots];
    __shared__ __align__(4) short s_slots[kMdMaxSlots][kMdN];
    __shared__ uint64_t s_bar[3 * kMdMaxStages + 6];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_groups, s_stop;

    const Mx4Params& p = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WLayout L = p.L;
    const int MT = L.mt_count, KT = L.kt_count, planes = (KT + 3) / 4, KS = (KT + kMdKt - 1) / kMdKt, NS = a.stages, S = a.S;
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_dyn + 1023) & ~(uintptr_t)1023);
    uint8_t* s_b = smem;                                        // [plane][16][128]
    uint8_t* ring = smem + (size_t)planes * kMdPlane;           // codes of the stages
    uint8_t* ring_s = ring + (size_t)NS * kMdCodes;             // scales of the stages
    uint32_t* s_bs = (uint32_t*)(ring_s + (size_t)NS * kMdScales);  // [K / 128][16]
    uint64_t* full = s_bar;
    uint64_t* sf_full = full + kMdMaxStages;
    uint64_t* empty = sf_full + kMdMaxStages;
    uint64_t* b_full = empty + kMdMaxStages;  // the group's rows and their scales are in place
    uint64_t* acc_full = b_full + 1;          // [2]
    uint64_t* acc_empty = acc_full + 2;       // [2]
    uint64_t* drained = acc_empty + 2;
    volatile int* abort_flag = &s_abort;
    int* status = p.hdr + kHdrStatus;

    if (tid == 0) {
        if (p.full_tiles) {
            ptx::prefetch_tensormap(&p.codes);
            ptx::prefetch_tensormap(&p.scales);
        }
        if (p.tail_subs) ptx::prefetch_tensormap(&p.t_codes);
        if (p.tail_r) ptx::prefetch_tensormap(&p.r_codes);
    }
    // (warp 0 goes straight for the ids)
    if (warp == 2) {
        if (lane < NS) {
            ptx::mbar_init(&full[lane], 1);
            ptx::mbar_init(&sf_full[lane], 4);
            ptx::mbar_init(&empty[lane], 1);
        }
        if (lane >= 16 && lane < 18) {
            ptx::mbar_init(&acc_full[lane - 16], 1);
            ptx::mbar_init(&acc_empty[lane - 16], 4);
        }
        if (lane == 18) ptx::mbar_init(b_full, 4);
        if (lane == 19) ptx::mbar_init(drained, 1);
        if (lane == 20) s_abort = 0;
        if (lane == 21 && S > 32) s_groups = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 3 && lane < 4) {
        // this CTA's share of x into L2, while the groups are found
        const int64_t all = (int64_t)(a.per_slot ? S : S / a.k) * a.n_in * (TYPE == MOE_F32 ? 4 : 2);
        const int64_t share = (all / gridDim.x + 127) / 128 * 128, x0 = share * blockIdx.x + lane * 65536;
        const int64_t x1 = min(all, share * (blockIdx.x + 1)), n = min(x1 - x0, (int64_t)65536);
        if (n > 0) ptx::bulk_prefetch_l2((const char*)a.x + x0, (uint32_t)n);
    }
    const int S4 = (S + 3) & ~3;
    if (S <= 32) {
        // one warp finds the groups: equal ids by a warp match
        if (warp == 0) {
            const bool stop = read_status(status) != 0;
            const int e = lane < S ? __ldg(a.ids + lane) : -1;
            const bool bad = lane < S && (unsigned)e >= (unsigned)a.E;
            if (bad) set_status(status, MOE_ERR_BAD_ID);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int before = __popc(same & ((1u << lane) - 1u)), all = __popc(same), first = __ffs(same) - 1;
            const int n = lane < S && before == 0 ? (all + kMdN - 1) / kMdN : 0;
            int base = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, base, o);
                if (lane >= o) base += v;
            }
            const bool none = __any_sync(0xffffffffu, bad || stop);
            if (lane == 31) s_groups = none ? 0 : base;
            base -= n;
            for (int g = 0; g < n; ++g) {
                s_expert[base + g] = e;
                s_count[base + g] = (short)min(kMdN, all - g * kMdN);
            }
            base = __shfl_sync(0xffffffffu, base, first);
            if (lane < S) s_slots[base + before / kMdN][before % kMdN] = (short)lane;
        }
    } else {
        // every slot against all others, four ids a load
        if (tid == 0) s_stop = read_status(status) != 0;
        int bad = 0;
        if (tid < S4) {
            const int e = tid < S ? __ldg(a.ids + tid) : -1;
            bad = tid < S && (unsigned)e >= (unsigned)a.E;
            s_ids[tid] = e;
            s_pass[tid] = 0;
        }
        if (bad) set_status(status, MOE_ERR_BAD_ID);
        const bool mine = !__syncthreads_or(bad) && !s_stop && tid < S;
        int before = 0, all = 0, first = tid, n = 0;
        if (mine) {
            const int e = s_ids[tid];
            for (int j = 0; j < S4; j += 4) {
                const int4 v = *(const int4*)(s_ids + j);
                const int m[4] = {v.x == e, v.y == e, v.z == e, v.w == e};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    all += m[q];
                    if (m[q] && j + q < tid) {
                        ++before;
                        first = min(first, j + q);
                    }
                }
            }
            if (before == 0) s_pass[tid] = n = (all + kMdN - 1) / kMdN;
        }
        __syncthreads();
        if (n > 0) {
            int base = 0;
            for (int j = 0; j < tid; j += 4) {
                const int4 v = *(const int4*)(s_pass + j);
                base += v.x + (j + 1 < tid ? v.y : 0) + (j + 2 < tid ? v.z : 0) + (j + 3 < tid ? v.w : 0);
            }
            s_base[tid] = base;
            for (int g = 0; g < n; ++g) {
                s_expert[base + g] = s_ids[tid];
                s_count[base + g] = (short)min(kMdN, all - g * kMdN);
            }
            atomicAdd(&s_groups, n);  // a count: the order does not matter
        }
        __syncthreads();
        if (mine) s_slots[s_base[first] + before / kMdN][before % kMdN] = (short)tid;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    const int items = uniform(s_groups) * MT;
    // (rounded up: CTA 0 has the first item however few there are)
    const int it0 = (int)(((int64_t)items * blockIdx.x + gridDim.x - 1) / gridDim.x);
    const int it1 = (int)(((int64_t)items * (blockIdx.x + 1) + gridDim.x - 1) / gridDim.x);

    if (warp == 0) {
        // ------------------------------------------------------------ weights
        const uint32_t issue = ptx::elect_one();
        int s = 0, q = 0;
        uint32_t ph = 0, used = 0, par = 0;
        bool ok = true;
        for (int it = it0; it < it1 && ok; ++it) {
            const int e = s_expert[it / MT], mt = it % MT;
            for (int ks = 0; ks < KS; ++ks, ++q) {
                ok = warp_wait(&empty[s], ph ^ 1, abort_flag, status, p.wait_limit);
                if (!ok) break;
                if (!((int)blockIdx.x == p.stall_cta && q == p.stall_stage)) {
                    if (issue)
                        load_weights<kMdKt>(p, L, ring + (size_t)s * kMdCodes, ring_s + (size_t)s * kMdScales, e, mt, ks,
                                            &full[s]);
                    used |= 1u << s;
                    par = (par & ~(1u << s)) | (ph << s);
                }
                __syncwarp();
                if (++s == NS) { s = 0; ph ^= 1; }
            }
        }
        // let every copy issued land before the CTA can exit (bounded)
        volatile int never = 0;
        for (int j = 0; j < NS; ++j)
            if (used >> j & 1) warp_wait(&full[j], (par >> j) & 1, &never, status, kWaitLimitCycles);
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        const uint32_t issue = ptx::elect_one(), ring_a = ptx::smem_u32(ring), b_a = ptx::smem_u32(s_b);
        const uint32_t id0 = ptx::idesc_mxf4(kMdN, 0), id1 = ptx::idesc_mxf4(kMdN, 1);
        int s = 0;
        uint32_t ph = 0, n = 0;
        bool ok = true;
        for (int it = it0; it < it1 && ok; ++it, ++n) {
            const uint32_t buf = n & 1;
            ok = warp_wait(b_full, n & 1, abort_flag, status, p.wait_limit) &&
                 warp_wait(&acc_empty[buf], ((n >> 1) & 1) ^ 1, abort_flag, status, p.wait_limit);
            if (!ok) break;
            for (int ks = 0; ks < KS; ++ks) {
                // (the scale warps arrive after they have seen the stage's copies land)
                ok = warp_wait(&sf_full[s], ph, abort_flag, status, p.wait_limit);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t ad = ptx::desc_k_sw32(ring_a + (uint32_t)s * kMdCodes);
                const uint64_t bd = ptx::desc_k_sw128(b_a + (uint32_t)ks * (kMdKt / 4 * kMdPlane));
                const uint32_t sfa = tmem + kMdColA + (uint32_t)s * (2 * kMdKt);
                const uint32_t sfb = tmem + kMdColB + (uint32_t)ks * (2 * kMdKt);
                const int kts = KT - ks * kMdKt;
                if (issue) {
                    auto step = [&](int j) {
                        ptx::mma_mxf4_ss(tmem + buf * kMdN, ad + (j * kMxCodes >> 4),
                                         bd + ((j >> 2) * kMdPlane >> 4) + (j & 3) * 2, j & 1 ? id1 : id0,
                                         sfa + (j >> 1) * 4, sfb + (j >> 1) * 4, (ks | j) != 0);
                    };
                    if (kts >= kMdKt) {
#pragma unroll
                        for (int j = 0; j < kMdKt; ++j) step(j);
                    } else {
                        for (int j = 0; j < kts; ++j) step(j);
                    }
                    ptx::mma_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == NS) { s = 0; ph ^= 1; }
            }
            if (!ok) break;
            if (issue) ptx::mma_commit(&acc_full[buf]);
            __syncwarp();
        }
        if (issue) {
            ptx::mma_commit(drained);
            volatile int never = 0;
            wait_bar(drained, 0, &never, status, kWaitLimitCycles);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // -------------------------------------------------- the weights' scales
        const uint32_t dst = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kMdColA;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int q = (it1 - it0) * KS; q > 0; --q) {
            ok = warp_wait(&full[s], ph, abort_flag, status, p.wait_limit);
            if (!ok) break;
            uint32_t v[2][8];
            const uint32_t src = ptx::smem_u32(ring_s + (size_t)s * kMdScales);
            weight_scales(src, lane, v[0]);
            weight_scales(src + kMxAScales, lane, v[1]);
            ptx::tc_fence_after();
            ptx::tmem_st_32x32b_x8(dst + (uint32_t)s * (2 * kMdKt), v[0]);
            ptx::tmem_st_32x32b_x8(dst + (uint32_t)s * (2 * kMdKt) + 8u, v[1]);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sf_full[s]);
            if (++s == NS) { s = 0; ph ^= 1; }
        }
    } else {
        // ---------------------------------------------- rows, then accumulators
        // Every warp here passes the same barriers: one that has given up says so at
        // the next, and all leave there.
        const int w = warp < 4 ? warp - 2 : warp - 6;
        const bool drains = warp >= 8 && warp < 12;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        constexpr int esz = TYPE == MOE_F32 ? 4 : 2;
        int group = -1;
        uint32_t n = 0;
        bool ok = true;
        for (int it = it0; it < it1; ++it, ++n) {
            const int g = it / MT, mt = it % MT, rows = s_count[g];
            if (g != group) {
                // warps 8-11 have seen the last item's MMAs complete
                ok = ptx::bar_red_and(kMdBarRed, kMdRounders * 32, ok);
                if (!ok) break;
                group = g;
                const int units = rows * planes;
                for (int u0 = w; u0 < units; u0 += kMdRounders * kMxPlanes) {
                    MxEight<TYPE> v[kMxPlanes];
#pragma unroll
                    for (int i = 0; i < kMxPlanes; ++i) {
                        const int u = u0 + kMdRounders * i, r = u / planes, col = (u - r * planes) * 256 + lane * 8;
                        if (u < units && col < a.n_in) {
                            const int slot = s_slots[g][r];
                            const int64_t row = a.per_slot ? slot : slot / a.k;
                            v[i].load((const char*)a.x + (row * a.n_in + col) * esz);
                        } else {
                            v[i].zero();
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kMxPlanes; ++i) {
                        const int u = u0 + kMdRounders * i, r = u / planes, kp = u - r * planes;
                        if (u >= units) break;
                        uint32_t m = v[i].amax_bits();
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        const uint32_t X = mx_scale_byte(m);
                        const uint32_t c = X == 255u ? 0u : v[i].codes(mx_inv_scale(X));
                        uint32_t sw = X << (8 * ((lane >> 2) & 3));
                        sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
                        sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
                        *(uint32_t*)(s_b + (size_t)kp * kMdPlane + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                     (lane & 3) * 4) = c;
                        if ((lane & 15) == 0) s_bs[(2 * kp + (lane >> 4)) * kMdN + r] = sw;
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::bar_red_and(kMdBarRed, kMdRounders * 32, true);
                if (drains) {
                    ptx::tc_fence_after();
#pragma unroll 4
                    for (int kp = 0; kp < planes; ++kp) {
                        const uint32_t* q = s_bs + 2 * kp * kMdN + (lane & 15);
                        const uint32_t v[8] = {q[0], 0u, 0u, 0u, q[kMdN], 0u, 0u, 0u};
                        ptx::tmem_st_32x32b_x8(lanes + kMdColB + kp * 8, v);
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                }
            }
            if (!drains) continue;
            const uint32_t buf = n & 1;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b_full);
            uint32_t slots[kMdN / 2];  // two a word
#pragma unroll
            for (int j = 0; j < kMdN / 2; ++j) slots[j] = ((const uint32_t*)s_slots[g])[j];
            const int m = mt * kTileM + 32 * (warp & 3) + perm_row(lane);
            ok = ok && warp_wait(&acc_full[buf], (n >> 1) & 1, abort_flag, status, p.wait_limit);
            if (ok) {
                ptx::tc_fence_after();
                uint32_t v[kMdN];
                ptx::tmem_ld_32x32b_x16(lanes + buf * kMdN, v);
                ptx::tmem_ld_wait();
                if (m < L.n_out) {
#pragma unroll
                    for (int j = 0; j < kMdN; ++j)
                        if (j < rows)
                            p.out[(int64_t)(slots[j / 2] >> (16 * (j & 1)) & 0xffffu) * p.out_ld + m] =
                                __uint_as_float(v[j]);
                }
                __syncwarp();
                ptx::tc_fence_before();
                if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
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
bool plan_weights(Mx4Params& p, int n_experts, int stage_kt) {
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
        const cuuint32_t cb[5] = {128, 8, (cuuint32_t)stage_kt * 4, 1, 1};
        const cuuint64_t sd[4] = {64, KT * 4, (cuuint64_t)p.full_tiles, (cuuint64_t)n_experts};
        const cuuint64_t ss[3] = {sub, tile, ex};
        const cuuint32_t sb[4] = {64, (cuuint32_t)stage_kt * 4, 1, 1};
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

// An ordinary launch: no kernel here starts before its stream's previous one has
// ended.  (As programmatic dependents, whose blocks set up and took tensor memory
// before that, calls on three streams at once came to a standstill after some
// hundred thousand.  The cause was not found; with ordinary launches no block holds
// an SM, or its tensor memory, waiting for another grid.)
template <typename A>
moe_status launch(void (*kernel)(A), unsigned grid, int threads, size_t smem, cudaStream_t stream, const A& args) {
    kernel<<<grid, threads, smem, stream>>>(args);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The kernel's shared-memory limit, set once a device.
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (bit & done.load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

template <int TYPE>
moe_status launch_place(const MxPlaceArgs& a, unsigned grid, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(mx4_place_kernel<TYPE>, (int)(34 * kRidMaxE * sizeof(int)), done)) return MOE_ERR_CUDA;
    return launch(mx4_place_kernel<TYPE>, grid, kMpThreads, smem, s, a);
}

template <int TYPE>
moe_status launch_decode(const MxDecodeArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(mx4_decode_kernel<TYPE>, (int)kMdSmem, done)) return MOE_ERR_CUDA;
    const int64_t items = (int64_t)a.S * a.w.L.mt_count;  // at most: a group has a slot
    const int sms = mx_sm_count();
    return launch(mx4_decode_kernel<TYPE>, (unsigned)(items < sms ? items : sms), kMdThreads, kMdSmem, s, a);
}

moe_status launch_mx4_gemm(const Mx4Params& p, int64_t max_coltiles, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(mx4_gemm_kernel, (int)kMxSmem, done)) return MOE_ERR_CUDA;
    const int64_t units = max_coltiles * ((p.L.mt_count + 1) / 2);
    const int pairs = mx_sm_count() / 2;
    const unsigned grid = 2u * (unsigned)(units < pairs ? units : pairs);
    return launch(mx4_gemm_kernel, grid, kMxThreads, kMxSmem, stream, p);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mul_mat_id_mx4(const void* W_prepared, int n_experts, int n_out, int n_in, const void* x,
                                         moe_dtype x_type, const int32_t* ids, int64_t n_tokens, int k, moe_mode mode,
                                         float* dst, void* workspace, moe_stream stream) {
    if (n_tokens < 0 || k < 1 || n_experts < 1) return MOE_ERR_INVALID;
    if (n_tokens >= kMaxTokens || k >= kMaxK || k > n_experts) return MOE_ERR_RANGE;
    if (n_experts > kMaxExperts || !slots_in_range(n_tokens * (int64_t)k, n_experts)) return MOE_ERR_RANGE;
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
    const int planes = (n_in + 255) / 256;
    // One launch for few slots, unless they crowd on few experts: a group holds kMdN
    // slots and streams its expert's weights again, and every CTA rounds its groups'
    // rows itself (so by slots an expert times planes; the slots' square takes in that
    // with more of them the other form's launches matter less).  us, one launch / two:
    // 256 experts, 2048 -> 512: 9.2 / 18.7 at 32 slots, 20.9 / 27.7 at 128, 30.5 / 34.7
    // at 256; 7168 -> 2048: 91.3 / 99.0 at 64, 163 / 163 at 160; 32 experts, 2048 ->
    // 1024: 20.3 / 22.3 at 192, 22.2 / 22.2 at 256; 8 experts, 4096 -> 4096: 26.7 / 30.3
    // at 80 slots, 31.9 / 30.1 at 96; 8192 -> 4096: 40.3 / 43.9 at 40, 42.8 / 44.2 at 48;
    // 1024 -> 1024: 10.5 / 15.8 at 128; one, 4096 -> 4096: 12.9 / 18.1 at 8, 17.2 / 18.3
    // at 16.
    const int64_t E = n_experts;
    const bool few = S <= kMdMaxSlots && S <= kMdN * E && S * planes <= 200 * E && S * S * planes <= 12800 * E &&
                     planes <= kMdMaxPlanes;
    if (!plan_weights(p, n_experts, few ? kMdKt : kMxStageKt)) return MOE_ERR_CUDA;
    p.out = dst;
    p.out_ld = n_out;
    p.hdr = hdr;
    p.wait_limit = kWaitLimitCycles;
    p.stall_cta = -1;
    long long limit = 0;
    if (testing_stall_state(&p.stall_cta, &p.stall_stage, &limit)) p.wait_limit = limit;
    if (few) {
        MxDecodeArgs a = {};
        a.w = p;
        a.ids = ids;
        a.x = x;
        a.n_in = n_in;
        a.S = (int)S;
        a.k = k;
        a.E = n_experts;
        a.per_slot = mode == MOE_PER_SLOT;
        const int room = (int)((kMdSmem - 1024 - planes * (kMdPlane + kMdPlaneScales)) / kMdStage);
        a.stages = room < kMdMaxStages ? room : kMdMaxStages;
        prof_begin(s);
        const moe_status st = x_type == MOE_BF16  ? launch_decode<MOE_BF16>(a, s)
                              : x_type == MOE_F16 ? launch_decode<MOE_F16>(a, s)
                                                  : launch_decode<MOE_F32>(a, s);
        prof_mark(s, "decode");
        return st;
    }
    // The rounded rows take the workspace of the 16-bit ones: 128 bytes per 256
    // values and 8 of scales where those take 128 per 64.  Only up to 64 values do
    // the scales not fit behind the codes; there they take the rows' factors.
    MxRows o;
    o.rows_pad = W.rows_pad;
    o.scale_ld = (W.rows_pad + 3) / 4 * 4;  // bulk copies start on 16 bytes
    o.codes = (uint8_t*)(ws + W.xt);
    o.scales = n_in <= kTileK ? (uint2*)(ws + W.xs) : (uint2*)(o.codes + (size_t)planes * W.rows_pad * 128u);
    const bool broadcast = mode == MOE_BROADCAST;
    prof_begin(s);
    moe_status st;
    if (n_experts <= kRidMaxE) {
        const unsigned G = (unsigned)(n_tokens < kMpMaxCtas ? n_tokens : kMpMaxCtas);
        int32_t* counts = S > kMpSelfSlots ? (int32_t*)(ws + W.rid) : nullptr;
        if (counts) {
            mx4_count_kernel<<<(G + kMpParts - 1) / kMpParts, kMpThreads, (size_t)n_experts * sizeof(int), s>>>(
                ids, n_tokens, k, n_experts, (int)G, counts, hdr);
            if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
            prof_mark(s, "row_ids");
        }
        MxPlaceArgs a = {ids, x, n_in, n_tokens, k, n_experts, !broadcast, counts, (int32_t*)(ws + W.bounds),
                         (int32_t*)(ws + W.tiles), (int32_t*)(ws + W.pad), (int32_t*)(ws + W.dst),
                         (int32_t*)(ws + W.sprow), hdr, o};
        const int Ep = (n_experts + 31) & ~31;
        const size_t rows = 32 * (size_t)n_experts, sums = 2 * (size_t)(kMpThreads / Ep) * Ep;
        const size_t smem = (2 * (size_t)n_experts + (rows > sums ? rows : sums)) * sizeof(int);
        st = x_type == MOE_BF16  ? launch_place<MOE_BF16>(a, G, smem, s)
             : x_type == MOE_F16 ? launch_place<MOE_F16>(a, G, smem, s)
                                 : launch_place<MOE_F32>(a, G, smem, s);
    } else {
        int n_rid = 1;
        st = launch_row_ids(ids, S, k, n_experts, mode, (int32_t*)(ws + W.src1), (int32_t*)(ws + W.dst),
                            (int32_t*)(ws + W.bounds), (int32_t*)(ws + W.active), (int32_t*)(ws + W.tiles),
                            (int32_t*)(ws + W.pad), (int32_t*)(ws + W.sprow), kMxBN, hdr, nullptr, s, &n_rid);
        if (st) return st;
        prof_mark(s, "row_ids", n_rid);
        const int64_t rows = broadcast ? n_tokens : S, blocks = (rows + 7) / 8, cap = (int64_t)mx_sm_count() * 8;
        const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
        const int32_t* prow = (const int32_t*)(ws + W.sprow);
        const int copies = broadcast ? k : 1;
        if (x_type == MOE_BF16) mx4_gather_kernel<MOE_BF16><<<grid, 256, 0, s>>>(x, n_in, prow, copies, rows, o, hdr);
        else if (x_type == MOE_F16) mx4_gather_kernel<MOE_F16><<<grid, 256, 0, s>>>(x, n_in, prow, copies, rows, o, hdr);
        else mx4_gather_kernel<MOE_F32><<<grid, 256, 0, s>>>(x, n_in, prow, copies, rows, o, hdr);
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (st) return st;
    prof_mark(s, "gather");
    p.n_groups = n_experts;
    p.bounds = (const int32_t*)(ws + W.bounds);
    p.ntile_prefix = (const int32_t*)(ws + W.tiles);
    p.pad_start = (const int32_t*)(ws + W.pad);
    p.B = o.codes;
    p.BS = o.scales;
    p.rows_pad = o.rows_pad;
    p.scale_ld = o.scale_ld;
    p.dst_rows = (const int32_t*)(ws + W.dst);
    st = launch_mx4_gemm(p, (S + kMxBN - 1) / kMxBN + (S < n_experts ? S : n_experts), s);
    prof_mark(s, "gemm");
    return st;
}
