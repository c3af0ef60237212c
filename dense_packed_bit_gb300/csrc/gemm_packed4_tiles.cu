// gemm_packed4_tiles.cu -- Y = X W^T for 4-bit W with group scales and many rows of X per matrix, on tcgen05:
//
//     Y[m][r] = sum_g scale[r][g] * D_g[r][m],   D_g[r][m] = sum_{k in g} (code[r][k] - zero[r][g]) * X[m][k]
//
// 128 rows of W are the MMA's M (256 for a pair of CTAs that share it, cta_group::2), up to 256 rows of X its N.  The
// codes less their zeros are whole numbers of -15 .. 15, exact in X's type, so the tensor cores sum exact products in
// fp32; a group's sum is taken out of tensor memory, multiplied by the group's scale in fp32 and added up in registers.
// Scaled weights are never rounded, and no sum in the tensor core is longer than a group.  Taking D_g out costs a read of
// tensor memory and an FMA for each of its elements against G MMA steps of each.  With groups of 128 it mostly hides behind
// the MMAs (two accumulators of 256 columns); with groups of 64 and 32 it is what bounds the kernel: 2048 x 4096 to 4096 takes
// 66, 100 and 171 us, of which the MMAs 36.
//
// Roles of a CTA's 20 warps, over a ring of stages of 64 columns:
//   warp 0          X by TMA, 64 rows to a box; where `order` names the rows, warps 0 and 3 gather them four at a time;
//   warp 1          issues the MMAs (in a pair: the even CTA's, for both);
//   warp 2          codes by TMA, 128 rows x 128 codes to a box, into a ring of their own that is CRING boxes deep;
//   warps 4 - 11    make 16-bit numbers of them and store them as the MMA's A (128-byte swizzle), a thread to 32 codes of a
//                   row.  Three instructions for two codes: a byte and the same byte shifted are put into the halves of
//                   a register, masked into the mantissa of 1024 (bf16: 128), and that number and the zero are subtracted;
//   warps 12 - 19   a thread to a row of D and half of its columns: scale and add, at the end the activation and the store
//                   (at a fixed row of X a warp writes 32 neighbouring columns of Y).
// Persistent: the units of work -- a chunk of an expert's slots times a tile of rows of W -- are dealt to the CTAs in
// turn, tiles of rows first, so that X is read once and the codes, 4 bits a weight, come from L2.  The slots of an expert
// are cut into chunks of one size, of up to 256, 128 or 64, whichever takes the least time in whole rounds of units.
// Where one matrix gives few units, K is cut over the CTAs of a cluster, whose sums are added in order through shared memory
// (20 x 4096 to 4096: 11.6 us, uncut 25.3).
//
// Measured on a GB300 (groups of 128): 4096 x 4096 to 8192 in bf16 222 us = 1,240 TFLOP/s, 64% of a library product, where the
// MMAs alone take 145: the ends of units, sums and numbers do not all hide behind them.  4096 tokens of 2 of 8 experts of 8192 x
// 2048 with SwiGLU 416 us, bound by the gathers of X.  222 x 776 to 2304 9.2 us: latency, 0.4 us a stage.
#include "packed4.cuh"
#include "smem_limit.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace mm {

__device__ unsigned int g_packed4_tiles_err;

namespace {

constexpr int BM = 128;        // rows of W per CTA: the TMEM lanes
constexpr int BK = 64;         // columns per stage: 128 bytes of X's type
constexpr int BN = 256;        // rows of X per unit, at most: columns of an accumulator
constexpr int CBOX = BM * 64;  // bytes of a box: 128 rows of two stages' codes
constexpr int NTHREADS = 640;
constexpr int WARP_X = 0, WARP_MMA = 1, WARP_CODES = 2, WARP_X2 = 3, WARP_DEC0 = 4, WARP_EPI0 = 12;
constexpr int DEC_WARPS = 8, EPI_WARPS = 8;
constexpr int MAX_EXPERTS = 1024;
constexpr int BOX = 64;        // rows of X per TMA box

// A row's group sums are added one after another in fp32, each addition off by 2^-24 of the sum so far at most.  Where a CTA adds
// more than LONG_GROUPS (32,768 columns in groups of 32), units are of LONG_BN rows of X, which leaves a thread registers for a
// compensated total (Kahan's) to which its sums of FOLD groups go: the error stays that of FOLD groups at any length.  (64 x
// 2^20 in groups of 32, the first group large and the others just below half a place: 1.2e-4 of the terms without.)
constexpr int LONG_GROUPS = 1024, LONG_BN = 64, FOLD = 512;

// Registers of a thread once the roles part, of the 96 at launch: 384 x 40 + 256 x 176 <= 640 x 96.
#define MM_PACKED4_REGS_FEW "40"
#define MM_PACKED4_REGS_EPI "176"

// What a stage of 256, 128 and 64 rows of X costs, about.  A stage of few rows costs nearly as much as one of many, so shorter
// chunks pay where they fill SMs that would be idle, and not in a second round.  Measured (us, chunks of up to 256, 128 and 64):
// 600 x 4096 to 4096 34, 54, 72; 512 x 2048 to 8192 21, 32, 54; of experts of 2048 columns, 2000 slots of 4 of 512 rows
// 29, 23, 20 (gathered 49, 34, 25); 4000 slots of 8 of 300 rows 32, 26, 37 (58, 38, 48); of 8 of 1024 rows 45, 44, 68 (75, 63, 85).
__device__ __forceinline__ int cost_of(bool gathered, int i) { return i == 0 ? (gathered ? 25 : 17) : i == 1 ? (gathered ? 15 : 13) : 10; }

template <int CG>
struct Plan {
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN / CG * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = CG == 2 ? 4 : 3;
    static constexpr int CRING = CG == 2 ? 6 : 5;              // boxes of codes on their way to shared memory
    static constexpr int CODES = STAGES * STAGE;
    static constexpr int OUT = CODES + CRING * CBOX;           // 32 x 32 results of each epilogue warp
    static constexpr int ROWS = OUT + EPI_WARPS * 4096;        // rows of X, where they are gathered: 128 to a warp
    static constexpr int BAR = ROWS + 2 * 128 * 4;
    static constexpr int PRE = BAR + 320;                      // chunks before each expert
    static constexpr int TOTAL = PRE + (MAX_EXPERTS + 1) * 4 + 12 + 1024;  // + alignment of the dynamic allocation
    static_assert((3 * STAGES + 2 * CRING + 5) * 8 + 8 <= 320, "barriers");
    static_assert(TOTAL + 512 <= 227 * 1024, "shared memory");
};

struct Shared {  // what follows the barriers
    uint32_t tmem;
    int abort;
};

// A unit of work: rows r0 .. of matrix e times n slots from `first`; N: n rounded up to what the MMA takes.
struct Unit {
    int e, first, n, N;
    int r0;
};

struct Work {
    const int *pre;    // chunks before expert e; pre[experts]: all
    int experts, tiles;
    int longest;       // slots of a chunk, at most
    int units;
};

__device__ __forceinline__ int chunks_of(int n, int longest) { return (n + longest - 1) / longest; }

template <int CG>
__device__ __forceinline__ Unit unit_at(const Packed4MmArgs &a, const Work &w, int u, unsigned int *err) {
    const int chunk = u / w.tiles, tile = u - chunk * w.tiles;
    int lo = 0, hi = w.experts;  // pre[lo] <= chunk < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.pre[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    const Slots s = slots_of(a, lo, err);
    const int many = chunks_of(s.count, w.longest), part = chunk - w.pre[lo];
    const int each = (((s.count + many - 1) / many) + 15) / 16 * 16;  // of equal chunks, rounded up: at most `longest`
    Unit r;
    // (many - 1) each <= (many - 1) longest < count: the last chunk has slots too
    r.e = lo, r.first = s.first + part * each, r.n = min(each, s.count - part * each);
    r.N = (r.n + 16 * CG - 1) / (16 * CG) * (16 * CG);
    r.r0 = tile * BM * CG;
    return r;
}

template <int CG>
__device__ __forceinline__ void fail(volatile int *abort_flag, unsigned int code) {
    atomicOr(&g_packed4_tiles_err, code);
    *abort_flag = 1;
    if constexpr (CG == 2)
        st_cluster_u32(cluster_map(smem_u32(const_cast<int *>(abort_flag)), cluster_ctarank() ^ 1u), 1u);
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 2) umma_f16_pair(d, da, db, idesc, accumulate);
    else umma_f16(d, da, db, idesc, accumulate);
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// mbar_try_wait and mbar_wait of a barrier by its address
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (try_wait(bar, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) return false;
    }
}

template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
    if constexpr (CG == 2) mbar_arrive_cluster(cluster_map(smem_u32(bar), 0));
    else mbar_arrive(bar);
}

// 32 codes as 16-bit numbers in order, 16 bytes for each word: chunks first .. first + 3 of the row's 128 bytes
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t *row, int r, int first, const uint4 &v, uint32_t z) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w}, zero = Code4<T>::zero(z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[j] = Code4<T>::sub(and_or(prmt(w[i], w[i] >> 4, 0x4400u + 0x1111u * j), 0x000F000Fu, Code4<T>::kBase), zero);
        *reinterpret_cast<uint4 *>(row + (((first + i) ^ (r & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
    }
}

// 8 columns of this thread's TMEM lane; tmem_wait8 waits for them (and every load before)
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// Slots first .. first + n - 1 and rows r0 .. r0 + 31 of Y from `out`, [32 slots][32 rows] of a warp: 16 bytes to a lane where
// Y allows it (vec), else element by element.
template <typename T>
__device__ __forceinline__ void store_block(const Packed4MmArgs &a, const float *out, int first, int n, int r0, int lane, bool vec) {
    const int left = min(32, a.rows - r0);
    if (a.swiglu) {
        const int per = 16;  // columns of Y
        if (vec && left == 32) {
            const int c = (lane & 3) * 4;
            for (int j = lane >> 2; j < n; j += 8) {
                const float4 p = *reinterpret_cast<const float4 *>(out + j * 32 + 2 * c), q = *reinterpret_cast<const float4 *>(out + j * 32 + 2 * c + 4);
                const int64_t at = (int64_t)(first + j) * a.y_stride + (r0 >> 1) + c;
                if (a.y_dtype == 2) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.Y) + at) =
                        make_float4(swiglu(p.x, p.y, true), swiglu(p.z, p.w, true), swiglu(q.x, q.y, true), swiglu(q.z, q.w, true));
                } else {
                    const uint32_t lo = Code4<T>::round(swiglu(p.x, p.y, false)) | (uint32_t)Code4<T>::round(swiglu(p.z, p.w, false)) << 16;
                    const uint32_t hi = Code4<T>::round(swiglu(q.x, q.y, false)) | (uint32_t)Code4<T>::round(swiglu(q.z, q.w, false)) << 16;
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.Y) + at) = make_uint2(lo, hi);
                }
            }
        } else {
            for (int i = lane; i < n * per; i += 32) {
                const int j = i / per, c = i % per;
                if (2 * c < left) store_y(a, first + j, (r0 >> 1) + c, swiglu(out[j * 32 + 2 * c], out[j * 32 + 2 * c + 1], a.y_dtype == 2));
            }
        }
    } else if (vec && left == 32) {
        if (a.y_dtype == 2) {
            const int c = (lane & 7) * 4;
            for (int j = lane >> 3; j < n; j += 4)
                *reinterpret_cast<float4 *>(static_cast<float *>(a.Y) + (int64_t)(first + j) * a.y_stride + r0 + c) =
                    *reinterpret_cast<const float4 *>(out + j * 32 + c);
        } else {
            const int c = (lane & 3) * 8;
            for (int j = lane >> 2; j < n; j += 8) {
                const float4 p = *reinterpret_cast<const float4 *>(out + j * 32 + c), q = *reinterpret_cast<const float4 *>(out + j * 32 + c + 4);
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.Y) + (int64_t)(first + j) * a.y_stride + r0 + c) =
                    make_uint4(Code4<T>::round(p.x) | (uint32_t)Code4<T>::round(p.y) << 16, Code4<T>::round(p.z) | (uint32_t)Code4<T>::round(p.w) << 16,
                               Code4<T>::round(q.x) | (uint32_t)Code4<T>::round(q.y) << 16, Code4<T>::round(q.z) | (uint32_t)Code4<T>::round(q.w) << 16);
            }
        }
    } else {
        for (int j = 0; j < n; ++j)
            if (lane < left) store_y(a, first + j, r0 + lane, out[j * 32 + lane]);
    }
}

template <typename T, int CG, bool LONG>
__global__ void __launch_bounds__(NTHREADS, 1)
    packed4_tiles_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ Packed4MmArgs a, const int ksplit) {
    using P = Plan<CG>;
    constexpr int STAGES = P::STAGES, CRING = P::CRING;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_aligned<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + P::BAR);  // X has arrived (a pair's other CTA's)
    uint64_t *ready = full + STAGES;   // the numbers and X are there (the leader's)
    uint64_t *empty = ready + STAGES;  // the stage's MMAs are done (every CTA's)
    uint64_t *cfull = empty + STAGES;  // codes have arrived (this CTA's)
    uint64_t *cempty = cfull + CRING;  // they have been read (this CTA's)
    uint64_t *accf = cempty + CRING;   // a group's sum is complete (every CTA's)
    uint64_t *acce = accf + 2;         // it has been taken (the leader's)
    uint64_t *last = acce + 2;
    Shared *sh = reinterpret_cast<Shared *>(last + 1);
    volatile int *abort_flag = &sh->abort;
    int *pre = reinterpret_cast<int *>(smem + P::PRE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u, part = CG == 1 && ksplit > 1 ? cluster_ctarank() : 0u;
    const int cid = blockIdx.x / (CG * ksplit), ncl = gridDim.x / (CG * ksplit);
    // this CTA's part of K, in whole boxes of codes: stages st0 .. st0 + stages - 1
    const int boxes = (a.cols + 2 * BK - 1) / (2 * BK), st0 = 2 * (boxes * (int)part / ksplit);
    const int stages = min((a.cols + BK - 1) / BK, 2 * (boxes * ((int)part + 1) / ksplit)) - st0;

    if (warp == WARP_MMA) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(&sh->tmem, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&sh->tmem, 512);
            tmem_relinquish();
        }
    }
    const int xwarps = a.order ? 2 : 1;
    uint64_t *const xbar = CG == 2 && rank == 1 ? full : ready;  // where this CTA's X arrives
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], xwarps);
            // the decode warps, the leader's X, and of a pair the other CTA, which tells that its X is there
            mbar_init(&ready[s], DEC_WARPS / 2 * CG + xwarps + CG - 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < CRING; ++s) {
            mbar_init(&cfull[s], 1);
            mbar_init(&cempty[s], DEC_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], EPI_WARPS * CG);
        }
        mbar_init(last, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    // weights laid out long ago are asked for before the kernel in front has ended, where that one does not say whose they are
    const bool early = a.weights_static && !a.offsets;
    if (!early) {
        pdl_wait();
        pdl_launch_dependents();
    }

    // chunks before each expert
    unsigned int err = 0;
    Work wk;
    wk.pre = pre, wk.experts = a.experts, wk.tiles = (a.rows + BM * CG - 1) / (BM * CG);
    {
        __shared__ int sums[3][NTHREADS / 32];
        const int e0 = 2 * threadIdx.x;
        int n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) n[i] = e0 + i < a.experts ? slots_of(a, e0 + i, &err).count : 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int v = chunks_of(n[0], 256 >> k) + chunks_of(n[1], 256 >> k), all = __reduce_add_sync(~0u, v);
            if (lane == 0) sums[k][warp] = all;
        }
        __syncthreads();
        // the longest chunk: the one whose rounds of units take the least time, of equal ones the largest (256 where K is cut)
        int of_warp = 0, all = 0;
        bool too_many = false;
        int64_t least = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            // (a warp's sum is 2^30 at most, the limit below less than 2^26)
            const int v = lane < NTHREADS / 32 ? min(sums[k][lane], 1 << 26) : 0, chunks = __reduce_add_sync(~0u, v);
            too_many = chunks > (a.slots + 63) / 64 + a.experts;  // of k = 2 in the end: the shortest
            const int64_t cost = (int64_t)((uint32_t)(chunks * wk.tiles + ncl - 1) / (uint32_t)ncl) * cost_of(a.order != nullptr, k);
            if (LONG ? k == 2 : k == 0 || (ksplit == 1 && cost < least)) least = cost, wk.longest = 256 >> k, of_warp = v, all = chunks;
        }
        // Ranges that overlap may hold more slots than there are: the numbers of units would pass 32 bits
        if (too_many) err = kDevErrRange, all = 0;
        const int c0 = chunks_of(n[0], wk.longest), c1 = chunks_of(n[1], wk.longest);
        int run = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += up;
        }
        const int before = __reduce_add_sync(~0u, lane < warp ? of_warp : 0) + run - c0 - c1;
        if (e0 < a.experts) pre[e0] = before;
        if (e0 + 1 < a.experts) pre[e0 + 1] = before + c0;
        if (threadIdx.x == 0) pre[a.experts] = all;
        wk.units = all * wk.tiles;
    }
    __syncwarp();
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh->tmem;

    const auto late_wait = [&] {
        if (early) {
            pdl_wait();
            pdl_launch_dependents();
        }
    };
    if (warp < WARP_DEC0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " MM_PACKED4_REGS_FEW ";");
        // every copy issued must land before this CTA's shared memory is released
        const auto drain = [&](int it) {
            for (int i = 0; i < STAGES && i < it; ++i) {
                const int lastit = i + ((it - 1 - i) / STAGES) * STAGES;
                if (!mbar_wait(&xbar[i], (uint32_t)(lastit / STAGES) & 1)) {
                    atomicOr(&g_packed4_tiles_err, kDevErrDrain);
                    break;
                }
            }
        };
        if (warp == WARP_X && !a.order) {
            late_wait();
            int b = 0, it = 0;
            uint32_t use = 0;
            bool stop = false;
            for (int u = cid; u < wk.units && !stop; u += ncl) {
                const Unit t = unit_at<CG>(a, wk, u, &err);
                const int mine = t.N / CG, from = (int)rank * mine;  // this CTA's rows of X
                // whole boxes: the rows behind the unit's are loaded too, into the rest of the stage
                const int boxes = (mine + BOX - 1) / BOX;
                for (int s = 0; s < stages; ++s, ++it) {
                    if (*abort_flag) { stop = true; break; }
                    if (use > 0 && !mbar_wait_sleep(&empty[b], (use - 1) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitEmpty);
                        stop = true;
                        break;
                    }
                    if (elected()) {
                        mbar_arrive_expect_tx(&xbar[b], (uint32_t)boxes * BOX * 128u);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(smem + b * P::STAGE + P::A_BYTES + i * BOX * 128, &tmX, &xbar[b], (st0 + s) * BK, t.first + from + i * BOX);
                    }
                    __syncwarp();
                    if (++b == STAGES) b = 0, ++use;
                }
            }
            drain(it);
        } else if (warp == WARP_X || (warp == WARP_X2 && a.order)) {
            // Gathered rows, four to an instruction, half of them to each of two warps: 27 clocks an instruction for both, which
            // is what the TMA unit takes.  (One lane for each four rows: 70 clocks; three warps, the third of which asks for
            // codes too: the whole call 6 to 16% slower; copies of 16 bytes: 60 for four rows, and beside gathers no sooner.)
            const int half = warp == WARP_X2;
            int *const rows = reinterpret_cast<int *>(smem + P::ROWS) + half * 128;  // this warp's own
            int b = 0, it = 0;
            uint32_t use = 0;
            bool stop = false;
            for (int u = cid; u < wk.units && !stop; u += ncl) {
                const Unit t = unit_at<CG>(a, wk, u, &err);
                const int mine = t.N / CG, n = mine / 2;  // a multiple of 8
                const int g0 = half * n, from = (int)rank * mine + g0;
                for (int i = lane; i < n; i += 32) {  // rows that are none, or behind the chunk: any row, not stored
                    const int64_t row = from + i < t.n ? x_row(a, t.first + from + i, &err) : 0;
                    rows[i] = row < 0 ? 0 : (int)row;
                }
                __syncwarp();
                for (int s = 0; s < stages; ++s, ++it) {
                    if (*abort_flag) { stop = true; break; }
                    if (use > 0 && !mbar_wait_sleep(&empty[b], (use - 1) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitEmpty);
                        stop = true;
                        break;
                    }
                    __syncwarp();
                    if (elected()) {
                        uint8_t *dst = smem + b * P::STAGE + P::A_BYTES + g0 * 128;
                        mbar_arrive_expect_tx(&xbar[b], (uint32_t)n * 128u);
#pragma unroll 4
                        for (int i = 0; i < n; i += 4) {
                            const int4 r = *reinterpret_cast<const int4 *>(rows + i);
                            tma_gather4(dst + i * 128, &tmX, &xbar[b], (st0 + s) * BK, r.x, r.y, r.z, r.w);
                        }
                    }
                    __syncwarp();
                    if (++b == STAGES) b = 0, ++use;
                }
            }
            if (half == 0) drain(it);
        } else if (warp == WARP_CODES) {
            if (lane == 0) {
                int b = 0, it = 0;
                uint32_t use = 0;
                bool stop = false;
                for (int u = cid; u < wk.units && !stop; u += ncl) {
                    const Unit t = unit_at<CG>(a, wk, u, &err);
                    for (int s = 0; s < stages; s += 2, ++it) {
                        if (*abort_flag) { stop = true; break; }
                        // The warps that empty the ring wait for the kernel in front, however long that runs: so does this
                        // one once the ring is full, before the first wait that has a limit.
                        if (it == CRING) late_wait();
                        if (use > 0 && !mbar_wait_sleep(&cempty[b], (use - 1) & 1)) {
                            fail<CG>(abort_flag, kDevErrWaitEmpty);
                            stop = true;
                            break;
                        }
                        mbar_arrive_expect_tx(&cfull[b], CBOX);
                        tma_load_3d(smem + P::CODES + b * CBOX, &tmW, &cfull[b], (st0 + s) * (BK / 2), t.r0 + (int)rank * BM, t.e);
                        if (++b == CRING) b = 0, ++use;
                    }
                }
                for (int i = 0; i < CRING && i < it; ++i) {
                    const int lastit = i + ((it - 1 - i) / CRING) * CRING;
                    if (!mbar_wait(&cfull[i], (uint32_t)(lastit / CRING) & 1)) {
                        atomicOr(&g_packed4_tiles_err, kDevErrDrain);
                        break;
                    }
                }
            }
            __syncwarp();
            late_wait();
        } else if (warp == WARP_MMA && rank == 0) {
            late_wait();
            constexpr uint32_t fmt = __is_same(T, __half) ? kFmtF16 : kFmtBF16;
            if (elected()) {
                // One thread issues all MMAs, and a stage of few rows of X takes no longer than its instructions: addresses
                // are 32-bit numbers, a stage's parity turns with the ring, and a descriptor is its lower word.
                const uint32_t ready0 = smem_u32(ready), empty0 = smem_u32(empty), accf0 = smem_u32(accf), acce0 = smem_u32(acce);
                const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(smem)), db0 = sdesc_kmajor_sw128(smem_u32(smem) + P::A_BYTES);
                const int steps = a.group / 32;  // half stages of a group: 1, 2 or 4
                uint32_t b = 0, parity = 0;      // stage of the ring, its barriers' parity
                uint32_t acc = 0, taken = 1;     // accumulator in turn, the parity of its being taken (at first it is free)
                bool stop = false;
                const auto wait = [&](uint32_t bar, uint32_t at, unsigned int code) {
                    if (!try_wait(bar, at) && !slow_wait(bar, at)) {
                        fail<CG>(abort_flag, code);
                        stop = true;
                    }
                };
                for (int u = cid; u < wk.units && !stop; u += ncl) {
                    const Unit t = unit_at<CG>(a, wk, u, &err);
                    const uint32_t idesc = make_idesc(fmt, fmt, (uint32_t)t.N, BM * CG);
                    int left = (min(a.cols, (st0 + stages) * BK) - st0 * BK + 31) / 32, in_group = 0;  // half stages
                    for (; left > 0; left -= 2) {
                        if (in_group == 0) wait(acce0 + 8 * acc, taken, kDevErrWaitEmpty);  // a group's accumulator is free
                        wait(ready0 + 8 * b, parity, kDevErrWaitFull);
                        if (stop) break;
                        tc_fence_after_sync();
                        const uint64_t da = da0 + b * (P::STAGE >> 4), db = db0 + b * (P::STAGE >> 4);
                        // the first MMA of a group clears the accumulator
                        mma<CG>(tmem + acc * BN, da, db, idesc, in_group);
                        mma<CG>(tmem + acc * BN, da + 2, db + 2, idesc, 1);
                        if (steps == 1 && left > 1) {  // groups of 32: the second half is another
                            commit<CG>(accf0 + 8 * acc);
                            acc ^= 1, taken ^= acc ^ 1;
                            wait(acce0 + 8 * acc, taken, kDevErrWaitEmpty);
                            if (stop) break;
                            tc_fence_after_sync();
                            mma<CG>(tmem + acc * BN, da + 4, db + 4, idesc, 0);
                            mma<CG>(tmem + acc * BN, da + 6, db + 6, idesc, 1);
                        } else if (steps > 1) {
                            mma<CG>(tmem + acc * BN, da + 4, db + 4, idesc, 1);
                            mma<CG>(tmem + acc * BN, da + 6, db + 6, idesc, 1);
                        }
                        commit<CG>(empty0 + 8 * b);
                        in_group += 2;
                        if (in_group >= steps || left <= 2) {
                            commit<CG>(accf0 + 8 * acc);
                            acc ^= 1, taken ^= acc ^ 1, in_group = 0;
                        }
                        if (++b == STAGES) b = 0, parity ^= 1;
                    }
                    if (*abort_flag) stop = true;
                }
                // every MMA issued must be complete before the tensor memory is freed
                commit<CG>(smem_u32(last));
                if (!mbar_wait(last, 0)) atomicOr(&g_packed4_tiles_err, kDevErrWaitMma);
            }
            __syncwarp();
        } else if (warp == WARP_MMA) {
            // the pair's other CTA: the leader's MMAs read its X too
            late_wait();
            if (elected()) {
                int b = 0;
                uint32_t use = 0;
                bool stop = false;
                for (int u = cid; u < wk.units && !stop; u += ncl)
                    for (int s = 0; s < stages; ++s) {
                        if (*abort_flag || !mbar_wait_sleep(&full[b], use & 1)) {
                            if (!*abort_flag) fail<CG>(abort_flag, kDevErrWaitFull);
                            stop = true;
                            break;
                        }
                        arrive_leader<CG>(&ready[b]);
                        if (++b == STAGES) b = 0, ++use;
                    }
            }
            __syncwarp();
        } else {
            late_wait();
        }
    } else if (warp < WARP_EPI0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " MM_PACKED4_REGS_FEW ";");
        late_wait();
        // four warps take the even stages, four the odd ones: a box of codes holds one of each
        const int odd = (warp - WARP_DEC0) >> 2, r = ((warp - WARP_DEC0) & 3) * 32 + lane;  // row of the tile
        uint8_t *const row = smem + r * 128;
        const uint8_t *const box = smem + P::CODES + r * 64;
        // chunk j of row r lies at j ^ (r / 2 % 4) of its 64 bytes
        const int lo = (odd * 2 ^ ((r >> 1) & 3)) << 4, hi = lo ^ 16;
        int b = 0, cb = 0;
        uint32_t use = 0, cuse = 0;
        bool stop = false;
        const auto next_stage = [&] { if (++b == STAGES) b = 0, ++use; };
        if (odd) next_stage();
        const int shift = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
        for (int u = cid; u < wk.units && !stop; u += ncl) {
            const uint8_t *zeros = nullptr;
            if (a.zeros) {
                const Unit t = unit_at<CG>(a, wk, u, &err);
                zeros = a.zeros + t.e * a.scales_expert + min(t.r0 + (int)rank * BM + r, a.rows - 1) * a.scales_row;
            }
            const auto zeros_at = [&](int s) {  // low half: of the stage's first 32 columns, high half: of the others
                if (!zeros || s >= stages) return 0x00080008u;
                const int j = ((st0 + s) * BK) >> shift;
                const uint32_t z = __ldg(zeros + j) & 15u;
                return z | (a.group == 32 ? __ldg(zeros + min(j + 1, a.groups - 1)) & 15u : z) << 16;
            };
            uint32_t z0 = zeros_at(odd), z1 = zeros_at(odd + 2);  // two stages ahead
            for (int s = odd;; s += 2) {
                const bool box_only = s >= stages;  // an odd number of stages: the last box is passed over
                if (box_only && !(odd && s == stages)) break;
                const uint32_t z = z0;
                z0 = z1;
                z1 = zeros_at(s + 4);
                if (*abort_flag || !mbar_wait_sleep(&cfull[cb], cuse & 1)) {
                    if (!*abort_flag) fail<CG>(abort_flag, kDevErrWaitFull);
                    stop = true;
                    break;
                }
                const uint4 v = *reinterpret_cast<const uint4 *>(box + cb * CBOX + lo), w = *reinterpret_cast<const uint4 *>(box + cb * CBOX + hi);
                __syncwarp();
                if (lane == 0) mbar_arrive(&cempty[cb]);
                if (!box_only) {
                    if (use > 0 && !mbar_wait_sleep(&empty[b], (use - 1) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitEmpty);
                        stop = true;
                        break;
                    }
                    store_codes<T>(row + b * P::STAGE, r, 0, v, z & 0xFFFFu);
                    store_codes<T>(row + b * P::STAGE, r, 4, w, z >> 16);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&ready[b]);
                }
                if (!box_only) next_stage(), next_stage();
                if (++cb == CRING) cb = 0, ++cuse;
            }
            // with an odd number of stages a unit's first one falls to the other place of the ring
            if (stages & 1) {
                if (odd) next_stage();
                else {
                    b = b == 0 ? STAGES - 1 : b - 1;
                    if (b == STAGES - 1) --use;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 " MM_PACKED4_REGS_EPI ";");
        late_wait();
        const int quarter = warp & 3, half = (warp - WARP_EPI0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        constexpr int SC = 2;  // scales on their way
        int gi = 0;
        bool stop = false;
        const int size = a.y_dtype == 2 ? 4 : 2;
        const bool vec = reinterpret_cast<uintptr_t>(a.Y) % 16 == 0 && a.y_stride * size % 16 == 0;
        Unit t = {0, 0, 0, 0, 0};
        const uint16_t *sc = nullptr;
        uint16_t next[SC];
        const int gfirst = st0 * BK / a.group, glast = (min(a.cols, (st0 + stages) * BK) + a.group - 1) / a.group;
        const auto enter = [&](int u) {  // the unit's first scales
            if (u >= wk.units) return;
            t = unit_at<CG>(a, wk, u, &err);
            sc = static_cast<const uint16_t *>(a.scales) + t.e * a.scales_expert +
                 min(t.r0 + (int)rank * BM + 32 * quarter + lane, a.rows - 1) * a.scales_row;
#pragma unroll
            for (int i = 0; i < SC; ++i) next[i] = gfirst + i < glast ? __ldg(sc + gfirst + i) : 0;
        };
        enter(cid);
        for (int u = cid; u < wk.units; u += ncl) {
            const int cols = (t.N + 63) / 64 * 32, c0 = half * cols;  // this half's columns of D
            constexpr int ACC = LONG ? LONG_BN / 2 : BN / 2;
            float acc[ACC], all[LONG ? ACC : 1], lost[LONG ? ACC : 1];
#pragma unroll
            for (int i = 0; i < ACC; ++i) {
                acc[i] = 0.f;
                if constexpr (LONG) all[i] = lost[i] = 0.f;
            }
            const auto fold = [&] {  // all += acc; lost: what that addition, and those before it, added too much
                if constexpr (LONG) {
#pragma unroll
                    for (int i = 0; i < ACC; ++i) {
                        const float y = acc[i] - lost[i], t = all[i] + y, c = (t - all[i]) - y;
                        all[i] = t, lost[i] = fabsf(c) < INFINITY ? c : 0.f, acc[i] = 0.f;  // of an infinity it is NaN
                    }
                }
            };
            for (int g0 = gfirst; g0 < glast && !stop; g0 += SC) {
                float now[SC];
#pragma unroll
                for (int i = 0; i < SC; ++i) {
                    now[i] = Code4<T>::f32(next[i]);
                    next[i] = g0 + SC + i < glast ? __ldg(sc + g0 + SC + i) : 0;
                }
#pragma unroll 1
                for (int i = 0; i < SC; ++i, ++gi) {
                    if (g0 + i >= glast) break;
                    const float f = i == 0 ? now[0] : now[1];
                    if (*abort_flag) { stop = true; break; }
                    if (!mbar_wait_sleep(&accf[gi & 1], (uint32_t)(gi / 2) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitMma);
                        stop = true;
                        break;
                    }
                    __syncwarp();  // the reads below are the whole warp's
                    tc_fence_after_sync();
                    const uint32_t d = lanes + (uint32_t)((gi & 1) * BN + c0);
                    // 8 columns are read while the 8 before them are added
                    uint32_t v[2][8];
                    tmem_ld8(d, v[0]);
#pragma unroll
                    for (int c = 0; c < ACC / 8; ++c) {
                        if (c % 4 == 0 && c * 8 >= cols) break;
                        tmem_wait8(v[c & 1]);
                        if (c < ACC / 8 - 1 && (c + 1) * 8 < cols) tmem_ld8(d + (c + 1) * 8, v[(c + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
                            fma2_bcast(acc[c * 8 + j], acc[c * 8 + j + 1], f, __uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1]));
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&acce[gi & 1]);
                }
                if (LONG && (g0 - gfirst) % FOLD == FOLD - SC) fold();
            }
            if constexpr (LONG) {
                fold();
#pragma unroll
                for (int i = 0; i < ACC; ++i) acc[i] = all[i];
            }
            if (CG == 1 && ksplit > 1) {
                // The cluster's CTAs have a part of K each, of this one unit.  Every MMA and copy of the CTA has ended: its ring
                // takes the partial sums, [slot][128 rows], and the CTAs add up a share of the slots each, in order.
                float *sums = reinterpret_cast<float *>(smem);
                const int row = 32 * quarter + lane;
#pragma unroll
                for (int j = 0; j < ACC; ++j)
                    if (j < cols) sums[(c0 + j) * BM + row] = acc[j];
                __syncwarp();
                cluster_sync();
                const int share = (t.n + ksplit - 1) / ksplit, n0 = (int)part * share, n1 = min(t.n, n0 + share);
                const int quad = lane * 4;
                for (int n = n0 + warp - WARP_EPI0; n < n1; n += EPI_WARPS) {
                    const uint32_t from = smem_u32(sums + n * BM + quad);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), p[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < ksplit) p[k] = ld_cluster_v4(cluster_map(from, k));
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < ksplit) v.x += p[k].x, v.y += p[k].y, v.z += p[k].z, v.w += p[k].w;
                    if (t.r0 + quad < a.rows) store4<T>(a, t.first + n, t.r0 + quad, v, vec);
                }
                __syncwarp();
                cluster_sync();  // nobody leaves before its sums have been read
                break;
            }
            if (stop) break;
            const Unit done = t;
            enter(u + ncl);  // its scales come while this one is stored
            float *const out = reinterpret_cast<float *>(smem + P::OUT) + (warp - WARP_EPI0) * 1024;
            const int r0 = done.r0 + (int)rank * BM + 32 * quarter;
#pragma unroll
            for (int c = 0; c < ACC / 32; ++c) {
                const int base = c0 + c * 32;
                if (c * 32 >= cols || base >= done.n || r0 >= a.rows) break;
                if (a.order) {  // a slot whose row of X does not exist (reported where X was loaded) counts as 0s
                    unsigned int seen = 0;
                    const uint32_t ok = __ballot_sync(~0u, base + lane >= done.n || x_row(a, done.first + base + lane, &seen) >= 0);
                    if (ok != ~0u)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(ok >> j & 1)) acc[c * 32 + j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) out[j * 32 + lane] = acc[c * 32 + j];
                __syncwarp();
                store_block<T>(a, out, done.first + base, min(32, done.n - base), r0, lane, vec);
                __syncwarp();
            }
        }
    }
    if (CG == 1 && ksplit > 1 && warp < WARP_EPI0) {  // the epilogue's two barriers count every thread
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    if (err) atomicOr(&g_packed4_tiles_err, err);
    __syncwarp();
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after_sync();
    if (warp == WARP_MMA) {
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

int64_t units_of(const Packed4MmArgs &a, int64_t rows, int64_t longest) {
    return (a.slots + longest - 1) / longest * ((a.rows + rows - 1) / rows);
}

// One matrix that gives few units: K is cut over a cluster first (codes are then made numbers once), to at least one and a
// half boxes of codes (192 columns) a CTA, as far as all CTAs run at once; chunks stay whole then.
int ksplit_of(const Packed4MmArgs &a, int sms, int64_t longest) {
    const int boxes = (a.cols + 2 * BK - 1) / (2 * BK);
    int ksplit = 1;
    while (!a.offsets && ksplit < 8 && units_of(a, BM, longest) * ksplit * 2 <= sms && ksplit * 3 <= boxes) ksplit *= 2;
    return ksplit;
}

template <typename T, int CG, bool LONG>
cudaError_t launch(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    using P = Plan<CG>;
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void *)packed4_tiles_kernel<T, CG, LONG>, P::TOTAL);
    if (e != cudaSuccess) return e;
    CUtensorMap tx, tw;
    e = packed4_tmap_x(&tx, a, a.order ? 1 : BOX);
    if (e == cudaSuccess) e = packed4_tmap_w(&tw, a, BK, BM, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.rows + BM * CG - 1) / (BM * CG), longest = LONG ? LONG_BN : BN;
    const int ksplit = CG == 1 ? ksplit_of(a, sms, longest) : 1;
    // no more CTAs than units of the shortest chunks
    const int64_t most = ksplit > 1 ? units_of(a, BM, longest) : ((a.slots + 63) / 64 + (a.offsets ? a.experts : 0)) * tiles;
    const int64_t clusters = most < sms / CG ? most : sms / CG;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(clusters * CG * ksplit));
    lc.blockDim = dim3(NTHREADS);
    lc.dynamicSmemBytes = P::TOTAL;
    lc.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)(CG * ksplit), attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = CG * ksplit > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, packed4_tiles_kernel<T, CG, LONG>, tx, tw, a, ksplit);
}

}  // namespace

cudaError_t launch_packed4_tiles(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    // Pairs of CTAs share X where they fill the SMs (us, single CTAs and pairs, bf16 in groups of 128: 2048 x 4096 to 4096 70 and 67,
    // 512 x 4096 to 12288 70 and 66), else single ones have twice the units (512 x 4096 to 4096 26 and 32; 1024 x 4096 to 4096,
    // with 64 pairs, 37 and 36).
    const bool pairs = units_of(a, 2 * BM, BN) >= sms / 2;
    // groups that a CTA adds at most, of equal shares in whole boxes
    const int ksplit = pairs ? 1 : ksplit_of(a, sms, BN);
    const int64_t each = ((a.cols + 2 * BK - 1) / (2 * BK) + ksplit - 1) / ksplit * (2 * BK) / a.group;
    if (each > LONG_GROUPS) return a.dtype == 0 ? launch<__half, 1, true>(a, sms, s) : launch<__nv_bfloat16, 1, true>(a, sms, s);
    if (pairs) return a.dtype == 0 ? launch<__half, 2, false>(a, sms, s) : launch<__nv_bfloat16, 2, false>(a, sms, s);
    return a.dtype == 0 ? launch<__half, 1, false>(a, sms, s) : launch<__nv_bfloat16, 1, false>(a, sms, s);
}

unsigned int packed4_tiles_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_packed4_tiles_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_packed4_tiles_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
