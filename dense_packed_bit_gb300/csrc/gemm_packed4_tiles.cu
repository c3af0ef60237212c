// gemm_packed4_tiles.cu -- Y = X W^T for 4-bit W with group scales and many rows of X per matrix, on tcgen05:
//
//     Y[m][r] = sum_g scale[r][g] * D_g[r][m],   D_g[r][m] = sum_{k in g} (code[r][k] - zero[r][g]) * X[m][k]
//
// 128 rows of W are the MMA's M (256 for a pair of CTAs that share it, cta_group::2), up to 256 rows of X its N.  The
// codes less their zeros are whole numbers of -15 .. 15, exact in X's type, so the tensor cores sum exact products in
// fp32; a group's sum is taken out of tensor memory, multiplied by the group's scale in fp32 and added up in registers.
// Scaled weights are never rounded, and no sum in the tensor core is longer than a group.  Taking D_g out costs a read of
// tensor memory and an FMA for each of its elements against G MMA steps of each: with groups of 128 a quarter of the time
// of the MMAs, beside which it runs (two accumulators of 256 columns), with groups of 32 all of it.
//
// Roles of a CTA's 16 warps, over a ring of stages of 64 columns:
//   warp 0          X by TMA, 16 rows to a box, or four gathered rows at a time where `order` names them;
//   warp 1          issues the MMAs (in a pair: the even CTA's, for both);
//   warps 4 - 7     a thread to a row of W: codes AHEAD stages ahead from memory into registers, made 16-bit numbers and
//                   stored as the MMA's A (128-byte swizzle).  Three instructions for two codes: a byte and the same byte
//                   shifted are put into the halves of a register, masked into the mantissa of 1024 (bf16: 128), and that
//                   number and the zero are subtracted;
//   warps 8 - 15    a thread to a row of D and half of its columns: scale and add, at the end the activation and the store
//                   (at a fixed row of X a warp writes 32 neighbouring columns of Y).
// Persistent: the units of work -- a chunk of an expert's slots times a tile of rows of W -- are dealt to the CTAs in
// turn, tiles of rows first, so that X is read once and the codes, 4 bits a weight, come from L2.  The slots of an expert
// are cut into chunks of one size; the longest chunk is the largest of 256, 128 and 64 that leaves no SM without work.
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
constexpr int AHEAD = 4;       // stages of codes on their way to registers
constexpr int NTHREADS = 512;
constexpr int WARP_TMA = 0, WARP_MMA = 1, WARP_DEC0 = 4, WARP_EPI0 = 8;
constexpr int DEC_WARPS = 4, EPI_WARPS = 8;
constexpr int MAX_EXPERTS = 1024;
constexpr int BOX = 16;        // rows of X per TMA box

// Registers of a thread after the roles part, of the 128 at launch: 256 x 80 + 256 x 176 = 512 x 128.
#define MM_PACKED4_REGS_FEW "80"
#define MM_PACKED4_REGS_EPI "176"

template <int CG>
struct Plan {
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN / CG * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = CG == 2 ? 6 : 4;
    static constexpr int BAR = STAGES * STAGE;                 // 3 barriers a stage, 4 of the accumulators, 1 at the end
    static constexpr int PRE = BAR + 256;                      // chunks before each expert
    static constexpr int TOTAL = PRE + (MAX_EXPERTS + 1) * 4 + 12 + 1024;  // + alignment of the dynamic allocation
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
    int64_t units;
};

__device__ __forceinline__ int chunks_of(int n, int longest) { return (n + longest - 1) / longest; }

template <int CG>
__device__ __forceinline__ Unit unit_at(const Packed4MmArgs &a, const Work &w, int64_t u, unsigned int *err) {
    const int chunk = (int)(u / w.tiles), tile = (int)(u - (int64_t)chunk * w.tiles);
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
    atomicExch(&g_packed4_tiles_err, code);
    *abort_flag = 1;
    if constexpr (CG == 2)
        st_cluster_u32(cluster_map(smem_u32(const_cast<int *>(abort_flag)), cluster_ctarank() ^ 1u), 1u);
}

template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
    if constexpr (CG == 2) mbar_arrive_cluster(cluster_map(smem_u32(bar), 0));
    else mbar_arrive(bar);
}

// 64 codes of one row and their zeros (one, or of groups of 32 two)
struct Codes {
    uint4 lo, hi;
    uint32_t z;  // low half: of the first 32 columns, high half: of the others
};

__device__ __forceinline__ void load_codes(const Packed4MmArgs &a, const uint8_t *codes, const uint8_t *zeros, int s, Codes &c) {
    const int col = s * BK;
    c.lo = ld_stream_v4(codes + s * (BK / 2));
    c.hi = col + 32 < a.cols ? ld_stream_v4(codes + s * (BK / 2) + 16) : make_uint4(0, 0, 0, 0);
    if (zeros) {
        const uint32_t z0 = __ldg(zeros + col / a.group) & 15;
        const uint32_t z1 = a.group == 32 && col + 32 < a.cols ? __ldg(zeros + col / 32 + 1) & 15 : z0;
        c.z = z0 | z1 << 16;
    } else {
        c.z = 0x00080008u;
    }
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

// Column `row` of Y, slots first .. first + n - 1: this thread's values of one row of D
template <typename T, typename Y>
__device__ __forceinline__ void store_rows(const Packed4MmArgs &a, int64_t first, int row, int n, const float (&v)[32]) {
    if (row >= a.rows) return;
    Y *p = static_cast<Y *>(a.Y) + first * a.y_stride + row;
#pragma unroll
    for (int j = 0; j < 32; ++j, p += a.y_stride) {
        if (j >= n) break;
        if constexpr (sizeof(Y) == 4) *p = v[j];
        else *p = Code4<T>::round(v[j]);
    }
}

// silu(gate) * up of the rows of neighbouring lanes: the even lane takes the even slots, the odd lane the others
template <typename T, typename Y>
__device__ __forceinline__ void store_pairs(const Packed4MmArgs &a, int64_t first, int row, int n, const float (&v)[32]) {
    const int odd = row & 1;
    Y *p = static_cast<Y *>(a.Y) + (first + odd) * a.y_stride + (row >> 1);
#pragma unroll
    for (int j = 0; j < 32; j += 2, p += 2 * a.y_stride) {
        if (j >= n) break;
        const float got = __shfl_xor_sync(~0u, odd ? v[j] : v[j + 1], 1);
        const float gate = odd ? got : v[j], up = odd ? v[j + 1] : got;
        if (j + odd >= n || row >= a.rows) continue;
        const float z = silu(gate) * up;
        if constexpr (sizeof(Y) == 4) *p = z;
        else *p = Code4<T>::round(z);
    }
}

template <typename T, int CG>
__global__ void __launch_bounds__(NTHREADS, 1)
    packed4_tiles_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ Packed4MmArgs a) {
    using P = Plan<CG>;
    constexpr int STAGES = P::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_aligned<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + P::BAR);  // X has arrived (this CTA's)
    uint64_t *ready = full + STAGES;   // codes and X are there (the leader's)
    uint64_t *empty = ready + STAGES;  // the stage's MMAs are done (every CTA's)
    uint64_t *accf = empty + STAGES;   // a group's sum is complete (every CTA's)
    uint64_t *acce = accf + 2;         // it has been taken (the leader's)
    uint64_t *last = acce + 2;
    Shared *sh = reinterpret_cast<Shared *>(last + 1);
    volatile int *abort_flag = &sh->abort;
    int *pre = reinterpret_cast<int *>(smem + P::PRE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int64_t cid = blockIdx.x / CG, ncl = gridDim.x / CG;

    if (warp == WARP_MMA) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(&sh->tmem, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&sh->tmem, 512);
            tmem_relinquish();
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&ready[s], DEC_WARPS * CG);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], EPI_WARPS * CG);
        }
        mbar_init(last, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
    }
    pdl_wait();
    pdl_launch_dependents();

    // chunks before each expert, for the longest chunk that leaves no SM idle
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
        int k = 0;
        for (; k < 2; ++k) {
            int64_t all = 0;
            for (int w = 0; w < NTHREADS / 32; ++w) all += sums[k][w];
            if (all * wk.tiles >= ncl) break;
        }
        wk.longest = 256 >> k;
        const int c0 = chunks_of(n[0], wk.longest), c1 = chunks_of(n[1], wk.longest);
        int run = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += up;
        }
        int before = run - c0 - c1, all = 0;
        for (int w = 0; w < NTHREADS / 32; ++w) {
            if (w < warp) before += sums[k][w];
            all += sums[k][w];
        }
        if (e0 < a.experts) pre[e0] = before;
        if (e0 + 1 < a.experts) pre[e0 + 1] = before + c0;
        if (threadIdx.x == 0) pre[a.experts] = all;
        wk.units = (int64_t)all * wk.tiles;
    }
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh->tmem;
    const int stages = (a.cols + BK - 1) / BK;

    if (warp < WARP_DEC0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " MM_PACKED4_REGS_FEW ";");
        if (warp == WARP_TMA) {
            int it = 0;
            bool stop = false;
            for (int64_t u = cid; u < wk.units && !stop; u += ncl) {
                const Unit t = unit_at<CG>(a, wk, u, &err);
                const int mine = t.N / CG, from = (int)rank * mine;  // this CTA's rows of X
                int rows[2][4];
                if (a.order) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // rows that are none, or behind the chunk: any row, not stored
                            const int i = from + (h * 32 + lane) * 4 + j;
                            const int64_t row = i < t.n ? x_row(a, t.first + i, &err) : 0;
                            rows[h][j] = row < 0 ? 0 : (int)row;
                        }
                }
                for (int s = 0; s < stages; ++s, ++it) {
                    const int b = it % STAGES;
                    const uint32_t use = it / STAGES;
                    if (*abort_flag) { stop = true; break; }
                    if (use > 0 && !mbar_wait(&empty[b], (use - 1) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitEmpty);
                        stop = true;
                        break;
                    }
                    uint8_t *dst = smem + b * P::STAGE + P::A_BYTES;
                    if (lane == 0) mbar_arrive_expect_tx(&full[b], (uint32_t)mine * 128u);
                    __syncwarp();
                    if (a.order) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if ((h * 32 + lane) * 4 < mine)
                                tma_gather4(dst + (h * 32 + lane) * 512, &tmX, &full[b], s * BK, rows[h][0], rows[h][1], rows[h][2], rows[h][3]);
                    } else if (lane * BOX < mine) {
                        tma_load_2d(dst + lane * BOX * 128, &tmX, &full[b], s * BK, t.first + from + lane * BOX);
                    }
                }
            }
            // every copy issued must land before this CTA's shared memory is released
            for (int b = 0; b < STAGES && b < it; ++b) {
                const int lastit = b + ((it - 1 - b) / STAGES) * STAGES;
                if (!mbar_wait(&full[b], (uint32_t)(lastit / STAGES) & 1)) {
                    atomicExch(&g_packed4_tiles_err, kDevErrDrain);
                    break;
                }
            }
        } else if (warp == WARP_MMA && rank == 0) {
            if (lane == 0) {
                constexpr uint32_t fmt = sizeof(T) && __is_same(T, __half) ? kFmtF16 : kFmtBF16;
                constexpr uint16_t both = (uint16_t)((1u << CG) - 1u);
                const int steps = a.group / 16;  // MMAs of a group
                int it = 0, gi = 0;              // stages, groups so far
                bool stop = false;
                for (int64_t u = cid; u < wk.units && !stop; u += ncl) {
                    const Unit t = unit_at<CG>(a, wk, u, &err);
                    const uint32_t idesc = make_idesc(fmt, fmt, (uint32_t)t.N, BM * CG);
                    const int total = (a.cols + 15) / 16;  // MMAs of the unit
                    int done = 0;                          // of them, those of whole or begun groups so far
                    for (int s = 0; s < stages && !stop; ++s, ++it) {
                        const int b = it % STAGES;
                        const uint32_t use = it / STAGES;
                        if (*abort_flag) { stop = true; break; }
                        if (!mbar_wait(&ready[b], use & 1)) {
                            fail<CG>(abort_flag, kDevErrWaitFull);
                            stop = true;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t at = smem_u32(smem + b * P::STAGE);
#pragma unroll 1
                        for (int k = 0; k < BK / 16 && done < total; ++k, ++done) {
                            const int in_group = done & (steps - 1);
                            if (in_group == 0 && gi >= 2 && !mbar_wait(&acce[gi & 1], (uint32_t)(gi / 2 - 1) & 1)) {
                                fail<CG>(abort_flag, kDevErrWaitEmpty);
                                stop = true;
                                break;
                            }
                            if (in_group == 0) tc_fence_after_sync();
                            const uint32_t d = tmem + (uint32_t)((gi & 1) * BN);
                            const uint64_t da = sdesc_kmajor_sw128(at + 32u * k), db = sdesc_kmajor_sw128(at + P::A_BYTES + 32u * k);
                            if constexpr (CG == 2) umma_f16_pair(d, da, db, idesc, in_group > 0);
                            else umma_f16(d, da, db, idesc, in_group > 0);
                            if (in_group == steps - 1 || done == total - 1) {
                                if constexpr (CG == 2) umma_commit_pair(&accf[gi & 1], both);
                                else umma_commit(&accf[gi & 1]);
                                ++gi;
                            }
                        }
                        if constexpr (CG == 2) umma_commit_pair(&empty[b], both);
                        else umma_commit(&empty[b]);
                    }
                }
                // every MMA issued must be complete before the tensor memory is freed
                if constexpr (CG == 2) umma_commit_pair(last, 1);
                else umma_commit(last);
                if (!mbar_wait(last, 0)) atomicExch(&g_packed4_tiles_err, kDevErrWaitMma);
            }
        }
    } else if (warp < WARP_EPI0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " MM_PACKED4_REGS_FEW ";");
        const int r = threadIdx.x - 32 * WARP_DEC0;  // the row of the tile
        // the cursor of the loads runs AHEAD stages before the one that decodes, over the ends of units
        int64_t lu = cid;
        int ls = 0;
        const uint8_t *lc = nullptr, *lz = nullptr;
        const auto point = [&] {
            if (lu >= wk.units) return;
            const Unit t = unit_at<CG>(a, wk, lu, &err);
            const int row = min(t.r0 + (int)rank * BM + r, a.rows - 1);
            lc = a.codes + t.e * a.codes_expert + row * a.codes_row;
            lz = a.zeros ? a.zeros + t.e * a.scales_expert + row * a.scales_row : nullptr;
        };
        const auto load = [&](Codes &c) {
            if (lu >= wk.units) return;
            load_codes(a, lc, lz, ls, c);
            if (++ls == stages) ls = 0, lu += ncl, point();
        };
        Codes c[AHEAD];
        point();
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load(c[i]);
        const int64_t mine = cid < wk.units ? (wk.units - cid + ncl - 1) / ncl : 0, all = mine * stages;
        bool stop = false;
        int b = 0;
        uint32_t use = 0;
        for (int64_t it = 0; it < all && !stop; it += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (it + i >= all || stop) break;
                if (*abort_flag) { stop = true; break; }
                if (use > 0 && !mbar_wait(&empty[b], (use - 1) & 1)) {
                    fail<CG>(abort_flag, kDevErrWaitEmpty);
                    stop = true;
                    break;
                }
                uint8_t *row = smem + b * P::STAGE + r * 128;
                store_codes<T>(row, r, 0, c[i].lo, c[i].z & 0xFFFFu);
                store_codes<T>(row, r, 4, c[i].hi, c[i].z >> 16);
                load(c[i]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // the stage is ready when X is there too: one warp of each CTA waits for it
                    if (warp == WARP_DEC0 && !mbar_wait(&full[b], use & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitFull);
                    }
                    arrive_leader<CG>(&ready[b]);
                }
                if (++b == STAGES) b = 0, ++use;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 " MM_PACKED4_REGS_EPI ";");
        const int quarter = warp & 3, half = (warp - WARP_EPI0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        int gi = 0;
        bool stop = false;
        for (int64_t u = cid; u < wk.units && !stop; u += ncl) {
            const Unit t = unit_at<CG>(a, wk, u, &err);
            const int cols = (t.N + 63) / 64 * 32, c0 = half * cols;  // this half's columns of D
            const int row = t.r0 + (int)rank * BM + 32 * quarter + lane;
            const uint16_t *sc = static_cast<const uint16_t *>(a.scales) + t.e * a.scales_expert + (int64_t)min(row, a.rows - 1) * a.scales_row;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.f;
            constexpr int SC = 4;  // scales on their way
            uint16_t next[SC];
#pragma unroll
            for (int i = 0; i < SC; ++i) next[i] = i < a.groups ? __ldg(sc + i) : 0;
            for (int g0 = 0; g0 < a.groups && !stop; g0 += SC) {
                float now[SC];
#pragma unroll
                for (int i = 0; i < SC; ++i) {
                    now[i] = Code4<T>::f32(next[i]);
                    next[i] = g0 + SC + i < a.groups ? __ldg(sc + g0 + SC + i) : 0;
                }
#pragma unroll 1
                for (int i = 0; i < SC; ++i, ++gi) {
                    if (g0 + i >= a.groups) break;
                    const float f = i == 0 ? now[0] : i == 1 ? now[1] : i == 2 ? now[2] : now[3];
                    if (*abort_flag) { stop = true; break; }
                    if (!mbar_wait(&accf[gi & 1], (uint32_t)(gi / 2) & 1)) {
                        fail<CG>(abort_flag, kDevErrWaitMma);
                        stop = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d = lanes + (uint32_t)((gi & 1) * BN + c0);
                    // 8 columns are read while the 8 before them are added
                    uint32_t v[2][8];
                    tmem_ld8(d, v[0]);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (c % 4 == 0 && c * 8 >= cols) break;
                        tmem_wait8(v[c & 1]);
                        if (c < 15 && (c + 1) * 8 < cols) tmem_ld8(d + (c + 1) * 8, v[(c + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
                            fma2_bcast(acc[c * 8 + j], acc[c * 8 + j + 1], f, __uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1]));
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&acce[gi & 1]);
                }
            }
            if (stop) break;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int base = c0 + c * 32;
                if (c * 32 >= cols || base >= t.n) break;
                if (a.order) {  // a slot whose row of X does not exist (reported where X was loaded) counts as 0s
                    unsigned int seen = 0;
                    const uint32_t ok = __ballot_sync(~0u, base + lane >= t.n || x_row(a, t.first + base + lane, &seen) >= 0);
                    if (ok != ~0u)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(ok >> j & 1)) acc[c * 32 + j] = 0.f;
                }
                const int n = min(32, t.n - base);
                const float(&v)[32] = *reinterpret_cast<const float(*)[32]>(&acc[c * 32]);
                if (a.y_dtype == 2) {
                    if (a.swiglu) store_pairs<T, float>(a, t.first + base, row, n, v);
                    else store_rows<T, float>(a, t.first + base, row, n, v);
                } else {
                    if (a.swiglu) store_pairs<T, uint16_t>(a, t.first + base, row, n, v);
                    else store_rows<T, uint16_t>(a, t.first + base, row, n, v);
                }
            }
        }
    }
    if (err) atomicExch(&g_packed4_tiles_err, err);
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

template <typename T, int CG>
cudaError_t launch(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    using P = Plan<CG>;
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void *)packed4_tiles_kernel<T, CG>, P::TOTAL);
    if (e != cudaSuccess) return e;
    CUtensorMap tm;
    // a single row may have any stride: the map wants one of whole 16 bytes that holds the row
    const uint64_t stride = a.x_rows > 1 ? (uint64_t)a.x_stride * 2 : ((uint64_t)a.cols * 2 + 15) / 16 * 16;
    e = make_tmap_2d(&tm, a.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.X, (uint64_t)a.cols,
                     (uint64_t)a.x_rows, stride, BK, a.order ? 1 : BOX, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    // no more CTAs than units of the shortest chunks
    const int64_t tiles = (a.rows + BM * CG - 1) / (BM * CG);
    const int64_t most = ((a.slots + 63) / 64 + (a.offsets ? a.experts : 0)) * tiles;
    const int64_t clusters = most < sms / CG ? most : sms / CG;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(clusters * CG));
    lc.blockDim = dim3(NTHREADS);
    lc.dynamicSmemBytes = P::TOTAL;
    lc.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = CG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, packed4_tiles_kernel<T, CG>, tm, a);
}

}  // namespace

cudaError_t launch_packed4_tiles(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    return a.dtype == 0 ? launch<__half, 1>(a, sms, s) : launch<__nv_bfloat16, 1>(a, sms, s);
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
