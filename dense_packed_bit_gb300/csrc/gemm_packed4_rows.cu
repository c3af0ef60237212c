// gemm_packed4_rows.cu -- Y = X W^T for 4-bit W with group scales and few rows of X per matrix:
//
//     Y[m][r] = sum_g scale[r][g] * sum_{k in g} (code[r][k] - zero[r][g]) * X[m][k]
//
// "Kernel 0112", section "What the kernel costs in a whole token": the products of a token are bound by reading
// 4-bit weights.  What a call cannot do without is the codes, half a byte each, and 2 or 3 bytes a group.
//
// A unit of work is 64 rows of W times 8 (or 16) rows of X.  One warp of a CTA brings it by TMA, 512 columns at a time,
// through a ring that does not stop at a unit's end: the codes, and as many columns of the rows of X (gathered where
// `order` names them).  Eight warps multiply, four tiles of 16 rows by two halves of the columns.  The codes become
// exact 16-bit whole numbers in registers and are the A operand of mma.sync m16n8k16, whose k slots are dealt so that no
// data moves between lanes: a word of 8 codes holds in one masked step the codes 0 and 4, in the next 1 and 5, and X is
// paired the same way.  The tensor cores add the products of one group in fp32; the group's scale is applied to that sum
// in fp32, so neither scaled weights nor partial sums are ever rounded to 16 bits.
//
// K is cut over a cluster of CTAs where the rows alone would leave SMs idle; all parts are added in a fixed order through
// shared memory, so results repeat bit for bit.  More rows of X than 8 (16) go around again with the codes read from L2.
//
// Measured on a GB300: 1 x 1536 to 12288 5.2 us, of which most is latency; 13 x 4096 to 10240 15.1 us = 1.48 TB/s, bound by
// dependent instructions of 8 warps an SM; 64 tokens of 8 of 64 experts of 2048 x 1408 54 us = 1.96 TB/s, issue 53% of cycles.
#include "packed4.cuh"
#include "smem_limit.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace mm {

__device__ unsigned int g_packed4_rows_err;

namespace {

constexpr int TILE = 16;       // rows of W per warp
constexpr int ROWS = 64;       // per unit
constexpr int BK = 512;        // columns per stage
constexpr int HALF = 256;      // per warp
constexpr int CODES = ROWS * BK / 2;
constexpr int CONSUMERS = 256, NTHREADS = CONSUMERS + 32;
constexpr int AHEAD = 2;       // stages of scales on their way to registers
constexpr int MAX_CLUSTER = 8, MAX_EXPERTS = 1024;

template <int NT>
struct Plan {
    static constexpr int TOKENS = 8 * NT;
    static constexpr int X = TOKENS * BK * 2, STAGE = CODES + X;   // codes: two boxes of 256 columns, X: eight of 64
    static constexpr int DEPTH = NT == 1 ? 3 : 2;
    static constexpr int CTAS = 2;                                 // of an SM: 2 x 72 KB, 2 x 64 KB and the partial tiles
    static constexpr int STRIDE = ROWS + 4;                        // floats between tokens of a partial tile
    static constexpr int RED = DEPTH * STAGE;                      // [2 turns][2 halves][TOKENS][STRIDE]
    static constexpr int PART = RED + 4 * TOKENS * STRIDE * 4;     // [TOKENS][ROWS], of a cluster's CTA
    static constexpr int BAR = PART + TOKENS * ROWS * 4;
    static constexpr int TOTAL = BAR + 2 * DEPTH * 8 + 16 + 1024;  // + alignment of the dynamic allocation
    static_assert(CTAS * (TOTAL + MAX_EXPERTS * 10 + 1024 + 64) <= 227 * 1024, "shared memory");
};

// d += a b, or with FIRST d = a b
template <typename T, bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float c0 = FIRST ? 0.f : d[0], c1 = FIRST ? 0.f : d[1], c2 = FIRST ? 0.f : d[2], c3 = FIRST ? 0.f : d[3];
    if constexpr (sizeof(T) && __is_same(T, __half))
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The 8 codes of w less z as pairs (0, 4), (1, 5), (2, 6), (3, 7); zero: Zero4<T>::of(z).  In fp16 the second field of a
// byte is used where it is: 1024 + 16 c, a sixteenth of which, less 64 + z, is one exact FMA, so a word takes one shift.
template <typename T>
struct Zero4;
template <>
struct Zero4<__nv_bfloat16> {
    uint32_t z;
    static __device__ __forceinline__ Zero4 of(uint32_t z) { return {Code4<__nv_bfloat16>::zero(z)}; }
    __device__ __forceinline__ void decode(uint32_t w, uint32_t (&p)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = Code4<__nv_bfloat16>::sub(and_or(w >> (4 * i), 0x000F000Fu, Code4<__nv_bfloat16>::kBase), z);
    }
};
template <>
struct Zero4<__half> {
    uint32_t z, z16;  // 1024 + z; -(64 + z)
    static __device__ __forceinline__ Zero4 of(uint32_t z) { return {Code4<__half>::zero(z), 0xD400D400u + z * 0x00100010u}; }
    __device__ __forceinline__ void decode(uint32_t w, uint32_t (&p)[4]) const {
        const uint32_t v = w >> 8, sixteenth = 0x2C002C00u;
        const auto high = [&](uint32_t x) {
            const uint32_t f = and_or(x, 0x00F000F0u, Code4<__half>::kBase);
            const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&f), *reinterpret_cast<const __half2 *>(&sixteenth),
                                      *reinterpret_cast<const __half2 *>(&z16));
            return *reinterpret_cast<const uint32_t *>(&r);
        };
        p[0] = Code4<__half>::sub(and_or(w, 0x000F000Fu, Code4<__half>::kBase), z);
        p[1] = high(w);
        p[2] = Code4<__half>::sub(and_or(v, 0x000F000Fu, Code4<__half>::kBase), z);
        p[3] = high(v);
    }
};

// Which 8 columns of 128 (of 16 such) the lanes with q = lane % 4 take in the i-th of four turns.  A group of 32 columns takes
// all lanes: chunk 4 i + q.  Wider ones let a lane have two neighbours, 8 (i / 2) + 2 q + i % 2, so that the eight lanes that
// read X together meet no bank twice.  Where they lie, 16 bytes j of row r at j ^ r % 8, an XOR of a lane's own offset tells:
struct Place {
    uint32_t codes, x;  // offsets of turn 0 in the half's codes and X
    template <int G>
    static __device__ __forceinline__ Place of(int lane) {
        const uint32_t g = lane >> 2, q = lane & 3;
        if (G == 32) return {g * 128 + (g << 4) + q * 4, g * 128 + ((q ^ g) << 4)};
        return {g * 128 + (((q >> 1) ^ g) << 4) + (q & 1) * 8, g * 128 + (((q * 2) ^ g) << 4)};
    }
    // 128 columns further: four 16-byte pieces of codes; two boxes of X (added by the caller)
    template <int G>
    __device__ __forceinline__ uint32_t code(int i, int part) const {
        if (G == 32) return codes ^ (uint32_t)((part * 4 + i) << 4);
        return (codes ^ (uint32_t)((part * 4 + (i >> 1) * 2) << 4)) + (i & 1) * 4;
    }
    template <int G>
    __device__ __forceinline__ uint32_t column(int i) const {
        return x ^ (uint32_t)(G == 32 ? (i & 1) << 6 : (i & 1) << 4);
    }
};

// Scales (low half) and zeros (high half) of rows g and g + 8 for a half of a stage: lane q holds group q (and, of 32 columns,
// group q + 4) of it.
template <int G>
struct Scales {
    static constexpr int N = G == 32 ? 2 : 1;
    uint32_t g[N], h[N];
};

// A half of a stage: 16 rows times 256 columns.  codes: the tile's rows of a box; x: the half's four boxes; left: columns of the
// half that exist (TAIL: not all).
template <typename T, int NT, int G, bool TAIL>
__device__ __forceinline__ void half_stage(const uint8_t *codes, const uint8_t *x, const Place &at, const Scales<G> &sz, int left,
                                           int lane, float (&acc)[NT][4]) {
    constexpr int GROUPS = 128 / G, TURNS = 4 / GROUPS;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        if (TAIL && part * 128 >= left) break;
        uint32_t wg[4], wh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *from = codes + at.code<G>(i, part);
            wg[i] = *reinterpret_cast<const uint32_t *>(from);
            wh[i] = *reinterpret_cast<const uint32_t *>(from + 8 * 128);
        }
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            constexpr int LANES = HALF / G < 4 ? HALF / G : 4;
            const int group = part * GROUPS + j, from = (lane & ~3) | (group & (LANES - 1));
            const uint32_t sg = __shfl_sync(~0u, sz.g[group / 4], from), sh = __shfl_sync(~0u, sz.h[group / 4], from);
            const Zero4<T> zg = Zero4<T>::of(sg >> 16), zh = Zero4<T>::of(sh >> 16);
            float d[NT][4];
#pragma unroll
            for (int i = j * TURNS; i < (j + 1) * TURNS; ++i) {
                uint32_t pg[4], ph[4];
                zg.decode(wg[i], pg);
                zh.decode(wh[i], ph);
                const uint32_t a0[4] = {pg[0], ph[0], pg[1], ph[1]}, a1[4] = {pg[2], ph[2], pg[3], ph[3]};
                const int box = part * 2 + (i >> 1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 v = *reinterpret_cast<const uint4 *>(x + box * (NT * 1024) + n * 1024 + at.column<G>(i));
                    if (TAIL && box * 64 >= left) v = make_uint4(0, 0, 0, 0);  // a box that was not loaded
                    if (i == j * TURNS) mma<T, true>(d[n], a0, prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632));
                    else mma<T, false>(d[n], a0, prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632));
                    mma<T, false>(d[n], a1, prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
                }
            }
            const float fg = Code4<T>::f32((uint16_t)sg), fh = Code4<T>::f32((uint16_t)sh);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(fg, d[n][0], acc[n][0]);
                acc[n][1] = fmaf(fg, d[n][1], acc[n][1]);
                acc[n][2] = fmaf(fh, d[n][2], acc[n][2]);
                acc[n][3] = fmaf(fh, d[n][3], acc[n][3]);
            }
        }
    }
}

// Where a warp is in the CTA's work: units in turn, of each its slots TOKENS at a time, of those its stages.
struct Cursor {
    int unit;
    int e, r0, first, count;  // the unit's expert, rows and slots
    int t0, s;                // slots already done, stage
};

// Grid: clusters that take units in turn; a cluster's CTAs take consecutive parts of K.
template <typename T, int NT, int G>
__global__ void __launch_bounds__(NTHREADS, Plan<NT>::CTAS)
    packed4_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ Packed4MmArgs a, const int cluster, const int xbox) {
    using P = Plan<NT>;
    constexpr int DEPTH = P::DEPTH, TOKENS = P::TOKENS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_aligned<1024>(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + P::BAR), *empty = full + DEPTH;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(empty + DEPTH);
    __shared__ int16_t listed[MAX_EXPERTS];  // the experts that have slots
    __shared__ int listed_n, first[MAX_EXPERTS], count[MAX_EXPERTS];  // and their slots
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
    const int cid = blockIdx.x / cluster, clusters = gridDim.x / cluster;
    const int tiles = (a.rows + ROWS - 1) / ROWS, stages = (a.cols + BK - 1) / BK;
    const int s0 = stages * rank / cluster, s1 = stages * (rank + 1) / cluster;
    unsigned int err = 0;
    int units = tiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < DEPTH; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], CONSUMERS / 32);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    // weights laid out long ago are asked for before the kernel in front has ended, where that one does not say whose they are
    const bool early = a.weights_static && !a.offsets;
    if (a.offsets) {
        pdl_wait();
        pdl_launch_dependents();
        if (warp == 0) {
            int n = 0;
            for (int e0 = 0; e0 < a.experts; e0 += 32) {
                const Slots s = e0 + lane < a.experts ? slots_of(a, e0 + lane, &err) : Slots{0, 0};
                const bool some = s.count > 0;
                const uint32_t m = __ballot_sync(~0u, some);
                if (some) {
                    const int at = n + __popc(m & ((1u << lane) - 1u));
                    listed[at] = (int16_t)(e0 + lane);
                    first[at] = s.first, count[at] = s.count;
                }
                n += __popc(m);
            }
            if (lane == 0) listed_n = n;
        }
    }
    __syncthreads();
    if (a.offsets) units = listed_n * tiles;

    const auto enter = [&](Cursor &c) {  // c.unit is set
        c.t0 = 0, c.s = s0;
        if (c.unit >= units) return;
        const int at = a.offsets ? c.unit / tiles : 0;
        c.r0 = (c.unit - at * tiles) * ROWS;
        c.e = a.offsets ? listed[at] : 0, c.first = a.offsets ? first[at] : 0, c.count = a.offsets ? count[at] : (int)a.slots;
    };
    const auto next_chunk = [&](Cursor &c) {
        c.s = s0, c.t0 += TOKENS;
        if (c.t0 >= c.count) c.unit += clusters, enter(c);
    };

    if (warp == CONSUMERS / 32) {
        // the producer: lane i holds the row of X of slot t0 + i
        Cursor c;
        c.unit = cid;
        enter(c);
        int row = 0;
        const auto rows_of_chunk = [&] {
            if (!a.order || c.unit >= units) return;
            const int64_t r = lane < TOKENS && c.t0 + lane < c.count ? x_row(a, c.first + c.t0 + lane, &err) : 0;
            row = r < 0 ? 0 : (int)r;
        };
        const auto boxes_of = [&](int s) { return min(8, (a.cols - s * BK + 63) / 64); };
        const auto codes = [&](const Cursor &k, int b) {
            const int rows = a.order ? min(TOKENS, (k.count - k.t0 + 3) & ~3) : xbox;
            const int wide = a.cols - k.s * BK > HALF ? 2 : 1;
            mbar_arrive_expect_tx(&full[b], (uint32_t)wide * (CODES / 2) + (uint32_t)(boxes_of(k.s) * rows) * 128u);
            for (int i = 0; i < wide; ++i)
                tma_load_3d(smem + b * P::STAGE + i * (CODES / 2), &tmW, &full[b], k.s * (BK / 2) + i * 128, k.r0, k.e);
        };
        const auto xs = [&](const Cursor &k, int b) {
            uint8_t *dst = smem + b * P::STAGE + CODES;
            const int boxes = boxes_of(k.s);
            if (a.order) {
                const int rows = min(TOKENS, (k.count - k.t0 + 3) & ~3);
                for (int i = 0; i < rows; i += 4) {
                    const int r0 = __shfl_sync(~0u, row, i), r1 = __shfl_sync(~0u, row, i + 1), r2 = __shfl_sync(~0u, row, i + 2),
                              r3 = __shfl_sync(~0u, row, i + 3);
                    if (elected())
                        for (int j = 0; j < boxes; ++j) tma_gather4(dst + j * (NT * 1024) + i * 128, &tmX, &full[b], k.s * BK + j * 64, r0, r1, r2, r3);
                }
            } else if (elected()) {
                for (int j = 0; j < boxes; ++j) tma_load_2d(dst + j * (NT * 1024), &tmX, &full[b], k.s * BK + j * 64, k.first + k.t0);
            }
        };
        int b = 0, n = 0;
        uint32_t use = 0;
        bool stop = false;
        const auto more = [&] { return c.unit < units && s0 < s1; };
        if (early) {
            // the first stages' codes, then what waits for the kernel in front
            Cursor f = c;
            for (int i = 0; i < DEPTH && f.unit < units && s0 < s1; ++i) {
                if (elected()) codes(f, i);
                __syncwarp();
                if (++f.s == s1) next_chunk(f);
            }
        }
        if (!a.offsets) {
            pdl_wait();
            pdl_launch_dependents();
        }
        rows_of_chunk();
        while (more() && !stop) {
            if (use > 0) {
                if (*abort_flag || !mbar_wait_sleep(&empty[b], (use - 1) & 1)) {
                    if (lane == 0 && !*abort_flag) atomicOr(&g_packed4_rows_err, kDevErrWaitEmpty);
                    *abort_flag = 1;
                    stop = true;
                    break;
                }
            }
            __syncwarp();
            if (!early || use > 0) {
                if (elected()) codes(c, b);
                __syncwarp();
            }
            xs(c, b);
            __syncwarp();
            ++n;
            if (++b == DEPTH) b = 0, ++use;
            if (++c.s == s1) {
                if (cluster > 1) {  // the consumers' barriers count every thread; a cluster seldom has a second chunk
                    __syncwarp();
                    cluster_sync();
                    cluster_sync();
                }
                next_chunk(c);
                rows_of_chunk();
            }
        }
        // every copy issued must land before this CTA's shared memory is released
        for (int i = 0; i < DEPTH && i < n; ++i) {
            const int lastn = i + ((n - 1 - i) / DEPTH) * DEPTH;
            if (!mbar_wait(&full[i], (uint32_t)(lastn / DEPTH) & 1)) {
                if (lane == 0) atomicOr(&g_packed4_rows_err, kDevErrDrain);
                break;
            }
        }
    } else {
        const int g = lane >> 2, q = lane & 3, tile = warp & 3, half = warp >> 2;
        const Place place = Place::of<G>(lane);
        // scales and zeros AHEAD stages ahead, with a cursor of their own
        constexpr int LANES = HALF / G < 4 ? HALF / G : 4, N = Scales<G>::N;
        Cursor sc;
        uint32_t rg = 0, rh = 0;  // the rows' first scale in their matrix
        const uint16_t *scales = nullptr;
        const uint8_t *zeros = nullptr;
        sc.unit = cid;
        const int j0 = (s0 * BK + half * HALF) / G + (q & (LANES - 1));  // this lane's first group
        int j = j0;
        const auto point = [&] {
            if (sc.unit >= units) return;
            scales = static_cast<const uint16_t *>(a.scales) + sc.e * a.scales_expert;
            if (a.zeros) zeros = a.zeros + sc.e * a.scales_expert;
            rg = (uint32_t)min(sc.r0 + tile * TILE + g, a.rows - 1) * (uint32_t)a.scales_row;
            rh = (uint32_t)min(sc.r0 + tile * TILE + g + 8, a.rows - 1) * (uint32_t)a.scales_row;
        };
        Scales<G> sz[AHEAD];
        const auto fetch = [&](Scales<G> &x) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                x.g[n] = x.h[n] = 8u << 16;
                if (sc.unit < units && j + 4 * n < a.groups) {
                    const uint32_t k = (uint32_t)(j + 4 * n);
                    x.g[n] = __ldg(scales + (rg + k)) | (zeros ? (uint32_t)(__ldg(zeros + (rg + k)) & 15) : 8u) << 16;
                    x.h[n] = __ldg(scales + (rh + k)) | (zeros ? (uint32_t)(__ldg(zeros + (rh + k)) & 15) : 8u) << 16;
                }
            }
            j += BK / G;
            if (++sc.s == s1) {
                const int unit = sc.unit;
                next_chunk(sc);
                j = j0;
                if (sc.unit != unit) point();
            }
        };
        enter(sc);
        point();
        if (early) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) fetch(sz[i]);
        }
        if (!a.offsets) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if (!early) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) fetch(sz[i]);
        }
        float *const red = reinterpret_cast<float *>(smem + P::RED), *const part = reinterpret_cast<float *>(smem + P::PART);
        int b = 0, turn = 0, ahead = 0;
        uint32_t use = 0;
        bool stop = false;
        Cursor c;
        c.unit = cid;
        enter(c);
        const int size = a.y_dtype == 2 ? 4 : 2;
        const bool vec = reinterpret_cast<uintptr_t>(a.Y) % 16 == 0 && a.y_stride * size % 16 == 0;
        while (c.unit < units) {
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
            for (int s = s0; s < s1;) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (i < ahead || s >= s1) continue;
                    const Scales<G> now = sz[i];
                    fetch(sz[i]);
                    if (!stop && !mbar_wait(&full[b], use & 1)) {
                        if (lane == 0) atomicOr(&g_packed4_rows_err, kDevErrWaitFull);
                        *abort_flag = 1;
                        stop = true;  // nothing waits any more, the warps' barriers are still met
                    }
                    __syncwarp();
                    const uint8_t *st = smem + b * P::STAGE;
                    const uint8_t *w = st + half * (CODES / 2) + tile * (TILE * 128), *x = st + CODES + half * (4 * NT * 1024);
                    const int left = a.cols - s * BK - half * HALF;
                    if (left >= HALF) half_stage<T, NT, G, false>(w, x, place, now, left, lane, acc);
                    else half_stage<T, NT, G, true>(w, x, place, now, left, lane, acc);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[b]);
                    if (++b == DEPTH) b = 0, ++use;
                    ++s;
                    ahead = i + 1;
                }
                if (ahead == AHEAD) ahead = 0;
            }
            float *mine = red + (turn * 2 + half) * (TOKENS * P::STRIDE) + tile * TILE;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) mine[(8 * n + 2 * q + (i & 1)) * P::STRIDE + g + 8 * (i >> 1)] = acc[n][i];
            __syncwarp();
            bar_sync(1, CONSUMERS);
            const float *sum = red + turn * 2 * (TOKENS * P::STRIDE);
            // four rows to a thread
            constexpr int QUADS = ROWS / 4;
            const int n = min(TOKENS, c.count - c.t0) * QUADS;
            const auto total = [&](int i) {
                const float *p = sum + i / QUADS * P::STRIDE + i % QUADS * 4;
                const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + TOKENS * P::STRIDE);
                return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            };
            if (cluster > 1) {
                for (int i = threadIdx.x; i < n; i += CONSUMERS) reinterpret_cast<float4 *>(part)[i] = total(i);
                __syncwarp();
                cluster_sync();
            }
            if (rank == 0) {
                for (int i = threadIdx.x; i < n; i += CONSUMERS) {
                    const int t = c.t0 + i / QUADS, r = c.r0 + i % QUADS * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (cluster > 1) {
                        const uint32_t from = smem_u32(part + i * 4);
                        float4 p[MAX_CLUSTER];
#pragma unroll
                        for (int k = 0; k < MAX_CLUSTER; ++k)
                            if (k < cluster) p[k] = ld_cluster_v4(cluster_map(from, k));
#pragma unroll
                        for (int k = 0; k < MAX_CLUSTER; ++k)
                            if (k < cluster) v.x += p[k].x, v.y += p[k].y, v.z += p[k].z, v.w += p[k].w;
                    } else {
                        v = total(i);
                    }
                    // a slot whose row of X does not exist (reported where X was loaded) counts as 0s
                    unsigned int seen = 0;
                    if (a.order && x_row(a, c.first + t, &seen) < 0) v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < a.rows) store4<T>(a, c.first + t, r, v, vec);
                }
            }
            __syncwarp();
            if (cluster > 1) cluster_sync();  // nobody leaves, or writes part again, before it has been read
            turn ^= 1;  // of two buffers the other is free: the barrier above was behind its last reader
            next_chunk(c);
        }
    }
    if (err) atomicOr(&g_packed4_rows_err, err);
}

// K is cut over as many CTAs of a cluster as the GPU holds beside each other (us, cut and uncut: 1 x 12288
// to 1536 in fp16 and groups of 128 7.3 and 22; 8 x 4096 to 4096 6.7 and 8.7)
struct Cut {
    int64_t units;
    int cluster, ctas;  // ctas: that the GPU holds
};
Cut cut_of(const Packed4MmArgs &a, int sms) {
    const int tiles = (a.rows + ROWS - 1) / ROWS, stages = (a.cols + BK - 1) / BK;
    const int64_t units = tiles * (a.offsets ? (a.slots < a.experts ? a.slots : a.experts) : 1);
    const int ctas = sms * 2;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && cluster * 2 <= stages && units * cluster * 2 <= ctas) cluster *= 2;
    return {units, cluster, ctas};
}

template <typename T, int NT, int G>
cudaError_t launch(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    using P = Plan<NT>;
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void *)packed4_rows_kernel<T, NT, G>, P::TOTAL);
    if (e != cudaSuccess) return e;
    const int xbox = a.slots < P::TOKENS ? (int)a.slots : P::TOKENS;
    CUtensorMap tx, tw;
    e = packed4_tmap_x(&tx, a, a.order ? 1 : xbox);
    if (e == cudaSuccess) e = packed4_tmap_w(&tw, a, HALF / 2, ROWS, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const auto [units, cluster, ctas] = cut_of(a, sms);
    static_assert(P::CTAS == 2, "as cut_of counts");
    const int64_t fit = ctas / cluster, clusters = units < fit ? units : fit;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(clusters * cluster));
    lc.blockDim = dim3(NTHREADS);
    lc.dynamicSmemBytes = P::TOTAL;
    lc.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, packed4_rows_kernel<T, NT, G>, tx, tw, a, cluster, xbox);
}

template <typename T, int NT>
cudaError_t launch_g(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    if (a.group == 128) return launch<T, NT, 128>(a, sms, s);
    if (a.group == 64) return launch<T, NT, 64>(a, sms, s);
    return launch<T, NT, 32>(a, sms, s);
}

template <typename T>
cudaError_t launch_t(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    // 16 at a time where a matrix has more than 8 rows of X; of experts some have twice the average (us, 8 and 16 at a time: 8 x
    // 4096 to 4096 6.2 and 7.0, 13 rows 11.0 and 7.3; 64 experts of 2048 x 2048 with 3 slots each 48 and 50, with 4 58 and 57)
    return a.slots > (a.offsets ? 3 * (int64_t)a.experts : 8) ? launch_g<T, 2>(a, sms, s) : launch_g<T, 1>(a, sms, s);
}

}  // namespace

// A warp adds the sums of half of a CTA's groups one after another in fp32, each addition off by 2^-24 of the sum so far at most:
// 1,024 of them (65,536 columns in groups of 32, more where K is cut) are what the bound of the error allows.
bool packed4_rows_holds(const Packed4MmArgs &a, int sms) {
    const Cut c = cut_of(a, sms);
    const int64_t stages = ((a.cols + BK - 1) / BK + c.cluster - 1) / c.cluster;
    return stages * (HALF / a.group) <= 1024;
}

cudaError_t launch_packed4_rows(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    return a.dtype == 0 ? launch_t<__half>(a, sms, s) : launch_t<__nv_bfloat16>(a, sms, s);
}

unsigned int packed4_rows_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_packed4_rows_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_packed4_rows_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
