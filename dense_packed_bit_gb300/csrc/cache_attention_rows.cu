// cache_attention_rows.cu -- attention of few new tokens over a paged cache: up to 16 rows (new
// tokens x query heads of one kv head) per sequence, the form of a decode step and of small trees.
//
// Mathematics.  Online softmax: per row the running reference m (in base-2 units, scale log2(e)
// folded into one multiply), l = sum 2^(s - m) and O = sum 2^(s - m) v.  O and l are only rescaled
// when a row's maximum passes its reference by more than 8 (probabilities stay below 2^8, far inside
// fp16), so most blocks cost no rescaling; the final O / l does not depend on the reference.
//
// Bound: reading K and V once (4 D bytes a key and kv head; 16 rows x 4 D operations for them are a
// twentieth of what the tensor cores could do meanwhile).  So the layout is made for loads in flight and
// few instructions per key: blocks of 64 keys pass through a ring of TMA boxes (one per page and 64 columns,
// 128-byte swizzle) that one warp fills; four warps take 16 keys of each block, with no barrier between them
// but the ring's; two CTAs per SM with 192 KB of rings between them.  The 16 x D rows of Q stay in registers as the A operand of
// mma.sync.m16n8k16 (K rows read by ldmatrix are B as they lie, V rows by ldmatrix.trans); the probabilities
// go from accumulator registers to A registers without shared memory.
//
// Split.  Two CTAs per SM, each with an even share of all units' blocks (share_of); ragged lengths cost no more
// than their sum.  A unit that several CTAs share is joined by the last of them to finish, in the order of its
// parts (a ticket per unit, reset by the last), so the result does not depend on which one is last.
//
// Measured, one call: 48 sequences of 100 to 16,000 tokens, one new, 32 heads over 8 of 128 columns, bf16, pages of
// 64: 100 us = 6.07 TB/s, 89% of a plain copy's.  Small calls are a latency of launch, share, first loads and join:
// 1 x 513 (12 heads of 64) 7.9 us, 8 sequences of 32,000 under a window of 1,024 12.6, trees of 4 x 7 tokens 9.1.
//
// What a row does not see: its score is replaced, not added to.  In blocks that the mask cuts,
// infinities and NaN in V are taken out of the product (0 x NaN) and added to the rows that do see them.
#include "cache_attention.cuh"
#include "tcgen05.cuh"

namespace mm {

namespace {

__device__ unsigned int g_rows_err;

constexpr int WARPS = 4, NT = (WARPS + 1) * 32;  // four warps compute, the fifth loads
constexpr int SUB = 16, B = WARPS * SUB;         // keys of a warp's part of a block, of a block
constexpr int MIN_BLOCKS = 1;    // blocks of a part, at least (see least_part)
constexpr int WHOLE_BLOCKS = 8;  // units up to this are not cut when there are many (30 x 100 to 500 tokens: 13.7 us, cut 19.2)
constexpr int JOIN = 8;          // parts joined at a time
constexpr int UNIT_COST = 12;    // what beginning and ending a unit takes, in blocks of a full GPU (48 ragged: 100 us, with 0 135)
constexpr int HALF = B * 128;          // bytes of a block's 64 columns

struct RowsArgs {
    CacheAttnArgs a;
    int box;           // keys of one TMA box
    int force_whole;
    int32_t *tickets;  // [kTickets]
    float2 *ml;        // [CTAs][2][16]
    float *part;       // [CTAs][2][16][head_dim]
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// What the rows of one sequence need between them: the blocks, and where the mask cuts between rows
struct SeqKeys {
    SeqView v;
    int end, whole, low, high;
    KeyBlocks kb;  // count 0: no rows
};
__device__ __forceinline__ SeqKeys seq_keys(const CacheAttnArgs &a, int seq) {
    SeqKeys k;
    k.v = seq_view(a, seq, &g_rows_err);
    const int len = k.v.len, count = k.v.count;
    k.end = len + count;
    k.whole = a.mask ? len : len + 1;
    // a drafted token's depth is between 0 and count; a causal row i is at len + i
    k.low = a.window ? (a.mask ? len - a.window : len - a.window + 1) : 0;
    k.high = a.window ? len + count - a.window : 0;
    k.kb = key_blocks<B>(k.low, a.sinks, k.end);
    if (count == 0 || count * a.group > kRowsMax) k.kb.count = 0;  // the latter: max_q said otherwise
    return k;
}

// KS: 16-element steps of the head dimension held (head_dim <= 16 KS, the rest zero)
template <typename T, int KS>
__global__ void __launch_bounds__(NT, 2) rows_kernel(const __grid_constant__ CUtensorMap kmap,
                                                     const __grid_constant__ CUtensorMap vmap, const RowsArgs p) {
    constexpr int HALVES = KS / 4, STAGES = 6 / HALVES;  // 3 stages of 32 KB, or 6 of 16 KB
    constexpr int TILE = HALVES * HALF;                  // K or V of one block
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[STAGES], empty[STAGES];
    __shared__ float2 sm_ml[WARPS][16];
    __shared__ float sm_p[WARPS][16][SUB];  // probabilities of a block whose V holds an infinity or NaN
    __shared__ ShareScratch sm_share;
    __shared__ int sm_last;
    uint8_t *sm = smem_aligned<1024>(raw);
    const CacheAttnArgs &a = p.a;
    const CacheView &c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], WARPS);
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_launch_dependents();

    Share share;
    const auto blocks = [&](int s) { return s < c.seqs ? seq_keys(a, s).kb.count : 0; };
    const ShareRules rules = {MIN_BLOCKS, WHOLE_BLOCKS, UNIT_COST, p.force_whole};
    if (!share_of<NT>(c.seqs, c.kv_heads, rules, blocks, sm_share, share)) return;
    int at = share.at, seq = share.item, seq_first = share.first;
    SeqKeys k = seq_keys(a, seq);

    const uint32_t ring_s = smem_u32(sm);
    const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // > 0: a masked score stays -infinity
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;       // of Q, for a negative scale
    const int D = c.head_dim, pairs = D / 2;
    uint32_t it = 0;  // blocks that have passed through the ring
    bool ok = true;

    while (at < share.stop) {
        const int n = k.kb.count;
        const UnitPart u = unit_part(share, at, seq_first, n, MIN_BLOCKS);
        const int head = u.head, b0 = u.b0, b1 = u.b1;
        if (b1 <= b0) break;  // nothing of the unit but its cost, or a part that a short unit does not have
        const SeqView sv = k.v;
        const int rows = sv.count * a.group;
        constexpr int OS = KS * 16 + 4;  // the warps' O side by side, fp32, rows padded by 4 words
        float *so = reinterpret_cast<float *>(sm);

        if (warp == WARPS) {
            // a lane to each box: page lane / (2 HALVES) of the block, K or V, 64 columns
            const int boxes = B / p.box * 2 * HALVES, x = lane % (2 * HALVES), row = lane / (2 * HALVES) * p.box;
            const CUtensorMap *map = x < HALVES ? &kmap : &vmap;
            uint8_t *dst = sm + x * HALF + row * 128;
            const int unheld = last_unheld(a, k.low, p.box);
            const auto page_at = [&](int b) {
                const int key = k.kb.block(b) * B + row;
                if (b >= b1 || lane >= boxes || key >= k.end) return -1;
                const int page = page_of(c, seq, key >> c.page_shift);
                if (page < 0 && (key < a.sinks || key > unheld)) g_rows_err = kDevErrRange;
                return page;
            };
            int page = page_at(b0), page2 = page_at(b0 + 1);
            for (int b = b0; b < b1; ++b, ++it) {
                const int page3 = page_at(b + 2);
                const uint32_t st = it % STAGES;
                if (it >= STAGES && !__all_sync(0xffffffffu, mbar_wait(&empty[st], (it / STAGES - 1) & 1))) {
                    atomicExch(&g_rows_err, kDevErrWaitEmpty);
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[st], 2 * TILE);
                __syncwarp();
                if (lane < boxes)  // no page: out of the tensor, reads as zeros
                    tma_load_4d(dst + st * 2 * TILE, map, &full[st], x % HALVES * 64, (k.kb.block(b) * B + row) & (c.page_size - 1),
                                head, page < 0 ? (int)min(c.pages, (int64_t)0x7fffffff) : page);
                page = page2, page2 = page3;
            }
            if (!ok)  // nothing of this CTA's may be in flight when it ends
                for (uint32_t y = it > STAGES ? it - STAGES : 0; y < it; ++y) mbar_wait(&full[y % STAGES], (y / STAGES) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (__syncthreads_or(!ok)) return;
        } else {
            // this thread's rows: lane / 4 and 8 later
            RowView rv[2];
            uint32_t tree[2], q[KS][4];
            const uint32_t *src[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = min((lane >> 2) + 8 * h, rows - 1), i = r / a.group;
                rv[h] = row_view(a, sv.len, sv.first, sv.count, i);
                check_held(a, seq, sv, rv[h], &g_rows_err);
                tree[h] = rv[h].bits ? __ldg(rv[h].bits) & ((1u << sv.count) - 1u) : 0u;  // count <= 16
                src[h] = reinterpret_cast<const uint32_t *>(
                    static_cast<const char *>(a.Q) +
                    ((int64_t)(sv.first + i) * a.q_stride + (int64_t)(head * a.group + r - i * a.group) * D) * 2);
            }
#pragma unroll
            for (int e = 0; e < KS; ++e)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int d = e * 16 + (x >> 1) * 8 + 2 * (lane & 3);
                    q[e][x] = d < D ? __ldg(src[x & 1] + d / 2) ^ flip : 0u;
                }
            const auto in = [&](int h, int j) {
                const int t = j - sv.len;
                return j < rv[h].end ? j >= rv[h].low || j < a.sinks : t < 32 && (tree[h] >> t & 1u);
            };
            float o[2 * KS][4];
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            // ldmatrix: this lane's row of K and V, its chunk 2 e + (0 or 1) swizzled by the row's low bits
            const int kr = (lane & 7) + ((lane >> 4) << 3), vr = (lane & 7) + (((lane >> 3) & 1) << 3), x6 = lane & 6;
            const int kb0 = (((lane >> 3) ^ lane) & 1) << 4, vb0 = (((lane >> 4) ^ lane) & 1) << 4;

            for (int b = b0; b < b1; ++b, ++it) {
                const uint32_t st = it % STAGES;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (it / STAGES) & 1))) {
                    atomicExch(&g_rows_err, kDevErrWaitFull);
                    ok = false;  // the loader waits for what is in flight
                    break;
                }
                const uint32_t kt = ring_s + st * 2 * TILE + warp * SUB * 128, vt = kt + TILE;
                const int key0 = k.kb.block(b) * B + warp * SUB;
                if (key0 >= k.end || (key0 + SUB <= k.low && key0 >= a.sinks)) {  // no row sees any of these
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[st]);
                    continue;
                }

                // four ldmatrix at a time, so that their latency is paid once
                float s[2][4] = {};
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    uint32_t f[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) ldsm4(f[e], kt + h * HALF + kr * 128 + kb0 + ((2 * e ^ x6) << 4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        mma16<T>(s[0], q[4 * h + e], f[e][0], f[e][1]);
                        mma16<T>(s[1], q[4 * h + e], f[e][2], f[e][3]);
                    }
                }
                uint32_t fv[4][4];  // V's first half, on its way during the softmax
#pragma unroll
                for (int e = 0; e < 4; ++e) ldsm4t(fv[e], vt + vr * 128 + vb0 + ((2 * e ^ x6) << 4));
                // whether some row does not see some of these keys
                const bool cut = key0 + SUB > k.whole || (key0 < k.high && key0 + SUB > a.sinks);
                if (cut) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (!in(x >> 1, key0 + n * 8 + 2 * (lane & 3) + (x & 1))) s[n][x] = -INFINITY;
                }
                float mx[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1])) * scale2;
                if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                        const float now = fmaxf(m[h], mx[h]);
                        const float f = now == -INFINITY ? 1.f : ex2(m[h] - now);
                        m[h] = now;
                        l[h] *= f;
#pragma unroll
                        for (int n = 0; n < 2 * KS; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
                    }
                }
                // a row that has seen nothing yet has scores of -infinity here: 2^-infinity = 0
                const float base[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[n][x] = ex2(fmaf(s[n][x], scale2, base[x >> 1]));
                        l[x >> 1] += s[n][x];
                    }
                uint32_t pr[4];
                pr[0] = Pair<T>::pack(s[0][0], s[0][1]);
                pr[1] = Pair<T>::pack(s[0][2], s[0][3]);
                pr[2] = Pair<T>::pack(s[1][0], s[1][1]);
                pr[3] = Pair<T>::pack(s[1][2], s[1][3]);
                bool special = false;
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    if (h > 0)
#pragma unroll
                        for (int e = 0; e < 4; ++e) ldsm4t(fv[e], vt + h * HALF + vr * 128 + vb0 + ((2 * e ^ x6) << 4));
                    if (cut) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                special |= any_special<T>(fv[e][i]);
                                fv[e][i] = without_special<T>(fv[e][i]);
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        mma16<T>(o[8 * h + 2 * e], pr, fv[e][0], fv[e][1]);
                        mma16<T>(o[8 * h + 2 * e + 1], pr, fv[e][2], fv[e][3]);
                    }
                }
                if (cut && __any_sync(0xffffffffu, special)) {  // rare: added where they are seen, key by key
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            sm_p[warp][(lane >> 2) + 8 * (x >> 1)][n * 8 + 2 * (lane & 3) + (x & 1)] = s[n][x];
                    __syncwarp();
                    for (int i = 0; i < SUB; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!in(h, key0 + i)) continue;
                            const float pv = sm_p[warp][(lane >> 2) + 8 * h][i];
#pragma unroll
                            for (int n = 0; n < 2 * KS; ++n) {
                                const uint32_t w = *reinterpret_cast<const uint32_t *>(
                                    sm + st * 2 * TILE + TILE + (n >> 3) * HALF + (warp * SUB + i) * 128 + (((n & 7) ^ (i & 7)) << 4) + 4 * (lane & 3));
                                const uint16_t lo = (uint16_t)w, hi = (uint16_t)(w >> 16);
                                if ((lo & Pair<T>::kExp) == Pair<T>::kExp) o[n][2 * h] += pv * Pair<T>::one(lo);
                                if ((hi & Pair<T>::kExp) == Pair<T>::kExp) o[n][2 * h + 1] += pv * Pair<T>::one(hi);
                            }
                        }
                }
                __syncwarp();  // the warp is through with this stage
                if (lane == 0) mbar_arrive(&empty[st]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                if ((lane & 3) == 0) sm_ml[warp][(lane >> 2) + 8 * h] = make_float2(m[h], l[h]);
            }
            if (__syncthreads_or(!ok)) return;
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(so + (warp * 16 + (lane >> 2) + 8 * h) * OS + n * 8 + 2 * (lane & 3)) =
                        make_float2(o[n][2 * h], o[n][2 * h + 1]);
        }
        __syncthreads();

        const bool alone = b0 == 0 && b1 == n;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + u.second) * 16;
        const auto out_at = [&](int r, int d) {
            const int i = r / a.group;
            return reinterpret_cast<uint32_t *>(
                static_cast<char *>(a.O) +
                ((int64_t)(sv.first + i) * a.o_stride + (int64_t)(head * a.group + r - i * a.group) * D + d) * 2);
        };
        for (int e = threadIdx.x; e < rows * pairs; e += NT) {
            const int r = e / pairs, d = 2 * (e - r * pairs);
            float mt = -INFINITY, lt = 0.f;
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mt = fmaxf(mt, sm_ml[w][r].x);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = sm_ml[w][r];
                if (saw_nothing(ml)) continue;
                const float f = ex2(ml.x - mt);
                const float2 x = *reinterpret_cast<const float2 *>(so + (w * 16 + r) * OS + d);
                lt += f * ml.y;
                v.x += f * x.x, v.y += f * x.y;
            }
            if (alone) {
                const float inv = lt != 0.f ? 1.f / lt : 0.f;
                *out_at(r, d) = Pair<T>::pack(v.x * inv, v.y * inv);
            } else {
                *reinterpret_cast<float2 *>(p.part + (slot + r) * D + d) = v;
                if (d == 0) p.ml[slot + r] = make_float2(mt, lt);
            }
        }
        if (!alone) {
            __syncthreads();
            if (threadIdx.x == 0) {
                __threadfence();  // the block's partial results before its ticket, the others' after it
                sm_last = atomicAdd(p.tickets + u.g0, 1) == u.used - 1;
                if (sm_last) p.tickets[u.g0] = 0;  // ready for the next call
                __threadfence();
            }
            __syncthreads();
            if (sm_last) {
                const int used = u.used;
                const int64_t slot0 = ((int64_t)u.g0 * 2 + u.first_second) * 16;
                const int quads = D / 4;
                for (int e = threadIdx.x; e < rows * quads; e += NT) {
                    const int r = e / quads, d = 4 * (e - r * quads);
                    float mt = -INFINITY, lt = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int y = 0; y < used; y += JOIN) {  // so many parts' loads at a time
                        float2 ml[JOIN];
                        float4 x[JOIN];
#pragma unroll
                        for (int i = 0; i < JOIN; ++i) {
                            const int64_t sl = (y + i == 0 ? slot0 : (int64_t)(u.g0 + min(y + i, used - 1)) * 32) + r;
                            ml[i] = __ldcg(&p.ml[sl]);
                            x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part + sl * D + d));
                            if (y + i >= used) ml[i] = make_float2(-INFINITY, 0.f);
                        }
                        float now = mt;
#pragma unroll
                        for (int i = 0; i < JOIN; ++i) now = fmaxf(now, ml[i].x);
                        const float f = now == -INFINITY ? 1.f : ex2(mt - now);
                        mt = now;
                        lt *= f, v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
                        for (int i = 0; i < JOIN; ++i) {
                            if (saw_nothing(ml[i])) continue;
                            const float w = ex2(ml[i].x - now);
                            lt += w * ml[i].y;
                            v.x += w * x[i].x, v.y += w * x[i].y, v.z += w * x[i].z, v.w += w * x[i].w;
                        }
                    }
                    const float inv = lt != 0.f ? 1.f / lt : 0.f;
                    *reinterpret_cast<uint2 *>(out_at(r, d)) =
                        make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
                }
            }
        }
        at = share.parts ? at + 1 : min(share.stop, u.u1);
        if (at >= share.stop) break;
        if (at >= seq_first + (share.parts ? share.parts : n + share.cost) * c.kv_heads) {  // the next sequence that has rows
            seq_first = at;
            do k = seq_keys(a, ++seq);
            while (k.kb.count == 0);
        }
        fence_proxy_async_smem();  // the ring was written by threads; TMA writes it next
        __syncthreads();
    }
}

template <typename T, int KS>
cudaError_t launch(const RowsArgs &p, int ctas, cudaStream_t s) {
    constexpr int SMEM = 6 * 2 * HALF + 1024;  // the ring, and alignment
    static_assert(SMEM - 1024 >= WARPS * 16 * (KS * 16 + 4) * 4, "the warps' O fit in the rings");
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void *)rows_kernel<T, KS>, SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap k, v;
    e = cache_tmap(&k, p.a.c, p.a.c.k, p.box);
    if (e == cudaSuccess) e = cache_tmap(&v, p.a.c, p.a.c.v, p.box);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_kernel<T, KS>, dim3((unsigned)ctas), NT, SMEM, s, k, v, p);
}

template <typename T>
cudaError_t launch_t(const RowsArgs &p, int ctas, cudaStream_t s) {
    return p.a.c.head_dim <= 64 ? launch<T, 4>(p, ctas, s) : launch<T, 8>(p, ctas, s);
}

}  // namespace

int cache_attention_rows_ctas(const CacheView &c, int sms) {
    const int64_t most = (int64_t)c.seqs * c.kv_heads * (((c.max_pages << c.page_shift) + B - 1) / B);  // blocks
    const int64_t ctas = (most + MIN_BLOCKS - 1) / MIN_BLOCKS;
    const int64_t cap = 2 * sms < kTickets ? 2 * sms : kTickets;
    return (int)(ctas < cap ? ctas : cap);
}

int64_t cache_attention_rows_workspace(const CacheView &c, int ctas) {
    return kTickets * 4 + (int64_t)ctas * 32 * (8 + (int64_t)c.head_dim * 4);
}

cudaError_t launch_cache_attention_rows(const CacheAttnArgs &a, int ctas, cudaStream_t s) {
    char *w = static_cast<char *>(a.ws);
    const int64_t most = (int64_t)a.c.seqs * a.c.kv_heads * (((a.c.max_pages << a.c.page_shift) + B - 1) / B + UNIT_COST);
    RowsArgs p{a, a.c.page_size < B ? a.c.page_size : B, most >= kShareLimit, nullptr, nullptr, nullptr};
    p.tickets = reinterpret_cast<int32_t *>(w);
    w += kTickets * 4;
    p.part = reinterpret_cast<float *>(w);
    p.ml = reinterpret_cast<float2 *>(w + (int64_t)ctas * 32 * a.c.head_dim * 4);
    return a.c.dtype == 0 ? launch_t<__half>(p, ctas, s) : launch_t<__nv_bfloat16>(p, ctas, s);
}

unsigned int cache_attention_rows_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_rows_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_rows_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
