// cache_attention_tiles.cu -- attention of many rows over a paged cache: chunks of prompts, wide draft
// trees, many query heads of one kv head.  Both products on the tensor cores (tcgen05), S, P and O in
// tensor memory.
//
// Rows.  The rows of a (sequence, kv head) are its new tokens times its query heads, row r being token
// r / group, head r % group, so grouped heads share every key they read.  A unit is 256 of them, as two
// tiles of 128 rows ("streams" 0 and 1), each with its own S (128 x 128 fp32, TMEM columns 0 and 128) and
// O (columns 256 and 384).  With 128 rows or fewer both streams take the same tile and every other block of
// keys, and are joined at the end: the tensor core then has a product to do while a softmax runs, as it
// has with two tiles.
//
// Mathematics.  Online softmax in base-2 units with a lazy reference: per block of 128 keys and stream
// S = Q K^T (A, B from shared memory); one thread per row reads its 128 scores and writes P = 2^(S - m),
// rounded to the cache's type, over S, with the reference m that it has; only if a score passed m by more than 8
// is m raised, O and l rescaled and P written again (so P stays below 2^8, and the maximum costs no latency of its
// own).  O += P V takes P from TMEM as A and V from shared memory as an MN-major B (V rows lie as the
// cache has them; nothing is transposed).
//
// Roles (384 threads, one CTA per SM): warps 0-3 and 4-7 the softmax of stream 0 and 1, warp 8 issues the MMAs,
// warp 9 the TMA loads (one box per page and 64 columns; a page past the end reads as zeros), warps 10 and 11 look
// after V where the mask cuts, as it arrives: they see every slot of the ring before the MMA warp does.  The MMA order
// PV(i), QK(i + 1) per stream, streams in turn, lets the tensor core work on one stream while the other is in its
// softmax.  (One issuing warp per stream was 9% slower: the streams' products then share the tensor core instead of
// taking turns, and their softmaxes coincide.  P handed over in halves was 15% slower: the MMA warp then waits inside
// a product with the other stream's ready.)  The MMA warp runs as one, with operands the compiler knows to be uniform:
// issued from one thread's branch the same products took 12% longer.
//
// Split.  One CTA per SM, each with an even share of all units' blocks (share_of), the ring of K and V blocks
// running through its units; the last CTA of a shared unit to finish joins the partial results in order.
//
// Bound: the tensor core and the softmax in turn, and the beginning and end of each unit.  Per pair of blocks (two
// streams, 128 keys) the products take 2,050 cycles at the rated speed; a stream's softmax is about 1,100 (128
// exponentials a thread) and with its waits 1,500.  Measured, one call: a chunk of 4,096 tokens on 12,289 under a window
// of 4,096, 32 heads over 8 of 128 columns, bf16: 256 us = 1,090 TFLOP/s, 58% of a library product's rate.  Of a CTA's
// 500,000 cycles there (by time stamps of one warp, which made the call 3% longer) 66% are 102 pairs at 3,280, 9% ten
// pairs that the mask cuts at 4,650, 7% the beginning of 4.2 units (the walk, Q, the first scores), 11% their last blocks,
// O and joins, 6% the launch, its wait and the share.  16 trees of 64 tokens on 2,500 to 8,000: 89 us, of which the
// pairs are 58%, beginnings 10%, ends 15%, the launch 15%; 4 chunks of 150 to 1,024 tokens on up to 700, 12 heads of 64:
// 22.3 us (45%, 10%, 15%, 28%); a chunk of 64 on 500: 18.5.
//
// What a row does not see: its score is replaced.  V rows that no row of the unit sees are zeroed in shared
// memory (0 x NaN), and where the mask cuts between rows V is looked through: infinities and NaN are taken out of the
// product and, when the unit's O is stored, added to the rows that see them (add_special).
#include "cache_attention.cuh"
#include "tcgen05.cuh"

namespace mm {

namespace {

__device__ unsigned int g_tiles_err;

constexpr int NT = 384, B = 128, ROWS = 256;
// blocks of a part, at least: joining takes as long as several (a chunk of 64 tokens on 500, 5 blocks: cut 23.3 us, whole
// 19.0; of 200 on 1,000, 10 blocks: 3 parts 19.5, 2 20.8, whole 24)
constexpr int MIN_BLOCKS = 4;
constexpr int WHOLE_BLOCKS = 8;  // units up to this are not cut when there are many (the 4 chunks: 22.3 us, cut 28.3)
constexpr int UNIT_COST = 4;     // what beginning and ending a unit takes, in blocks (16 trees: 89 us, with 0 98, with 8 92)
constexpr int HALF = 16384;      // 128 rows of 64 elements, 128-byte swizzle

template <int HALVES>
struct Plan {
    static constexpr int TILE = HALVES * HALF;  // Q tile, K or V block
    static constexpr int STAGES = HALVES == 2 ? 5 : 8;
    static constexpr int RING = 2 * TILE;       // behind Q; Q's place also holds a stream's O when two are joined
    static constexpr int BARS = RING + STAGES * TILE;
    static constexpr int ML = BARS + (3 * STAGES + 16) * 8;  // (m, l) of a stream's rows for the join
    static constexpr int BYTES = ML + 1024 + 1024;  // alignment slack
    static_assert(STAGES / 2 + 1 < 8 && BYTES + 512 <= 232448 && RING >= 128 * HALVES * 64 * 4, "shared memory");
};

struct TilesArgs {
    CacheAttnArgs a;
    int tiles;  // 256-row units of a (sequence, kv head), at most
    int box;    // keys of one TMA box
    int force_whole;
    FastDiv by_group, by_tiles;
    uint32_t *tickets;  // [kTickets]: parts done, and 2^16 for each whose V holds an infinity or NaN
    float2 *ml;                 // [CTAs][2][256]
    float4 *part;               // [CTAs][2][head_dim / 4][256]
};

// 32 fp32 columns of this thread's TMEM lane, begun: v holds them after the next tmem_ld_done.
__device__ __forceinline__ void tmem_ld32_begin(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
// Waits for the loads begun.  What is then computed from them is computed with the values that pass through
// here (a scale, two maxima), so that none of it can be moved in front of the wait.
__device__ __forceinline__ void tmem_ld_done(float2 &scale, float &m0, float &m1) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(scale.x), "+f"(scale.y), "+f"(m0), "+f"(m1) : : "memory");
}

// 16 columns of this thread's lane (the caller waits with tmem_wait_st)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The MMA warp runs as one, and what its instructions take is the same in all lanes and known to be (a reduction's
// result is): the lane that issues is a predicate, not a branch.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// D[tmem] (+)= A[smem] * B[smem], by the lane with `lead`.  The descriptors share their high word.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// bits of [0, 32) below n
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// which of keys j0 .. j0 + 31 the row sees
__device__ __forceinline__ uint32_t seen_bits(const RowView &r, int j0, int sinks, int len, int count) {
    uint32_t s = below(r.end - j0) & (~below(r.low - j0) | below(sinks - j0));
    if (r.bits) {
        const int t0 = j0 - len;
        if (t0 > -32 && t0 < count) {
            const int w = t0 >> 5, words = (count + 31) >> 5;
            const uint32_t lo = w >= 0 ? __ldg(r.bits + w) : 0u, hi = w + 1 < words ? __ldg(r.bits + w + 1) : 0u;
            s |= __funnelshift_r(lo, hi, (unsigned)(t0 & 31)) & below(count - t0);
        }
    }
    return s;
}

// What the 256 rows of tile item % tiles of sequence item / tiles need between them
struct UnitKeys {
    SeqView v;
    int row0, rows;            // rows 0: none
    int end, whole, low, high; // keys needed, and where the mask cuts between rows (see cut())
    KeyBlocks kb;              // count 0: no rows
    __device__ __forceinline__ bool cut(int key0, int sinks) const {
        return key0 + B > whole || (key0 < high && key0 + B > sinks);
    }
};
__device__ __forceinline__ UnitKeys unit_keys(const TilesArgs &p, int item) {
    UnitKeys k;
    const CacheAttnArgs &a = p.a;
    const int seq = p.by_tiles.div(item);
    k.v = seq_view(a, seq, &g_tiles_err);
    k.row0 = (item - seq * p.tiles) * ROWS;
    k.rows = min(k.v.count * a.group - k.row0, ROWS);
    k.kb = {0, 0, 0};
    k.end = k.whole = k.low = k.high = 0;
    if (k.rows <= 0) return k;
    const int i0 = p.by_group.div(k.row0), i1 = p.by_group.div(k.row0 + k.rows - 1), len = k.v.len;
    if (a.mask) {  // a row's depth is between 0 and count drafted tokens
        k.end = len + k.v.count, k.whole = len;
        if (a.window) k.low = len - a.window, k.high = len + k.v.count - a.window;
    } else {
        k.end = len + i1 + 1, k.whole = len + i0 + 1;
        if (a.window) k.low = len + i0 - a.window + 1, k.high = len + i1 - a.window + 1;
    }
    k.kb = key_blocks<B>(k.low, a.sinks, k.end);
    return k;
}

// The infinities and NaN that were taken out of V, added to the stored O of the unit's rows that see them.  The weight
// of a key that a row sees is above 0, so an infinity stays one whatever it is multiplied with.  By the 256 threads of
// the softmax; the keys are looked for again, a block at a time, into list[0 .. 127] (list[128]: how many).
// (As a function of its own it cost the kernel registers over the call: 48 sequences of 100 to 16,000 tokens, 8 new each,
// 142 us, inlined 132.)
template <typename T>
__device__ __forceinline__ void add_special(const CacheAttnArgs &a, const UnitKeys &k, const FastDiv &by_group, int seq, int head,
                                         volatile int *list) {
    const CacheView &c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool mine = 4 * lane < c.head_dim;
    const auto values = [&](int j) {  // of key j, this lane's four
        uint2 v = make_uint2(0, 0);
        const int page = page_of(c, seq, j >> c.page_shift);
        if (mine && page >= 0)
            v = *reinterpret_cast<const uint2 *>(c.v + ((int64_t)page * c.page_stride + head * c.head_stride +
                                                        (j & (c.page_size - 1)) * c.token_stride + 4 * lane) * 2);
        return v;
    };
    for (int b = 0; b < k.kb.count; ++b) {
        const int key0 = k.kb.block(b) * B;
        if (!k.cut(key0, a.sinks)) continue;
        if (threadIdx.x == 0) list[128] = 0;
        __syncwarp();
        bar_sync(1, 256);
        for (int j = key0 + warp; j < min(key0 + B, k.end); j += 8) {
            if (j >= a.sinks && j < k.low) continue;
            const uint2 v = values(j);
            if (__any_sync(0xffffffffu, any_special<T>(v.x) || any_special<T>(v.y)) && lane == 0)
                list[atomicAdd(const_cast<int *>(list) + 128, 1)] = j;
        }
        __syncwarp();
        bar_sync(1, 256);
        const int n = list[128];
        for (int r = warp; n > 0 && r < k.rows; r += 8) {
            const int i = by_group.div(k.row0 + r);
            const RowView rv = row_view(a, k.v.len, k.v.first, k.v.count, i);
            float add[4] = {-0.f, -0.f, -0.f, -0.f};  // what leaves every other value as it is
            bool any = false;
            for (int x = 0; x < n; ++x) {
                const int j = list[x];
                if (!sees(rv, j, a.sinks, k.v.len, k.v.count)) continue;
                const uint2 v = values(j);
                const uint16_t h[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y, (uint16_t)(v.y >> 16)};
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if ((h[y] & Pair<T>::kExp) == Pair<T>::kExp) add[y] += Pair<T>::one(h[y]), any = true;
            }
            if (any) {  // never a lane past head_dim, whose values are 0
                uint2 *out = reinterpret_cast<uint2 *>(
                    static_cast<char *>(a.O) + ((int64_t)(k.v.first + i) * a.o_stride +
                                                (int64_t)(head * a.group + k.row0 + r - i * a.group) * c.head_dim + 4 * lane) * 2);
                const uint2 o = *out;
                *out = make_uint2(Pair<T>::pack(Pair<T>::one((uint16_t)o.x) + add[0], Pair<T>::one((uint16_t)(o.x >> 16)) + add[1]),
                                  Pair<T>::pack(Pair<T>::one((uint16_t)o.y) + add[2], Pair<T>::one((uint16_t)(o.y >> 16)) + add[3]));
            }
        }
        __syncwarp();
        bar_sync(1, 256);  // before the list is written again
    }
}

// The units of one CTA, in order; every role walks them by itself.
struct Walk {
    Share share;
    int at, item, first;  // where the walk is, the item there and its beginning
    UnitKeys k;
    // the unit at hand: its head, the first of its blocks here and how many, the parts it is joined of
    int head, b0, n, used, g0;
    bool alone, second, first_second;

    __device__ __forceinline__ bool here(const TilesArgs &p) {  // false: no more
        if (at >= share.stop) return false;
        const int kv_heads = p.a.c.kv_heads;
        const int size = share.parts ? share.parts : k.kb.count + share.cost;
        if (at >= first + size * kv_heads) {
            first += size * kv_heads;
            do k = unit_keys(p, ++item);
            while (k.kb.count == 0);
        }
        const UnitPart u = unit_part(share, at, first, k.kb.count, MIN_BLOCKS);
        head = u.head, b0 = u.b0, n = u.b1 - u.b0, used = u.used, g0 = u.g0;
        alone = u.b0 == 0 && u.b1 == k.kb.count;
        second = u.second, first_second = u.first_second;
        at = share.parts ? at + 1 : min(share.stop, u.u1);
        return n > 0;  // else nothing of the unit but its cost, or a part that a short unit does not have
    }
};

template <typename T, int HALVES>
__global__ void __launch_bounds__(NT, 1) tiles_kernel(const __grid_constant__ CUtensorMap kmap,
                                                      const __grid_constant__ CUtensorMap vmap, const TilesArgs p) {
    using P = Plan<HALVES>;
    constexpr int ST = P::STAGES;
    extern __shared__ uint8_t raw[];
    __shared__ ShareScratch sm_share;
    __shared__ Walk sm_walk;  // of the softmax warps, which have no registers for it
    __shared__ int sm_last, sm_more;
    uint8_t *sm = smem_aligned<1024>(raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + P::BARS);
    uint64_t *full = bars, *empty = bars + ST, *seen = bars + 2 * ST, *s_full = bars + 3 * ST, *p_full = s_full + 2,
             *o_done = s_full + 4, *drain = s_full + 6, *q_full = s_full + 7;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 8);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // V of the CTA's unit i holds an infinity or NaN: poisons[i % 8] (warps 10 and 11 are at most ST / 2 + 1 units ahead)
    volatile int *poisons = reinterpret_cast<volatile int *>(tmem_slot + 2);

    const CacheAttnArgs &a = p.a;
    const CacheView &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31;
    // through a shuffle: the role branches below hold warp-wide instructions, and a compiler that can relate the
    // warp's number to tid may merge them with single-thread blocks before them
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int sinks = a.sinks;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1), mbar_init(seen + i, 2);
        for (int i = 0; i < 2; ++i) mbar_init(s_full + i, 1), mbar_init(p_full + i, 4), mbar_init(o_done + i, 1);
        mbar_init(drain, 1), mbar_init(q_full, 8);
        *fail = 0;
        for (int i = 0; i < 8; ++i) poisons[i] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();

    Walk w;
    {
        const int items = c.seqs * p.tiles;
        const auto blocks = [&](int i) { return i < items ? unit_keys(p, i).kb.count : 0; };
        const ShareRules rules = {MIN_BLOCKS, WHOLE_BLOCKS, UNIT_COST, p.force_whole};
        if (!share_of<NT>(items, c.kv_heads, rules, blocks, sm_share, w.share)) return;
        w.at = w.share.at, w.item = w.share.item, w.first = w.share.first;
        w.k = unit_keys(p, w.item);
    }
    __syncwarp();
    if (warp == 8) tmem_alloc(tmem_slot, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (tid == 0) sm_walk = w;
    __syncthreads();
    pdl_launch_dependents();  // not before: the next kernel's CTAs may take tensor memory, and then wait for this one
    const uint32_t tmem = *tmem_slot;
    const int steps = (c.head_dim + 15) / 16;  // 16-element steps of the head dimension
    const auto wait = [&](uint64_t *bar, uint32_t parity, unsigned code, bool asleep = false) {
        if (mbar_try_wait(bar, parity) || (!*fail && (asleep ? mbar_wait_sleep(bar, parity) : mbar_wait(bar, parity)))) return true;
        if (!*fail) atomicExch(&g_tiles_err, code);
        *fail = 1;
        return false;
    };
    // A unit's loads in the order of their use: K 0, V 0, K 1, ...; where the streams take turns K 0, then K i + 1
    // and V i.  The slots of the ring count on over the CTA's units.  The block whose V load y is, -1 for K:
    const auto block_of_v = [](int y, int n, bool single) {
        return !single ? (y & 1 ? y >> 1 : -1) : y == 2 * n - 1 ? n - 1 : y > 0 && !(y & 1) ? y / 2 - 1 : -1;
    };

    if (warp < 8) {
        const int s = warp >> 2, t = tid & 127;                 // stream, row of its tile
        const uint32_t quarter = (uint32_t)(warp & 3) << 21;    // this warp's 32 TMEM lanes
        const uint32_t ts = tmem + quarter + s * 128, to = tmem + quarter + 256 + s * 128;
        const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // > 0: a masked score stays -infinity
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;       // of Q, for a negative scale
        const int D = c.head_dim;
        uint32_t task = 0;  // blocks this stream has done
        bool ok = true;
        for (uint32_t units = 0;; ++units) {
            volatile int *poison = poisons + (units & 7);
            if (tid == 0) {
                Walk next = sm_walk;
                sm_more = !*fail && next.here(p);
                sm_walk = next;
            }
            __syncwarp();
            bar_sync(1, 256);
            if (!sm_more) break;
            const Walk &u = sm_walk;
            const SeqView sv = u.k.v;
            const int row0 = u.k.row0, nrows = u.k.rows, n = u.n, head = u.head;
            const KeyBlocks kb = u.k.kb;
            const int b0 = u.b0, whole = u.k.whole, high = u.k.high;
            const bool single = nrows <= 128;
            // Q into shared memory (both streams share a tile where one holds all rows), zeros past its rows and columns
            if (!single || s == 0) {
                constexpr int PER = HALVES * 8;  // 16-byte vectors of a row: this thread's is the same in all its rows
                const int x = t % PER, r1 = t / PER;
                const char *Q = static_cast<const char *>(a.Q) + ((int64_t)sv.first * a.q_stride + (int64_t)head * a.group * D + x * 8) * 2;
                uint8_t *to_sm = sm + s * P::TILE + (x >> 3) * HALF;
#pragma unroll 1
                for (int j0 = 0; j0 < PER; j0 += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = s * 128 + r1 + (j0 + j) * (128 / PER);
                        v[j] = make_uint4(0, 0, 0, 0);
                        if (r < nrows && x * 8 < D) {
                            const int i = p.by_group.div(row0 + r), h = row0 + r - i * a.group;
                            v[j] = __ldg(reinterpret_cast<const uint4 *>(Q + ((int64_t)i * a.q_stride + h * D) * 2));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = r1 + (j0 + j) * (128 / PER);
                        v[j].x ^= flip, v[j].y ^= flip, v[j].z ^= flip, v[j].w ^= flip;
                        *reinterpret_cast<uint4 *>(to_sm + r * 128 + (((x & 7) ^ (r & 7)) << 4)) = v[j];
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);

            const int r = single ? t : s * 128 + t;  // row of the unit's 256
            const int rc = min(r, nrows - 1), i = p.by_group.div(row0 + rc);
            const RowView rv = row_view(a, sv.len, sv.first, sv.count, i);
            check_held(a, p.by_tiles.div(u.item), sv, rv, &g_tiles_err);
            float m = -INFINITY, l = 0.f;
            int done = 0;
            for (int blk = single ? s : 0; blk < n; blk += single ? 2 : 1, ++done, ++task) {
                ok = __all_sync(0xffffffffu, wait(s_full + s, task & 1, kDevErrWaitMma));
                if (!ok) break;
                tc_fence_after_sync();
                const int key0 = kb.block(b0 + blk) * B;
                const bool cut = key0 + B > whole || (key0 < high && key0 + B > sinks);  // as UnitKeys::cut()
                float mx = -INFINITY;
                // The first block, or rows that have seen nothing yet: the maximum.  Where the mask cuts: -infinity into
                // S first.  (In the loop below the same took more code than the instruction cache likes, in every block.)
                if (cut || __any_sync(0xffffffffu, m == -INFINITY)) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float v[32];
                        tmem_ld32(ts + 32 * q, v);
                        if (cut) {
                            const uint32_t bits = seen_bits(rv, key0 + 32 * q, sinks, sv.len, sv.count);
                            uint32_t u0[16], u1[16];
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = bits >> x & 1u ? v[x] : -INFINITY;
#pragma unroll
                            for (int x = 0; x < 16; ++x) u0[x] = __float_as_uint(v[x]), u1[x] = __float_as_uint(v[16 + x]);
                            __syncwarp();
                            tmem_st16(ts + 32 * q, u0);
                            tmem_st16(ts + 32 * q + 16, u1);
                        }
#pragma unroll
                        for (int x = 0; x < 32; ++x) mx = fmaxf(mx, v[x]);
                    }
                    tmem_wait_st();
                    mx *= scale2;
                }
                // P in the cache's type, two to a register: S stays in TMEM until it is known to hold
                uint32_t pk[64];
                float2 sum;
#pragma unroll 1
                for (bool raise = __any_sync(0xffffffffu, mx > m + 8.f);; raise = true) {
                    if (raise) {
                        const float now = fmaxf(m, mx);
                        const float f = now == -INFINITY ? 1.f : ex2(m - now);
                        m = now;
                        l *= f;
                        if (done > 0) {
                            ok = __all_sync(0xffffffffu, wait(o_done + s, (task - 1) & 1, kDevErrWaitMma));
                            if (!ok) break;
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int d = 0; d < steps * 16; d += 32) {  // columns past head_dim hold nothing that is used
                                float o[32];
                                tmem_ld32(to + d, o);
                                uint32_t u0[16], u1[16];
#pragma unroll
                                for (int x = 0; x < 16; ++x) u0[x] = __float_as_uint(o[x] * f), u1[x] = __float_as_uint(o[16 + x] * f);
                                tmem_st16(to + d, u0);
                                tmem_st16(to + d + 16, u1);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : -m;
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                    float a0 = -INFINITY, a1 = -INFINITY;
                    const float2 one = make_float2(1.f, 1.f), bs = make_float2(base, base);
                    float2 sc = make_float2(scale2, scale2);
                    const auto probs = [&](float (&v)[32], int q) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            float2 e = ffma2(make_float2(v[2 * x], v[2 * x + 1]), sc, bs);
                            e.x = ex2(e.x), e.y = ex2(e.y);
                            pk[16 * q + x] = Pair<T>::pack(e.x, e.y);
                            if (x & 1)
                                sum1 = ffma2(e, one, sum1), a1 = fmaxf(fmaxf(a1, v[2 * x]), v[2 * x + 1]);
                            else
                                sum0 = ffma2(e, one, sum0), a0 = fmaxf(fmaxf(a0, v[2 * x]), v[2 * x + 1]);
                        }
                    };
                    // the next 32 columns are on their way while 32 are worked on
                    float va[32], vb[32];
                    tmem_ld32_begin(ts, va);
                    tmem_ld_done(sc, a0, a1);
                    tmem_ld32_begin(ts + 32, vb);
                    probs(va, 0);
                    tmem_ld_done(sc, a0, a1);
                    tmem_ld32_begin(ts + 64, va);
                    probs(vb, 1);
                    tmem_ld_done(sc, a0, a1);
                    tmem_ld32_begin(ts + 96, vb);
                    probs(va, 2);
                    tmem_ld_done(sc, a0, a1);
                    probs(vb, 3);
                    sum = make_float2(sum0.x + sum1.x, sum0.y + sum1.y);
                    mx = fmaxf(a0, a1) * scale2;
                    if (!__any_sync(0xffffffffu, mx > m + 8.f)) break;
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t u[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) u[x] = pk[16 * q + x];
                    tmem_st16(ts + 16 * q, u);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + s);
                l += sum.x + sum.y;
            }
            __syncwarp();
            if (ok && done > 0) ok = __all_sync(0xffffffffu, wait(o_done + s, (task - 1) & 1, kDevErrWaitMma));
            tc_fence_after_sync();
            const auto store = [&](int d, const float (&o)[32], float f) {
                char *out = static_cast<char *>(a.O) + ((int64_t)(sv.first + i) * a.o_stride +
                                                        (int64_t)(head * a.group + row0 + rc - i * a.group) * D) * 2;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (d + 8 * x < D)
                        *reinterpret_cast<uint4 *>(out + (d + 8 * x) * 2) =
                            make_uint4(Pair<T>::pack(o[8 * x] * f, o[8 * x + 1] * f), Pair<T>::pack(o[8 * x + 2] * f, o[8 * x + 3] * f),
                                       Pair<T>::pack(o[8 * x + 4] * f, o[8 * x + 5] * f), Pair<T>::pack(o[8 * x + 6] * f, o[8 * x + 7] * f));
            };
            bool special = false;  // V of the unit holds infinities or NaN that were taken out of it
            if (!u.alone) {
                // partial results: both streams' of the same rows where they share a tile
                const int64_t slot = (int64_t)blockIdx.x * 2 + u.second;
                for (int d = 0; d < D; d += 32) {
                    float o[32];
                    if (done > 0) {
                        tmem_ld32(to + d, o);
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = 0.f;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (d + 4 * x < D)
                            p.part[(slot * (D / 4) + d / 4 + x) * ROWS + s * 128 + t] =
                                make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                }
                p.ml[slot * ROWS + s * 128 + t] = make_float2(m, l);
                tc_fence_before_sync();
                bar_sync(1, 256);
                if (tid == 0) {
                    __threadfence();  // the unit's partial results before its ticket, the others' after it
                    const uint32_t mine = *poison ? 0x10001u : 1u, all = atomicAdd(p.tickets + u.g0, mine) + mine;
                    const bool last = (all & 0xffffu) == (uint32_t)u.used;
                    sm_last = last ? (all >> 16 ? 2 : 1) : 0;
                    if (last) {
                        __threadfence();
                        p.tickets[u.g0] = 0;  // ready for the next call
                    }
                    *poison = 0;
                }
                __syncwarp();
                bar_sync(1, 256);
                const int last = sm_last;
                special = last == 2;
                if (last) {
                    const int per = single ? 2 : 1, sources = per * u.used;
                    const auto slot_of = [&](int y) {  // source y: slot * 256 + its rows' first
                        const int g = y / per;
                        return (int64_t)((u.g0 + g) * 2 + (g == 0 && u.first_second)) * ROWS;
                    };
                    const int64_t half = tid & 255;
                    if (half < nrows) {
                        float mt = -INFINITY, lt = 0.f;
                        for (int y = 0; y < sources; ++y) {
                            const float2 q = __ldcg(p.ml + slot_of(y) + (single ? (y & 1) * 128 : 0) + half);
                            if (saw_nothing(q)) continue;
                            const float now = fmaxf(mt, q.x);
                            lt = lt * (mt == -INFINITY ? 1.f : ex2(mt - now)) + q.y * ex2(q.x - now);
                            mt = now;
                        }
                        const float inv = lt != 0.f ? 1.f / lt : 0.f;
                        const int ri = p.by_group.div(row0 + (int)half), rh = row0 + (int)half - ri * a.group;
                        uint4 *out = reinterpret_cast<uint4 *>(static_cast<char *>(a.O) +
                                                               ((int64_t)(sv.first + ri) * a.o_stride + (int64_t)(head * a.group + rh) * D) * 2);
#pragma unroll 1
                        for (int x = 0; x < D / 8; x += 4) {  // 32 columns at a time, so that many loads are in flight
                            float o[32] = {};
#pragma unroll 1
                            for (int y = 0; y < sources; y += 2) {
                                float f[2];
                                float4 g[2][8];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int yk = min(y + k, sources - 1);
                                    const int64_t at = slot_of(yk), row = (single ? (yk & 1) * 128 : 0) + half;
                                    const float2 q = __ldcg(p.ml + at + row);
                                    f[k] = q.x > -INFINITY && y + k < sources ? ex2(q.x - mt) * inv : 0.f;
                                    const float4 *src = p.part + at * (D / 4) + (int64_t)(2 * x) * ROWS + row;
#pragma unroll
                                    for (int z = 0; z < 8; ++z)
                                        // a part past the last adds 0, not 0 times what the last one holds (an infinity, say)
                                        g[k][z] = 2 * x + z < D / 4 && y + k < sources ? __ldcg(src + z * ROWS) : make_float4(0.f, 0.f, 0.f, 0.f);
                                }
#pragma unroll
                                for (int k = 0; k < 2; ++k)
#pragma unroll
                                    for (int z = 0; z < 8; ++z) {
                                        o[4 * z] += f[k] * g[k][z].x, o[4 * z + 1] += f[k] * g[k][z].y;
                                        o[4 * z + 2] += f[k] * g[k][z].z, o[4 * z + 3] += f[k] * g[k][z].w;
                                    }
                            }
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (x + z < D / 8)
                                    out[x + z] = make_uint4(Pair<T>::pack(o[8 * z], o[8 * z + 1]), Pair<T>::pack(o[8 * z + 2], o[8 * z + 3]),
                                                            Pair<T>::pack(o[8 * z + 4], o[8 * z + 5]), Pair<T>::pack(o[8 * z + 6], o[8 * z + 7]));
                        }
                    }
                }
            } else if (single) {
                float *so = reinterpret_cast<float *>(sm);  // [d][row], in Q's place
                float2 *sm_ml = reinterpret_cast<float2 *>(sm + P::ML);
                bar_sync(1, 256);                           // both streams are through with Q
                if (s == 1) {
                    if (done > 0)
                        for (int d = 0; d < D; d += 32) {
                            float o[32];
                            tmem_ld32(to + d, o);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (d + x < D) so[(d + x) * 128 + t] = o[x];
                        }
                    sm_ml[t] = make_float2(m, l);
                }
                tc_fence_before_sync();
                bar_sync(1, 256);
                if (s == 0) {
                    const float2 other = sm_ml[t];
                    const float mt = fmaxf(m, other.x);
                    const float f0 = m == -INFINITY ? 0.f : ex2(m - mt), f1 = other.x == -INFINITY ? 0.f : ex2(other.x - mt);
                    const float lt = l * f0 + other.y * f1, inv = lt != 0.f ? 1.f / lt : 0.f;
                    for (int d = 0; d < D; d += 32) {
                        float o[32];
                        tmem_ld32(to + d, o);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = o[x] * (f0 * inv) + (f1 > 0.f && d + x < D ? so[(d + x) * 128 + t] * (f1 * inv) : 0.f);
                        if (r < nrows) store(d, o, 1.f);
                        __syncwarp();
                    }
                    tc_fence_before_sync();
                }
                if (tid == 0) sm_last = *poison, *poison = 0;
                __syncwarp();
                bar_sync(1, 256);  // before Q's place is written again
                special = sm_last != 0;
            } else {
                const float inv = l != 0.f ? 1.f / l : 0.f;
                for (int d = 0; d < D; d += 32) {
                    float o[32];
                    tmem_ld32(to + d, o);
                    if (r < nrows) store(d, o, inv);
                    __syncwarp();
                }
                tc_fence_before_sync();
                if (tid == 0) sm_last = *poison, *poison = 0;
                __syncwarp();
                bar_sync(1, 256);
                special = sm_last != 0;
            }
            // (the same for all 256 threads, also where a wait has failed: there are barriers inside)
            if (special) add_special<T>(a, u.k, p.by_group, p.by_tiles.div(u.item), head, reinterpret_cast<volatile int *>(sm));
            __syncwarp();
            bar_sync(1, 256);  // the walk may go on
        }
        tc_fence_before_sync();
        __syncthreads();  // tensor memory has been read
    } else {
        if (warp == 8) {
            const uint32_t lead = lane == 0, full_warp = 0xffffffffu;
            const uint32_t fmt = c.dtype == 0 ? kFmtF16 : kFmtBF16;
            const uint32_t iqk = make_idesc(fmt, fmt, B, 128);
            const uint32_t ipv = make_idesc(fmt, fmt, (uint32_t)steps * 16, 128) | 1u << 16;  // V: MN-major
            // descriptors differ in their address alone (bytes / 16 in the low bits)
            const uint64_t dk = sdesc_kmajor_sw128(0), dv = sdesc_make(0, HALF, 1024, kSdescSw128);
            const uint32_t k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
            const uint32_t base = uniform((smem_u32(sm) & 0x3FFFFu) >> 4), ring = base + P::RING / 16;
            const uint32_t acc = uniform(tmem), bar = uniform(smem_u32(bars));
            const auto signal = [&](const uint64_t *b) { commit(bar + (uint32_t)(b - bars) * 8, lead); };
            const auto signal_empty = [&](uint32_t stage) { commit(bar + (ST + stage) * 8, lead); };
            uint32_t units = 0, task0 = 0, task1 = 0;
            uint32_t st = 0, ph = 0;  // the ring's next slot: its stage, the parity of its barrier
            bool ok = true;
            const auto all = [&](uint64_t *b, uint32_t parity) { return __all_sync(full_warp, wait(b, parity, kDevErrWaitFull)) != 0; };
            while (ok && __all_sync(full_warp, w.here(p))) {
                const int n = (int)uniform((uint32_t)w.n);
                const bool single = __any_sync(full_warp, w.k.rows <= 128);
                // a lane to each of what has to be there
                const auto there = [&]() { return all(lane == 0 ? full + st : seen + st, ph); };
                const auto on = [&]() {
                    const uint32_t wrap = st + 1 == ST;
                    st = uniform(wrap ? 0 : st + 1), ph ^= wrap;
                };
                const auto qk = [&](int s, uint32_t stage) {
                    const uint32_t q = (uint32_t)dk + base + (single ? 0 : s * (P::TILE / 16));
                    const uint32_t k = (uint32_t)dk + ring + stage * (P::TILE / 16);
#pragma unroll
                    for (int e = 0; e < HALVES * 4; ++e) {  // columns past head_dim are zeros in Q and K
                        const uint32_t off = (e >> 2) * (HALF / 16) + (e & 3) * 2;
                        // n > 0: the flag of the first one has to be a value of the run.  As a constant 0, in the
                        // unrolled loop, the product came out added to what was in tensor memory.
                        mma_ss(acc + s * 128, q + off, k + off, k_hi, iqk, e > 0 || n <= 0, lead);
                    }
                    signal(s_full + s);
                };
                const auto pv = [&](int s, uint32_t stage, int begun) {
                    const uint32_t v = (uint32_t)dv + ring + stage * (P::TILE / 16);
#pragma unroll
                    for (int e = 0; e < B / 16; ++e)
                        mma_ts(acc + 256 + s * 128, acc + s * 128 + e * 8, v + e * 128, v_hi, ipv, begun > 0 || e > 0, lead);
                    signal(o_done + s);
                };
                const auto probs = [&](int s) { return all(p_full + s, (s ? task1++ : task0++) & 1); };
                ok = all(q_full, units++ & 1) && there();
                if (!ok) break;
                tc_fence_after_sync();
                qk(0, st);
                if (!single) qk(1, st);
                signal_empty(st);
                on();
                if (single && n > 1) {
                    ok = there();
                    if (!ok) break;
                    tc_fence_after_sync();
                    qk(1, st);
                    signal_empty(st);
                    on();
                }
                if (single) {  // blocks in turn: V i and K i + 2
                    for (int i = 0; ok && i < n; ++i) {
                        ok = there() && (i & 1 ? probs(1) : probs(0));
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (i & 1)
                            pv(1, st, i > 1);
                        else
                            pv(0, st, i > 1);
                        signal_empty(st);
                        on();
                        if (i + 2 < n) {
                            ok = there();
                            if (!ok) break;
                            tc_fence_after_sync();
                            if (i & 1)
                                qk(1, st);
                            else
                                qk(0, st);
                            signal_empty(st);
                            on();
                        }
                    }
                } else {
                    for (int i = 0; i < n; ++i) {  // V i and K i + 1, for one stream and then the other
                        const bool more = i + 1 < n;
                        const uint32_t sv = st, pv_there = ph;
                        on();
                        const uint32_t sk = st;
                        // a lane to each of what has to be there: V i, K i + 1, P
                        uint64_t *b = p_full;
                        uint32_t parity = task0++ & 1;
                        if (lane < 2) b = (lane ? seen : full) + sv, parity = pv_there;
                        if ((lane == 2 || lane == 3) && more) b = (lane == 3 ? seen : full) + sk, parity = ph;
                        ok = all(b, parity);
                        if (!ok) break;
                        tc_fence_after_sync();
                        pv(0, sv, i);
                        if (more) qk(0, sk);
                        ok = probs(1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        pv(1, sv, i);
                        if (more) qk(1, sk);
                        signal_empty(sv);
                        if (more) {
                            signal_empty(sk);
                            on();
                        }
                    }
                }
            }
            signal(drain);
            if (!mbar_wait(drain, 0) && lead) atomicExch(&g_tiles_err, kDevErrDrain);
            __syncwarp();
        } else if (warp == 9) {
            // a lane to each box: page lane / HALVES of the block, 64-column half lane % HALVES
            const int ops = B / p.box * HALVES;
            const int row = lane / HALVES * p.box, col = lane % HALVES * 64;
            uint8_t *dst = sm + P::RING + (lane % HALVES) * HALF + row * 128;
            uint32_t x = 0;
            bool ok = true;
            while (ok && w.here(p)) {
                const int n = w.n, seq = w.item / p.tiles;
                const int unheld = last_unheld(a, w.k.low, p.box);
                const auto page_at = [&](int blk) {
                    const int key = w.k.kb.block(w.b0 + blk) * B + row;
                    if (blk >= n || lane >= ops || key >= w.k.end) return -1;
                    const int page = page_of(c, seq, key >> c.page_shift);
                    if (page < 0 && (key < sinks || key > unheld)) g_tiles_err = kDevErrRange;
                    return page;
                };
                const auto load = [&](const CUtensorMap *map, int blk, int page) {
                    const uint32_t st = x % ST;
                    if (x >= ST && !__all_sync(0xffffffffu, wait(empty + st, (x / ST - 1) & 1, kDevErrWaitEmpty))) return false;
                    if (lane == 0) mbar_arrive_expect_tx(full + st, P::TILE);
                    __syncwarp();
                    if (lane < ops)  // no page: out of the tensor, reads as zeros
                        tma_load_4d(dst + st * P::TILE, map, full + st, col, (w.k.kb.block(w.b0 + blk) * B + row) & (c.page_size - 1),
                                    w.head, page < 0 ? (int)min(c.pages, (int64_t)0x7fffffff) : page);
                    ++x;
                    return true;
                };
                // pages of block i, i + 1 and, ahead of their use, i + 2
                int pg0 = page_at(0), pg1 = page_at(1);
                ok = load(&kmap, 0, pg0);
                const bool single = w.k.rows <= 128;
                for (int i = 0; ok && i < n; ++i) {
                    const int pg2 = page_at(i + 2);
                    if (!single) ok = load(&vmap, i, pg0);
                    if (ok && i + 1 < n) ok = load(&kmap, i + 1, pg1);
                    if (ok && single) ok = load(&vmap, i, pg0);
                    pg0 = pg1, pg1 = pg2;
                }
            }
            // nothing of this CTA's may be in flight when it ends
            for (uint32_t y = x > ST ? x - ST : 0; y < x; ++y)
                if (!mbar_wait(full + y % ST, (y / ST) & 1)) atomicExch(&g_tiles_err, kDevErrDrain);
            __syncwarp();
        } else {
            // Every slot of the ring is waited for in order (a barrier's phase may not pass unseen), and passed on
            uint32_t st = 0, ph = 0;
            bool ok = true;
            for (uint32_t units = 0; ok && w.here(p); ++units) {
                const int n = w.n, end = w.k.end, low = w.k.low;
                const bool single = w.k.rows <= 128;
                for (int y = 0; y < 2 * n; ++y) {
                    ok = __all_sync(0xffffffffu, wait(full + st, ph, kDevErrWaitFull, true));
                    if (!ok) break;
                    const int i = block_of_v(y, n, single), key0 = i < 0 ? 0 : w.k.kb.block(w.b0 + i) * B;
                    if (i >= 0 && w.k.cut(key0, sinks)) {
                        uint8_t *v = sm + P::RING + st * P::TILE;
                        // infinite or NaN: the magnitude's bits are kExp or more, and adding this carries into bit 15
                        constexpr uint32_t up = (0x8000u - Pair<T>::kExp) * 0x10001u;
#pragma unroll 1
                        for (int e0 = tid - 320; e0 < P::TILE / 16; e0 += 8 * 64) {
                            uint4 u[8];
                            uint32_t special = 0;
#pragma unroll
                            for (int k = 0; k < 8; ++k) u[k] = *reinterpret_cast<const uint4 *>(v + (e0 + 64 * k) * 16);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int e = e0 + 64 * k, j = key0 + ((e & 1023) >> 3);
                                if (j >= end || (j >= sinks && j < low)) {
                                    *reinterpret_cast<uint4 *>(v + e * 16) = make_uint4(0, 0, 0, 0);
                                } else {
                                    special |= (u[k].x & 0x7fff7fffu) + up;
                                    special |= (u[k].y & 0x7fff7fffu) + up;
                                    special |= (u[k].z & 0x7fff7fffu) + up;
                                    special |= (u[k].w & 0x7fff7fffu) + up;
                                }
                            }
                            if (special & 0x80008000u) {
                                poisons[units & 7] = 1;
#pragma unroll 1
                                for (int e = e0; e < e0 + 8 * 64; e += 64) {
                                    uint4 *at = reinterpret_cast<uint4 *>(v + e * 16);
                                    uint4 x = *at;
                                    x.x = without_special<T>(x.x), x.y = without_special<T>(x.y);
                                    x.z = without_special<T>(x.z), x.w = without_special<T>(x.w);
                                    *at = x;
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(seen + st);
                    if (++st == ST) st = 0, ph ^= 1;
                }
            }
            __syncwarp();
        }
        __syncthreads();  // tensor memory has been read
        if (warp == 8) {
            tc_fence_after_sync();
            tmem_relinquish();
            tmem_dealloc(tmem, 512);
        }
    }
}

int tile_count(int group, int64_t max_q) { return (int)((max_q * group + ROWS - 1) / ROWS); }

template <typename T, int HALVES>
cudaError_t launch(const TilesArgs &p, int ctas, cudaStream_t s) {
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void *)tiles_kernel<T, HALVES>, Plan<HALVES>::BYTES);
    if (e != cudaSuccess) return e;
    CUtensorMap k, v;
    e = cache_tmap(&k, p.a.c, p.a.c.k, p.box);
    if (e == cudaSuccess) e = cache_tmap(&v, p.a.c, p.a.c.v, p.box);
    if (e != cudaSuccess) return e;
    return launch_pdl(tiles_kernel<T, HALVES>, dim3((unsigned)ctas), NT, Plan<HALVES>::BYTES, s, k, v, p);
}

}  // namespace

int cache_attention_tiles_ctas(const CacheView &c, int group, int64_t max_q, int sms) {
    const int64_t blocks = ((c.max_pages << c.page_shift) + B - 1) / B;
    const int64_t most = (int64_t)tile_count(group, max_q) * c.seqs * c.kv_heads * ((blocks + MIN_BLOCKS - 1) / MIN_BLOCKS);
    const int cap = sms < kTickets ? sms : kTickets;
    return (int)(most < cap ? most : cap);
}

int64_t cache_attention_tiles_workspace(const CacheView &c, int ctas) {
    return kTickets * 4 + (int64_t)ctas * 2 * ROWS * (8 + (int64_t)c.head_dim * 4);
}

cudaError_t launch_cache_attention_tiles(const CacheAttnArgs &a, int ctas, cudaStream_t s) {
    const int tiles = tile_count(a.group, a.max_q);
    const int64_t units = (int64_t)tiles * a.c.seqs * a.c.kv_heads;
    const int64_t most = units * (((a.c.max_pages << a.c.page_shift) + B - 1) / B + UNIT_COST);
    TilesArgs p{a, tiles, a.c.page_size < B ? a.c.page_size : B, most >= kShareLimit, fast_div(a.group), fast_div(tiles),
                nullptr, nullptr, nullptr};
    char *w = static_cast<char *>(a.ws);
    p.tickets = reinterpret_cast<uint32_t *>(w);
    w += kTickets * 4;
    p.part = reinterpret_cast<float4 *>(w);
    w += (int64_t)ctas * 2 * ROWS * a.c.head_dim * 4;
    p.ml = reinterpret_cast<float2 *>(w);
    if (a.c.dtype == 0) return a.c.head_dim <= 64 ? launch<__half, 1>(p, ctas, s) : launch<__half, 2>(p, ctas, s);
    return a.c.head_dim <= 64 ? launch<__nv_bfloat16, 1>(p, ctas, s) : launch<__nv_bfloat16, 2>(p, ctas, s);
}

unsigned int cache_attention_tiles_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_tiles_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_tiles_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
