// cache_attention_tiles.cu -- attention of many rows over a paged cache: chunks of prompts, wide draft
// trees, many query heads of one kv head.  Both products on the tensor cores (tcgen05), S, P and O in
// tensor memory.
//
// Rows.  The rows of a (sequence, kv head) are its new tokens times its query heads, row r being token
// r / group, head r % group, so grouped heads share every key they read.  A CTA takes 256 of them as two
// tiles of 128 rows ("streams" 0 and 1), each with its own S (128 x 128 fp32, TMEM columns 0 and 128) and
// O (columns 256 and 384).  With 128 rows or fewer both streams take the same tile and every other block of
// keys, and are joined at the end: the tensor core then has a product to do while a softmax runs, as it
// has with two tiles.
//
// Mathematics.  Online softmax in base-2 units with a lazy reference: O and l are rescaled only where a
// row's maximum passes its reference by more than 8 (P stays below 2^8).  Per block of 128 keys and stream:
// S = Q K^T (A, B from shared memory), one thread per row reads its 128 scores, P = 2^(S - m) rounded to
// the cache's type goes back to TMEM over S, and O += P V takes P from TMEM as A and V from shared memory as
// an MN-major B (V rows lie as the cache has them; nothing is transposed).
//
// Roles (384 threads, one CTA per SM): warps 0-3 and 4-7 the softmax of stream 0 and 1, warp 8 issues the MMAs, warp 9 the TMA loads (one box per page and 64 columns; a page past
// the end reads as zeros), warps 10 and 11 look after V where the mask cuts.  The MMA order PV(i), QK(i + 1)
// per stream lets the tensor core work on one stream while the other is in its softmax.
//
// What a row does not see: its score is replaced.  V rows that no row of the CTA sees are zeroed in shared
// memory (0 x NaN), and where the mask cuts between rows V is looked through: if it holds an infinity or NaN,
// the CTA's rows are computed again by the definition, key by key.
//
// The keys of a unit (256 rows) are split over CTAs where there are few units; the last CTA to finish joins
// the partial results in the order of the splits.
#include "cache_attention.cuh"
#include "tcgen05.cuh"

namespace mm {

namespace {

__device__ unsigned int g_tiles_err;

constexpr int NT = 384, B = 128, ROWS = 256;
constexpr int MIN_BLOCKS = 4;   // blocks of a split, at least
constexpr int MAX_SPLITS = 32;
constexpr int HALF = 16384;     // 128 rows of 64 elements, 128-byte swizzle

template <int HALVES>
struct Plan {
    static constexpr int TILE = HALVES * HALF;  // Q tile, K or V block
    static constexpr int STAGES = HALVES == 2 ? 5 : 8;
    static constexpr int RING = 2 * TILE, BARS = RING + STAGES * TILE;
    static constexpr int BYTES = BARS + 512 + 1024;  // barriers and flags; alignment slack
    static constexpr int ML = RING + 128 * 128 * 4;  // after the loop: rows' (m, l), behind a stream's O
    static_assert(BYTES + 1024 <= 232448 && ML + ROWS * 8 <= BARS, "shared memory");
};

struct TilesArgs {
    CacheAttnArgs a;
    int splits, tiles;  // 256-row units per (sequence, kv head)
    int box;            // keys of one TMA box
    int32_t *tickets, *poison;  // per unit
    float2 *ml;                 // [units][splits][256]
    float4 *part;               // [units][splits][head_dim / 4][256]
};

// All 128 fp32 columns of this thread's TMEM lane; the wait is part of the statement, so that no register
// is read early.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]),
          "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]),
          "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]),
          "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]),
          "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]), "=f"(v[64]),
          "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]), "=f"(v[72]),
          "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]), "=f"(v[80]),
          "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]), "=f"(v[88]),
          "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]), "=f"(v[96]),
          "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]), "=f"(v[104]),
          "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
          "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]),
          "=f"(v[119]), "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]),
          "=f"(v[126]), "=f"(v[127])
        : "r"(taddr)
        : "memory");
}

// 32 columns of this thread's lane (the caller waits with tmem_wait_st)
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

template <typename T, int HALVES>
__global__ void __launch_bounds__(NT, 1) tiles_kernel(const __grid_constant__ CUtensorMap kmap,
                                                      const __grid_constant__ CUtensorMap vmap, const TilesArgs p) {
    using P = Plan<HALVES>;
    constexpr int ST = P::STAGES;
    extern __shared__ uint8_t raw[];
    __shared__ int sm_last;
    uint8_t *sm = smem_aligned<1024>(raw);
    float2 *sm_ml = reinterpret_cast<float2 *>(sm + P::ML);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + P::BARS);
    uint64_t *full = bars, *empty = bars + ST, *s_full = bars + 2 * ST, *p_full = s_full + 2, *o_done = s_full + 4,
             *drain = s_full + 6, *fix = s_full + 7, *fixed = s_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 9);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *poison = reinterpret_cast<int *>(tmem_slot + 2);

    const CacheAttnArgs &a = p.a;
    const CacheView &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x % p.splits, unit = blockIdx.x / p.splits;
    const int head = unit % c.kv_heads, seq = unit / c.kv_heads % c.seqs;
    const int tile = p.tiles - 1 - unit / c.kv_heads / c.seqs;  // the later rows, with more keys, first

    pdl_launch_dependents();
    pdl_wait();
    const SeqView sv = seq_view(a, seq, &g_tiles_err);
    const int row0 = tile * ROWS;
    const int nrows = min(sv.count * a.group - row0, ROWS);
    if (nrows <= 0) return;
    const bool single = nrows <= 128;
    const int i_first = row0 / a.group, i_last = (row0 + nrows - 1) / a.group;
    // keys the rows need between them, and where the mask cuts between rows: see KeyBlocks and cut()
    int end, whole, low = 0, high = 0;
    if (a.mask) {  // a row's depth is between 0 and count drafted tokens
        end = sv.len + sv.count, whole = sv.len;
        if (a.window) low = sv.len - a.window, high = sv.len + sv.count - a.window;
    } else {
        end = sv.len + i_last + 1, whole = sv.len + i_first + 1;
        if (a.window) low = sv.len + i_first - a.window + 1, high = sv.len + i_last - a.window + 1;
    }
    const int sinks = a.sinks;
    const KeyBlocks kb = key_blocks<B>(low, sinks, end);
    const int per = max((kb.count + p.splits - 1) / p.splits, MIN_BLOCKS);
    const int used = (kb.count + per - 1) / per;
    if (split >= used) return;
    const int b0 = split * per;
    const int n = min(kb.count, b0 + per) - b0;
    const auto key_of = [&](int i) { return kb.block(b0 + i) * B; };
    const auto cut = [&](int key0) { return key0 + B > whole || (key0 < high && key0 + B > sinks); };
    // loads in the order of their use: K 0, then K i + 1 and V i
    const auto slot_k = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
    const auto slot_v = [&](int i) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

    const int steps = (c.head_dim + 15) / 16;  // 16-element steps of the head dimension
    if (warp == 8) tmem_alloc(tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(s_full + i, 1), mbar_init(p_full + i, 128), mbar_init(o_done + i, 1);
        mbar_init(drain, 1), mbar_init(fix, 1), mbar_init(fixed, 64);
        *fail = 0, *poison = 0;
        fence_mbar_init();
    }
    // Q: both tiles (one where the streams share it), columns past head_dim zero, negated for a negative scale
    {
        const int per_row = HALVES * 8, total = (single ? 128 : ROWS) * per_row;
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        for (int e = tid; e < total; e += NT) {
            const int r = e / per_row, x = e - r * per_row;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < nrows && x * 8 < c.head_dim) {
                const int i = (row0 + r) / a.group, h = row0 + r - i * a.group;
                v = __ldg(reinterpret_cast<const uint4 *>(
                    static_cast<const char *>(a.Q) +
                    ((int64_t)(sv.first + i) * a.q_stride + (int64_t)(head * a.group + h) * c.head_dim + x * 8) * 2));
                v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
            }
            *reinterpret_cast<uint4 *>(sm + (r >> 7) * P::TILE + (x >> 3) * HALF + (r & 127) * 128 +
                                       (((x & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const auto wait = [&](uint64_t *bar, uint32_t parity, unsigned code) {
        if (!*fail && mbar_wait(bar, parity)) return true;
        if (!*fail) atomicExch(&g_tiles_err, code);
        *fail = 1;
        return false;
    };

    if (warp < 8) {
        const int s = warp >> 2, t = tid & 127;  // stream, row of its tile
        const int r = single ? t : s * 128 + t;  // row of the unit's 256
        const int rc = min(r, nrows - 1), i = (row0 + rc) / a.group;
        const RowView rv = row_view(a, sv.len, sv.first, sv.count, i);
        const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
        const uint32_t ts = tmem + quarter + s * 128, to = tmem + quarter + 256 + s * 128;
        const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // > 0: a masked score stays -infinity
        float m = -INFINITY, l = 0.f;
        int done = 0;
        bool ok = true;
        for (int blk = single ? s : 0; blk < n; blk += single ? 2 : 1, ++done) {
            ok = __all_sync(0xffffffffu, wait(s_full + s, done & 1, kDevErrWaitMma));
            if (!ok) break;
            tc_fence_after_sync();
            float v[128];
            tmem_ld128(ts, v);
            const int key0 = key_of(blk);
            if (cut(key0)) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t bits = seen_bits(rv, key0 + 32 * w, sinks, sv.len, sv.count);
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[32 * w + x] = bits >> x & 1u ? v[32 * w + x] : -INFINITY;
                }
            }
            float mx0 = v[0], mx1 = v[1];
#pragma unroll
            for (int x = 2; x < 128; x += 4) {
                mx0 = fmaxf(fmaxf(mx0, v[x]), v[x + 1]);
                if (x + 2 < 128) mx1 = fmaxf(fmaxf(mx1, v[x + 2]), v[x + 3]);
            }
            const float mx = fmaxf(mx0, mx1) * scale2;
            if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                const float now = fmaxf(m, mx);
                const float f = now == -INFINITY ? 1.f : ex2(m - now);
                m = now;
                l *= f;
                if (done > 0) {
                    ok = __all_sync(0xffffffffu, wait(o_done + s, (done - 1) & 1, kDevErrWaitMma));
                    if (!ok) break;
                    tc_fence_after_sync();
                    for (int d = 0; d < steps * 16; d += 32) {
                        float o[32];
                        uint32_t u[32];
                        tmem_ld32(to + d, o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(o[x] * f);
                        tmem_st32(to + d, u);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : -m;
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t u[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    float2 e = ffma2(make_float2(v[64 * h + 2 * x], v[64 * h + 2 * x + 1]), make_float2(scale2, scale2),
                                     make_float2(base, base));
                    e.x = ex2(e.x), e.y = ex2(e.y);
                    u[x] = Pair<T>::pack(e.x, e.y);
                    if (x & 1)
                        sum1.x += e.x, sum1.y += e.y;
                    else
                        sum0.x += e.x, sum0.y += e.y;
                }
                tmem_st32(ts + 32 * h, u);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive(p_full + s);
            l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
        }
        if (ok && done > 0) ok = __all_sync(0xffffffffu, wait(o_done + s, (done - 1) & 1, kDevErrWaitMma));
        tc_fence_after_sync();
        const auto store = [&](char *out, int d, const float (&o)[32], float f) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (d + 8 * x < c.head_dim)
                    *reinterpret_cast<uint4 *>(out + (d + 8 * x) * 2) =
                        make_uint4(Pair<T>::pack(o[8 * x] * f, o[8 * x + 1] * f), Pair<T>::pack(o[8 * x + 2] * f, o[8 * x + 3] * f),
                                   Pair<T>::pack(o[8 * x + 4] * f, o[8 * x + 5] * f), Pair<T>::pack(o[8 * x + 6] * f, o[8 * x + 7] * f));
        };
        char *out = static_cast<char *>(a.O) + ((int64_t)(sv.first + i) * a.o_stride +
                                                (int64_t)(head * a.group + row0 + rc - i * a.group) * c.head_dim) * 2;
        if (used > 1) {
            // partial results: both streams' of the same rows where they share a tile
            const int64_t at = (int64_t)unit * p.splits + split;
            for (int d = 0; d < c.head_dim; d += 32) {
                float o[32];
                if (done > 0) {
                    tmem_ld32(to + d, o);
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0.f;
                }
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (d + 4 * x < c.head_dim)
                        p.part[(at * (c.head_dim / 4) + d / 4 + x) * ROWS + s * 128 + t] =
                            make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            }
            p.ml[at * ROWS + s * 128 + t] = make_float2(m, l);
            __threadfence();
        } else if (!single) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            for (int d = 0; d < c.head_dim; d += 32) {
                float o[32];
                tmem_ld32(to + d, o);
                if (r < nrows) store(out, d, o, inv);
            }
        }
        tc_fence_before_sync();
        __syncthreads();  // 1: every role is through, the ring is free
        if (used == 1 && single) {
            float *so = reinterpret_cast<float *>(sm + P::RING);  // [d][row]
            tc_fence_after_sync();
            if (s == 1 && done > 0)
                for (int d = 0; d < c.head_dim; d += 32) {
                    float o[32];
                    tmem_ld32(to + d, o);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (d + x < c.head_dim) so[(d + x) * 128 + t] = o[x];
                }
            if (s == 1) sm_ml[t] = make_float2(m, l);
            bar_sync(1, 256);
            if (s == 0) {
                const float2 other = sm_ml[t];
                const float mt = fmaxf(m, other.x);
                const float f0 = m == -INFINITY ? 0.f : ex2(m - mt), f1 = other.x == -INFINITY ? 0.f : ex2(other.x - mt);
                const float lt = l * f0 + other.y * f1, inv = lt > 0.f ? 1.f / lt : 0.f;
                for (int d = 0; d < c.head_dim; d += 32) {
                    float o[32];
                    tmem_ld32(to + d, o);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        o[x] = o[x] * (f0 * inv) + (f1 > 0.f && d + x < c.head_dim ? so[(d + x) * 128 + t] * (f1 * inv) : 0.f);
                    if (r < nrows) store(out, d, o, 1.f);
                }
            }
            tc_fence_before_sync();
        }
    } else {
        if (warp == 8) {
            if (lane == 0) {
                const uint32_t fmt = c.dtype == 0 ? kFmtF16 : kFmtBF16;
                const uint32_t iqk = make_idesc(fmt, fmt, B, 128);
                const uint32_t ipv = make_idesc(fmt, fmt, (uint32_t)steps * 16, 128) | 1u << 16;  // V: MN-major
                const uint32_t smb = smem_u32(sm);
                uint32_t looked = 0;
                const auto qk = [&](int s, int i) {
                    const int x = slot_k(i), st = x % ST;
                    if (!wait(full + st, (x / ST) & 1, kDevErrWaitFull)) return false;
                    tc_fence_after_sync();
                    const uint32_t q = smb + (single ? 0 : s * P::TILE), k = smb + P::RING + st * P::TILE;
                    for (int e = 0; e < steps; ++e) {
                        const uint32_t off = (e >> 2) * HALF + (e & 3) * 32;
                        umma_f16(tmem + s * 128, sdesc_kmajor_sw128(q + off), sdesc_kmajor_sw128(k + off), iqk, e > 0);
                    }
                    umma_commit(s_full + s);
                    if (single || s == 1) umma_commit(empty + st);
                    return true;
                };
                const auto pv = [&](int s, int i, int round) {
                    const int x = slot_v(i), st = x % ST;
                    if (!wait(full + st, (x / ST) & 1, kDevErrWaitFull)) return false;
                    const bool look = (single || s == 0) && cut(key_of(i));
                    if (look) mbar_arrive(fix);  // while the softmax runs
                    if (!wait(p_full + s, round & 1, kDevErrWaitFull)) return false;
                    if (look && !wait(fixed, looked++ & 1, kDevErrWaitFull)) return false;
                    tc_fence_after_sync();
                    const uint32_t v = smb + P::RING + st * P::TILE;
                    for (int e = 0; e < B / 16; ++e)
                        umma_f16_ta(tmem + 256 + s * 128, tmem + s * 128 + e * 8,
                                    sdesc_make(v + e * 2048, HALF, 1024, kSdescSw128), ipv, round > 0 || e > 0);
                    umma_commit(o_done + s);
                    if (single || s == 1) umma_commit(empty + st);
                    return true;
                };
                bool ok = qk(0, 0);
                if (ok && (!single || n > 1)) ok = qk(1, single ? 1 : 0);
                for (int i = 0; ok && i < n; ++i) {
                    if (single) {
                        ok = pv(i & 1, i, i >> 1) && (i + 2 >= n || qk(i & 1, i + 2));
                    } else {
                        for (int s = 0; ok && s < 2; ++s) ok = pv(s, i, i) && (i + 1 >= n || qk(s, i + 1));
                    }
                }
                umma_commit(drain);
                if (!mbar_wait(drain, 0)) atomicExch(&g_tiles_err, kDevErrDrain);
            }
            __syncwarp();
        } else if (warp == 9) {
            // page lane / HALVES of the block, 64-column half lane % HALVES
            const int ops = B / p.box * HALVES;
            int x = 0;
            for (; x < 2 * n; ++x) {
                const bool is_v = x == 2 * n - 1 || (x > 0 && !(x & 1));
                const int blk = x == 0 ? 0 : x == 2 * n - 1 ? n - 1 : x & 1 ? (x + 1) / 2 : x / 2 - 1;
                const int key = key_of(blk) + lane / HALVES * p.box;
                int page = -1;
                if (lane < ops && key < end) {
                    page = page_of(c, seq, key >> c.page_shift);
                    if (page < 0) atomicExch(&g_tiles_err, kDevErrRange);
                }
                const int st = x % ST;
                if (x >= ST && !__all_sync(0xffffffffu, wait(empty + st, (x / ST - 1) & 1, kDevErrWaitEmpty))) break;
                if (lane == 0) mbar_arrive_expect_tx(full + st, P::TILE);
                __syncwarp();
                if (lane < ops)  // a page out of range is out of the tensor: zeros
                    tma_load_4d(sm + P::RING + st * P::TILE + (lane % HALVES) * HALF + lane / HALVES * p.box * 128,
                                is_v ? &vmap : &kmap, full + st, (lane % HALVES) * 64, key & (c.page_size - 1), head,
                                page < 0 ? (int)min(c.pages, (int64_t)0x7fffffff) : page);
            }
            // nothing of this CTA's may be in flight when it ends
            for (int y = max(0, x - ST); y < x; ++y)
                if (!mbar_wait(full + y % ST, (y / ST) & 1)) atomicExch(&g_tiles_err, kDevErrDrain);
            __syncwarp();
        } else {
            const int ft = tid - 320;
            uint32_t looked = 0;
            for (int i = 0; i < n; ++i) {
                const int key0 = key_of(i);
                if (!cut(key0)) continue;
                const int x = slot_v(i), st = x % ST;
                if (!__all_sync(0xffffffffu, wait(fix, looked++ & 1, kDevErrWaitFull) &&
                                                 wait(full + st, (x / ST) & 1, kDevErrWaitFull)))
                    break;
                uint8_t *v = sm + P::RING + st * P::TILE;
                bool special = false;
#pragma unroll 4
                for (int e = ft; e < P::TILE / 16; e += 64) {
                    const int j = key0 + ((e & 1023) >> 3);
                    uint4 *at = reinterpret_cast<uint4 *>(v + e * 16);
                    if (j >= end || (j >= sinks && j < low)) {
                        *at = make_uint4(0, 0, 0, 0);
                    } else {
                        const uint4 u = *at;
                        special |= any_special<T>(u.x) || any_special<T>(u.y) || any_special<T>(u.z) || any_special<T>(u.w);
                    }
                }
                if (special) *poison = 1;
                fence_proxy_async_smem();
                mbar_arrive(fixed);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncthreads();  // 1
    }
    __syncthreads();  // 2: tensor memory has been read
    if (warp == 8) {
        tc_fence_after_sync();
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
    if (*fail) return;
    bool again = *poison != 0;
    if (used > 1) {
        if (tid == 0) {
            if (again) atomicOr(p.poison + unit, 1);
            __threadfence();
            const int k = atomicAdd(p.tickets + unit, 1);
            sm_last = k == used - 1;
            if (sm_last) {
                __threadfence();
                *poison = atomicExch(p.poison + unit, 0);
                p.tickets[unit] = 0;  // ready for the next call
            }
        }
        __syncthreads();
        if (!sm_last) return;
        __threadfence();
        again = *poison != 0;
        if (!again) {
            const int sources = single ? 2 * used : used;
            const int64_t at0 = (int64_t)unit * p.splits;
            const auto ml_of = [&](int y, int r) {
                return __ldcg(p.ml + (at0 + (single ? y >> 1 : y)) * ROWS + (single ? (y & 1) * 128 : 0) + r);
            };
            if (tid < nrows) {
                float mt = -INFINITY, lt = 0.f;
                for (int y = 0; y < sources; ++y) mt = fmaxf(mt, ml_of(y, tid).x);
                for (int y = 0; y < sources && mt > -INFINITY; ++y) {
                    const float2 q = ml_of(y, tid);
                    if (q.x > -INFINITY) lt += q.y * ex2(q.x - mt);
                }
                sm_ml[tid] = make_float2(mt, lt > 0.f ? 1.f / lt : 0.f);
            }
            __syncthreads();
            const int d8 = c.head_dim / 8;
            for (int e = tid; e < ROWS * d8; e += NT) {
                const int r = e & (ROWS - 1), x = e / ROWS;
                if (r >= nrows) continue;
                const float2 t = sm_ml[r];
                float o[8] = {};
#pragma unroll 2
                for (int y = 0; y < sources; ++y) {
                    const float2 q = ml_of(y, r);
                    const float f = q.x > -INFINITY ? ex2(q.x - t.x) * t.y : 0.f;
                    const float4 *src = p.part + ((at0 + (single ? y >> 1 : y)) * (c.head_dim / 4) + 2 * x) * ROWS +
                                        (single ? (y & 1) * 128 : 0) + r;
                    const float4 u = __ldcg(src), w = __ldcg(src + ROWS);
                    o[0] += f * u.x, o[1] += f * u.y, o[2] += f * u.z, o[3] += f * u.w;
                    o[4] += f * w.x, o[5] += f * w.y, o[6] += f * w.z, o[7] += f * w.w;
                }
                const int i = (row0 + r) / a.group, h = row0 + r - i * a.group;
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.O) +
                                           ((int64_t)(sv.first + i) * a.o_stride + (int64_t)(head * a.group + h) * c.head_dim + 8 * x) * 2) =
                    make_uint4(Pair<T>::pack(o[0], o[1]), Pair<T>::pack(o[2], o[3]), Pair<T>::pack(o[4], o[5]), Pair<T>::pack(o[6], o[7]));
            }
        }
    }
    if (again)
        for (int r = warp; r < nrows; r += NT / 32) {
            const int i = (row0 + r) / a.group;
            attend_row<T>(a, seq, sv, i, head * a.group + row0 + r - i * a.group, &g_tiles_err);
        }
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

int64_t unit_count(const CacheView &c, int group, int64_t max_q, int *tiles) {
    *tiles = (int)((max_q * group + ROWS - 1) / ROWS);
    return (int64_t)*tiles * c.seqs * c.kv_heads;
}

template <typename T, int HALVES>
cudaError_t launch(const TilesArgs &p, cudaStream_t s) {
    static const cudaError_t once = cudaFuncSetAttribute(
        tiles_kernel<T, HALVES>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<HALVES>::BYTES);
    if (once != cudaSuccess) return once;
    CUtensorMap k, v;
    cudaError_t e = cache_tmap(&k, p.a.c, p.a.c.k, p.box);
    if (e == cudaSuccess) e = cache_tmap(&v, p.a.c, p.a.c.v, p.box);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)p.tiles * p.a.c.seqs * p.a.c.kv_heads;
    return launch_pdl(tiles_kernel<T, HALVES>, dim3((unsigned)(units * p.splits)), NT, Plan<HALVES>::BYTES, s, k, v, p);
}

}  // namespace

int cache_attention_tiles_splits(const CacheView &c, int group, int64_t max_q, int sms) {
    int tiles;
    const int64_t units = unit_count(c, group, max_q, &tiles);
    // four CTAs per SM in turn even out ragged lengths; none below MIN_BLOCKS blocks of keys
    int64_t s = units >= 2 * (int64_t)sms ? 1 : (4 * (int64_t)sms + units - 1) / units;
    const int64_t most = ((c.max_pages << c.page_shift) + B * MIN_BLOCKS - 1) / (B * MIN_BLOCKS);
    if (s > most) s = most;
    if (s > MAX_SPLITS) s = MAX_SPLITS;
    return (int)(s < 1 ? 1 : s);
}

int64_t cache_attention_tiles_workspace(const CacheView &c, int group, int64_t max_q, int splits) {
    if (splits <= 1) return 0;
    int tiles;
    const int64_t units = unit_count(c, group, max_q, &tiles);
    return 2 * round256(units * 4) + units * splits * ROWS * (8 + (int64_t)c.head_dim * 4);
}

cudaError_t launch_cache_attention_tiles(const CacheAttnArgs &a, int splits, cudaStream_t s) {
    TilesArgs p{a, splits, 0, a.c.page_size < B ? a.c.page_size : B, nullptr, nullptr, nullptr, nullptr};
    const int64_t units = unit_count(a.c, a.group, a.max_q, &p.tiles);
    if (units * splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (splits > 1) {
        char *w = static_cast<char *>(a.ws);
        p.tickets = reinterpret_cast<int32_t *>(w);
        w += round256(units * 4);
        p.poison = reinterpret_cast<int32_t *>(w);
        w += round256(units * 4);
        p.part = reinterpret_cast<float4 *>(w);
        w += units * splits * ROWS * (int64_t)a.c.head_dim * 4;
        p.ml = reinterpret_cast<float2 *>(w);
    }
    if (a.c.dtype == 0) return a.c.head_dim <= 64 ? launch<__half, 1>(p, s) : launch<__half, 2>(p, s);
    return a.c.head_dim <= 64 ? launch<__nv_bfloat16, 1>(p, s) : launch<__nv_bfloat16, 2>(p, s);
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
