// cache_attention.cuh -- what the kernels of attention over a paged cache share: which keys a row
// sees, the blocks of keys that a set of rows needs, the split's workspace and its join.
#pragma once

#include "cache_view.cuh"
#include "tmap.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

namespace mm {

constexpr float kLog2e = 1.4426950408889634f;

// Positions are 32-bit: a sequence holds at most 2^30 tokens.
//
// The keys a row sees: those before `end` (its own position and what precedes it, or with a tree
// the tokens before the drafts) that are below `sinks` or at `low` and later, and the drafted tokens
// whose bit is set.
struct RowView {
    int low, end;
    const uint32_t *bits;  // null: none
};

__device__ __forceinline__ bool sees(const RowView &r, int j, int sinks, int len, int count) {
    if (j < r.end) return j >= r.low || j < sinks;
    if (!r.bits) return false;
    const int t = j - len;
    return t < count && (__ldg(r.bits + (t >> 5)) >> (t & 31) & 1u);
}

// Bits of the row's mask below `count`
__device__ __forceinline__ int mask_depth(const uint32_t *bits, int count) {
    int n = 0;
    for (int w = 0; w * 32 < count; ++w) {
        uint32_t b = __ldg(bits + w);
        if (count - w * 32 < 32) b &= (1u << (count - w * 32)) - 1u;
        n += __popc(b);
    }
    return n;
}

// new token i of a sequence with `len` tokens before it
__device__ __forceinline__ RowView row_view(const CacheAttnArgs &a, int len, int first, int count, int i) {
    RowView r;
    int p = len + i;
    if (a.mask) {
        r.bits = a.mask + (int64_t)(first + i) * a.mask_words;
        p = len + mask_depth(r.bits, count) - 1;
        r.end = len;
    } else {
        r.bits = nullptr;
        r.end = p + 1;
    }
    r.low = a.window > 0 ? p - a.window + 1 : 0;
    return r;
}

// One sequence of the call, checked: its rows of Q, its cached tokens.
struct SeqView {
    int first, count, len;
};
__device__ __forceinline__ SeqView seq_view(const CacheAttnArgs &a, int seq, unsigned int *err) {
    SeqView s;
    const RowRange r = rows_of(a.q_start, seq, a.tokens, a.max_q, err);
    s.first = r.first, s.count = r.count;
    s.len = __ldg(a.c.lens + seq);
    if (s.len < 0 || (int64_t)s.len + s.count > row_capacity(a.c)) {
        *err = kDevErrRange;
        s.count = 0;
        s.len = 0;
    }
    // a mask narrower than the tree leaves the drafts past it unseen
    if (a.mask && s.count > a.mask_words * 32) *err = kDevErrRange, s.count = 0;
    return s;
}

// Blocks of B keys that rows with their lowest window start at `low` need, of `end` keys: the blocks of
// the sinks, then those from low on.  block(i) is the i-th one's number.
struct KeyBlocks {
    int sink_blocks, first, count;
    __device__ __forceinline__ int block(int i) const {
        return i < sink_blocks ? i : first + (i - sink_blocks);
    }
};
template <int B>
__device__ __forceinline__ KeyBlocks key_blocks(int low, int sinks, int end) {
    KeyBlocks k;
    if (low < 0) low = 0;
    if (low > end) low = end;
    k.first = low / B;
    k.sink_blocks = min((min(sinks, end) + B - 1) / B, k.first);
    k.count = k.sink_blocks + (end + B - 1) / B - k.first;
    return k;
}

template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    __device__ static uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static float one(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static constexpr uint32_t kExp = 0x7c00u;  // all ones: infinity or NaN
};
template <>
struct Pair<__nv_bfloat16> {
    __device__ static uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static float one(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static constexpr uint32_t kExp = 0x7f80u;
};

// either 16-bit half of v infinite or NaN
template <typename T>
__device__ __forceinline__ bool any_special(uint32_t v) {
    return (v & Pair<T>::kExp) == Pair<T>::kExp || ((v >> 16) & Pair<T>::kExp) == Pair<T>::kExp;
}
// v with such halves replaced by 0
template <typename T>
__device__ __forceinline__ uint32_t without_special(uint32_t v) {
    if ((v & Pair<T>::kExp) == Pair<T>::kExp) v &= 0xffff0000u;
    if (((v >> 16) & Pair<T>::kExp) == Pair<T>::kExp) v &= 0x0000ffffu;
    return v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A warp's, stream's or part's share (m, l) of a row that saw no key, so that it adds nothing.  m alone does not tell: a
// maximum passes over NaN, so a share whose scores are all NaN has m = -infinity too, and its l, which is NaN, has to
// reach the row.  Joined, ex2(-infinity - m) l is NaN for it whatever m is.
__device__ __forceinline__ bool saw_nothing(float2 ml) { return ml.x == -INFINITY && ml.y == 0.f; }

// Division by a number that is known at the launch: n / d = (n m) >> (31 + s) for 0 <= n < 2^31, with 2^s >= d
// and m = ceil(2^(31 + s) / d) <= 2^32 - 1 (d = 1: m 0).
struct FastDiv {
    uint32_t m, s;
    int d;
    __device__ __forceinline__ int div(int n) const { return m ? (int)(__umulhi((uint32_t)n, m) >> s) : n; }
};
inline FastDiv fast_div(int d) {
    if (d <= 1) return {0, 0, 1};
    uint32_t s = 0;
    while ((1ll << s) < d) ++s;
    return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s - 1, d};
}

// ---------------------------------------------------------------- which CTA does what
//
// An item is what a kernel's units are grouped by (a sequence, or 256 rows of one); each item that has n > 0
// blocks of keys has kv_heads units of n blocks.  The units are laid end to end in one of two measures and cut
// at multiples of `chunk`:
//   parts > 0: a unit measures `parts`, and its blocks are cut into as many parts (or whole: 1);
//   parts = 0: a unit measures cost + n, its blocks last; the cost stands for what beginning and ending a unit
//   takes, so that CTAs with many short units get fewer blocks.
// With at least two CTAs to a unit every unit is cut into equal parts, one to a CTA; with more to do the second
// measure, or whole units where all are short.
struct Share {
    int at, stop;     // this CTA's part
    int item, first;  // the item that `at` lies in, and where it begins
    int parts, cost, chunk;
};

struct ShareRules {
    int min_blocks, whole_blocks, unit_cost;
    int force_whole;  // the sums could pass 31 bits: whole units only
};
// All units end to end, at most: the last CTA's end, before it is cut, passes the sum by less than one for each CTA
constexpr int64_t kShareLimit = ((int64_t)1 << 31) - 4096;

// A shared unit's ticket is that of the CTA with its first part: a CTA begins one unit at most that it does not finish.  So
// the tickets take the same place in the workspace whatever the call's sizes, and no call's partial results lie there.
constexpr int kTickets = 1024;

struct ShareScratch {
    int a[32], b[32], most[32];
    int item, first;
};

// One unit of a CTA, or one part of it
struct UnitPart {
    int head, u0, u1;    // its place in the measure
    int b0, b1;          // its blocks here (b1 <= b0: none)
    int used, g0;        // the parts it is joined of: in CTA g0 and those that follow
    bool second;         // this part goes to the CTA's second slot (it begins a unit here that it does not finish)
    bool first_second;   // the same for the unit's first part
};

// The fewest blocks of a part of n: p parts take about n / p blocks' time and p parts' time to join, least at some
// multiple of sqrt(n).  (Rows kernel, 94 blocks: 8 parts 16.4 us, 12 14.4, 31 12.9, 38 13.1; 17 blocks: 5 12.4, 8 12.5,
// 17 13.4; 9 blocks: 3 8.7, 9 8.2.)
__device__ __forceinline__ int least_part(int n, int min_blocks) { return max(min_blocks, (int)(0.5f * sqrtf((float)n))); }

// at: a place in the item that begins at `first` and has n blocks
__device__ __forceinline__ UnitPart unit_part(const Share &s, int at, int first, int n, int min_blocks) {
    UnitPart u;
    const int size = s.parts ? s.parts : n + s.cost;
    u.head = (int)((uint32_t)(at - first) / (uint32_t)size);
    u.u0 = first + u.head * size, u.u1 = u.u0 + size;
    if (s.parts) {
        const int cut = min(s.parts, max((int)((uint32_t)n / (uint32_t)least_part(n, min_blocks)), 1));
        const int per = (int)((uint32_t)(n + cut - 1) / (uint32_t)cut);
        u.b0 = (at - u.u0) * per, u.b1 = min(n, u.b0 + per);
        u.used = s.parts == 1 ? 1 : (int)((uint32_t)(n + per - 1) / (uint32_t)per);
        u.g0 = u.u0;  // with more than one part, each CTA has one
        u.second = u.first_second = false;
    } else {
        u.b0 = max(at - u.u0 - s.cost, 0), u.b1 = min(s.stop, u.u1) - u.u0 - s.cost;
        u.g0 = (int)((uint32_t)(u.u0 + s.cost) / (uint32_t)s.chunk);
        u.used = (int)((uint32_t)(u.u1 - 1) / (uint32_t)s.chunk) - u.g0 + 1;
        u.second = u.b0 == 0 && (int)blockIdx.x * s.chunk < u.u0;
        u.first_second = u.g0 * s.chunk < u.u0;
    }
    return u;
}

// Sums over the block's NT values: inclusive ones in a and b (b is 0 or 1), totals in ta, tb, the largest a in most
template <int NT>
__device__ __forceinline__ void share_scan(int &a, int &b, ShareScratch &sh, int &ta, int &tb, int &most) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m = __reduce_max_sync(0xffffffffu, a);
    b = __popc(__ballot_sync(0xffffffffu, b != 0) & (0xffffffffu >> (31 - lane)));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o);
        if (lane >= o) a += x;
    }
    __syncthreads();
    if (lane == 31) sh.a[warp] = a, sh.b[warp] = b, sh.most[warp] = m;
    __syncthreads();
    // the warps' sums, one to a lane
    int wa = lane < NT / 32 ? sh.a[lane] : 0, wb = lane < NT / 32 ? sh.b[lane] : 0;
    most = __reduce_max_sync(0xffffffffu, lane < NT / 32 ? sh.most[lane] : 0);
    ta = __reduce_add_sync(0xffffffffu, wa), tb = __reduce_add_sync(0xffffffffu, wb);
    a += __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    b += __reduce_add_sync(0xffffffffu, lane < warp ? wb : 0);
}

// blocks(i): the blocks of item i (0 past the last).  Every thread of the block calls it and gets the same
// Share; false: nothing to do here.
template <int NT, typename Blocks>
__device__ __forceinline__ bool share_of(int items, int kv_heads, const ShareRules &rules, const Blocks &blocks,
                                         ShareScratch &sh, Share &s) {
    int total = 0, count = 0, most = 0, mine = 0, a = 0, b = 0;
    for (int i0 = 0; i0 < items; i0 += NT) {
        mine = a = blocks(i0 + threadIdx.x);
        b = mine > 0;
        int ta, tb, m;
        share_scan<NT>(a, b, sh, ta, tb, m);
        total += ta, count += tb, most = max(most, m);
    }
    const int units = count * kv_heads, grid = (int)gridDim.x;
    if (units == 0) return false;
    s.parts = s.cost = 0;
    if (rules.force_whole)
        s.parts = 1;
    else if (2 * (int64_t)units <= grid)
        s.parts = min((int)((uint32_t)grid / (uint32_t)units), (most + rules.min_blocks - 1) / rules.min_blocks);
    else if (most <= rules.whole_blocks)
        s.parts = 1;
    // the cost is no more than half of what a CTA gets
    if (!s.parts) s.cost = min((int)((uint32_t)(total * kv_heads) / (uint32_t)(2 * grid)), rules.unit_cost);
    const int all = s.parts ? units * s.parts : (total + s.cost * count) * kv_heads;
    s.chunk = (int)((uint32_t)(all + grid - 1) / (uint32_t)grid);
    if (!s.parts) s.chunk = max(s.chunk, rules.min_blocks);
    s.at = (int)blockIdx.x * s.chunk;  // this and the end below: < 2^31 (kShareLimit)
    if (s.at >= all) return false;
    s.stop = min(s.at + s.chunk, all);
    int before = 0;
    for (int i0 = 0; i0 < items; i0 += NT) {
        if (items > NT) {  // else the sums are still in registers
            mine = a = blocks(i0 + threadIdx.x);
            b = mine > 0;
            int ta, tb, m;
            share_scan<NT>(a, b, sh, ta, tb, m);
            const int here = s.parts ? tb * s.parts : ta + s.cost * tb;
            if (s.at >= (before + here) * kv_heads) {  // the same for all threads
                before += here;
                continue;
            }
        }
        const int w = s.parts ? s.parts : mine + s.cost;
        const int first = (before + (s.parts ? b * s.parts : a + s.cost * b) - w) * kv_heads;
        if (mine > 0 && s.at >= first && s.at < first + w * kv_heads) sh.item = i0 + threadIdx.x, sh.first = first;
        break;
    }
    __syncthreads();
    s.item = sh.item, s.first = sh.first;
    return true;
}

// A block reaches into pages that a window has released.  A box of keys needs its page if it begins in the sinks or
// behind this key; `low`: the lowest key that a row may see outside them (a drafted token sees itself, so one more).
__device__ __forceinline__ int last_unheld(const CacheAttnArgs &a, int low, int box) { return low + (a.mask ? 1 : 0) - box; }
// The exception, a row of a tree with no bit at all: it sits at len - 1 and sees key len - window, whose page may be gone.
__device__ __forceinline__ void check_held(const CacheAttnArgs &a, int seq, const SeqView &sv, const RowView &r, unsigned int *err) {
    if (a.mask && a.window > 0 && r.low == sv.len - a.window && r.low >= a.sinks && page_of(a.c, seq, r.low >> a.c.page_shift) < 0)
        *err = kDevErrRange;
}

// CTAs of the rows kernel (the blocks of all units are cut evenly over them)
int cache_attention_rows_ctas(const CacheView &c, int sms);
int64_t cache_attention_rows_workspace(const CacheView &c, int ctas);
cudaError_t launch_cache_attention_rows(const CacheAttnArgs &a, int ctas, cudaStream_t s);
unsigned int cache_attention_rows_take_device_error(cudaError_t *err);
// CTAs of the tiles kernel, one per SM at most
int cache_attention_tiles_ctas(const CacheView &c, int group, int64_t max_q, int sms);
int64_t cache_attention_tiles_workspace(const CacheView &c, int ctas);
cudaError_t launch_cache_attention_tiles(const CacheAttnArgs &a, int ctas, cudaStream_t s);
unsigned int cache_attention_tiles_take_device_error(cudaError_t *err);
constexpr int kRowsMax = 16;  // rows (new tokens x heads of a kv head) of one sequence in the rows kernel

// The pages of k or v: boxes of `box` tokens of one head, 64 columns, 128-byte swizzle; what is past
// head_dim, and pages past the last, read as zeros.
inline cudaError_t cache_tmap(CUtensorMap *map, const CacheView &c, const void *base, int box) {
    cudaError_t err;
    auto enc = tmap_encoder(&err);
    if (err != cudaSuccess) return err;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads, (cuuint64_t)c.pages};
    const auto bytes = [](int64_t stride, int64_t count) { return (cuuint64_t)(count > 1 ? stride * 2 : 16); };
    const cuuint64_t strides[3] = {bytes(c.token_stride, c.page_size), bytes(c.head_stride, c.kv_heads), bytes(c.page_stride, c.pages)};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, c.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void *>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace mm
