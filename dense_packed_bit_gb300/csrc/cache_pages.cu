// cache_pages.cu -- the bookkeeping of a paged cache of keys and values: reserving, writing,
// compacting, forking, releasing and copying pages.
//
// Everything stays on the device: a page is free where refs[page] == 0, and a call that needs
// n pages takes the n lowest free ones in order, so the result is a function of the state alone
// (no free list whose order depends on history, no atomics whose order shows).  One CTA finds
// them: 4 refs per thread and step, a block scan of the free counts, and the page of rank r put
// at place r of a shared-memory list.  The scan stops at the last page needed.  What moves data
// runs over the whole GPU in a second kernel of the same call (a programmatic dependent launch:
// its CTAs are resident when the first kernel ends).
//
// Bound: bytes moved (each token's K and V once in and once out) for fork, append and compact;
// the launch itself for small ones.  16-byte accesses, rows of one head contiguous.
//
// Measured, a call: 8 sequences forked into 64 (16 layers, 8 heads of 128, a partial page each: 170 MB written) 46 us with
// the children's release, of which the copy is 39 (131 MB of DRAM traffic: a parent's page is read once, part of what is
// written stays in L2) and the rest two kernels of one CTA in a row; 4,096 tokens of 8 heads of 128 appended 8.3 us,
// reserved 4.8; reserve, append and compact for 16 sequences of 12 drafts 22 us, four launches' host time.
#include "cache_view.cuh"

namespace mm {

namespace {

__device__ unsigned int g_pages_err;

constexpr int NT = 1024;      // allocating CTA
constexpr int LIST = 8192;    // pages it hands out per sweep of refs
constexpr int CT = 256;       // copying CTAs

__device__ __forceinline__ void range_error() { g_pages_err = kDevErrRange; }

// Inclusive scan over the block's NT values; `part` has 32 ints of shared memory.  Every thread
// gets its inclusive sum and the block total.
__device__ __forceinline__ int block_scan(int v, int *part, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // part may still be read from the scan before
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int p = lane < NT / 32 ? part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) p += u;
        }
        part[lane] = p;
    }
    __syncthreads();
    *total = part[NT / 32 - 1];
    return v + (warp ? part[warp - 1] : 0);
}

// Sum over the block's NT values, each at most 2^24 (a row of the table): a warp's fits 32 bits, the block's does not.
__device__ __forceinline__ int64_t block_sum(int v, int *part) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();  // part may still be read from the sum before
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t s = 0;
    for (int i = 0; i < NT / 32; ++i) s += part[i];
    return s;
}

constexpr int PER = 16;  // refs per thread and step of the search: four 16-byte loads in flight

// From page `from` on: puts the free pages of rank 0 .. want - 1 into list (want <= LIST) and
// returns how many there are of them; *next is the page to go on from.  list null: counts only.
__device__ __forceinline__ int64_t free_pages(const CacheView &c, int64_t from, int64_t want, int *list, int *part,
                                              int64_t *next) {
    int64_t found = 0;
    // steps begin at a multiple of 4 pages, so that a 16-byte aligned refs is read in 16-byte loads
    const bool wide = (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0;
    for (int64_t p0 = from & ~(int64_t)3; p0 < c.pages && found < want; p0 += (int64_t)PER * NT) {
        const int64_t p = p0 + (int64_t)PER * threadIdx.x;
        int r[PER];
#pragma unroll
        for (int q = 0; q < PER; q += 4) {
            if (wide && p + q + 3 < c.pages) {
                const int4 v = *reinterpret_cast<const int4 *>(c.refs + p + q);
                r[q] = v.x, r[q + 1] = v.y, r[q + 2] = v.z, r[q + 3] = v.w;
            } else {
#pragma unroll
                for (int i = q; i < q + 4; ++i) r[i] = p + i < c.pages ? c.refs[p + i] : 1;
            }
        }
        int n = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) n += r[i] == 0 && p + i >= from;
        int total;
        int64_t rank = found + block_scan(n, part, &total) - n;
        if (list && n) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (r[i] == 0 && p + i >= from) {
                    if (rank < want) list[rank] = (int)(p + i);
                    ++rank;
                }
        }
        found += total;
    }
    __syncthreads();
    if (list && found >= want && want > 0) {  // go on behind the last one taken
        *next = (int64_t)list[want - 1] + 1;
        found = want;
    }
    return found;
}

struct AllocShared {
    int list[LIST];
    int count[NT];  // pages each item of a step wants, then the rank of its first one within the batch
    int part[32];
};

// Gives every item i < n the pages it wants, in order.  count(i0) fills sh.count for items
// i0 .. i0 + NT - 1; give(i0, batch) assigns sh.list[r] to the items' wants of rank r, for 0 <= r <
// batch, sh.count[i - i0] being the rank of item i's first (negative ones were given in an earlier
// batch).  All or nothing: returns the number of pages lacking.
template <typename Count, typename Give>
__device__ __forceinline__ int64_t allocate(const CacheView &c, int64_t n, AllocShared &sh, const Count &count,
                                            const Give &give) {
    int64_t total = 0, base = 0, next = 0;
    for (int64_t i0 = 0; i0 < n; i0 += NT) {
        count(i0);
        __syncthreads();
        total += block_sum(sh.count[threadIdx.x], sh.part);
    }
    if (total == 0) return 0;
    // (from here on total is at most the number of pages, so that the ranks below fit 32 bits)
    const int64_t have = free_pages(c, 0, min(total, (int64_t)LIST), sh.list, sh.part, &next);
    if (have < total) {
        int64_t more = 0, end;
        if (have == LIST) more = free_pages(c, next, total - LIST, nullptr, sh.part, &end);
        if (have + more < total) return total - have - more;
    }
    for (int64_t done = 0; done < total;) {
        const int64_t batch = min(total - done, (int64_t)LIST);
        base = 0;
        for (int64_t i0 = 0; i0 < n; i0 += NT) {
            __syncthreads();
            count(i0);
            __syncthreads();
            int sum;
            const int m = sh.count[threadIdx.x];
            const int64_t first = base + block_scan(m, sh.part, &sum) - m - done;
            sh.count[threadIdx.x] = (int)max(min(first, (int64_t)LIST), -(int64_t)0x40000000);
            __syncthreads();
            give(i0, (int)batch);
            base += sum;
        }
        done += batch;
        __syncthreads();
        if (done < total) free_pages(c, next, min(total - done, (int64_t)LIST), sh.list, sh.part, &next);
    }
    return 0;
}

// table columns of sequence s that reserve looks at: [first, upto)
__device__ __forceinline__ void reserve_range(const CacheView &c, const int32_t *need, int64_t s, int64_t *first,
                                              int64_t *upto) {
    const int64_t len = c.lens[s], more = need[s];
    *first = *upto = 0;
    if (len < 0 || more < 0) {
        range_error();
        return;
    }
    *first = len >> c.page_shift;  // pages before it may have been released under a window
    *upto = (len + more + c.page_size - 1) >> c.page_shift;
    if (*upto > c.max_pages) {
        range_error();
        *upto = c.max_pages;
    }
}

// One warp per sequence.  An entry given in an earlier batch is marked -2 - page, so that it still
// counts as wanted and the ranks stay; the marks are turned into pages at the end.
__global__ void __launch_bounds__(NT, 1) reserve_kernel(const CacheView c, const int32_t *need, int32_t *missing) {
    __shared__ AllocShared sh;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // f(seq, entry, rank of the entry among the sequence's wanted ones)
    const auto each_wanted = [&](int64_t s, const auto &f) {
        int64_t first, upto;
        reserve_range(c, need, s, &first, &upto);
        int n = 0;
        for (int64_t j0 = first; j0 < upto; j0 += 32) {
            int32_t *e = c.table + s * c.max_pages + j0 + lane;
            const bool want = j0 + lane < upto && *e < 0;
            const unsigned m = __ballot_sync(0xffffffffu, want);
            if (want) f(e, n + __popc(m & ((1u << lane) - 1)));
            n += __popc(m);
        }
        return n;
    };
    const auto count = [&](int64_t i0) {
        for (int i = warp; i < NT; i += NT / 32) {
            const int n = i0 + i < c.seqs ? each_wanted(i0 + i, [](int32_t *, int) {}) : 0;
            if (lane == 0) sh.count[i] = n;
        }
    };
    const auto give = [&](int64_t i0, int batch) {
        for (int i = warp; i < NT && i0 + i < c.seqs; i += NT / 32) {
            const int first = sh.count[i];
            each_wanted(i0 + i, [&](int32_t *e, int j) {
                const int r = first + j;
                if (r >= 0 && r < batch) *e = -2 - sh.list[r];
            });
        }
    };
    const int64_t lacking = min(allocate(c, c.seqs, sh, count, give), (int64_t)0x7fffffff);
    __syncthreads();
    if (lacking == 0)
        for (int64_t s = warp; s < c.seqs; s += NT / 32)
            each_wanted(s, [&](int32_t *e, int) {
                const int page = -2 - *e;
                *e = page;
                c.refs[page] = 1;
            });
    if (threadIdx.x == 0) *missing = (int)lacking;
}

__device__ __forceinline__ bool fork_pair(const CacheView &c, const int32_t *parents, const int32_t *children, int64_t i,
                                          int *parent, int *child, int64_t *len) {
    *parent = parents[i];
    *child = children[i];
    if (*parent < 0 || *parent >= c.seqs || *child < 0 || *child >= c.seqs || *parent == *child) return false;
    *len = c.lens[*parent];
    return *len >= 0 && *len <= row_capacity(c);
}

// the last, partial pages of the children, and their lengths
__global__ void __launch_bounds__(NT, 1) fork_alloc_kernel(const CacheView c, const int32_t *parents,
                                                           const int32_t *children, int64_t n, int32_t *missing) {
    __shared__ AllocShared sh;
    pdl_wait();
    pdl_launch_dependents();
    const auto count = [&](int64_t i0) {
        const int64_t i = i0 + threadIdx.x;
        int p, ch, want = 0;
        int64_t len;
        if (i < n) {
            if (fork_pair(c, parents, children, i, &p, &ch, &len))
                want = (len & (c.page_size - 1)) ? 1 : 0;
            else
                range_error();
        }
        sh.count[threadIdx.x] = want;
    };
    const auto give = [&](int64_t i0, int batch) {
        const int64_t i = i0 + threadIdx.x;
        const int r = sh.count[threadIdx.x];
        int p, ch;
        int64_t len;
        if (i < n && r >= 0 && r < batch && fork_pair(c, parents, children, i, &p, &ch, &len) &&
            (len & (c.page_size - 1)))
            c.table[(int64_t)ch * c.max_pages + (len >> c.page_shift)] = sh.list[r];
    };
    const int64_t lacking = allocate(c, n, sh, count, give);
    __syncthreads();
    if (lacking == 0)
        for (int64_t i = threadIdx.x; i < n; i += NT) {
            int p, ch;
            int64_t len;
            if (!fork_pair(c, parents, children, i, &p, &ch, &len)) continue;
            c.lens[ch] = (int)len;
            if (len & (c.page_size - 1)) c.refs[c.table[(int64_t)ch * c.max_pages + (len >> c.page_shift)]] = 1;
        }
    if (threadIdx.x == 0) *missing = (int)lacking;
}

// n / d for 0 <= n < 2^31, 1 <= d <= 128 (a page's tokens, a row's vectors), by a product: a division for each
// 16-byte vector took more of the copy than its loads
struct Inverses {
    uint32_t m[129], s[129];
    constexpr Inverses() : m(), s() {
        for (uint32_t d = 2; d <= 128; ++d) {
            uint32_t bits = 0;
            while ((1u << bits) < d) ++bits;
            m[d] = (uint32_t)(((1ull << (31 + bits)) + d - 1) / d), s[d] = bits - 1;
        }
    }
};
__constant__ Inverses inverses = Inverses();
__device__ __forceinline__ int divided(int n, int d) {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, inverses.m[d]) >> inverses.s[d]);
}

// `tokens` rows of every head of one layer's page: 16-byte vectors, four in flight per thread
__device__ __forceinline__ void copy_page(const CacheView &c, char *base, int64_t src, int64_t dst, int tokens, int part,
                                          int parts) {
    const int vecs = c.head_dim / 8;  // 16-byte vectors per row
    const int all = tokens * vecs * c.kv_heads;
    const char *s = base + src * c.page_stride * 2;
    char *d = base + dst * c.page_stride * 2;
    const auto at = [&](int e) {
        const int row = divided(e, vecs), h = divided(row, tokens), t = row - h * tokens;
        return (h * c.head_stride + t * c.token_stride + (e - row * vecs) * 8) * 2;
    };
    for (int e = part * CT + threadIdx.x; e < all; e += 4 * parts * CT) {
        uint4 v[4];
        int64_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = e + i * parts * CT;
            if (x < all) {
                o[i] = at(x);
                v[i] = ld_stream_v4(s + o[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i * parts * CT < all) *reinterpret_cast<uint4 *>(d + o[i]) = v[i];
    }
}

// grid (n, 2 layers, parts): the partial page's tokens; the CTAs of layer 0's keys also share the
// full pages and fill the child's row of the table.  The children of one part of a page follow each other, so that
// what they share of it is read once and found in L2 by the others.
__global__ void __launch_bounds__(CT) fork_copy_kernel(const CacheView c, const int32_t *parents,
                                                       const int32_t *children, const int32_t *missing) {
    pdl_wait();
    pdl_launch_dependents();
    int p, ch;
    int64_t len;
    if (*missing != 0 || !fork_pair(c, parents, children, blockIdx.x, &p, &ch, &len)) return;
    const int64_t full = len >> c.page_shift;
    const int rest = (int)(len & (c.page_size - 1));
    const int32_t *from = c.table + (int64_t)p * c.max_pages;
    int32_t *to = c.table + (int64_t)ch * c.max_pages;
    if (blockIdx.y == 0) {
        for (int64_t j = blockIdx.z * CT + threadIdx.x; j < c.max_pages; j += gridDim.z * CT) {
            if (j == full && rest) continue;
            int page = -1;
            if (j < full) {
                page = from[j];
                if (page >= 0 && page < c.pages) {
                    atomicAdd(c.refs + page, 1);
                } else {
                    if (page >= c.pages) range_error();
                    page = -1;  // released under a window
                }
            }
            to[j] = page;
        }
    }
    if (!rest) return;
    const int src = from[full], dst = to[full];
    if (src < 0 || src >= c.pages || dst < 0 || dst >= c.pages) {
        range_error();
        return;
    }
    char *base = (blockIdx.y & 1 ? c.v : c.k) + (blockIdx.y >> 1) * c.layer_stride * 2;
    copy_page(c, base, src, dst, rest, blockIdx.z, gridDim.z);
}

__global__ void __launch_bounds__(CT) copy_pages_kernel(const CacheView c, const int32_t *src, const int32_t *dst) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = src[blockIdx.x], d = dst[blockIdx.x];
    if (s < 0 || s >= c.pages || d < 0 || d >= c.pages) {
        range_error();
        return;
    }
    char *base = (blockIdx.y & 1 ? c.v : c.k) + (blockIdx.y >> 1) * c.layer_stride * 2;
    copy_page(c, base, s, d, c.page_size, blockIdx.z, gridDim.z);
}

// takes the page out of a table entry and drops one reference to it
__device__ __forceinline__ void release(const CacheView &c, int32_t *entry) {
    const int page = atomicExch(entry, -1);
    if (page < 0) return;
    if (page >= c.pages || atomicSub(c.refs + page, 1) <= 0) {
        if (page < c.pages) atomicAdd(c.refs + page, 1);
        range_error();
    }
}

__global__ void __launch_bounds__(CT) free_kernel(const CacheView c, const int32_t *list, int64_t window,
                                                  int64_t sinks) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = list[blockIdx.x];
    if (s < 0 || s >= c.seqs) {
        range_error();
        return;
    }
    const int64_t len = c.lens[s];
    __syncthreads();  // before lens is cleared below
    for (int64_t j = threadIdx.x; j < c.max_pages; j += CT) {
        const int64_t first = j << c.page_shift, last = first + c.page_size - 1;
        if (window == 0 || (first >= sinks && last <= len - window)) release(c, c.table + (int64_t)s * c.max_pages + j);
    }
    if (window == 0 && threadIdx.x == 0) c.lens[s] = 0;
}

// grid (blocks over max_new rows, seqs): row i of sequence s, all kv heads, K then V
__global__ void __launch_bounds__(CT) append_kernel(const CacheView c, const char *K, const char *V,
                                                    int64_t token_stride, const int32_t *q_start, int64_t tokens,
                                                    int64_t max_new) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.y;
    const RowRange r = rows_of(q_start, s, tokens, max_new, &g_pages_err);
    const int64_t len = c.lens[s];
    if (len < 0 || len + r.count > row_capacity(c)) {
        range_error();
        return;
    }
    const int vecs = c.head_dim / 8, row = vecs * c.kv_heads;
    const int64_t all = (int64_t)r.count * row * 2;
    for (int64_t e = (int64_t)blockIdx.x * CT + threadIdx.x; e < all; e += (int64_t)gridDim.x * CT) {
        const int64_t kv = e / row;
        const int i = (int)(kv >> 1), x = (int)(e - kv * row), h = x / vecs, w = x - h * vecs;
        const int64_t t = len + i;
        const int page = page_of(c, s, t >> c.page_shift);
        if (page < 0) {
            range_error();
            continue;
        }
        const char *src = (kv & 1 ? V : K) + (((int64_t)r.first + i) * token_stride + h * c.head_dim + w * 8) * 2;
        char *dst = (kv & 1 ? c.v : c.k) + (page * c.page_stride + h * c.head_stride +
                                            (t & (c.page_size - 1)) * c.token_stride + w * 8) * 2;
        *reinterpret_cast<uint4 *>(dst) = ld_stream_v4(src);
    }
}

// kept new tokens of sequence s; -1: out of range, and the sequence is left as it is
__device__ __forceinline__ int kept_of(const int32_t *kept, int s, int count) {
    if (!kept) return count;
    const int k = kept[s];
    if (k < 0 || k > count) {
        range_error();
        return -1;
    }
    return k;
}

// grid (kv heads x layers x 2, seqs).  Token i comes from keep[i] >= i, so a step of CT / vecs
// tokens read before they are written leaves what later steps read alone: their sources are at
// or past the first token of their own step.
__global__ void __launch_bounds__(CT) compact_move_kernel(const CacheView c, const int32_t *q_start,
                                                          const int32_t *keep, const int32_t *kept, int64_t tokens,
                                                          int64_t max_new) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.y;
    const RowRange r = rows_of(q_start, s, tokens, max_new, &g_pages_err);
    const int n = kept_of(kept, s, r.count);
    const int64_t len = c.lens[s];
    if (len < 0 || len + r.count > row_capacity(c)) {
        range_error();
        return;
    }
    const int which = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.kv_heads, layer = (blockIdx.x >> 1) / c.kv_heads;
    char *base = (which ? c.v : c.k) + (layer * c.layer_stride + h * c.head_stride) * 2;
    const int vecs = c.head_dim / 8, step = CT / vecs;
    const int t = threadIdx.x / vecs, w = threadIdx.x - t * vecs;
    const auto row = [&](int64_t tok, bool write) -> char * {
        const int page = page_of(c, s, tok >> c.page_shift);
        if (page < 0 || (write && c.refs[page] > 1)) {
            range_error();
            return nullptr;
        }
        return base + (page * c.page_stride + (tok & (c.page_size - 1)) * c.token_stride + w * 8) * 2;
    };
    for (int i0 = 0; i0 < n; i0 += step) {
        const int i = i0 + t;
        char *dst = nullptr;
        uint4 v;
        if (t < step && i < n) {
            const int from = keep[r.first + i];
            if (from < i || from >= r.count || (i > 0 && keep[r.first + i - 1] >= from)) {
                range_error();
            } else if (from != i) {
                const char *src = row(len + from, false);
                dst = row(len + i, true);
                if (src && dst) {
                    v = *reinterpret_cast<const uint4 *>(src);
                } else {
                    dst = nullptr;
                }
            }
        }
        __syncthreads();
        if (dst) *reinterpret_cast<uint4 *>(dst) = v;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(CT) compact_table_kernel(const CacheView c, const int32_t *q_start,
                                                           const int32_t *kept, int64_t tokens, int64_t max_new) {
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.x;
    const RowRange r = rows_of(q_start, s, tokens, max_new, &g_pages_err);
    const int64_t len = c.lens[s];
    if (len < 0 || len + r.count > row_capacity(c)) {
        range_error();
        return;
    }
    const int n = r.ok ? kept_of(kept, s, r.count) : -1;
    if (n < 0) return;
    const int64_t now = len + n;
    __syncthreads();  // before lens changes
    if (threadIdx.x == 0) c.lens[s] = (int)now;
    for (int64_t j = ((now + c.page_size - 1) >> c.page_shift) + threadIdx.x; j < c.max_pages; j += CT)
        release(c, c.table + (int64_t)s * c.max_pages + j);
}

// CTAs that share one layer's page: about 32 KB each
unsigned copy_parts(const CacheView &c) {
    const int64_t bytes = (int64_t)c.kv_heads * c.page_size * c.head_dim * 2;
    return (unsigned)(bytes <= 32768 ? 1 : bytes >= 32768 * 16 ? 16 : (bytes + 32767) / 32768);
}

}  // namespace

cudaError_t launch_cache_reserve(const CacheView &c, const int32_t *need, int32_t *missing, cudaStream_t s) {
    return launch_pdl(reserve_kernel, dim3(1), NT, 0, s, c, need, missing);
}

cudaError_t launch_cache_append(const CacheView &c, const void *K, const void *V, int64_t token_stride,
                                const int32_t *q_start, int64_t tokens, int64_t max_new, cudaStream_t s) {
    const int64_t vecs = max_new * c.kv_heads * (c.head_dim / 8) * 2;
    const int64_t blocks = (vecs + CT - 1) / CT;
    return launch_pdl(append_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)c.seqs), CT, 0, s, c,
                      static_cast<const char *>(K), static_cast<const char *>(V), token_stride, q_start, tokens, max_new);
}

cudaError_t launch_cache_compact(const CacheView &c, const int32_t *q_start, const int32_t *keep, const int32_t *kept,
                                 int64_t tokens, int64_t max_new, cudaStream_t s) {
    const dim3 seqs((unsigned)c.seqs);
    if (keep) {
        const cudaError_t e =
            launch_pdl(compact_move_kernel, dim3((unsigned)(2 * c.kv_heads * c.layers), (unsigned)c.seqs), CT, 0, s, c,
                       q_start, keep, kept, tokens, max_new);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(compact_table_kernel, seqs, CT, 0, s, c, q_start, kept, tokens, max_new);
}

cudaError_t launch_cache_fork(const CacheView &c, const int32_t *parents, const int32_t *children, int64_t n,
                              int32_t *missing, cudaStream_t s) {
    const cudaError_t e = launch_pdl(fork_alloc_kernel, dim3(1), NT, 0, s, c, parents, children, n, missing);
    if (e != cudaSuccess) return e;
    return launch_pdl(fork_copy_kernel, dim3((unsigned)n, (unsigned)(2 * c.layers), copy_parts(c)), CT, 0, s, c, parents,
                      children, missing);
}

cudaError_t launch_cache_free(const CacheView &c, const int32_t *list, int64_t n, int64_t window, int64_t sinks,
                              cudaStream_t s) {
    return launch_pdl(free_kernel, dim3((unsigned)n), CT, 0, s, c, list, window, sinks);
}

cudaError_t launch_cache_copy_pages(const CacheView &c, const int32_t *src, const int32_t *dst, int64_t n,
                                    cudaStream_t s) {
    return launch_pdl(copy_pages_kernel, dim3((unsigned)n, (unsigned)(2 * c.layers), copy_parts(c)), CT, 0, s, c, src, dst);
}

unsigned int cache_pages_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_pages_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_pages_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
