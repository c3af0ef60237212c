// sample.cu -- the next token of each row of logits by temperature, top-k, top-p and min-p, from a
// given uniform number per row.
//
// Mathematics.  A token's weight is a whole number, w_i = rint(2^30 exp((x_i - m) r)), so every sum
// of weights is exact in 64 bits and no result depends on the order of summation or on how a row is
// split over threads.  In the order (w descending, index ascending) each filter keeps a prefix; the
// token is the first in index order at which the running sum of the kept weights exceeds floor(u S).
//
// Bound: one pass over the logits.  With top-k on, that pass is all: the k-th largest of the maxima
// of disjoint groups of 8 logits is a lower bound of the k-th largest logit (k groups hold a logit at
// least as large), so a bound t from the row's first part lets the pass put the few logits >= t into a
// shared-memory list, and everything else happens there.  (The bound is read off a histogram of the group
// maxima; a bisection over the block took 9,000 to 13,000 cycles of barriers.)  What the list must hold is all tokens whose
// weight reaches that of the k-th (equal weights can have different logits: t is lowered by 1/16 of a
// temperature and the list is used only if the weight of the lowered bound is smaller).  Tokens more than
// 22 temperatures below a logit weigh 0 and are left out.  The list is cut to the k-th largest by a
// histogram of the weights, then every token's rank and the weight before it are counted against all
// others (k^2 comparisons, no sort).  256 threads do this, whatever the block: their barriers are cheaper.
//
// Rows that the list cannot serve (top-k off or above kMaxListK, a list that overflows) select by a
// radix descent on the weights: 512 bins by exponent and 4 leading bits, filled in one pass over the row (from L2);
// the weights of the chosen bin go to shared memory in a second one, and linear bins narrow them there.  The token
// is then found by sums over ever smaller stretches (general_row).
//
// Measured, one call: 1 x 50257 fp32 10 to 12 us and 64 x 50257 bf16 15.5 us, both latency (a dozen phases of barriers);
// 512 x 128000 fp32 69 us = 3.8 TB/s, of which the pass is 43 us at 6.1 TB/s and finding the bound, ranks and
// sums the rest.  General path, the same three sizes: temperature alone 20, 25 and 137 us; top-p 42, 48 and 333;
// top-k 1000 and top-p 52, 58 and 416 (with one 64-bit addition per token in shared memory and every level a
// pass over the row top-k and top-p took 278, 434 and 2,930).
#include "cache_view.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

namespace mm {

namespace {

constexpr int CAP = 4096;       // list entries
constexpr int CUT = 1024;       // entries left after the histogram's cut (3 CUT <= CAP)
// top-k served by the list, as far as it has room (CUT).  List and general path, top-k 500: 1 x 50257 30 and 52 us,
// 512 x 128000 132 and 417; top-k 200: 14 and 52, 76 and 416
constexpr int kMaxListK = 512;
constexpr int BINS = 512;
constexpr float kOne = 1073741824.0f;  // 2^30

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void get(uint4 v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    __device__ static float one(float x) { return x; }
};
template <>
struct Vec<__half> {
    static constexpr int N = 8;
    __device__ static void get(uint4 v, float (&x)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ static float one(__half x) { return __half2float(x); }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void get(uint4 v, float (&x)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    __device__ static float one(__nv_bfloat16 x) { return __bfloat162float(x); }
};

struct Shared {
    float x[CAP];
    int idx[CAP];
    unsigned long long mass[BINS];
    unsigned long long key[CUT];  // w << 32 | ~index: larger is earlier in the order
    int count[BINS];
    unsigned long long part[32];
    float2 fpart[32];
    int wsum[32];
    int n, cut, picked, bin;
    unsigned long long acc_mass;
    int acc_count;
};

// whole numbers from floats ordered as the floats are (no NaN)
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ uint32_t weight(float x, float m, float rate) {
    if (!(x > -INFINITY)) return 0;  // NaN and -infinity
    const float z = x == m ? 0.f : (x - m) * rate;
    return __float2uint_rn(expf(z) * kOne);
}

// All NT threads of the block, or (BAR 1) the first NT of it
template <int NT, int BAR>
__device__ __forceinline__ void sync() {
    if (BAR == 0) {
        __syncthreads();
    } else {
        __syncwarp();
        bar_sync(BAR, NT);
    }
}

// maxima of two values over the block
template <int NT>
__device__ __forceinline__ float2 block_max(float2 v, Shared &sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
        v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.fpart[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh.fpart[(threadIdx.x & 31) % (NT / 32)];
#pragma unroll
    for (int o = NT / 64; o; o >>= 1) {
        v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
        v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    }
    return v;
}

// The first bin of sh.count at which the running count reaches `target`, BINS if none does.  The counts must be
// complete (a barrier before); a barrier ends it.
template <int NT, int BAR>
__device__ __forceinline__ int first_bin(Shared &sh, int target) {
    constexpr int EACH = NT >= BINS ? 1 : BINS / NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = threadIdx.x * EACH;
    int c[EACH], n = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) c[i] = b0 + i < BINS ? sh.count[b0 + i] : 0, n += c[i];
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
    }
    if (lane == 31) sh.wsum[warp] = run;
    if (threadIdx.x == 0) sh.bin = BINS;
    sync<NT, BAR>();
    run += __reduce_add_sync(0xffffffffu, lane < warp ? sh.wsum[lane] : 0) - n;  // in front of this thread's bins
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (run < target && run + c[i] >= target) sh.bin = b0 + i;
        run += c[i];
    }
    sync<NT, BAR>();
    return sh.bin;
}

template <int NT, int BAR>
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, Shared &sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    sync<NT, BAR>();
    if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
    sync<NT, BAR>();
    unsigned long long s = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s += sh.part[i];
    return s;
}

struct Row {
    float rate;
    int k;           // 0: off
    float top_p, u;
    uint32_t floor_w;  // min-p
};

// floor(f n) and whether there is a rest, exactly, for 0 < f < 1 and n < 2^63 (in whole numbers: a block's worth
// of fp64 products takes this GPU thousands of cycles)
__device__ __forceinline__ unsigned long long times(float f, unsigned long long n, bool *rest) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;
    const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);  // f = m 2^-shift
    const int shift = 150 - (int)max(e, 1u);                                  // 24 .. 149
    const unsigned long long lo = m * n, hi = __umul64hi(m, n);
    if (shift >= 128) {
        *rest = (lo | hi) != 0;
        return 0;
    }
    if (shift >= 64) {
        *rest = lo != 0 || (hi & ((1ull << (shift - 64)) - 1)) != 0;
        return hi >> (shift - 64);
    }
    *rest = (lo & ((1ull << shift) - 1)) != 0;
    return hi << (64 - shift) | lo >> shift;
}
__device__ __forceinline__ unsigned long long top_p_target(float p, unsigned long long mass) {
    if (!(p < 1.f)) return mass;
    if (!(p > 0.f)) return 1;
    bool rest;
    const unsigned long long t = times(p, mass, &rest);
    return t + rest;
}
__device__ __forceinline__ unsigned long long wanted(float u, unsigned long long total) {
    if (!(u > 0.f)) return 0;
    bool rest;
    return u < 1.f ? times(u, total, &rest) : total - 1;
}

__device__ __forceinline__ void put(const SampleArgs &a, int64_t row, int token, uint32_t w, unsigned long long total) {
    a.tokens[row] = token;
    // log(w / S) = -log1p((S - w) / w): exact near probability 1
    if (a.logprobs) a.logprobs[row] = token < 0 ? -INFINITY : -log1pf((float)(total - w) / (float)w);
}

__device__ __forceinline__ int bin_of(uint32_t w) { return (int)(__float_as_uint(__uint2float_rz(w)) >> 19) - (127 << 4); }
__device__ __forceinline__ uint32_t bin_low(int b) {
    return (uint32_t)ceilf(__uint_as_float((uint32_t)(b + (127 << 4)) << 19));
}

// The first bin from the top at which the running count (or mass) reaches the target; what lies
// above it is added to acc.  All of warp 0; 16 bins a lane.
__device__ __forceinline__ void find_bin(Shared &sh, bool by_mass, unsigned long long target) {
    const int lane = threadIdx.x;
    const int top = BINS - 1 - 16 * lane;  // this lane's bins: top, top - 1, ..., top - 15
    unsigned long long mine_m = 0;
    int mine_c = 0;
    for (int i = 0; i < 16; ++i) mine_m += sh.mass[top - i], mine_c += sh.count[top - i];
    unsigned long long m = mine_m;
    int c = mine_c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long um = __shfl_up_sync(0xffffffffu, m, o);
        const int uc = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) m += um, c += uc;
    }
    const unsigned long long have_m = sh.acc_mass;
    const int have_c = sh.acc_count;
    const bool reached = by_mass ? have_m + m >= target : (unsigned long long)(have_c + c) >= target;
    const unsigned at = __ballot_sync(0xffffffffu, reached);
    __syncwarp();
    if (at == 0) {
        if (lane == 0) sh.bin = -1;
    } else if (lane == __ffs(at) - 1) {
        unsigned long long am = have_m + m - mine_m;
        int ac = have_c + c - mine_c, b = top;
        for (; b > top - 15; --b) {
            if (by_mass ? am + sh.mass[b] >= target : (unsigned long long)(ac + sh.count[b]) >= target) break;
            am += sh.mass[b], ac += sh.count[b];
        }
        sh.bin = b, sh.acc_mass = am, sh.acc_count = ac;
    }
    __syncwarp();
}

// f(logit) for elements from .. to - 1, each by one of `count` threads (t is this one's number); 16-byte loads
template <typename T, typename F>
__device__ __forceinline__ void each(const T *x, int64_t from, int64_t to, int t, int count, const F &f) {
    constexpr int N = Vec<T>::N, U = 2;
    const T *p = x + from;
    const int64_t n = to - from;
    const int64_t head = min(n, (int64_t)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)));
    const uint4 *body = reinterpret_cast<const uint4 *>(p + head);
    const int64_t vecs = (n - head) / N, tail = head + vecs * N;
    for (int64_t v0 = t; v0 < vecs; v0 += U * count) {
        uint4 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (v0 + j * count < vecs) v[j] = __ldg(body + v0 + j * count);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (v0 + j * count >= vecs) continue;
            float e[N];
            Vec<T>::get(v[j], e);
#pragma unroll
            for (int i = 0; i < N; ++i) f(e[i]);
        }
    }
    for (int64_t i = t; i < head + n - tail; i += count) f(Vec<T>::one(p[i < head ? i : tail + i - head]));
}

// What the general path keeps in the list's places
struct General {
    uint32_t *list;                       // weights of one bin: sh.x
    unsigned long long *mass;             // the first level's bins: sh.idx
    int *count;
    uint32_t *mass_lo, *mass_hi;          // sums being made, by 15 bits: sh.key
    __device__ __forceinline__ explicit General(Shared &sh)
        : list(reinterpret_cast<uint32_t *>(sh.x)), mass(reinterpret_cast<unsigned long long *>(sh.idx)),
          count(reinterpret_cast<int *>(mass + BINS)), mass_lo(reinterpret_cast<uint32_t *>(sh.key)), mass_hi(mass_lo + BINS) {}
};

// sh.mass and sh.count of weights by bin: visit(first, last, add) hands the weights of elements first .. last - 1 to
// add(w, bin).  Sums are made in 32-bit parts (shared memory has no 64-bit addition): a weight's low and high 15 bits,
// 2^16 elements at a time.
template <int NT, typename Visit>
__device__ __forceinline__ void fill_bins(Shared &sh, int64_t n, const Visit &visit) {
    const General g(sh);
    __syncthreads();
    for (int b = threadIdx.x; b < BINS; b += NT) sh.mass[b] = 0, sh.count[b] = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 1 << 16) {
        for (int b = threadIdx.x; b < BINS; b += NT) g.mass_lo[b] = 0, g.mass_hi[b] = 0;
        __syncthreads();
        visit(i0, min(n, i0 + (1 << 16)), [&](uint32_t w, int b) {
            atomicAdd(g.mass_lo + b, w & 0x7fffu);
            atomicAdd(g.mass_hi + b, w >> 15);
            atomicAdd(&sh.count[b], 1);
        });
        __syncthreads();
        for (int b = threadIdx.x; b < BINS; b += NT) sh.mass[b] += g.mass_lo[b] + ((unsigned long long)g.mass_hi[b] << 15);
    }
    __syncthreads();
}

// The cut of the row's order at `target` tokens (or so much mass): weights above *cut_w and the
// first *taken of those equal to it.  Returns the mass in front of the cut; *cut_w = 0 where the whole
// row does not reach the target.  The first level's bins are in General.
template <typename T, int NT>
__device__ unsigned long long find_cut(const T *x, int64_t n, float m, const Row &r, Shared &sh, bool by_mass,
                                       unsigned long long target, uint32_t *cut_w, unsigned long long *taken) {
    const General g(sh);
    __syncthreads();
    for (int b = threadIdx.x; b < BINS; b += NT) sh.mass[b] = g.mass[b], sh.count[b] = g.count[b];
    if (threadIdx.x == 0) sh.acc_mass = 0, sh.acc_count = 0;
    __syncthreads();
    if (threadIdx.x < 32) find_bin(sh, by_mass, target);
    __syncthreads();
    const int first = sh.bin;
    if (first < 0) {  // the row has less
        *cut_w = 0, *taken = 0;
        unsigned long long all = 0;
        for (int q = threadIdx.x; q < BINS; q += NT) all += sh.mass[q];
        return block_sum<NT, 0>(all, sh);
    }
    uint32_t lo = bin_low(first), hi = bin_low(first + 1) - 1;
    const int in_bin = sh.count[first];
    const bool listed = in_bin <= CAP;  // the bin's weights in shared memory, and no further pass over the row
    if (listed && lo < hi) {
        if (threadIdx.x == 0) sh.n = 0;
        __syncthreads();
        each(x, 0, n, threadIdx.x, NT, [&](float v) {
            const uint32_t w = weight(v, m, r.rate);
            if (w >= lo && w <= hi) g.list[atomicAdd(&sh.n, 1)] = w;
        });
    }
    while (lo < hi) {
        const int bits = 32 - __clz(hi - lo), shift = bits > 9 ? bits - 9 : 0;
        fill_bins<NT>(sh, listed ? in_bin : n, [&](int64_t i0, int64_t i1, const auto &add) {
            const auto offer = [&](uint32_t w) {
                if (w >= lo && w <= hi) add(w, (int)((w - lo) >> shift));
            };
            if (listed)
                for (int i = (int)i0 + threadIdx.x; i < i1; i += NT) offer(g.list[i]);
            else
                each(x, i0, i1, threadIdx.x, NT, [&](float v) { offer(weight(v, m, r.rate)); });
        });
        if (threadIdx.x < 32) find_bin(sh, by_mass, target);
        __syncthreads();
        lo += (uint32_t)sh.bin << shift;
        hi = min(hi, lo + (1u << shift) - 1);
    }
    *cut_w = lo;
    *taken = by_mass ? (target - sh.acc_mass + lo - 1) / lo : target - (unsigned long long)sh.acc_count;
    return sh.acc_mass + *taken * lo;
}

// Any row: the cuts by radix descent, then the token.  Of the kept weights only those equal to the cut depend on the
// index order, and they are all alike: the kept mass of a stretch is the mass above the cut and the cut times as many
// of its ties as are still to be taken.  So the stretch that holds the token is found by sums in any order, over a
// part of the row for each warp, then over parts of that part, until a warp walks the last 64 in order.
template <typename T, int NT>
__device__ __forceinline__ void general_row(const SampleArgs &a, int64_t row, const T *x, int64_t n, float m, const Row &r, Shared &sh) {
    constexpr int W = NT / 32;
    uint32_t cut = 0;
    unsigned long long taken = 0;
    if (r.k > 0 || r.top_p < 1.f) {
        const General g(sh);
        fill_bins<NT>(sh, n, [&](int64_t i0, int64_t i1, const auto &add) {
            each(x, i0, i1, threadIdx.x, NT, [&](float v) {
                const uint32_t w = weight(v, m, r.rate);
                if (w) add(w, bin_of(w));
            });
        });
        unsigned long long mass = 0;
        for (int b = threadIdx.x; b < BINS; b += NT) {
            mass += sh.mass[b];
            g.mass[b] = sh.mass[b], g.count[b] = sh.count[b];
        }
        if (r.k > 0)
            mass = find_cut<T, NT>(x, n, m, r, sh, false, (unsigned long long)r.k, &cut, &taken);
        else
            mass = block_sum<NT, 0>(mass, sh);
        if (r.top_p < 1.f && mass > 0) find_cut<T, NT>(x, n, m, r, sh, true, top_p_target(r.top_p, mass), &cut, &taken);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t above = max(max(cut + 1, r.floor_w), 1u);      // weights kept whatever their place
    const bool ties_stay = cut != 0 && cut >= r.floor_w;
    int64_t from = 0, to = n;
    unsigned long long before = 0, ties_before = 0, want = 0, total = 0;  // in front of `from`
    do {
        const int64_t share = ((to - from + W - 1) / W + 31) / 32 * 32;
        const int64_t f = min(to, from + warp * share), t = min(to, f + share);
        unsigned long long mine = 0;
        int ties = 0;
        each(x, f, t, lane, 32, [&](float v) {
            const uint32_t w = weight(v, m, r.rate);
            if (w >= above) mine += w;
            ties += ties_stay && w == cut;
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        ties = __reduce_add_sync(0xffffffffu, ties);
        __syncthreads();
        if (lane == 0) sh.part[warp] = mine, sh.wsum[warp] = ties;
        __syncthreads();
        const auto kept = [&](int i, unsigned long long tie) {
            const unsigned long long left = tie < taken ? taken - tie : 0;
            return sh.part[i] + cut * min(left, (unsigned long long)sh.wsum[i]);
        };
        if (total == 0) {
            unsigned long long tie = 0;
            for (int i = 0; i < W; tie += sh.wsum[i], ++i) total += kept(i, tie);
            if (total == 0) {
                if (threadIdx.x == 0) put(a, row, -1, 1, 1);
                return;
            }
            want = wanted(r.u, total);
        }
        int i = 0;
        for (; i < W - 1; ++i) {
            const unsigned long long here = kept(i, ties_before);
            if (want < before + here) break;
            before += here, ties_before += sh.wsum[i];
        }
        from = min(to, from + i * share), to = min(to, from + share);
    } while (to - from > 64);
    if (warp != 0) return;
    for (int64_t i = from + lane; i - lane < to; i += 32) {
        const uint32_t w0 = i < to ? weight(Vec<T>::one(x[i]), m, r.rate) : 0u;
        const unsigned eq = __ballot_sync(0xffffffffu, ties_stay && w0 == cut);
        const bool tie = ties_stay && w0 == cut && ties_before + __popc(eq & ((1u << lane) - 1)) < taken;
        const uint32_t w = w0 >= above || tie ? w0 : 0u;
        ties_before += __popc(eq);
        unsigned long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        const bool here = w != 0 && before + s > want && before + s - w <= want;
        if (here) put(a, row, (int)i, w, total);
        if (__any_sync(0xffffffffu, here)) return;
        before += __shfl_sync(0xffffffffu, s, 31);
    }
}

// The token from the list of `have` logits, by the first TAIL threads of the block; true: too many equal weights.
template <int TAIL, int BAR>
__device__ __forceinline__ bool from_list(const SampleArgs &a, int64_t row, int have, float m, const Row &r, Shared &sh) {
    // the k heaviest of the list, by bins of their weights
    for (int b = threadIdx.x; b < BINS; b += TAIL) sh.count[b] = 0;
    sync<TAIL, BAR>();
    for (int i = threadIdx.x; i < have; i += TAIL) {
        const uint32_t w = weight(sh.x[i], m, r.rate);
        sh.x[i] = __uint_as_float(w);
        if (w) atomicAdd(&sh.count[BINS - 1 - bin_of(w)], 1);
    }
    sync<TAIL, BAR>();
    const int last = first_bin<TAIL, BAR>(sh, r.k);
    const uint32_t least = last == BINS ? 1u : bin_low(BINS - 1 - last);
    for (int i = threadIdx.x; i < have; i += TAIL) {
        const uint32_t w = __float_as_uint(sh.x[i]);
        if (w >= least) {
            const int at = atomicAdd(&sh.cut, 1);
            if (at < CUT) sh.key[at] = (unsigned long long)w << 32 | (uint32_t)~sh.idx[i];
        }
    }
    sync<TAIL, BAR>();
    const int c = sh.cut;
    if (c > CUT) {  // very many equal weights
        return true;
    }
    // rank and weight in front of each, four lanes per token (kept in the list's place, which is free)
    unsigned long long *before = reinterpret_cast<unsigned long long *>(sh.x);
    int *rank = sh.idx;
    const int sub = threadIdx.x & 3;
    unsigned long long mass = 0;
    for (int e0 = 0; e0 < c; e0 += TAIL / 4) {
        const int e = e0 + (threadIdx.x >> 2);
        const unsigned long long key = e < c ? sh.key[e] : ~0ull;
        unsigned long long in_front = 0;
        int n_front = 0;
#pragma unroll 4
        for (int f = sub; f < c; f += 4) {
            const unsigned long long o = sh.key[f];
            if (o > key) in_front += o >> 32, ++n_front;
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            in_front += __shfl_xor_sync(0xffffffffu, in_front, o);
            n_front += __shfl_xor_sync(0xffffffffu, n_front, o);
        }
        if (e < c && sub == 0) {
            before[e] = in_front, rank[e] = n_front;
            if (n_front < r.k) mass += key >> 32;
        }
    }
    mass = block_sum<TAIL, BAR>(mass, sh);
    const unsigned long long target = top_p_target(r.top_p, mass);
    float *kept_w = sh.x + 2 * CUT;
    int *kept_i = sh.idx + CUT;
    unsigned long long total = 0;
    for (int e = threadIdx.x; e < c; e += TAIL) {
        const unsigned long long key = sh.key[e];
        if (rank[e] < r.k && (rank[e] == 0 || before[e] < target) && (uint32_t)(key >> 32) >= r.floor_w) {
            total += key >> 32;
            const int at = atomicAdd(&sh.picked, 1);
            kept_w[at] = __uint_as_float((uint32_t)(key >> 32));
            kept_i[at] = (int)~(uint32_t)key;
        }
    }
    total = block_sum<TAIL, BAR>(total, sh);
    if (total == 0) {
        if (threadIdx.x == 0) put(a, row, -1, 1, 1);
        return false;
    }
    const unsigned long long want = wanted(r.u, total);
    const int kept = sh.picked;
    for (int e0 = 0; e0 < kept; e0 += TAIL / 4) {
        const int e = e0 + (threadIdx.x >> 2);
        unsigned long long s = 0;
        const int me = e < kept ? kept_i[e] : 0;
#pragma unroll 4
        for (int f = sub; f < kept; f += 4)
            if (kept_i[f] < me) s += __float_as_uint(kept_w[f]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (e < kept && sub == 0) {
            const uint32_t w = __float_as_uint(kept_w[e]);
            if (s <= want && want < s + w) put(a, row, me, w, total);
        }
    }
    return false;
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    constexpr int N = Vec<T>::N, G = 8 / N;  // vectors per group of 8
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x, n = a.vocab;
    const T *x = static_cast<const T *>(a.logits) + row * a.stride;
    Row r;
    const float temp = a.temperature ? a.temperature[row] : 1.f;
    r.rate = 1.f / fmaxf(temp, 0.f);  // infinity for the greedy choice
    r.k = a.top_k ? max(a.top_k[row], 0) : 0;
    if (!(temp > 0.f)) r.k = 1;
    r.top_p = a.top_p ? a.top_p[row] : 1.f;
    r.u = a.u[row];
    const float fw = ceilf((a.min_p ? a.min_p[row] : 0.f) * kOne);
    r.floor_w = fw > 0.f ? (fw < 4e9f ? (uint32_t)fw : 0xffffffffu) : 0u;

    // 16-byte vectors from the first aligned element on; the few in front and behind are scalars
    const int64_t head = min(n, (int64_t)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
    const uint4 *body = reinterpret_cast<const uint4 *>(x + head);
    const int64_t vecs = (n - head) / N, tail = head + vecs * N;
    const int edge = (int)(head + n - tail);  // < 2 N
    const auto edge_index = [&](int i) { return i < head ? (int64_t)i : tail + i - head; };

    const bool listed = r.k > 0 && r.k <= kMaxListK;
    float low = INFINITY;  // logits >= low go to the list
    if (threadIdx.x == 0) sh.n = 0, sh.cut = 0, sh.picked = 0;
    float t0 = -INFINITY;
    bool all_heavy = false;  // what is below `low` weighs 0
    if (listed) {
        // The first part: GROUPS groups of 8 rep logits per thread, so long that the list holds about 2700 logits at most
        constexpr int GROUPS = NT >= 1024 ? 4 : 2048 / NT;
        const int rep = (int)min((long long)r.k * n / (2700ll * 8 * GROUPS * NT) + 1, 64ll);
        float g[GROUPS], gx = -INFINITY, gl = -INFINITY;  // their maxima, the largest, minus the least finite one
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            g[q] = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < rep; ++i)
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int64_t v = (int64_t)((q * rep + i) * G + j) * NT + threadIdx.x;
                    if (v < vecs) {
                        float f[N];
                        Vec<T>::get(__ldg(body + v), f);
#pragma unroll
                        for (int e = 0; e < N; ++e) g[q] = fmaxf(g[q], f[e]);
                    }
                }
            gx = fmaxf(gx, g[q]);
            if (g[q] > -INFINITY) gl = fmaxf(gl, -g[q]);
        }
        for (int b = threadIdx.x; b < BINS; b += NT) sh.count[b] = 0;
        const float2 ends = block_max<NT>(make_float2(gx, gl), sh);
        const float mx = ends.x;
        // bins of the maxima's distance from the largest, over the range that can weigh anything
        const float range = fminf(22.f / r.rate, mx + ends.y), inv = range > 0.f ? (BINS - 1) / range : 0.f;
        int bin[GROUPS];
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            bin[q] = g[q] == mx ? 0 : (int)fminf((mx - g[q]) * inv, (float)(BINS - 1));
            atomicAdd(&sh.count[bin[q]], 1);
        }
        __syncthreads();
        const int last = first_bin<NT, 0>(sh, r.k);
        // the least of the maxima up to that bin: at least k of them are not below it
        float least = -INFINITY;
#pragma unroll
        for (int q = 0; q < GROUPS; ++q)
            if (bin[q] <= last) least = fmaxf(least, -g[q]);
        t0 = -block_max<NT>(make_float2(least, -INFINITY), sh).x;
        // a sixteenth of a temperature lower, but not where every weight is 0 whatever the rest holds
        const float down = t0 - 0.0625f / r.rate;
        low = down < t0 ? down : from_key(max(order_key(t0 + 0.f), order_key(-FLT_MAX)) - 1);
        const float none = mx - 22.f / r.rate;
        all_heavy = none >= low;
        low = fmaxf(fmaxf(low, none), -FLT_MAX);
    }
    __syncthreads();

    // the pass over the row
    float m = -INFINITY;
    const auto offer = [&](float f, int64_t i) {
        if (f >= low) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < CAP) sh.x[at] = f, sh.idx[at] = (int)i;
        }
    };
    constexpr int U = 4;
    for (int64_t v0 = threadIdx.x; v0 < vecs; v0 += U * NT) {
        uint4 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (v0 + j * NT < vecs) v[j] = ld_stream_v4(body + v0 + j * NT);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (v0 + j * NT >= vecs) continue;
            float f[N], vm = -INFINITY;
            Vec<T>::get(v[j], f);
#pragma unroll
            for (int e = 0; e < N; ++e) vm = fmaxf(vm, f[e]);
            m = fmaxf(m, vm);
            if (vm >= low) {
#pragma unroll
                for (int e = 0; e < N; ++e) offer(f[e], head + (v0 + j * NT) * N + e);
            }
        }
    }
    if (threadIdx.x < edge) {
        const int64_t i = edge_index(threadIdx.x);
        const float f = Vec<T>::one(x[i]);
        m = fmaxf(m, f);
        offer(f, i);
    }
    m = block_max<NT>(make_float2(m, 0.f), sh).x;
    if (m == -INFINITY) {  // nothing is left of the row
        if (threadIdx.x == 0) put(a, row, -1, 1, 1);
        return;
    }
    const int have = sh.n;
    bool ok = listed && have <= CAP;
    if (ok && !all_heavy) {  // does the list hold every token that weighs as much as the k-th?
        const uint32_t wk = weight(t0, m, r.rate), wl = weight(low, m, r.rate);
        ok = wl == 0 || wl < wk - (wk >> 20);
    }
    if (ok) {
        constexpr int TAIL = 256;
        bool many;
        if (NT == TAIL) {
            many = from_list<TAIL, 0>(a, row, have, m, r, sh);
        } else {
            if (threadIdx.x < TAIL) {
                many = from_list<TAIL, 1>(a, row, have, m, r, sh);
                if (threadIdx.x == 0) sh.bin = many;
            }
            __syncthreads();
            many = sh.bin;
        }
        if (!many) return;
    }
    general_row<T, NT>(a, row, x, n, m, r, sh);
}

template <typename T, int NT>
cudaError_t launch(const SampleArgs &a, cudaStream_t s) {
    static SmemLimit limit;
    const cudaError_t e = limit.allow((const void *)sample_kernel<T, NT>, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    return launch_pdl(sample_kernel<T, NT>, dim3((unsigned)a.rows), NT, sizeof(Shared), s, a);
}

template <typename T>
cudaError_t launch_t(const SampleArgs &a, int sms, cudaStream_t s) {
    // Up to two rows per SM one after the other, all the SM's warps on each; more rows four to an SM at a time, some
    // streaming while others choose.  1024 threads against 256: 1 x 50257 11.8 and 18.2 us, 152 x 128000 25 and 56,
    // 300 x 50257 32.1 and 33.1, 512 x 128000 79 and 69.
    return a.rows <= 2 * sms ? launch<T, 1024>(a, s) : launch<T, 256>(a, s);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int sms, cudaStream_t s) {
    if (a.dtype == 0) return launch_t<__half>(a, sms, s);
    if (a.dtype == 1) return launch_t<__nv_bfloat16>(a, sms, s);
    return launch_t<float>(a, sms, s);
}

}  // namespace mm
