// experts_route.cu -- a mixture of experts' router behind its logits: the top k experts of each token, their weights,
// and the tokens' places in an order by expert, in which the ragged products run.
//
// A warp takes a token with E / 32 logits to a lane, as whole numbers that order like the logits; the largest is found
// by two reductions over the warp (the value, then the lowest index that has it), k times.  The order is a counting
// sort: how many picks of each expert come before a token's is the sum over the experts before, the blocks of tokens
// before and the warps before, and a warp then walks its own tokens.  Up to ONE tokens one CTA does it all; with more a
// first kernel leaves each block's counts in the workspace and a second adds them up and places.  Nothing is counted
// with atomics whose order could show, so the order by expert is by token within.
//
// What bounds it: the launches and the chains of dependent reductions for few tokens (1 x 8: 3.0 us); a call reads the logits
// once and writes 16 bytes a pick (8191 x 128, 8 picks: 14.1 us, half of it picks, half places).
#include "cache_view.cuh"
#include "mm_common.cuh"
#include "mm_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

namespace mm {

namespace {

// Tokens that one CTA takes (us, one CTA and two kernels: 64 x 64 6.2 and 7.0, 80 x 64 7.9 and 7.4, 128 x 64 9.0 and 7.3)
constexpr int ONE = 64;
constexpr int BLOCKS = 128;       // blocks of tokens otherwise, at most (more only above 2^22 tokens)
constexpr int MAX_PER = 1 << 15;  // tokens of a block
constexpr int COUNTS = 8448;      // shared counts: [warps][experts], rows an odd number of words apart

__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Whole numbers that order like the logits (both zeros alike); 0 for NaN and -infinity, which are never picked.  A logit of
// 16 bits leaves the lower half to the expert, lower ones larger, so that the largest number is the pick: one reduction finds
// the value and the lowest index that has it (with fp32 it takes a second one).
template <typename T>
struct Key {
    static constexpr bool kHasIndex = true;
    static __device__ __forceinline__ uint32_t of(T x, int expert) {
        if (!(widen(x) > -INFINITY)) return 0;
        uint32_t b = *reinterpret_cast<const uint16_t *>(&x);
        if (b == 0x8000u) b = 0;
        return ((b >> 15 ? ~b : b | 0x8000u) << 16) | (0xFFFFu - (uint32_t)expert);
    }
    static __device__ __forceinline__ float value(uint32_t k) {
        const uint16_t b = (uint16_t)(k >> 31 ? (k >> 16) & 0x7FFFu : ~(k >> 16));
        return widen(*reinterpret_cast<const T *>(&b));
    }
};
template <>
struct Key<float> {
    static constexpr bool kHasIndex = false;
    static __device__ __forceinline__ uint32_t of(float x, int) {
        if (!(x > -INFINITY)) return 0;
        const uint32_t b = __float_as_uint(x + 0.0f);
        return b >> 31 ? ~b : b | 0x80000000u;
    }
    static __device__ __forceinline__ float value(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A token's logits, those of experts lane, lane + 32, ... to a lane
template <typename T, int PER>
struct Logits {
    T v[PER];
    __device__ __forceinline__ void load(const RouteArgs &a, int64_t t, int lane) {
        const T *x = static_cast<const T *>(a.logits) + t * a.stride + lane;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < a.experts) v[i] = __ldg(x + 32 * i);
    }
};

// The picks of token t: lane j < top_k returns expert j (or -1) and its weight is written.
template <typename T, int PER>
__device__ __forceinline__ int pick(const RouteArgs &a, int64_t t, const Logits<T, PER> &x, int lane) {
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = lane + 32 * i < a.experts ? Key<T>::of(x.v[i], lane + 32 * i) : 0;
    const auto value = [](uint32_t k) { return Key<T>::value(k); };
    constexpr bool SHORT = Key<T>::kHasIndex;
    float sum = 0.f;  // of the softmax over all experts
    uint32_t first = 0;
    int id = -1;
    float mine = -INFINITY;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        const uint32_t top = __reduce_max_sync(~0u, best);
        if (top == 0) break;
        int at;
        if constexpr (SHORT) {
            at = (int)(0xFFFFu - (top & 0xFFFFu));
        } else {
            at = 1 << 30;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == top) at = lane + 32 * i;
            at = (int)__reduce_min_sync(~0u, (unsigned)at);
        }
        if (j == 0) {
            first = top;
            if (!a.sigmoid && !a.renorm) {
                const float m = value(top);
#pragma unroll
                for (int i = 0; i < PER; ++i) sum += key[i] ? expf(value(key[i]) - m) : 0.f;
                sum = warp_sum(sum);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (SHORT ? key[i] == top : at == lane + 32 * i) key[i] = 0;
        if (lane == j) id = at, mine = value(top);
    }
    // Softmax: exp(x - largest) over its sum; sigmoid: 1 / (1 + exp(-x)).  Normalised sigmoids are divided by the largest
    // one's exp(x) first where that is below 1, so that they do not all vanish.
    const float m = value(first);
    float w = 0.f;
    if (id >= 0) {
        if (!a.sigmoid) w = expf(mine - m);
        else if (a.renorm && m < 0.f) w = expf(mine - m) / (1.0f + expf(mine));
        else w = 1.0f / (1.0f + expf(-mine));
    }
    if (a.renorm) sum = warp_sum(w);
    if (a.renorm || !a.sigmoid) w /= sum;
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = id >= 0 ? w * a.scale : 0.f;
    }
    return id;
}

// Tokens [begin, end) of warp `warp` of `warps` in block b of `per` tokens.
struct Share {
    int64_t begin, end;
};
__device__ __forceinline__ Share share_of(int64_t tokens, int64_t per, int b, int warp, int warps) {
    const int64_t t0 = min(b * per, tokens), n = min(per, tokens - t0), each = (n + warps - 1) / warps;
    const int64_t begin = min(warp * each, n), end = min(begin + each, n);
    return {t0 + begin, t0 + end};
}

__device__ __forceinline__ int row_of(int experts) { return experts | 1; }

// From each expert's count over all blocks, and over the blocks before this one, to the first place of its picks in this
// block: base[e].  Whole block; scratch [33].
__device__ __forceinline__ void scan_experts(int *total, int *base, int experts, int32_t *offsets, int *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x, own = e < experts ? total[e] : 0;
        int run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) scratch[warp] = run;
        __syncthreads();
        int before = carry, all = 0;
        const int used = min(warps, (experts - e0 + 31) / 32);
        for (int w = 0; w < used; ++w) {
            const int v = scratch[w];
            if (w < warp) before += v;
            all += v;
        }
        if (e < experts) {
            base[e] += before + run - own;
            if (offsets) offsets[e] = before + run - own;
        }
        carry += all;
        __syncthreads();
    }
    if (offsets && threadIdx.x == 0) offsets[experts] = carry;
}

// Places: counts[warp][e] become the warps' first places from base[e] (a warp to an expert, a lane to a warp's count), then
// every warp walks its tokens.
__device__ __forceinline__ void place(const RouteArgs &a, const Share &s, int *counts, const int *base, int warps) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = a.top_k, row = row_of(a.experts);
    for (int e = warp; e < a.experts; e += blockDim.x >> 5) {
        const int n = lane < warps ? counts[lane * row + e] : 0;
        int run = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += up;
        }
        if (lane < warps) counts[lane * row + e] = base[e] + run - n;
    }
    __syncthreads();
    if (warp >= warps) return;
    int *next = counts + warp * row;
    int id = s.begin < s.end && lane < k ? a.ids[s.begin * k + lane] : -1;
    for (int64_t t = s.begin; t < s.end; ++t) {
        const int after = t + 1 < s.end && lane < k ? a.ids[(t + 1) * k + lane] : -1;
        if (lane < k) {
            int at = -1;
            if (id >= 0) {  // the experts of a token differ, so its lanes do not meet
                at = next[id];
                next[id] = at + 1;
                a.order[at] = (int)(t * k + lane);
            }
            a.slots[t * k + lane] = at;
        }
        __syncwarp();
        id = after;
    }
}

// Picks of a block's tokens; with one block the places too.
template <typename T, int PER>
__global__ void __launch_bounds__(PER > 8 ? 512 : 1024) route_pick_kernel(const __grid_constant__ RouteArgs a, const int64_t per, const int warps) {
    __shared__ int counts[COUNTS];
    __shared__ int total[32 * PER], scratch[33];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Share s = share_of(a.tokens, per, blockIdx.x, warp, warps);
    for (int i = threadIdx.x; i < warps * row_of(a.experts); i += blockDim.x) counts[i] = 0;
    __syncthreads();
    if (warp < warps) {
        Logits<T, PER> x, next;
        if (s.begin < s.end) x.load(a, s.begin, lane);
        for (int64_t t = s.begin; t < s.end; ++t) {
            if (t + 1 < s.end) next.load(a, t + 1, lane);
            const int id = pick<T, PER>(a, t, x, lane);
            x = next;
            if (id >= 0) ++counts[warp * row_of(a.experts) + id];
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = warp; e < a.experts; e += blockDim.x >> 5) {
        const int n = __reduce_add_sync(~0u, lane < warps ? counts[lane * row_of(a.experts) + e] : 0);
        if (lane == 0) {
            if (gridDim.x > 1) a.counts[(int64_t)blockIdx.x * a.experts + e] = n;
            total[e] = n;
        }
    }
    if (gridDim.x > 1) return;
    __shared__ int base[32 * PER];
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) base[e] = 0;
    __syncthreads();
    scan_experts(total, base, a.experts, a.offsets, scratch);
    __syncthreads();
    place(a, s, counts, base, warps);
}

template <int PER>
__global__ void __launch_bounds__(PER > 8 ? 512 : 1024) route_place_kernel(const __grid_constant__ RouteArgs a, const int64_t per, const int warps) {
    __shared__ int counts[COUNTS];
    __shared__ int total[32 * PER], base[32 * PER], scratch[33];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Share s = share_of(a.tokens, per, blockIdx.x, warp, warps);
    for (int i = threadIdx.x; i < warps * row_of(a.experts); i += blockDim.x) counts[i] = 0;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) total[e] = base[e] = 0;
    __syncthreads();
    // The blocks' counts: a thread to an expert and a stretch of the blocks, eight loads on their way; whole numbers, whose
    // sums any order of the additions gives.
    const int wide = (a.experts + 31) & ~31, teams = max(1, (int)blockDim.x / wide), team = threadIdx.x / wide;
    for (int e = threadIdx.x - team * wide; team < teams && e < a.experts; e += blockDim.x) {
        const int each = ((int)gridDim.x + teams - 1) / teams, b0 = team * each, b1 = min(b0 + each, (int)gridDim.x);
        int all = 0, before = 0;
        for (int b = b0; b < b1; b += 8) {
            int n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = b + i < b1 ? __ldg(a.counts + (int64_t)(b + i) * a.experts + e) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) all += n[i], before += b + i < (int)blockIdx.x ? n[i] : 0;
        }
        atomicAdd(&total[e], all);
        atomicAdd(&base[e], before);
    }
    if (warp < warps) {
        for (int64_t t = s.begin; t < s.end; ++t) {
            const int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
            if (id >= 0) ++counts[warp * row_of(a.experts) + id];
            __syncwarp();
        }
    }
    __syncthreads();
    scan_experts(total, base, a.experts, blockIdx.x == 0 ? a.offsets : nullptr, scratch);
    __syncthreads();
    place(a, s, counts, base, warps);
}

struct Split {
    int64_t per;
    int blocks;
};
Split split_of(int64_t tokens) {
    if (tokens <= ONE) return {tokens, 1};
    int64_t per = (tokens + BLOCKS - 1) / BLOCKS;
    if (per < 32) per = 32;
    if (per > MAX_PER) per = MAX_PER;
    return {per, (int)((tokens + per - 1) / per)};
}

template <typename T, int PER>
cudaError_t launch(const RouteArgs &a, cudaStream_t s) {
    const Split p = split_of(a.tokens);
    int64_t warps = COUNTS / (a.experts | 1), most = PER > 8 ? 16 : 32;
    if (warps > most) warps = most;
    if (warps > p.per) warps = p.per;
    // the scan takes an expert to a thread, so a CTA is not less than four warps
    const int threads = 32 * (int)(warps < 4 ? 4 : warps);
    const cudaError_t e = launch_pdl(route_pick_kernel<T, PER>, dim3((unsigned)p.blocks), threads, 0, s, a, p.per, (int)warps);
    if (e != cudaSuccess || p.blocks == 1) return e;
    return launch_pdl(route_place_kernel<PER>, dim3((unsigned)p.blocks), threads, 0, s, a, p.per, (int)warps);
}

template <typename T>
cudaError_t launch_t(const RouteArgs &a, cudaStream_t s) {
    if (a.experts <= 32) return launch<T, 1>(a, s);
    if (a.experts <= 64) return launch<T, 2>(a, s);
    if (a.experts <= 128) return launch<T, 4>(a, s);
    if (a.experts <= 256) return launch<T, 8>(a, s);
    return launch<T, 32>(a, s);
}

}  // namespace

int64_t experts_route_workspace(int64_t tokens, int experts) {
    const Split p = split_of(tokens);
    return p.blocks == 1 ? 0 : (int64_t)p.blocks * experts * (int64_t)sizeof(int32_t);
}

cudaError_t launch_experts_route(const RouteArgs &a, cudaStream_t s) {
    if (a.dtype == 0) return launch_t<__half>(a, s);
    if (a.dtype == 1) return launch_t<__nv_bfloat16>(a, s);
    return launch_t<float>(a, s);
}

}  // namespace mm
