// experts_combine.cu -- the weighted sum of a token's expert rows, added to the residual stream:
//
//     out[t] = residual[t] + sum_j weights[t][j] * Y[slots[t][j]]
//
// in fp32, j ascending, rounded once.  Bound by memory: a call reads tokens x top_k rows of Y, one of the residual and
// writes one.  A thread takes 16 bytes of Y's columns with up to 8 rows' loads on their way at once: 8191 x 2048 from 8 rows each
// 93.2 us = 6.44 TB/s, 96% of a copy (Y in fp32, out in bf16); from rows of 16 bits to fp32 61 us.
#include "cache_view.cuh"
#include "mm_common.cuh"
#include "mm_internal.h"
#include "packed4.cuh"

namespace mm {

__device__ unsigned int g_combine_err;

namespace {

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements, 16 bytes of them at a time
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
    T v[N];
};

// Rows of Y are read once, and stay as they lie in memory until they are added: elements of bf16 taken apart at the load made the
// eight loads wait for one another (8191 x 2048 from 8 rows each in bf16 to fp32 163 us, as words 61)
template <typename T, int N>
struct Row {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ float at(int) const { return widen<T>(v); }
};
template <typename T>
struct Row<T, 16 / sizeof(T)> {
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = ld_stream_v4(p); }
    __device__ __forceinline__ float at(int i) const {
        const int word = i * (int)sizeof(T) / 4;
        const uint32_t w = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
        if constexpr (sizeof(T) == 4) return __uint_as_float(w);
        else if constexpr (__is_same(T, __half)) return __half2float(__ushort_as_half((unsigned short)(w >> (16 * (i & 1)))));
        else return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

constexpr int THREADS = 256, AHEAD = 8;

// A block per token and THREADS N columns of it (1 where strides or pointers do not allow vectors)
template <typename TY, typename TO, int N>
__global__ void __launch_bounds__(THREADS) combine_kernel(const __grid_constant__ CombineArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    unsigned int err = 0;
    const int64_t t = blockIdx.x;
    for (int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N; c < a.cols; c += (int64_t)gridDim.y * blockDim.x * N) {
        float sum[N];
        if (a.residual) {
            const Pack<TO, N> r = *reinterpret_cast<const Pack<TO, N> *>(static_cast<const TO *>(a.residual) + t * a.r_stride + c);
#pragma unroll
            for (int x = 0; x < N; ++x) sum[x] = widen<TO>(r.v[x]);
        } else {
#pragma unroll
            for (int x = 0; x < N; ++x) sum[x] = 0.f;
        }
        for (int j0 = 0; j0 < a.top_k; j0 += AHEAD) {
            Row<TY, N> y[AHEAD];
            float w[AHEAD];
            bool have[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                have[j] = false;
                if (j0 + j >= a.top_k) continue;
                const int slot = __ldg(a.slots + t * a.top_k + j0 + j);
                if (slot >= a.y_rows || slot < -1) err = kDevErrRange;
                else have[j] = slot >= 0;
                if (!have[j]) continue;
                w[j] = __ldg(a.weights + t * a.top_k + j0 + j);
                y[j].load(static_cast<const TY *>(a.Y) + slot * a.y_stride + c);
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (have[j])
#pragma unroll
                    for (int x = 0; x < N; ++x) sum[x] = fmaf(w[j], y[j].at(x), sum[x]);
        }
        Pack<TO, N> o;
#pragma unroll
        for (int x = 0; x < N; ++x) o.v[x] = narrow<TO>(sum[x]);
        *reinterpret_cast<Pack<TO, N> *>(static_cast<TO *>(a.out) + t * a.out_stride + c) = o;
    }
    if (err) atomicExch(&g_combine_err, err);
}

// Rows of packs of n elements start where a pack may
bool fits(const void *p, int64_t stride, int64_t size, int n) {
    const int64_t bytes = size * n < 16 ? size * n : 16;
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0 && stride * size % bytes == 0;
}

template <typename TY, typename TO>
cudaError_t launch(const CombineArgs &a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(TY);
    const bool vec = a.cols % N == 0 && fits(a.Y, a.y_stride, sizeof(TY), N) && fits(a.out, a.out_stride, sizeof(TO), N) &&
                     (!a.residual || fits(a.residual, a.r_stride, sizeof(TO), N));
    const int64_t vecs = a.cols / (vec ? N : 1), blocks = (vecs + THREADS - 1) / THREADS;
    const int threads = vecs < THREADS ? (int)(vecs + 31) / 32 * 32 : THREADS;
    const dim3 grid((unsigned)a.tokens, (unsigned)(blocks < 65535 ? blocks : 65535));
    if (vec) return launch_pdl(combine_kernel<TY, TO, N>, grid, threads, 0, s, a);
    return launch_pdl(combine_kernel<TY, TO, 1>, grid, threads, 0, s, a);
}

template <typename TY>
cudaError_t launch_o(const CombineArgs &a, cudaStream_t s) {
    if (a.out_dtype == 0) return launch<TY, __half>(a, s);
    if (a.out_dtype == 1) return launch<TY, __nv_bfloat16>(a, s);
    return launch<TY, float>(a, s);
}

}  // namespace

cudaError_t launch_experts_combine(const CombineArgs &a, cudaStream_t s) {
    if (a.y_dtype == 0) return launch_o<__half>(a, s);
    if (a.y_dtype == 1) return launch_o<__nv_bfloat16>(a, s);
    return launch_o<float>(a, s);
}

unsigned int experts_combine_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_combine_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_combine_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
