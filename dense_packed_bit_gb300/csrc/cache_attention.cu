// cache_attention.cu -- attention over a paged cache: which kernel a call runs, and its workspace.
#include "cache_attention.cuh"

namespace mm {

namespace {

__device__ unsigned int g_attn_err;

template <typename T>
__global__ void __launch_bounds__(128) plain_kernel(const CacheAttnArgs a) {
    const int seq = blockIdx.y;
    const SeqView sv = seq_view(a, seq, &g_attn_err);
    const int64_t all = (int64_t)sv.count * a.heads;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); w < all; w += (int64_t)gridDim.x * 4)
        attend_row<T>(a, seq, sv, (int)(w / a.heads), (int)(w % a.heads), &g_attn_err);
}

bool few_rows(const CacheAttnArgs &a) { return a.max_q * a.group <= kRowsMax; }

}  // namespace

int64_t cache_attention_workspace(const CacheView &c, int heads, int64_t tokens, int64_t max_q, int sms) {
    (void)tokens;
    if (max_q * (heads / c.kv_heads) <= kRowsMax)
        return cache_attention_rows_workspace(c, cache_attention_rows_splits(c, sms));
    return 0;
}

cudaError_t launch_cache_attention(const CacheAttnArgs &a, int sms, cudaStream_t s) {
    if (few_rows(a)) return launch_cache_attention_rows(a, cache_attention_rows_splits(a.c, sms), s);
    const int64_t warps = a.max_q * a.heads;
    const dim3 grid((unsigned)((warps + 3) / 4 < 65535 ? (warps + 3) / 4 : 65535), (unsigned)a.c.seqs);
    if (a.c.dtype == 0)
        plain_kernel<__half><<<grid, 128, 0, s>>>(a);
    else
        plain_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

unsigned int cache_attention_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_attn_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_attn_err, &zero, sizeof(zero));
    }
    if (*err == cudaSuccess && v == 0) v = cache_attention_rows_take_device_error(err);
    return v;
}

}  // namespace mm
