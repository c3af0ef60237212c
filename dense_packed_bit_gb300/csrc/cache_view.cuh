// cache_view.cuh -- the paged cache of keys and values as the kernels see it.
//
// Token t of sequence s: page table[s][t >> page_shift], row t & (page_size - 1).  Everything
// read from device memory that becomes an address (page numbers, lengths, row ranges) is
// checked before its use: what is out of range is treated as absent and recorded in the
// translation unit's device error word (kDevErrRange).
#pragma once

#include "mm_common.cuh"
#include "mm_internal.h"
#include "smem_limit.h"

namespace mm {

constexpr unsigned int kDevErrRange = kCacheErrRange;

__device__ __forceinline__ int page_of(const CacheView &c, int seq, int64_t slot) {
    if (slot < 0 || slot >= c.max_pages) return -1;
    const int p = __ldg(c.table + (int64_t)seq * c.max_pages + slot);
    return p >= 0 && p < c.pages ? p : -1;
}

// tokens sequence `seq` can hold in its table row
__device__ __forceinline__ int64_t row_capacity(const CacheView &c) { return c.max_pages << c.page_shift; }

// [first, first + count) of sequence seq's rows of Q; out of range: no rows, and not ok
struct RowRange {
    int first, count;
    bool ok;
};
__device__ __forceinline__ RowRange rows_of(const int32_t *q_start, int seq, int64_t tokens, int64_t max_q,
                                            unsigned int *err) {
    const int64_t a = __ldg(q_start + seq), b = __ldg(q_start + seq + 1);
    if (a < 0 || b < a || b > tokens || b - a > max_q) {
        *err = kDevErrRange;
        return {0, 0, false};
    }
    return {(int)a, (int)(b - a), true};
}

// Launches a kernel whose first step is pdl_wait(): it may become resident while the kernel before it in
// the stream ends (that one's results are visible after the wait), which hides the launch itself.  The kernel calls
// pdl_launch_dependents() behind its wait, so that one that starts without a wait of its own has only this one beside it.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kern, args...);
}

}  // namespace mm
