// cache_attention.cu -- attention over a paged cache: which kernel a call runs, and its workspace.
//
// Up to 16 rows (new tokens x query heads of a kv head) of a sequence: the rows kernel, whose one m16 tile they fill.
// More: the tiles kernel, whose 128-row products are mostly zeros below that.  Measured, rows and tiles kernel: 48
// sequences of 100 to 16,000 tokens, 8 kv heads of 128 columns, 1 new token (4 rows) 100 and 131 us, 4 new (16 rows) 106 and 131; 8 x 100 to
// 1,000 tokens, 12 heads of 64, 16 rows 12.1 and 17.7; one sequence of 513, 1 row 7.9 and 13.4.
#include "cache_attention.cuh"

namespace mm {

int64_t cache_attention_workspace(const CacheView &c, int heads, int64_t tokens, int64_t max_q, int sms) {
    (void)tokens;
    const int group = heads / c.kv_heads;
    if (max_q * group <= kRowsMax) return cache_attention_rows_workspace(c, cache_attention_rows_ctas(c, sms));
    return cache_attention_tiles_workspace(c, cache_attention_tiles_ctas(c, group, max_q, sms));
}

cudaError_t launch_cache_attention(const CacheAttnArgs &a, int sms, cudaStream_t s) {
    if (a.max_q * a.group <= kRowsMax) return launch_cache_attention_rows(a, cache_attention_rows_ctas(a.c, sms), s);
    return launch_cache_attention_tiles(a, cache_attention_tiles_ctas(a.c, a.group, a.max_q, sms), s);
}

unsigned int cache_attention_take_device_error(cudaError_t *err) {
    const unsigned int v = cache_attention_rows_take_device_error(err);
    if (*err != cudaSuccess || v != 0) return v;
    return cache_attention_tiles_take_device_error(err);
}

}  // namespace mm
