// cache_attention_rows.cu -- attention of few new tokens over a paged cache: up to 16 rows (new
// tokens x query heads of one kv head) per sequence, the form of a decode step and of small trees.
//
// Mathematics.  Online softmax: per row the running reference m (in base-2 units, scale log2(e)
// folded into one multiply), l = sum 2^(s - m) and O = sum 2^(s - m) v.  O and l are only rescaled
// when a row's maximum passes its reference by more than 8 (probabilities stay below 2^8, far inside
// fp16), so most blocks cost no rescaling; the final O / l does not depend on the reference.
//
// Bound: reading K and V once (4 D bytes a key and kv head; 16 rows x 4 D operations for them are a
// twentieth of what the tensor cores could do meanwhile).  So the layout is made for loads in flight:
// a CTA of four warps owns a range of one kv head's keys; every warp streams its own 16-key blocks
// (whole rows, 16-byte cp.async) through a ring of three stages of its own, with no barrier between
// warps until the end; two CTAs are resident per SM, 128 KB in flight.  The 16 x D rows of Q stay in
// registers as the A operand of mma.sync.m16n8k16 (K rows read by ldmatrix are B as they lie, V rows by
// ldmatrix.trans); the probabilities go from accumulator registers to A registers without shared
// memory.  A block lies in one page (pages hold a multiple of 16 tokens).
//
// The keys of a unit (sequence, kv head) are split over CTAs when there are few units; the last CTA
// of a unit to finish adds the partial O in the order of the splits (a ticket per unit, reset by the
// last), so the result does not depend on which one is last.
//
// What a row does not see: its score is replaced, not added to.  Keys no row sees are not read (zero
// filled).  Where a block is cut differently for different rows, infinities and NaN in V are taken
// out of the product (0 x NaN) and added to the rows that do see them.
#include "cache_attention.cuh"

namespace mm {

namespace {

__device__ unsigned int g_rows_err;

constexpr int WARPS = 4, NT = WARPS * 32, B = 16, STAGES = 3;
constexpr int MIN_BLOCKS = 8;  // blocks of a split, at least

struct RowsArgs {
    CacheAttnArgs a;
    int splits;
    int32_t *tickets;  // [seqs][kv_heads]
    float2 *ml;        // [seqs][kv_heads][splits][16]
    float *part;       // [seqs][kv_heads][splits][16][head_dim]
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// KS: 16-element steps of the head dimension held (head_dim <= 16 KS, the rest zero)
template <typename T, int KS>
__global__ void __launch_bounds__(NT, 2) rows_kernel(const RowsArgs p) {
    constexpr int ROW = KS * 32;              // bytes of a key's row in shared memory
    constexpr int TILE = B * ROW;             // K or V of one block
    constexpr int RING = STAGES * 2 * TILE;   // one warp's
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float2 sm_ml[WARPS][16];
    __shared__ int sm_last;
    const CacheAttnArgs &a = p.a;
    const CacheView &c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
    const int seq = unit / c.kv_heads, head = unit - seq * c.kv_heads;
    const SeqView sv = seq_view(a, seq, &g_rows_err);
    const int rows = sv.count * a.group;
    if (rows == 0 || rows > 16) return;  // rows > 16: max_q said otherwise, recorded by seq_view

    // this thread's rows: lane / 4 and 8 later
    RowView rv[2];
    uint32_t tree[2];
    int64_t low = 0;
    const int64_t end = sv.len + sv.count;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = (lane >> 2) + 8 * h;
        rv[h] = row_view(a, sv.len, sv.first, sv.count, min(r, rows - 1) / a.group);
        tree[h] = rv[h].bits ? __ldg(rv[h].bits) & (sv.count < 32 ? (1u << sv.count) - 1u : ~0u) : 0u;
    }
    // the lowest window start of all rows, and the highest: keys from there on are cut by no window
    low = min(rv[0].low, rv[1].low);
    int64_t high = max(rv[0].low, rv[1].low);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
        high = max(high, __shfl_xor_sync(0xffffffffu, high, o));
    }
    if (a.mask) low = min(low, sv.len);  // the window does not cut drafted tokens
    const KeyBlocks kb = key_blocks<B>(low, a.sinks, end);
    int64_t per = (kb.count + p.splits - 1) / p.splits;
    if (per < MIN_BLOCKS) per = MIN_BLOCKS;
    const int used = (int)((kb.count + per - 1) / per);  // splits of this unit, >= 1
    if (split >= used) return;
    const int64_t b0 = split * per, b1 = min(kb.count, b0 + per);

    const int64_t whole = a.mask ? sv.len : sv.len + 1;  // keys before it are cut by no row's end
    const float scale2 = a.scale * kLog2e;
    uint32_t q[KS][4];
    {
        const char *Q = static_cast<const char *>(a.Q);
        const uint32_t *src[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min((lane >> 2) + 8 * h, rows - 1), i = r / a.group;
            src[h] = reinterpret_cast<const uint32_t *>(
                Q + ((int64_t)(sv.first + i) * a.q_stride + (int64_t)(head * a.group + r - i * a.group) * c.head_dim) * 2);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int d = k * 16 + (x >> 1) * 8 + 2 * (lane & 3);
                q[k][x] = d < c.head_dim ? __ldg(src[x & 1] + d / 2) : 0u;
            }
    }

    uint8_t *ring = sm + warp * RING;
    const uint32_t ring_s = smem_u32(ring);
    const int vecs = c.head_dim / 8;
    if (vecs < 2 * KS)  // columns past head_dim stay zero
        for (int e = lane; e < RING / 16; e += 32) *reinterpret_cast<uint4 *>(ring + e * 16) = make_uint4(0, 0, 0, 0);
    __syncwarp();

    const char *kbase = c.k + head * c.head_stride * 2, *vbase = c.v + head * c.head_stride * 2;
    // block i of this warp: b0 + warp + i WARPS
    const auto page_at = [&](int64_t b) {
        if (b >= b1) return -1;
        return page_of(c, seq, (kb.block(b) * B) >> c.page_shift);
    };
    const auto load = [&](int64_t b, int page, int stage) {
        if (b < b1) {
            const int64_t key0 = kb.block(b) * B;
            const uint32_t dst = ring_s + stage * 2 * TILE;
            const int64_t base = page < 0 ? 0 : (page * c.page_stride + (key0 & (c.page_size - 1)) * c.token_stride) * 2;
            if (page < 0) g_rows_err = kDevErrRange;
#pragma unroll
            for (int i = 0; i < B * 2 * KS / 32; ++i) {
                const int e = i * 32 + lane, r = e / (2 * KS), x = e % (2 * KS);
                const int64_t j = key0 + r;
                const bool read = page >= 0 && j < end && (j >= low || j < a.sinks);
                if (x < vecs) {
                    const int64_t off = read ? base + (r * c.token_stride + x * 8) * 2 : 0;
                    const uint32_t at = dst + r * ROW + ((x ^ (r & 7)) << 4);
                    cp16(at, kbase + off, read);
                    cp16(at + TILE, vbase + off, read);
                }
            }
        }
        cp_commit();
    };

    float o[2 * KS][4];
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int64_t b = b0 + warp;
    int page = page_at(b);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        const int next = page_at(b + (s + 1) * WARPS);
        load(b + s * WARPS, page, s);
        page = next;
    }
    int stage = 0;
    for (; b < b1; b += WARPS) {
        const int next = page_at(b + STAGES * WARPS);
        {
            const int to = stage + STAGES - 1;
            load(b + (STAGES - 1) * WARPS, page, to >= STAGES ? to - STAGES : to);
        }
        page = next;
        cp_wait<STAGES - 1>();
        __syncwarp();
        const uint32_t kt = ring_s + stage * 2 * TILE, vt = kt + TILE;
        const int64_t key0 = kb.block(b) * B;

        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            const int r = (lane & 7) + ((lane >> 4) << 3), x = 2 * k + ((lane >> 3) & 1);
            ldsm4(f, kt + r * ROW + ((x ^ (r & 7)) << 4));
            mma16<T>(s[0], q[k], f[0], f[1]);
            mma16<T>(s[1], q[k], f[2], f[3]);
        }
        // whether some row does not see some key of this block
        const bool cut = key0 + B > whole || (key0 < high && key0 + B > a.sinks);
        bool seen[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                seen[n][x] = true;
                if (cut) {
                    const int64_t j = key0 + n * 8 + 2 * (lane & 3) + (x & 1);
                    const RowView &r = rv[x >> 1];
                    if (j < r.end) {
                        seen[n][x] = j >= r.low || j < a.sinks;
                    } else {
                        const int64_t t = j - sv.len;
                        seen[n][x] = t < 32 && (tree[x >> 1] >> t & 1u);
                    }
                }
                s[n][x] = seen[n][x] ? s[n][x] * scale2 : -INFINITY;
            }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float now = fmaxf(m[h], mx[h]);
                const float f = now == -INFINITY ? 1.f : ex2(m[h] - now);
                m[h] = now;
                l[h] *= f;
#pragma unroll
                for (int n = 0; n < 2 * KS; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[n][x] = seen[n][x] ? ex2(s[n][x] - m[x >> 1]) : 0.f;
                l[x >> 1] += s[n][x];
            }
        uint32_t pr[4];
        pr[0] = Pair<T>::pack(s[0][0], s[0][1]);
        pr[1] = Pair<T>::pack(s[0][2], s[0][3]);
        pr[2] = Pair<T>::pack(s[1][0], s[1][1]);
        pr[3] = Pair<T>::pack(s[1][2], s[1][3]);
        bool special = false;
#pragma unroll
        for (int n = 0; n < KS; ++n) {
            uint32_t f[4];
            const int r = (lane & 7) + (((lane >> 3) & 1) << 3), x = 2 * n + (lane >> 4);
            ldsm4t(f, vt + r * ROW + ((x ^ (r & 7)) << 4));
            if (cut) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    special |= any_special<T>(f[i]);
                    f[i] = without_special<T>(f[i]);
                }
            }
            mma16<T>(o[2 * n], pr, f[0], f[1]);
            mma16<T>(o[2 * n + 1], pr, f[2], f[3]);
        }
        if (cut && __any_sync(0xffffffffu, special)) {  // rare: added where they are seen, key by key
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int64_t j = key0 + i;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = j < rv[h].end ? j >= rv[h].low || j < a.sinks
                                                  : j - sv.len < 32 && (tree[h] >> (j - sv.len) & 1u);
                    // the probability of key i lies with the lane of its column
                    const int owner = (lane & ~3) | ((i & 7) >> 1);
                    const float pv = __shfl_sync(0xffffffffu, s[i >> 3][2 * h + (i & 1)], owner);
                    if (!in) continue;
#pragma unroll
                    for (int n = 0; n < 2 * KS; ++n) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(
                            ring + stage * 2 * TILE + TILE + i * ROW + ((n ^ (i & 7)) << 4) + 4 * (lane & 3));
                        if (any_special<T>(w)) {
                            const uint16_t lo = (uint16_t)w, hi = (uint16_t)(w >> 16);
                            if ((lo & Pair<T>::kExp) == Pair<T>::kExp) o[n][2 * h] += pv * Pair<T>::one(lo);
                            if ((hi & Pair<T>::kExp) == Pair<T>::kExp) o[n][2 * h + 1] += pv * Pair<T>::one(hi);
                        }
                    }
                }
            }
        }
        __syncwarp();  // this stage is free
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if ((lane & 3) == 0) sm_ml[warp][(lane >> 2) + 8 * h] = make_float2(m[h], l[h]);
    }
    // the warps' O side by side in shared memory, fp32, rows padded by 4 words
    constexpr int OS = KS * 16 + 4;
    float *so = reinterpret_cast<float *>(sm);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2 *>(so + (warp * 16 + (lane >> 2) + 8 * h) * OS + n * 8 + 2 * (lane & 3)) =
                make_float2(o[n][2 * h], o[n][2 * h + 1]);
    __syncthreads();

    const int D = c.head_dim, pairs = D / 2;
    const int64_t slot = ((int64_t)unit * p.splits + split) * 16;
    const auto out_at = [&](int r, int d) {
        const int i = r / a.group;
        return reinterpret_cast<uint32_t *>(
            static_cast<char *>(a.O) +
            ((int64_t)(sv.first + i) * a.o_stride + (int64_t)(head * a.group + r - i * a.group) * D + d) * 2);
    };
    for (int e = threadIdx.x; e < rows * pairs; e += NT) {
        const int r = e / pairs, d = 2 * (e - r * pairs);
        float mt = -INFINITY, lt = 0.f;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mt = fmaxf(mt, sm_ml[w][r].x);
        if (mt > -INFINITY) {
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = sm_ml[w][r];
                if (ml.x == -INFINITY) continue;
                const float f = ex2(ml.x - mt);
                const float2 x = *reinterpret_cast<const float2 *>(so + (w * 16 + r) * OS + d);
                lt += f * ml.y;
                v.x += f * x.x, v.y += f * x.y;
            }
        }
        if (used == 1) {
            const float inv = mt > -INFINITY ? 1.f / lt : 0.f;
            *out_at(r, d) = Pair<T>::pack(v.x * inv, v.y * inv);
        } else {
            *reinterpret_cast<float2 *>(p.part + (slot + r) * D + d) = v;
            if (d == 0) p.ml[slot + r] = make_float2(mt, lt);
        }
    }
    if (used == 1) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int t = atomicAdd(p.tickets + unit, 1);
        sm_last = t == used - 1;
        if (sm_last) p.tickets[unit] = 0;  // ready for the next call
    }
    __syncthreads();
    if (!sm_last) return;
    __threadfence();
    const int64_t slot0 = (int64_t)unit * p.splits * 16;
    for (int e = threadIdx.x; e < rows * pairs; e += NT) {
        const int r = e / pairs, d = 2 * (e - r * pairs);
        float mt = -INFINITY, lt = 0.f;
        float2 v = make_float2(0.f, 0.f);
        for (int s = 0; s < used; ++s) mt = fmaxf(mt, __ldcg(&p.ml[slot0 + s * 16 + r]).x);
        if (mt > -INFINITY) {
#pragma unroll 4
            for (int s = 0; s < used; ++s) {
                const float2 ml = __ldcg(&p.ml[slot0 + s * 16 + r]);
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(p.part + (slot0 + s * 16 + r) * D + d));
                const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt);
                lt += f * ml.y;
                v.x += f * x.x, v.y += f * x.y;
            }
        }
        const float inv = mt > -INFINITY ? 1.f / lt : 0.f;
        *out_at(r, d) = Pair<T>::pack(v.x * inv, v.y * inv);
    }
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

template <typename T, int KS>
cudaError_t launch(const RowsArgs &p, cudaStream_t s) {
    constexpr int SMEM = WARPS * STAGES * 2 * B * KS * 32;
    static_assert(SMEM >= WARPS * 16 * (KS * 16 + 4) * 4, "the warps' O fit in the rings");
    static const cudaError_t once =
        cudaFuncSetAttribute(rows_kernel<T, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (once != cudaSuccess) return once;
    rows_kernel<T, KS><<<(unsigned)((int64_t)p.splits * p.a.c.seqs * p.a.c.kv_heads), NT, SMEM, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RowsArgs &p, cudaStream_t s) {
    return p.a.c.head_dim <= 64 ? launch<T, 4>(p, s) : launch<T, 8>(p, s);
}

}  // namespace

int cache_attention_rows_splits(const CacheView &c, int sms) {
    const int64_t units = (int64_t)c.seqs * c.kv_heads, blocks = (c.max_pages << c.page_shift) / B;
    // four CTAs for each resident one, so that ragged lengths even out, but no less than MIN_BLOCKS each
    int64_t s = (8 * (int64_t)sms + units - 1) / units;
    const int64_t most = (blocks + MIN_BLOCKS - 1) / MIN_BLOCKS;
    if (s > most) s = most;
    if (s > 64) s = 64;
    return (int)(s < 1 ? 1 : s);
}

int64_t cache_attention_rows_workspace(const CacheView &c, int splits) {
    if (splits <= 1) return 0;
    const int64_t units = (int64_t)c.seqs * c.kv_heads;
    return round256(units * 4) + round256(units * splits * 16 * 8) + units * splits * 16 * c.head_dim * 4;
}

cudaError_t launch_cache_attention_rows(const CacheAttnArgs &a, int splits, cudaStream_t s) {
    RowsArgs p{a, splits, nullptr, nullptr, nullptr};
    if (splits > 1) {
        const int64_t units = (int64_t)a.c.seqs * a.c.kv_heads;
        char *w = static_cast<char *>(a.ws);
        p.tickets = reinterpret_cast<int32_t *>(w);
        w += round256(units * 4);
        p.ml = reinterpret_cast<float2 *>(w);
        w += round256(units * splits * 16 * 8);
        p.part = reinterpret_cast<float *>(w);
    }
    return a.c.dtype == 0 ? launch_t<__half>(p, s) : launch_t<__nv_bfloat16>(p, s);
}

unsigned int cache_attention_rows_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_rows_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_rows_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
