// gemm_packed4_rows.cu -- Y = X W^T for 4-bit W with group scales and few rows of X per matrix:
//
//     Y[m][r] = sum_g scale[r][g] * sum_{k in g} (code[r][k] - zero[r][g]) * X[m][k]
//
// "Kernel 0112", section "What the kernel costs in a whole token": the products of a token are bound by reading
// 4-bit weights.  What a call cannot do without is the codes, half a byte each, and 2 or 3 bytes a group.
//
// A warp takes 16 rows of W and a part of K and streams it from memory into registers, 128 columns at a time: lane
// (g, q) = (lane / 4, lane % 4) loads 16 bytes (32 codes) of row g and of row g + 8, eight such loads ahead of their
// use.  The codes become exact 16-bit whole numbers in registers and are the A operand of mma.sync m16n8k16, whose
// k slots are dealt so that no data moves: a word of 8 codes holds in one masked step the codes 0 and 4, in the next 1
// and 5, and X is paired the same way.  The tensor cores add the products of one group in fp32; the group's scale is
// applied to that sum in fp32, so neither scaled weights nor partial sums are ever rounded to 16 bits.  Groups below
// 128 need the lanes of a row on the same group: they exchange words among the four lanes of a row first.
//
// K is cut over the warps of a CTA, and over a cluster of CTAs where the rows alone would leave SMs idle; the parts
// are added in a fixed order through shared memory, so results repeat bit for bit.  8 or 16 rows of X at a time (the
// MMA's n, once or twice); more of them go around again with the codes read from L2.
#include "packed4.cuh"
#include "smem_limit.h"

namespace mm {

__device__ unsigned int g_packed4_rows_err;

namespace {

constexpr int TILE = 16;      // rows of W per warp
constexpr int KBLOCK = 128;   // columns per step
constexpr int DEEP = 4;       // steps loaded ahead
constexpr int STRIDE = 20;    // floats between tokens of a staged partial tile: lanes' stores meet no bank twice
constexpr int MAX_WARPS = 8, MAX_CLUSTER = 8, MAX_EXPERTS = 1024;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a lane waits for of one step: its codes come to shared memory (its own 2 x 16 bytes of the warp's 1 KB), these to
// registers: the scale (low half) and zero (high half) of rows g and g + 8.
struct Scales {
    uint32_t g, h;
};

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// This lane's part of 16 rows of W.
struct Source {
    const uint8_t *g, *h;  // codes of rows g and g + 8, at this lane's 16 bytes of the first step
    const uint16_t *sg, *sh;
    const uint8_t *zg, *zh;

    __device__ __forceinline__ void point(const Packed4MmArgs &a, int e, int r0, int lane) {
        // rows past the last one read the last one and are not stored
        const int rg = min(r0 + (lane >> 2), a.rows - 1), rh = min(r0 + (lane >> 2) + 8, a.rows - 1);
        const uint8_t *c = a.codes + e * a.codes_expert + (lane & 3) * 16;
        g = c + rg * a.codes_row, h = c + rh * a.codes_row;
        const uint16_t *s = static_cast<const uint16_t *>(a.scales) + e * a.scales_expert;
        sg = s + rg * a.scales_row, sh = s + rh * a.scales_row;
        const uint8_t *z = a.zeros ? a.zeros + e * a.scales_expert : nullptr;
        zg = z ? z + rg * a.scales_row : nullptr, zh = z ? z + rh * a.scales_row : nullptr;
    }

    template <int G>
    __device__ __forceinline__ void load(int b, int cols, int q, uint4 *dst, Scales &s) const {
        const int col = b * KBLOCK + q * 32;
        if (col < cols) {
            copy16(dst, g + (int64_t)b * (KBLOCK / 2));
            copy16(dst + 32, h + (int64_t)b * (KBLOCK / 2));
        } else {
            dst[0] = dst[32] = make_uint4(0, 0, 0, 0);
        }
        if (G == KBLOCK || col < cols) {  // of a group of 128 every lane applies the scale, whether it has codes or not
            const int j = G == KBLOCK ? b : col / G;
            s.g = __ldg(sg + j) | (zg ? (uint32_t)(__ldg(zg + j) & 15) : 8u) << 16;
            s.h = __ldg(sh + j) | (zh ? (uint32_t)(__ldg(zh + j) & 15) : 8u) << 16;
        } else {
            s.g = s.h = 8u << 16;
        }
    }
};

// The words of a row's 128 codes (four to a lane, lane q those of columns 32 q on) redistributed so that word i of every
// lane lies in group i / (4 G / 128); chunk_of tells which 8 columns the word then holds.
template <int G>
__device__ __forceinline__ void exchange(uint4 &w, int q) {
    if constexpr (G == 64) {
        const bool low = q < 2;
        const uint32_t r0 = __shfl_xor_sync(~0u, low ? w.z : w.x, 2), r1 = __shfl_xor_sync(~0u, low ? w.w : w.y, 2);
        if (low) w.z = r0, w.w = r1;
        else w.x = r0, w.y = r1;
    } else if constexpr (G == 32) {
        const bool even = (q & 1) == 0, low = q < 2;
        uint32_t r0 = __shfl_xor_sync(~0u, even ? w.y : w.x, 1), r1 = __shfl_xor_sync(~0u, even ? w.w : w.z, 1);
        if (even) w.y = r0, w.w = r1;
        else w.x = r0, w.z = r1;
        r0 = __shfl_xor_sync(~0u, low ? w.z : w.x, 2), r1 = __shfl_xor_sync(~0u, low ? w.w : w.y, 2);
        if (low) w.z = r0, w.w = r1;
        else w.x = r0, w.y = r1;
    }
}
// 64: a lane below 2 keeps its words 0, 1 and gets those of lane q + 2; the others keep 2, 3 and get those of q - 2.
template <int G>
__device__ __forceinline__ int chunk_of(int i, int q) {
    if constexpr (G == 128) return q * 4 + i;
    if constexpr (G == 64) return (i >> 1) * 8 + (q & 1) * 4 + (q >> 1) * 2 + (i & 1);
    return i * 4 + q;
}

// The 8 codes of w less z as pairs (0, 4), (1, 5), (2, 6), (3, 7); zero: Zero4<T>::of(z).  In fp16 the second field of a
// byte is used where it is: 1024 + 16 c, a sixteenth of which, less 64 + z, is one exact FMA, so a word takes one shift.
template <typename T>
struct Zero4;
template <>
struct Zero4<__nv_bfloat16> {
    uint32_t z;
    static __device__ __forceinline__ Zero4 of(uint32_t z) { return {Code4<__nv_bfloat16>::zero(z)}; }
    __device__ __forceinline__ void decode(uint32_t w, uint32_t (&p)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = Code4<__nv_bfloat16>::sub(and_or(w >> (4 * i), 0x000F000Fu, Code4<__nv_bfloat16>::kBase), z);
    }
};
template <>
struct Zero4<__half> {
    uint32_t z, z16;  // 1024 + z; -(64 + z)
    static __device__ __forceinline__ Zero4 of(uint32_t z) { return {Code4<__half>::zero(z), 0xD400D400u + z * 0x00100010u}; }
    __device__ __forceinline__ void decode(uint32_t w, uint32_t (&p)[4]) const {
        const uint32_t v = w >> 8, sixteenth = 0x2C002C00u;
        const auto high = [&](uint32_t x) {
            const uint32_t f = and_or(x, 0x00F000F0u, Code4<__half>::kBase);
            const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&f), *reinterpret_cast<const __half2 *>(&sixteenth),
                                      *reinterpret_cast<const __half2 *>(&z16));
            return *reinterpret_cast<const uint32_t *>(&r);
        };
        p[0] = Code4<__half>::sub(and_or(w, 0x000F000Fu, Code4<__half>::kBase), z);
        p[1] = high(w);
        p[2] = Code4<__half>::sub(and_or(v, 0x000F000Fu, Code4<__half>::kBase), z);
        p[3] = high(v);
    }
};

// 8 columns from `col` of a row of X as the same pairs; columns at or past cols are 0
__device__ __forceinline__ void load_x(const uint16_t *x, int col, int cols, uint32_t (&p)[4]) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (x && col + 8 <= cols) {
        v = __ldg(reinterpret_cast<const uint4 *>(x + col));
    } else if (x && col < cols) {
        uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < cols) t[i >> 1] |= (uint32_t)__ldg(x + col + i) << (16 * (i & 1));
        v = make_uint4(t[0], t[1], t[2], t[3]);
    }
    p[0] = prmt(v.x, v.z, 0x5410), p[1] = prmt(v.x, v.z, 0x7632);
    p[2] = prmt(v.y, v.w, 0x5410), p[3] = prmt(v.y, v.w, 0x7632);
}

template <typename T, int NT, int G>
__device__ __forceinline__ void step(uint4 vg, uint4 vh, const Scales &in, int b, int cols, const uint16_t *const (&x)[NT], int lane,
                                     float (&acc)[NT][4]) {
    constexpr int GROUPS = KBLOCK / G, WORDS = 4 / GROUPS;
    const int q = lane & 3;
    exchange<G>(vg, q);
    exchange<G>(vh, q);
    const uint32_t wg[4] = {vg.x, vg.y, vg.z, vg.w}, wh[4] = {vh.x, vh.y, vh.z, vh.w};
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        uint32_t sg = in.g, sh = in.h;
        if constexpr (GROUPS > 1) {
            const int from = (lane & ~3) | j * (G / 32);
            sg = __shfl_sync(~0u, sg, from);
            sh = __shfl_sync(~0u, sh, from);
        }
        const Zero4<T> zg = Zero4<T>::of(sg >> 16), zh = Zero4<T>::of(sh >> 16);
        float d[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll
        for (int i = j * WORDS; i < (j + 1) * WORDS; ++i) {
            uint32_t pg[4], ph[4];
            zg.decode(wg[i], pg);
            zh.decode(wh[i], ph);
            const uint32_t a0[4] = {pg[0], ph[0], pg[1], ph[1]}, a1[4] = {pg[2], ph[2], pg[3], ph[3]};
            const int col = b * KBLOCK + chunk_of<G>(i, q) * 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t p[4];
                load_x(x[n], col, cols, p);
                mma<T>(d[n], a0, p[0], p[1]);
                mma<T>(d[n], a1, p[2], p[3]);
            }
        }
        const float fg = Code4<T>::f32((uint16_t)sg), fh = Code4<T>::f32((uint16_t)sh);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(fg, d[n][0], acc[n][0]);
            acc[n][1] = fmaf(fg, d[n][1], acc[n][1]);
            acc[n][2] = fmaf(fh, d[n][2], acc[n][2]);
            acc[n][3] = fmaf(fh, d[n][3], acc[n][3]);
        }
    }
}

// Where a warp is: its part of K of a unit (16 rows of an expert's matrix), for 8 NT of the expert's slots after the other.
struct Cursor {
    int64_t unit;
    int e, r0, first, count;  // the unit's expert, rows and slots
    int t0, b;                // slots already done, step
};

// Grid: clusters that take units in turn; a cluster's CTAs and their warps take consecutive parts of K.  The loads run DEEP
// steps ahead of the products and do not stop at a unit's end.
template <typename T, int NT, int G>
__global__ void __launch_bounds__(32 * MAX_WARPS, NT == 1 ? 3 : 2)
    packed4_rows_kernel(const __grid_constant__ Packed4MmArgs a, const int cluster) {
    extern __shared__ uint4 smem[];  // a ring of DEEP KB to each warp, and twice a partial tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    uint4(*ring)[64] = reinterpret_cast<uint4(*)[64]>(smem) + warp * DEEP;
    float(*red)[8 * NT * STRIDE] = reinterpret_cast<float(*)[8 * NT * STRIDE]>(smem + warps * DEEP * 64);  // [2][warps]
    __shared__ float part[8 * NT * TILE];
    __shared__ int16_t listed[MAX_EXPERTS];  // the experts that have slots
    __shared__ int listed_n;
    const int g = lane >> 2, q = lane & 3;
    const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
    const int64_t cid = blockIdx.x / cluster, clusters = gridDim.x / cluster;
    const int tiles = (a.rows + TILE - 1) / TILE, steps = (a.cols + KBLOCK - 1) / KBLOCK;
    const int parts = warps * cluster, mine = rank * warps + warp;
    const int b0 = (int)((int64_t)steps * mine / parts), b1 = (int)((int64_t)steps * (mine + 1) / parts);
    unsigned int err = 0;
    int64_t units = tiles;

    const auto enter = [&](Cursor &c) {  // c.unit is set
        c.t0 = 0, c.b = b0;
        if (c.unit >= units) return;
        const int at = a.offsets ? (int)(c.unit / tiles) : 0;
        c.e = a.offsets ? listed[at] : 0;
        c.r0 = (int)(c.unit - (int64_t)at * tiles) * TILE;
        const Slots s = slots_of(a, c.e, &err);
        c.first = s.first, c.count = s.count;
    };
    const auto past_chunk = [&](Cursor &c) {  // to the next slots, or the next unit
        c.b = b0, c.t0 += 8 * NT;
        if (c.t0 >= c.count) c.unit += clusters, enter(c);
    };
    Cursor ld;
    Source src;
    Scales sc[DEEP];
    ld.unit = cid;
    const auto load = [&](int u) {
        if (ld.unit < units && b0 < b1) {
            src.load<G>(ld.b, a.cols, q, &ring[u][lane], sc[u]);
            if (++ld.b == b1) {
                const int64_t unit = ld.unit;
                past_chunk(ld);
                if (ld.unit != unit && ld.unit < units) src.point(a, ld.e, ld.r0, lane);
            }
        }
        copies_commit();
    };
    const auto start = [&] {
        enter(ld);
        if (ld.unit < units) src.point(a, ld.e, ld.r0, lane);
#pragma unroll
        for (int u = 0; u < DEEP; ++u) load(u);
    };
    const bool early = a.weights_static && !a.offsets;
    if (early) start();
    pdl_wait();
    pdl_launch_dependents();
    if (a.offsets) {
        if (warp == 0) {
            int n = 0;
            for (int e0 = 0; e0 < a.experts; e0 += 32) {
                const bool some = e0 + lane < a.experts && slots_of(a, e0 + lane, &err).count > 0;
                const uint32_t m = __ballot_sync(~0u, some);
                if (some) listed[n + __popc(m & ((1u << lane) - 1u))] = (int16_t)(e0 + lane);
                n += __popc(m);
            }
            if (lane == 0) listed_n = n;
        }
        __syncthreads();
        units = (int64_t)listed_n * tiles;
    }
    if (!early) start();

    int slot = 0, turn = 0;
    Cursor at;
    at.unit = cid;
    enter(at);
    while (at.unit < units) {
        const uint16_t *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = at.t0 + 8 * n + g;
            const int64_t row = t < at.count ? x_row(a, at.first + t, &err) : -1;
            x[n] = row < 0 ? nullptr : static_cast<const uint16_t *>(a.X) + row * a.x_stride;
        }
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        for (int b = b0; b < b1;) {
#pragma unroll
            for (int u = 0; u < DEEP; ++u) {
                if (u < slot || b >= b1) continue;
                copies_wait<DEEP - 1>();
                const uint4 vg = ring[u][lane], vh = ring[u][lane + 32];
                const Scales now = sc[u];
                load(u);
                step<T, NT, G>(vg, vh, now, b, a.cols, x, lane, acc);
                ++b;
                slot = u + 1;
            }
            if (slot == DEEP) slot = 0;
        }
        float(&mine_red)[8 * NT * STRIDE] = red[turn * warps + warp];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine_red[(8 * n + 2 * q + (i & 1)) * STRIDE + g + 8 * (i >> 1)] = acc[n][i];
        __syncthreads();
        if (cluster > 1) {
            for (int i = threadIdx.x; i < 8 * NT * TILE; i += blockDim.x) {
                float v = 0.f;
                for (int w = 0; w < warps; ++w) v += red[turn * warps + w][(i / TILE) * STRIDE + i % TILE];
                part[i] = v;
            }
            cluster_sync();
        }
        if (rank == 0) {
            for (int i = threadIdx.x; i < 8 * NT * TILE; i += blockDim.x) {
                const int t = at.t0 + i / TILE, r = at.r0 + i % TILE;
                float v = 0.f;
                if (cluster > 1) {
                    const uint32_t from = smem_u32(&part[i]);
                    float p[MAX_CLUSTER];
#pragma unroll
                    for (int c = 0; c < MAX_CLUSTER; ++c)
                        if (c < cluster)
                            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[c]) : "r"(cluster_map(from, c)) : "memory");
#pragma unroll
                    for (int c = 0; c < MAX_CLUSTER; ++c)
                        if (c < cluster) v += p[c];
                } else {
                    for (int w = 0; w < warps; ++w) v += red[turn * warps + w][(i / TILE) * STRIDE + i % TILE];
                }
                // a row's neighbour is the lane beside it, and the loop's length a multiple of 32: whole warps are here
                const float up = __shfl_down_sync(~0u, v, 1);
                if (t < at.count && r < a.rows) {
                    if (!a.swiglu) store_y(a, at.first + t, r, v);
                    else if ((r & 1) == 0) store_y(a, at.first + t, r >> 1, silu(v) * up);
                }
            }
        }
        if (cluster > 1) cluster_sync();  // nobody leaves, or writes part again, before it has been read
        turn ^= 1;  // of two buffers the other is free: the barrier above was behind its last reader
        past_chunk(at);
    }
    copies_wait<0>();
    if (err) atomicExch(&g_packed4_rows_err, err);
}

template <typename T, int NT, int G>
cudaError_t launch(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    // K is cut into as many parts as keep all warps resident at once, but into no less than four (where it has as many
    // steps), so that a tile's parts are a CTA's warps; beyond a CTA's eight warps a cluster's CTAs share it.
    constexpr int RESIDENT = NT == 1 ? 24 : 16;  // warps of an SM: the launch bounds
    constexpr int bytes = DEEP * 1024 + 2 * 8 * NT * STRIDE * 4;  // of shared memory to a warp
    static SmemLimit limit;
    const cudaError_t e = limit.allow((const void *)packed4_rows_kernel<T, NT, G>, MAX_WARPS * bytes);
    if (e != cudaSuccess) return e;
    const int tiles = (a.rows + TILE - 1) / TILE, steps = (a.cols + KBLOCK - 1) / KBLOCK;
    const int64_t units = tiles * (a.offsets ? (a.slots < a.experts ? a.slots : a.experts) : 1);
    int parts = 1;
    while (parts * 2 <= steps && parts < MAX_WARPS * MAX_CLUSTER && (units * parts * 2 <= sms * RESIDENT || parts < 4)) parts *= 2;
    const int warps = parts < MAX_WARPS ? parts : MAX_WARPS, cluster = parts / warps;
    const int64_t fit = (int64_t)sms * (RESIDENT / warps) / cluster, clusters = units < fit ? units : fit;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(clusters * cluster));
    lc.blockDim = dim3(32u * warps);
    lc.dynamicSmemBytes = (size_t)warps * bytes;
    lc.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, packed4_rows_kernel<T, NT, G>, a, cluster);
}

template <typename T, int NT>
cudaError_t launch_g(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    if (a.group == 128) return launch<T, NT, 128>(a, sms, s);
    if (a.group == 64) return launch<T, NT, 64>(a, sms, s);
    return launch<T, NT, 32>(a, sms, s);
}

template <typename T>
cudaError_t launch_t(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    // 16 at a time where a matrix has more than 8 rows of X on average
    return a.slots > (a.offsets ? 8 * (int64_t)a.experts : 8) ? launch_g<T, 2>(a, sms, s) : launch_g<T, 1>(a, sms, s);
}

}  // namespace

cudaError_t launch_packed4_rows(const Packed4MmArgs &a, int sms, cudaStream_t s) {
    return a.dtype == 0 ? launch_t<__half>(a, sms, s) : launch_t<__nv_bfloat16>(a, sms, s);
}

unsigned int packed4_rows_take_device_error(cudaError_t *err) {
    unsigned int v = 0;
    *err = cudaMemcpyFromSymbol(&v, g_packed4_rows_err, sizeof(v));
    if (*err == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        *err = cudaMemcpyToSymbol(g_packed4_rows_err, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mm
