// packed4.cuh -- 4-bit weights with group scales as the kernels see them: whose rows a unit of work
// multiplies, and codes turned into 16-bit whole numbers.
//
// Everything read from device memory that becomes an address (expert offsets, rows of X) is checked
// before its use: what is out of range is treated as absent and recorded in the translation unit's
// device error word (kDevErrRange).
#pragma once

#include "cache_view.cuh"  // launch_pdl, kDevErrRange
#include "mm_common.cuh"
#include "mm_internal.h"
#include "tmap.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace mm {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// (a & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

// Codes become weights by placing them in the mantissa of a 16-bit number whose last place is 1 (1024 in fp16,
// 128 in bf16) and taking that number and the zero off again: c - z is a whole number of -15 .. 15, exact in
// both types, and the difference of two exact numbers is rounded nowhere.
template <typename T>
struct Code4;
template <>
struct Code4<__half> {
    static constexpr uint32_t kBase = 0x64006400u;  // 1024
    static __device__ __forceinline__ uint32_t zero(uint32_t z) { return 0x64006400u + z * 0x10001u; }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ float f32(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ uint16_t round(float v) { return __half_as_ushort(__float2half_rn(v)); }
};
template <>
struct Code4<__nv_bfloat16> {
    static constexpr uint32_t kBase = 0x43004300u;  // 128
    static __device__ __forceinline__ uint32_t zero(uint32_t z) { return 0x43004300u + z * 0x10001u; }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        const __nv_bfloat162 d =
            __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    static __device__ __forceinline__ float f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t round(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};

// silu(g) u, the same wherever Y lies.  For fp32 an exponential and a quotient of an ulp or two.  For results of 16 bits, of which
// half a step is 2^-11 of the value or more, few instructions: an exponential of 2 + 1.18 |g| ulp (1.3e-5 at a gate of -88)
// and a quotient of 2 ulp, whose divisor has to stay below 2^126: a quarter of 1 + exp(-g) does wherever that is finite.
__device__ __forceinline__ float swiglu(float g, float u, bool wide) {
    if (wide) return g / (1.0f + expf(-g)) * u;
    return __fdividef(0.25f * g, fmaf(0.25f, __expf(-g), 0.25f)) * u;
}

// Slots [first, first + count) of expert e.
struct Slots {
    int first, count;
};
__device__ __forceinline__ Slots slots_of(const Packed4MmArgs &a, int e, unsigned int *err) {
    if (!a.offsets) return {0, (int)a.slots};
    const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
    if (lo < 0 || hi < lo || hi > a.slots) {
        *err = kDevErrRange;
        return {0, 0};
    }
    return {lo, hi - lo};
}

// The row of X that slot i multiplies, -1 where order names none.
__device__ __forceinline__ int64_t x_row(const Packed4MmArgs &a, int64_t i, unsigned int *err) {
    if (!a.order) return i;
    const int pick = __ldg(a.order + i);
    const int row = pick < 0 ? -1 : pick / a.per_row;
    if (row < 0 || row >= a.x_rows) {
        *err = kDevErrRange;
        return -1;
    }
    return row;
}

// Y[slot][col] = v in Y's type (0 f16, 1 bf16, 2 f32)
__device__ __forceinline__ void store_y(const Packed4MmArgs &a, int64_t slot, int col, float v) {
    const int64_t i = slot * a.y_stride + col;
    if (a.y_dtype == 2) static_cast<float *>(a.Y)[i] = v;
    else if (a.y_dtype == 1) static_cast<uint16_t *>(a.Y)[i] = Code4<__nv_bfloat16>::round(v);
    else static_cast<uint16_t *>(a.Y)[i] = Code4<__half>::round(v);
}

// Columns r .. r + 3 of Y (rows of W) for a slot; vec: four of them are 16 (8) aligned bytes
template <typename T>
__device__ __forceinline__ void store4(const Packed4MmArgs &a, int64_t slot, int r, const float4 &v, bool vec) {
    const int64_t row = slot * a.y_stride;
    if (a.swiglu) {
        const bool wide = a.y_dtype == 2;
        const float p = swiglu(v.x, v.y, wide), q = swiglu(v.z, v.w, wide);
        if (vec && r + 3 < a.rows) {
            if (a.y_dtype == 2) *reinterpret_cast<float2 *>(static_cast<float *>(a.Y) + row + (r >> 1)) = make_float2(p, q);
            else *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.Y) + row + (r >> 1)) = Code4<T>::round(p) | (uint32_t)Code4<T>::round(q) << 16;
        } else {
            if (r < a.rows) store_y(a, slot, r >> 1, p);
            if (r + 2 < a.rows) store_y(a, slot, (r >> 1) + 1, q);
        }
    } else if (vec && r + 3 < a.rows) {
        if (a.y_dtype == 2) *reinterpret_cast<float4 *>(static_cast<float *>(a.Y) + row + r) = v;
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.Y) + row + r) =
                make_uint2(Code4<T>::round(v.x) | (uint32_t)Code4<T>::round(v.y) << 16, Code4<T>::round(v.z) | (uint32_t)Code4<T>::round(v.w) << 16);
    } else {
        if (r < a.rows) store_y(a, slot, r, v.x);
        if (r + 1 < a.rows) store_y(a, slot, r + 1, v.y);
        if (r + 2 < a.rows) store_y(a, slot, r + 2, v.z);
        if (r + 3 < a.rows) store_y(a, slot, r + 3, v.w);
    }
}

// True in one thread of the warp.  The compiler knows that of elect.sync, and puts the operands of TMA copies and MMAs behind
// it straight into uniform registers: four MMAs and a commit are issued in 160 clocks, behind a test of the lane in 700; a
// gather of four rows in a third of the 70 clocks that a lane for each takes.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// X in boxes of 64 columns (128 bytes, swizzled) and `rows` rows, W's codes in boxes of `bytes` by `rows`.  A matrix of one row
// may have any stride: the map is given one that holds it.
inline cudaError_t packed4_tmap_x(CUtensorMap *map, const Packed4MmArgs &a, int rows) {
    const uint64_t stride = a.x_rows > 1 ? (uint64_t)a.x_stride * 2 : ((uint64_t)a.cols * 2 + 15) / 16 * 16;
    return make_tmap_2d(map, a.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.X, (uint64_t)a.cols,
                        (uint64_t)a.x_rows, stride, 64, (uint32_t)rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
inline cudaError_t packed4_tmap_w(CUtensorMap *map, const Packed4MmArgs &a, int bytes, int rows, CUtensorMapSwizzle swizzle) {
    const uint64_t held = ((uint64_t)a.cols + 31) / 32 * 16, row = a.rows > 1 ? (uint64_t)a.codes_row : held;
    return make_tmap_3d(CU_TENSOR_MAP_DATA_TYPE_UINT8, map, a.codes, held, (uint64_t)a.rows, (uint64_t)a.experts, row,
                        a.experts > 1 ? (uint64_t)a.codes_expert : row, (uint32_t)bytes, (uint32_t)rows, swizzle);
}

}  // namespace mm
