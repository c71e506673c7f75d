// The 8-bit cache: its handle and the device helpers its kernels share.
#pragma once

#include "tq_paged.cuh"

namespace tq {

// Element conversions of the calls' dtypes.
struct F8Elem {
    static __device__ __forceinline__ float2 from_bf16x2(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float2 from_f16x2(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
};

__device__ __forceinline__ uint32_t f8_pack16(float x, float y, int dtype) {
    if (dtype == TQ_DTYPE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// two consecutive elements to row + i (i even)
__device__ __forceinline__ void f8_store2(void* row, int64_t i, float x, float y, int dtype) {
    if (dtype == TQ_DTYPE_F32)
        *reinterpret_cast<float2*>(static_cast<float*>(row) + i) = make_float2(x, y);
    else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(row) + i) = f8_pack16(x, y, dtype);
}

// 16 consecutive elements to row + i (16-byte aligned)
__device__ __forceinline__ void f8_store16(void* row, int64_t i, const float (&v)[16], int dtype) {
    if (dtype == TQ_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    } else {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + i);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            p[k] = make_uint4(f8_pack16(v[8 * k], v[8 * k + 1], dtype), f8_pack16(v[8 * k + 2], v[8 * k + 3], dtype),
                              f8_pack16(v[8 * k + 4], v[8 * k + 5], dtype), f8_pack16(v[8 * k + 6], v[8 * k + 7], dtype));
    }
}

// the power of two an exponent byte stands for (0: 2^-127, a subnormal; 255: NaN)
__device__ __forceinline__ float f8_scale(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FC00000u : e == 0u ? 0x00400000u : e << 23);
}

// two e4m3 codes (low, high byte) as fp16: exact
__device__ __forceinline__ uint32_t f8_to_f16x2(uint32_t two_codes) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(two_codes));
    return r;
}
__device__ __forceinline__ uint32_t f8_to_f16x2_hi(uint32_t four_codes) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(r) : "r"(four_codes));
    return r;
}

__host__ __device__ constexpr int f8_page_bytes(int d) { return 32 * d + 32; }

}  // namespace tq

struct tq_f8_cache {
    tq_f8_config cfg;
    tq::PagedGeom geom;
    uint32_t* err;
    uint32_t *cnt, *gcnt;
    float4 *part, *meta;
};
