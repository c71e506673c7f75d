// The 4-bit cache: its handle and the device helpers its kernels share.
#pragma once

#include "tq_f8.cuh"

namespace tq {

__host__ __device__ constexpr int i4_page_bytes(int d) { return 18 * d + 32; }
// places in a page: scales (keys' rows, then values'), then exponent bytes
__host__ __device__ constexpr int i4_scales_at(int d) { return 16 * d; }
__host__ __device__ constexpr int i4_exps_at(int d) { return 18 * d; }

// S(u) of a scale byte
__device__ __forceinline__ float i4_scale(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)(u << 7))); }

// Codes i and i + 4 (i = 0 .. 3) of the eight in w, as fp16 pair of code - 8.  A
// code under the fp16 exponent of 1024 is 1024 + code: exact, and so is the difference.
__device__ __forceinline__ __half2 i4_pair(uint32_t w, int i) {
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    return __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1032.f));
}

}  // namespace tq

struct tq_i4_cache {
    tq_i4_config cfg;
    tq::PagedGeom geom;
    uint32_t* err;
    uint32_t *cnt, *gcnt;
    float4 *part, *meta;
};
