// cache.cuh -- what the paged 8-bit cache's writer (cache_append.cu) and its
// reader (cache_attn.cu) share: the layout's rules and the e4m3 conversions.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "lidx.h"

namespace lidx {

constexpr int kCacheMaxD = 128;
constexpr int kCacheMinExp = -40;  // smallest scale a page is given: 2^-40

// Shape rules of a cache and its block table (see lidx.h).
inline int check_cache(int64_t B, int64_t S, int Hkv, int D, int page, int64_t max_pages, int64_t num_pages) {
    if (B < 1 || S < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1) return LIDX_ERR_SHAPE;
    if (B > (1 << 20) || S > (1 << 30) || Hkv > (1 << 16)) return LIDX_ERR_SHAPE;
    if (D < 16 || D % 16 || D > kCacheMaxD) return LIDX_ERR_SHAPE;
    if (page != 16 && page != 32 && page != 64 && page != 128) return LIDX_ERR_SHAPE;
    if (max_pages > (1 << 30) / page || num_pages > INT32_MAX / page / Hkv) return LIDX_ERR_SHAPE;
    return LIDX_OK;
}

// Two e4m3 codes (low byte first) <-> two floats; rounds to nearest even, saturates at +-448.
__device__ __forceinline__ uint32_t e4m3x2_from(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
__device__ __forceinline__ float f16_to_f32(uint16_t v) {
    float r;
    asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(v));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to(uint32_t v) {
    const uint32_t h = f16x2_from_e4m3x2(v & 0xffffu);
    return make_float2(f16_to_f32((uint16_t)(h & 0xffffu)), f16_to_f32((uint16_t)(h >> 16)));
}

}  // namespace lidx
