// cache.cuh -- what the paged caches' writers (cache_append.cu, rope_append.cu) and readers (cache_attn.cu,
// cache4_attn.cu) share: the layout's rules and the conversions of e4m3 and of 4-bit numbers.
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

// ---- 4-bit numbers.  A slot's codes are e2m1 (sign, two exponent bits, one fraction bit: 0 .5 1 1.5 2 3 4 6), dim i in bits
// 4 (i % 8) of word i / 8; each 16 dims have an exponent x of 4 bits, 0 .. 11, and 12 .. 15 where they are not numbers.
// code * 2^x is e4m3 times 2^5 exactly: codes of 1 and more add x to e4m3's exponent field, and so does .5, which is a
// power of two.  (e4m3's largest finite is 448; 6 * 2^11 / 2^5 = 384.)
constexpr int kCache4Exps = 12;
constexpr float kCache4Unit = 32.f;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// e4m3 codes of the eight sizes with exponent x: bytes of lo and hi.
__device__ __forceinline__ void cache4_table(uint32_t x, uint32_t& lo, uint32_t& hi) {
    lo = x * 0x08080800u + 0x14100800u;
    hi = x * 0x08080808u + 0x24201c18u;
    if (x >= kCache4Exps) lo = hi = 0x7f7f7f7fu;
}
// Eight 4-bit codes -> eight e4m3 codes: sizes by a byte lookup, signs by a byte's replicated top bit.
__device__ __forceinline__ uint2 cache4_widen(uint32_t w, uint32_t lo, uint32_t hi) {
    const uint32_t m = w & 0x77777777u, u = w << 4;
    const uint32_t a = prmt(lo, hi, m), b = prmt(lo, hi, m >> 16);
    return make_uint2(a | (prmt(u, w, 0xd9c8u) & 0x80808080u), b | (prmt(u, w, 0xfbeau) & 0x80808080u));
}
// The same with shifts that are products (by 16 and, the upper half, 2^16), for loops that the integer pipe bounds: products
// go to another.  The factors are registers that the compiler knows nothing of.
__device__ __forceinline__ uint2 cache4_widen_mul(uint32_t w, uint32_t lo, uint32_t hi, uint32_t f16, uint32_t f65536) {
    const uint32_t m = w & 0x77777777u, u = w * f16;
    const uint32_t a = prmt(lo, hi, m), b = prmt(lo, hi, __umulhi(m, f65536));
    return make_uint2(a | (prmt(u, w, 0xd9c8u) & 0x80808080u), b | (prmt(u, w, 0xfbeau) & 0x80808080u));
}
// Two floats -> two codes (lo in the low bits); rounds to nearest even, saturates at +-6.
__device__ __forceinline__ uint32_t e2m1x2_from(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace lidx
