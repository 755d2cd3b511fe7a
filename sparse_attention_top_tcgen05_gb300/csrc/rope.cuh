// rope.cuh -- what the rotary kernels share (rope.cu, norm_rope.cu, rope_append.cu): the angle of a position, quotients by
// sizes, vectors of 16 bytes.
//
// Frequencies are turns per position in 0.64 fixed point, so pos * freq mod 2^64 is the fraction of
// a turn exactly, whatever the position: a float angle would lose log2(pos) of its 24 bits.  The upper
// 32 bits of the product, read as signed, are the angle from half a turn back to half a turn.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <climits>

#include "kernels.h"
#include "lidx.h"

namespace lidx {

// n / d for n < 2^31: (hi(n * mul) + n) >> shift with shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1
// (division by an invariant integer through multiplication, Granlund and Montgomery 1994).
struct RopeDiv {
    uint32_t d, mul, shift;
};
inline RopeDiv rope_div(uint32_t d) {
    RopeDiv r;
    r.d = d;
    r.shift = 0;
    while ((1ull << r.shift) < d) ++r.shift;
    r.mul = (uint32_t)(((1ull << 32) * ((1ull << r.shift) - d)) / d + 1);
    return r;
}
__device__ __forceinline__ uint32_t rope_quot(uint32_t n, const RopeDiv& v) {
    return (__umulhi(n, v.mul) + n) >> v.shift;
}

// A rotation: pair i of a token turns by pos[axis of i] * freqs[i], scaled by mscale.
struct RopeTurn {
    const int32_t* pos;
    int64_t ps[3];        // strides of axis, T0, T1
    const uint64_t* freqs;
    const uint8_t* axis;  // nullable: every pair is of axis 0
    int axes, R, off, half;
    float mscale, sign;   // sign -1: the inverse
};

// Scaled cosine and sine of position pos of a pair.
__device__ __forceinline__ float2 rope_cs(int pos, uint64_t freq, float mscale, float sign) {
    const uint64_t t = (uint64_t)(int64_t)pos * freq;
    // half turns in [-1, 1): 32 bits of the fraction, rounded once
    const float h = (float)(int32_t)(t >> 32) * 0x1p-31f;
    float s, c;
    sincospif(h, &s, &c);
    return make_float2(c * mscale, s * mscale * sign);
}

__device__ __forceinline__ float2 rope_cs(const RopeTurn& r, int64_t t0, int64_t t1, int u) {
    int64_t at = t0 * r.ps[1] + t1 * r.ps[2];
    if (r.axis) at += min((int)r.axis[u], r.axes - 1) * r.ps[0];
    return rope_cs(r.pos[at], r.freqs[u], r.mscale, r.sign);
}

__device__ __forceinline__ float rope_get(const float* p) { return *p; }
__device__ __forceinline__ float rope_get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void rope_unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void rope_unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 rope_pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 rope_pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Angles in shared memory.  An item (a vector of the interleaved layout, a pair of vectors of the half layout) has A
// consecutive angles; two of them are a 16-byte word (two cosines, two sines: operands of packed arithmetic), and the items'
// k-th words follow each other, so that lanes with neighbouring items read neighbouring words: with an item's angles side by
// side their reads met in the same banks.
template <int A>
__device__ __forceinline__ void rope_put_angle(float2* token, int u, int items, const float2& c) {  // angle u of a token
    const int item = u / A, j = u % A;
    float* at = reinterpret_cast<float*>(token) + ((j >> 1) * items + item) * 4 + (j & 1);
    at[0] = c.x;
    at[2] = c.y;
}
template <int A>
__device__ __forceinline__ void rope_angles_of(const float2* token, int item, int items, float2 (&c)[A]) {
#pragma unroll
    for (int k = 0; k < A / 2; ++k) {
        const float4 v = reinterpret_cast<const float4*>(token)[k * items + item];
        c[2 * k] = make_float2(v.x, v.z);
        c[2 * k + 1] = make_float2(v.y, v.w);
    }
}

// Rules of a rotation's host arguments (see lidx.h), and its device form.  own_pos: pos may be NULL.
int rope_turn(const lidx_rope_turn* r, int D, int inverse, RopeTurn& out, bool own_pos = false);
int rope_turn_aligned(const lidx_rope_turn& r);

}  // namespace lidx
