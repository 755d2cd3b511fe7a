// rope_append.cuh -- the kernel that writes new keys and values into a paged cache with the norm and the rotary positions of
// the keys on the way (rope_append.cu: 8 bits and the entries, cache4_append.cu: 4 bits).
//
// Keys: k' = turn(k r w) as in norm_rope.cu (both parts optional), in fp32; then k' and v are rounded once, to the cache's
// numbers.  8 bits: as cache_append.cu.  4 bits: a page of one head has a scale 2^e, the smallest (e >= -40) with
// |x| <= 6 * 2^11 * 2^e, kept or grown as there; each 16 dims of a slot have an exponent x, the smallest of 0 .. 11 with
// |x| <= 6 * 2^x * 2^e, and codes e2m1 (cache.cuh).  A page's groups reach over 2^11 of size with one fraction bit each; what
// is smaller yet keeps steps of half a scale.  When the scale grows by 2^d, exponents fall by d and the codes stay, unless
// the exponent would fall below 0.  A group with an infinity or a NaN has exponent 15 (not numbers) and changes no scale.
//
// One block per (sequence, page it touches, some heads, k or v); LANES lanes a token, 16 dims each, so that a group's
// maximum is a lane's own.  A page's tokens stay in registers between the page's maximum and the conversion.  Angles of the
// page's tokens are computed once a block into shared memory and serve its heads.
//
// What bounds it.  8 bits, 4 x 4097 tokens of 8 heads of 128, half of each key turned: 26.5 us (25.5 us for cache_append.cu, which
// turns nothing), a block's dependent reads and barriers.  4 bits, the same with a norm and all of each key turned by three axes:
// 32.5 us, 67 % of issue slots busy.  One token of 64 sequences, normed and turned: 8.7 us, in 4 bits 9.5 us; passes go by the page,
// so its 1024 blocks of 256 threads run in three waves.
//
// Blocks an SM: two of four passes (128 registers), three of fewer (80).  With that the kernels of half layouts spill 44 to 128
// bytes and those of pairs side by side up to 48 (-Xptxas -v).  One and two blocks spill nothing and take longer: the prompts above 29.3
// and 35.4 us.
#pragma once
#include "cache.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace lidx {

constexpr int kRaThreads = 256;
constexpr int kRaStatic = kRaThreads / 32 * (int)sizeof(uint32_t);  // bytes of s_top

struct RopeAppendParams {
    const uint16_t* x[2];  // k, v
    int64_t xs[2][3];
    uint8_t* cache[2];
    int32_t* exps[2];
    float* scale[2];
    RopeTurn r;
    int turn;              // 0: no rotation
    const void* w;         // nullable: no norm
    int w32;
    float eps, inv_d;
    const int32_t* table;
    const int32_t* start;
    const int32_t* count;
    int64_t num_pages;
    int S, Hkv, D, page, max_pages, J;
    int page_shift;        // page = 1 << page_shift
    int heads;             // of a block
    RopeDiv pairs;
};

// How pairs lie in the lanes' 16 dims: neighbours, the same places of two lanes (both with offset and rotated part of whole
// lanes), or anyhow: then rows go through shared memory.
enum { kRaPairs = 0, kRaHalf = 1, kRaAny = 2 };

// |bits| of a float; infinities and NaN become NaN and do not count.
__device__ __forceinline__ uint32_t ra_finite(float& v) {
    const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
    if (u < 0x7f800000u) return u;
    v = __uint_as_float(0x7fffffffu);
    return 0;
}
// Smallest e with amax <= top * 2^e, top = mt * 2^et, mt in [1/2, 1).
__device__ __forceinline__ int ra_exp(float amax, float mt, int et) {
    int ex;
    const float m = frexpf(amax, &ex);
    return ex - et + (m > mt ? 1 : 0);
}
// Maximum over the block; s: a word a warp.  Two barriers.
__device__ __forceinline__ uint32_t ra_block_max(uint32_t m, uint32_t* s) {
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRaThreads / 32; ++i) m = max(m, s[i]);
    return m;
}

// Largest size of a lane's 16 dims; NaN where one is.
__device__ __forceinline__ float ra_size(const float (&y)[16]) {
    float g = fabsf(y[0]);
#pragma unroll
    for (int i = 1; i < 15; i += 2) g = max3_nan(g, fabsf(y[i]), fabsf(y[i + 1]));
    return max_nan(g, fabsf(y[15]));
}
// Two neighbouring dims times f.
__device__ __forceinline__ void ra_times(float& a, float& b, uint64_t f) { unpack2(mul2(pack2(a, b), f), a, b); }

template <int BITS, int LANES, int MODE, int PER>
__global__ void __launch_bounds__(kRaThreads, PER == 4 ? 2 : 3) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
    constexpr int G = kRaThreads / LANES;                                // tokens a pass, PER passes
    constexpr int A = MODE == kRaPairs ? 8 : (MODE == kRaHalf ? 16 : 2);  // angles of a lane (rope.cuh)
    extern __shared__ __align__(16) float s_ra[];
    __shared__ uint32_t s_top[kRaThreads / 32];
    const int b = blockIdx.x / p.J, j = blockIdx.x % p.J, which = blockIdx.z;
    const int64_t start = p.start[b];
    int64_t count = p.count ? p.count[b] : p.S;
    count = count < 0 ? 0 : (count > p.S ? p.S : count);
    // page slots are counted from the page of the first position that is not negative
    const int64_t from = start < 0 ? 0 : start;
    const int64_t slot = (from >> p.page_shift) + j;
    const int64_t p0 = slot * p.page;
    const int64_t lo = from > p0 ? from : p0;  // new tokens: positions [lo, hi)
    int64_t hi = start + count;
    hi = hi < p0 + p.page ? hi : p0 + p.page;
    if (hi <= lo || slot >= p.max_pages) return;
    const int64_t pid = p.table[(int64_t)b * p.max_pages + slot];
    const int n = (int)(hi - lo), nk = p0 < start ? (int)(lo - p0) : 0;  // new tokens, tokens the page holds
    const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES, d0 = 16 * l;
    const bool on = d0 < p.D;
    const bool turns = which == 0 && p.turn, norms = which == 0 && p.w != nullptr;
    const int R2 = p.r.R / 2;
    float* const s_w = s_ra;                                // [4][LANES] words of 16 bytes
    float2* const s_cs = (float2*)(s_ra + 16 * LANES);      // [n][R2]
    const uint16_t* const x0 = p.x[which] + b * p.xs[which][0] + (lo - start) * p.xs[which][1] + d0;
    const int h0 = blockIdx.y * p.heads, hz = min(h0 + p.heads, p.Hkv);
    uint4 va[PER], vb[PER];
    auto load = [&](int h) {
        const uint16_t* x = x0 + h * p.xs[which][2];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = grp + k * G;
            va[k] = vb[k] = make_uint4(0, 0, 0, 0);
            if (e < n && on) {
                const uint4* src = reinterpret_cast<const uint4*>(x + e * p.xs[which][1]);
                va[k] = src[0];
                vb[k] = src[1];
            }
        }
    };
    load(h0);
    if (turns) {
        for (int i = threadIdx.x; i < n * R2; i += kRaThreads) {
            const int e = rope_quot(i, p.pairs), u = i - e * R2;
            const int64_t at = lo - start + e;
            const float2 c = p.r.pos ? rope_cs(p.r, b, at, u) : rope_cs((int)(lo + e), p.r.freqs[u], p.r.mscale, 1.f);
            if constexpr (MODE == kRaAny)
                s_cs[e * R2 + u] = c;
            else
                rope_put_angle<A>(s_cs + e * R2, u, R2 / A, c);
        }
    }
    if (norms && threadIdx.x < LANES && on) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s_w[(i / 4 * LANES + l) * 4 + i % 4] = p.w32 ? ((const float*)p.w)[d0 + i] : rope_get((const __nv_bfloat16*)p.w + d0 + i);
    }
    if (pid < 0 || pid >= p.num_pages) return;  // (the same in all threads; the loads did not wait for it)
    __syncthreads();
    for (int h = h0; h < hz; ++h) {
        const int64_t cell = pid * p.Hkv + h;
        const float old = p.scale[which][cell];
        float f[PER][16];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            rope_unpack(va[k], reinterpret_cast<float(&)[8]>(f[k][0]));
            rope_unpack(vb[k], reinterpret_cast<float(&)[8]>(f[k][8]));
        }
        if (h + 1 < hz) load(h + 1);
        uint32_t top = 0;
        float size[PER];  // of the lane's dims
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            size[k] = 0.f;
            if (k * G >= n) continue;
            const int e = grp + k * G;
            float(&y)[16] = f[k];
            if (norms) {
                uint64_t s2 = pack2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; i += 2) s2 = fma2(pack2(y[i], y[i + 1]), pack2(y[i], y[i + 1]), s2);
                float ss, odd;
                unpack2(s2, ss, odd);
                ss += odd;
#pragma unroll
                for (int i = 1; i < LANES; i <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, i);
                const float r = __frsqrt_rn(ss * p.inv_d + p.eps);
                if (on) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 w = reinterpret_cast<const float4*>(s_w)[i / 4 * LANES + l];
                        ra_times(y[i], y[i + 1], mul2(pack2(r, r), pack2(w.x, w.y)));
                        ra_times(y[i + 2], y[i + 3], mul2(pack2(r, r), pack2(w.z, w.w)));
                    }
                }
            }
            if (turns) {
                const float2* cs = s_cs + (e < n ? e : 0) * R2;
                const int at = d0 - p.r.off;
                if constexpr (MODE == kRaPairs) {
                    if (at >= 0 && at < p.r.R) {
                        float2 c[A];
                        rope_angles_of<A>(cs, at / 16, R2 / A, c);
#pragma unroll
                        for (int i = 0; i < A; ++i) {
                            const float s = y[2 * i], t = y[2 * i + 1];
                            y[2 * i] = s * c[i].x - t * c[i].y;
                            y[2 * i + 1] = t * c[i].x + s * c[i].y;
                        }
                    }
                } else if constexpr (MODE == kRaHalf) {
                    // a pair's other element is at the same place of another lane
                    const int hop = R2 / 16;
                    const bool first = at >= 0 && at < R2, second = at >= R2 && at < p.r.R;
                    const int lane = threadIdx.x & 31, peer = first ? lane + hop : (second ? lane - hop : lane);
                    const int item = first ? at / 16 : (second ? (at - R2) / 16 : 0);
                    const float sign = first ? -1.f : 1.f;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float4 v = reinterpret_cast<const float4*>(cs)[i / 2 * (R2 / A) + item];  // two cosines, two sines
                        const float t0 = __shfl_sync(0xffffffffu, y[i], peer), t1 = __shfl_sync(0xffffffffu, y[i + 1], peer);
                        const uint64_t t = mul2(pack2(t0 * sign, t1 * sign), pack2(v.z, v.w));
                        if (first || second) unpack2(fma2(pack2(y[i], y[i + 1]), pack2(v.x, v.y), t), y[i], y[i + 1]);
                    }
                } else {
                    float* row = (float*)(s_cs + min(p.page, p.S) * R2) + grp * p.D;
                    __syncwarp();  // the pass before is read
                    if (on) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) row[d0 + i] = y[i];
                    }
                    __syncwarp();
                    for (int u = l; u < R2; u += LANES) {
                        const int ia = p.r.half ? p.r.off + u : p.r.off + 2 * u, ib = p.r.half ? ia + R2 : ia + 1;
                        const float s = row[ia], t = row[ib];
                        row[ia] = s * cs[u].x - t * cs[u].y;
                        row[ib] = t * cs[u].x + s * cs[u].y;
                    }
                    __syncwarp();
                    if (on) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = row[d0 + i];
                    }
                }
            }
            size[k] = ra_size(y);
            if (e < n) top = max(top, __float_as_uint(size[k]));
        }
        top = ra_block_max(top, s_top);
        if (top >= 0x7f800000u) {  // (the same in all threads) what is not finite does not count
            top = 0;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (grp + k * G < n) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = max(top, ra_finite(f[k][i]));
                }
            top = ra_block_max(top, s_top);
        }
        const float amax = __uint_as_float(top);
        const int e = amax > 0.f ? (BITS == 8 ? ra_exp(amax, 0.875f, 9) : ra_exp(amax, 0.75f, 14)) : kCacheMinExp;
        float now = ldexpf(1.f, max(e, kCacheMinExp));
        if (nk > 0) now = fmaxf(now, old);
        const float inv = 1.f / now;  // exact: a power of two (an old scale that is none rounds)
        const bool grows = nk > 0 && now > old;
        const float ratio = old / now;
        const int64_t row0 = cell * p.page;  // first slot of the page and head
        if constexpr (BITS == 8) {
            uint8_t* out = p.cache[which] + row0 * p.D;
            if (grows) {
                // the earlier tokens' codes move to the new scale
                for (int i = threadIdx.x; i < nk * p.D / 8; i += kRaThreads) {
                    uint2 c = reinterpret_cast<const uint2*>(out)[i];
                    uint32_t q[2] = {c.x, c.y};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 a = e4m3x2_to(q[k]), z = e4m3x2_to(q[k] >> 16);
                        q[k] = e4m3x2_from(a.x * ratio, a.y * ratio) | (e4m3x2_from(z.x * ratio, z.y * ratio) << 16);
                    }
                    reinterpret_cast<uint2*>(out)[i] = make_uint2(q[0], q[1]);
                }
            }
            out += (lo - p0) * p.D + d0;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (grp + k * G < n && on) {
                    uint32_t q[4];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) ra_times(f[k][i], f[k][i + 1], pack2(inv, inv));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[i] = e4m3x2_from(f[k][4 * i], f[k][4 * i + 1]) | (e4m3x2_from(f[k][4 * i + 2], f[k][4 * i + 3]) << 16);
                    *reinterpret_cast<uint4*>(out + (grp + k * G) * p.D) = make_uint4(q[0], q[1], q[2], q[3]);
                }
            }
        } else {
            uint8_t* const out = p.cache[which] + row0 * (p.D / 2) + l * 8;
            int32_t* const ex = p.exps[which] + row0;
            auto nibbles = [&](uint32_t x) {  // the lanes' exponents, of a slot
                x = on ? x << (4 * l) : 0u;
#pragma unroll
                for (int i = 1; i < LANES; i <<= 1) x |= __shfl_xor_sync(0xffffffffu, x, i);
                return x;
            };
            if (grows) {
                const int rise = ra_exp(ratio, 0.5f, 1);  // smallest r with ratio <= 2^r, r <= 0
                for (int t0 = 0; t0 < nk; t0 += G) {
                    const int t = t0 + grp;
                    uint32_t x = 0;
                    if (t < nk && on) {
                        x = ((uint32_t)ex[t] >> (4 * l)) & 15u;
                        if (x < kCache4Exps) {
                            const int to = max((int)x + rise, 0);
                            uint2* at = reinterpret_cast<uint2*>(out + t * (p.D / 2));
                            const float m = ldexpf(ratio, (int)x - to) * kCache4Unit;  // (a table of exponent 0 holds 2^-5 of the codes)
                            uint32_t lut0, lut1;
                            cache4_table(0, lut0, lut1);
                            uint32_t q[2] = {at->x, at->y};
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint2 wide = cache4_widen(q[k], lut0, lut1);
                                const float2 a = e4m3x2_to(wide.x), c = e4m3x2_to(wide.x >> 16);
                                const float2 g = e4m3x2_to(wide.y), z = e4m3x2_to(wide.y >> 16);
                                q[k] = e2m1x2_from(a.x * m, a.y * m) | (e2m1x2_from(c.x * m, c.y * m) << 8) |
                                       (e2m1x2_from(g.x * m, g.y * m) << 16) | (e2m1x2_from(z.x * m, z.y * m) << 24);
                            }
                            *at = make_uint2(q[0], q[1]);
                            x = to;
                        }
                    }
                    x = nibbles(x);
                    if (t < nk && l == 0) ex[t] = (int32_t)x;
                    __syncwarp();
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (k * G >= n) break;
                const int t = (int)(lo - p0) + grp + k * G;
                const bool live = grp + k * G < n;
                const bool number = size[k] <= 3.4028235e38f;
                int x = size[k] > 0.f ? ra_exp(size[k] * inv, 0.75f, 3) : 0;
                x = !number ? 15 : max(0, min(x, kCache4Exps - 1));
                const float m = number ? ldexpf(inv, -x) : 0.f;
                if (live && on) {
                    uint32_t q[2];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) ra_times(f[k][i], f[k][i + 1], pack2(m, m));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        q[i] = 0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) q[i] |= e2m1x2_from(f[k][8 * i + 2 * c], f[k][8 * i + 2 * c + 1]) << (8 * c);
                        if (!number) q[i] = 0;
                    }
                    *reinterpret_cast<uint2*>(out + t * (p.D / 2)) = make_uint2(q[0], q[1]);
                }
                const uint32_t all = nibbles((uint32_t)x);
                if (live && l == 0) ex[t] = (int32_t)all;
            }
        }
        if (threadIdx.x == 0) p.scale[which][cell] = now;
    }
}

template <int BITS, int LANES, int MODE, int PER>
static cudaError_t ra_launch_passes(const RopeAppendParams& p, int64_t B, int smem, cudaStream_t st) {
    auto* kernel = rope_append_kernel<BITS, LANES, MODE, PER>;
    if (smem + kRaStatic > 48 * 1024) {  // what every kernel may have is counted with s_top
        const cudaError_t e = set_smem_attr((const void*)kernel, smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)(B * p.J), (unsigned)((p.Hkv + p.heads - 1) / p.heads), 2);
    kernel<<<grid, kRaThreads, smem, st>>>(p);
    return cudaGetLastError();
}
template <int BITS, int LANES, int MODE>
static cudaError_t ra_launch_mode(const RopeAppendParams& p, int64_t B, int smem, cudaStream_t st) {
    constexpr int G = kRaThreads / LANES;
    smem += 64 * LANES;
    if (p.page <= G) return ra_launch_passes<BITS, LANES, MODE, 1>(p, B, smem, st);
    if (p.page <= 2 * G) return ra_launch_passes<BITS, LANES, MODE, 2>(p, B, smem, st);
    if constexpr (LANES == 8) return ra_launch_passes<BITS, LANES, MODE, 4>(p, B, smem, st);
    return cudaErrorInvalidValue;
}
template <int BITS, int LANES>
static cudaError_t ra_launch(const RopeAppendParams& p, int64_t B, cudaStream_t st) {
    const RopeTurn& r = p.r;
    const int R2 = r.R / 2, rows = p.page < p.S ? p.page : p.S, angles = p.turn ? rows * R2 * 8 : 0;
    if (!p.turn || (!r.half && r.off % 16 == 0 && r.R % 16 == 0)) return ra_launch_mode<BITS, LANES, kRaPairs>(p, B, angles, st);
    if (r.half && r.off % 16 == 0 && R2 % 16 == 0) return ra_launch_mode<BITS, LANES, kRaHalf>(p, B, angles, st);
    return ra_launch_mode<BITS, LANES, kRaAny>(p, B, angles + kRaThreads / LANES * p.D * 4, st);
}
template <int BITS>
static cudaError_t ra_launch_bits(const RopeAppendParams& p, int64_t B, cudaStream_t st) {
    return p.D <= 64 ? ra_launch<BITS, 4>(p, B, st) : ra_launch<BITS, 8>(p, B, st);
}
cudaError_t cache4_append_launch(const RopeAppendParams& p, int64_t B, cudaStream_t st);  // 4 bits

}  // namespace lidx
