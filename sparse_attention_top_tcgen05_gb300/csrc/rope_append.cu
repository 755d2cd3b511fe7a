// rope_append.cu -- new keys and values into a paged cache with the norm and the rotary positions of the keys on the way, into
// 8 or 4 bits; and the 4-bit cache as an 8-bit one.
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
#include "cache.cuh"
#include "rope.cuh"

namespace lidx {

constexpr int kRaThreads = 256;

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
    int S, Hkv, D, page, max_pages, J, heads;  // heads of a block
    RopeDiv pairs;
};

enum { kRaPlain = 0, kRaPairs = 1, kRaHalf = 2, kRaAny = 3 };  // how pairs lie in the lanes' 16 dims

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

template <int BITS, int LANES, int MODE>
__global__ void __launch_bounds__(kRaThreads) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
    constexpr int G = kRaThreads / LANES, PER = 128 / G;  // tokens a pass, passes of the longest page
    extern __shared__ __align__(16) float s_ra[];
    __shared__ uint32_t s_top[kRaThreads / 32];
    const int b = blockIdx.x / p.J, j = blockIdx.x % p.J, which = blockIdx.z;
    const int64_t start = p.start[b];
    int64_t count = p.count ? p.count[b] : p.S;
    count = count < 0 ? 0 : (count > p.S ? p.S : count);
    // page slots are counted from the page of the first position that is not negative
    const int64_t from = start < 0 ? 0 : start;
    const int64_t slot = from / p.page + j;
    const int64_t p0 = slot * p.page;
    const int64_t lo = from > p0 ? from : p0;  // new tokens: positions [lo, hi)
    int64_t hi = start + count;
    hi = hi < p0 + p.page ? hi : p0 + p.page;
    if (hi <= lo || slot >= p.max_pages) return;
    const int64_t pid = p.table[(int64_t)b * p.max_pages + slot];
    if (pid < 0 || pid >= p.num_pages) return;
    const int n = (int)(hi - lo), nk = p0 < start ? (int)(lo - p0) : 0;  // new tokens, tokens the page holds
    const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES, d0 = 16 * l;
    const bool on = d0 < p.D;
    const bool turns = MODE != kRaPlain && which == 0, norms = which == 0 && p.w != nullptr;
    const int R2 = p.r.R / 2;
    float* const s_w = s_ra;                                    // [D]
    float2* const s_cs = (float2*)(s_ra + p.D);                 // [n][R2]
    if (turns) {
        for (int i = threadIdx.x; i < n * R2; i += kRaThreads) {
            const int e = rope_quot(i, p.pairs), u = i - e * R2;
            const int64_t at = lo - start + e;
            s_cs[i] = p.r.pos ? rope_cs(p.r, b, at, u) : rope_cs((int)(lo + e), p.r.freqs[u], p.r.mscale, 1.f);
        }
    }
    if (norms)
        for (int d = threadIdx.x; d < p.D; d += kRaThreads)
            s_w[d] = p.w32 ? ((const float*)p.w)[d] : rope_get((const __nv_bfloat16*)p.w + d);
    const int h0 = blockIdx.y * p.heads, hz = min(h0 + p.heads, p.Hkv);
    for (int h = h0; h < hz; ++h) {
        const uint16_t* x = p.x[which] + b * p.xs[which][0] + (lo - start) * p.xs[which][1] + h * p.xs[which][2] + d0;
        const int64_t cell = pid * p.Hkv + h;
        const float old = p.scale[which][cell];
        float f[PER][16];
        uint4 va[PER], vb[PER];
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
        if (h == h0) __syncthreads();  // angles and weights are there
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (k * G >= n) break;
            const int e = grp + k * G;
            float(&y)[16] = f[k];
            rope_unpack(va[k], reinterpret_cast<float(&)[8]>(y[0]));
            rope_unpack(vb[k], reinterpret_cast<float(&)[8]>(y[8]));
            if (norms) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) ss += y[i] * y[i];
#pragma unroll
                for (int i = 1; i < LANES; i <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, i);
                const float r = __frsqrt_rn(ss * p.inv_d + p.eps);
                if (on) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] *= r * s_w[d0 + i];
                }
            }
            if (turns) {
                const float2* cs = s_cs + (e < n ? e : 0) * R2;
                if constexpr (MODE == kRaPairs) {
                    // pairs (2i, 2i + 1) of an even offset
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const int u = (d0 + i - p.r.off) / 2;
                        if (d0 + i >= p.r.off && u < R2) {
                            const float2 c = cs[u];
                            const float s = y[i], t = y[i + 1];
                            y[i] = s * c.x - t * c.y;
                            y[i + 1] = t * c.x + s * c.y;
                        }
                    }
                } else if constexpr (MODE == kRaHalf) {
                    // halves and offset of whole groups: a pair's other element is at the same place of another lane
                    const int at = d0 - p.r.off, hop = R2 / 16;
                    const bool first = at >= 0 && at < R2, second = at >= R2 && at < p.r.R;
                    const int lane = threadIdx.x & 31, peer = first ? lane + hop : (second ? lane - hop : lane);
                    const float2* c = cs + (first ? at : (second ? at - R2 : 0));
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float t = __shfl_sync(0xffffffffu, y[i], peer);
                        if (first || second) y[i] = y[i] * c[i].x + (first ? -t : t) * c[i].y;
                    }
                } else if constexpr (MODE == kRaAny) {
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
            if (e < n) {
#pragma unroll
                for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
            }
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
                    for (int i = 0; i < 4; ++i)
                        q[i] = e4m3x2_from(f[k][4 * i] * inv, f[k][4 * i + 1] * inv) |
                               (e4m3x2_from(f[k][4 * i + 2] * inv, f[k][4 * i + 3] * inv) << 16);
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
                uint32_t g = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) g = max(g, __float_as_uint(f[k][i]) & 0x7fffffffu);
                const bool number = g < 0x7f800000u;
                int x = g > 0 ? ra_exp(__uint_as_float(g) * inv, 0.75f, 3) : 0;
                x = !number ? 15 : max(0, min(x, kCache4Exps - 1));
                const float m = number ? ldexpf(inv, -x) : 0.f;
                if (live && on) {
                    uint32_t q[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        q[i] = 0;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            q[i] |= e2m1x2_from(f[k][8 * i + 2 * c] * m, f[k][8 * i + 2 * c + 1] * m) << (8 * c);
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

// Codes and exponents of a 4-bit cache -> e4m3 of number / 32: a thread a group.
struct WidenParams {
    const uint2* codes[2];
    const int32_t* exps[2];
    uint4* out[2];
    int64_t groups;
    int per;  // groups of a slot
};
__global__ void __launch_bounds__(256) cache4_widen_kernel(const __grid_constant__ WidenParams p) {
    const int which = blockIdx.y;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < p.groups; i += gridDim.x * 256ll) {
        const int64_t slot = i / p.per;
        const uint2 c = p.codes[which][i];
        const uint32_t x = ((uint32_t)p.exps[which][slot] >> (4 * (int)(i - slot * p.per))) & 15u;
        uint32_t lo, hi;
        cache4_table(x, lo, hi);
        const uint2 a = cache4_widen(c.x, lo, hi), b = cache4_widen(c.y, lo, hi);
        p.out[which][i] = make_uint4(a.x, a.y, b.x, b.y);
    }
}

// ------------------------------------------------------------------- host

template <int BITS, int LANES, int MODE>
static cudaError_t ra_launch_mode(const RopeAppendParams& p, int64_t B, int smem, cudaStream_t st) {
    auto* kernel = rope_append_kernel<BITS, LANES, MODE>;
    if (smem > 48 * 1024) {
        const cudaError_t e = set_smem_attr((const void*)kernel, smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)(B * p.J), (unsigned)((p.Hkv + p.heads - 1) / p.heads), 2);
    kernel<<<grid, kRaThreads, smem, st>>>(p);
    return cudaGetLastError();
}
template <int BITS, int LANES>
static cudaError_t ra_launch(const RopeAppendParams& p, int64_t B, cudaStream_t st) {
    const RopeTurn& r = p.r;
    const int R2 = r.R / 2, rows = p.page < p.S ? p.page : p.S;
    int smem = p.D * 4 + (p.turn ? rows * R2 * 8 : 0);
    if (!p.turn) return ra_launch_mode<BITS, LANES, kRaPlain>(p, B, smem, st);
    if (!r.half && r.off % 2 == 0) return ra_launch_mode<BITS, LANES, kRaPairs>(p, B, smem, st);
    if (r.half && r.off % 16 == 0 && R2 % 16 == 0) return ra_launch_mode<BITS, LANES, kRaHalf>(p, B, smem, st);
    smem += kRaThreads / LANES * p.D * 4;
    return ra_launch_mode<BITS, LANES, kRaAny>(p, B, smem, st);
}

// Both entries; bits 8: exps NULL.  r NULL: no rotation.
static int ra_append(int bits, const void* k, const void* v, const int64_t* ks, const int64_t* vs, const lidx_rope_turn* r,
                     const void* w, int w_dtype, float eps, const int32_t* block_table, const int32_t* start,
                     const int32_t* count, int64_t B, int64_t S, int Hkv, int D, int page, int64_t max_pages,
                     int64_t num_pages, void* k_cache, void* v_cache, int32_t* k_exps, int32_t* v_exps, float* k_scale,
                     float* v_scale, void* stream) {
    if (!k || !v || !ks || !vs || !block_table || !start || !k_cache || !v_cache || !k_scale || !v_scale ||
        (bits == 4 && (!k_exps || !v_exps)))
        return LIDX_ERR_NULL;
    int rc = check_cache(B, S, Hkv, D, page, max_pages, num_pages);
    if (rc) return rc;
    RopeAppendParams p;
    p.r = RopeTurn{nullptr, {0, 0, 0}, nullptr, nullptr, 1, 2, 0, 0, 1.f, 1.f};
    if (r) {
        rc = rope_turn(r, D, 0, p.r, true);
        if (rc) return rc;
    }
    if ((w_dtype != 0 && w_dtype != 1) || (w && (!(eps >= 0.f) || !isfinite(eps)))) return LIDX_ERR_SHAPE;
    const int64_t J = (S + page - 2) / page + 1;  // pages S tokens can touch
    if (B * J > INT_MAX || Hkv > 65535) return LIDX_ERR_SHAPE;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15u) return LIDX_ERR_ALIGN;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)k_exps | (uintptr_t)v_exps | (uintptr_t)block_table |
         (uintptr_t)start | (uintptr_t)count) & 3u)
        return LIDX_ERR_ALIGN;
    if (w && (uintptr_t)w % (w_dtype == 0 ? 4 : 2)) return LIDX_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if ((ks[i] | vs[i]) & 7) return LIDX_ERR_ALIGN;
    if (r) {
        rc = rope_turn_aligned(*r);
        if (rc) return rc;
    }
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    p.x[0] = (const uint16_t*)k;
    p.x[1] = (const uint16_t*)v;
    for (int i = 0; i < 3; ++i) {
        p.xs[0][i] = ks[i];
        p.xs[1][i] = vs[i];
    }
    p.cache[0] = (uint8_t*)k_cache;
    p.cache[1] = (uint8_t*)v_cache;
    p.exps[0] = k_exps;
    p.exps[1] = v_exps;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.turn = r != nullptr;
    p.w = w;
    p.w32 = w_dtype == 0;
    p.eps = eps;
    p.inv_d = 1.f / D;
    p.table = block_table;
    p.start = start;
    p.count = count;
    p.num_pages = num_pages;
    p.S = (int)S;
    p.Hkv = Hkv;
    p.D = D;
    p.page = page;
    p.max_pages = (int)max_pages;
    p.J = (int)J;
    p.heads = 1;
    p.pairs = rope_div(p.r.R / 2);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (bits == 8)
        e = D <= 64 ? ra_launch<8, 4>(p, B, st) : ra_launch<8, 8>(p, B, st);
    else
        e = D <= 64 ? ra_launch<4, 4>(p, B, st) : ra_launch<4, 8>(p, B, st);
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // namespace lidx

using namespace lidx;

extern "C" {

int lidx_rope_cache_append(const void* k, const void* v, const int64_t* ks, const int64_t* vs, const lidx_rope_turn* r,
                           const void* w, int w_dtype, float eps, const int32_t* block_table, const int32_t* start,
                           const int32_t* count, int64_t B, int64_t S, int Hkv, int D, int page, int64_t max_pages,
                           int64_t num_pages, void* k_cache, void* v_cache, float* k_scale, float* v_scale, void* stream) {
    if (!r) return LIDX_ERR_NULL;
    return ra_append(8, k, v, ks, vs, r, w, w_dtype, eps, block_table, start, count, B, S, Hkv, D, page, max_pages, num_pages,
                     k_cache, v_cache, nullptr, nullptr, k_scale, v_scale, stream);
}

int lidx_cache4_append(const void* k, const void* v, const int64_t* ks, const int64_t* vs, const lidx_rope_turn* r,
                       const void* w, int w_dtype, float eps, const int32_t* block_table, const int32_t* start,
                       const int32_t* count, int64_t B, int64_t S, int Hkv, int D, int page, int64_t max_pages,
                       int64_t num_pages, void* k_cache, void* v_cache, int32_t* k_exps, int32_t* v_exps, float* k_scale,
                       float* v_scale, void* stream) {
    return ra_append(4, k, v, ks, vs, r, w, w_dtype, eps, block_table, start, count, B, S, Hkv, D, page, max_pages, num_pages,
                     k_cache, v_cache, k_exps, v_exps, k_scale, v_scale, stream);
}

int lidx_cache4_to_8(const void* k_cache, const void* v_cache, const int32_t* k_exps, const int32_t* v_exps, int Hkv, int D,
                     int page, int64_t num_pages, void* k8, void* v8, void* stream) {
    if (!k_cache || !v_cache || !k_exps || !v_exps || !k8 || !v8) return LIDX_ERR_NULL;
    const int rc = check_cache(1, 1, Hkv, D, page, 1, num_pages);
    if (rc) return rc;
    if (((uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)k8 | (uintptr_t)v8) & 15u) return LIDX_ERR_ALIGN;
    if (((uintptr_t)k_exps | (uintptr_t)v_exps) & 3u) return LIDX_ERR_ALIGN;
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    WidenParams p;
    p.codes[0] = (const uint2*)k_cache;
    p.codes[1] = (const uint2*)v_cache;
    p.exps[0] = k_exps;
    p.exps[1] = v_exps;
    p.out[0] = (uint4*)k8;
    p.out[1] = (uint4*)v8;
    p.per = D / 16;
    p.groups = num_pages * Hkv * page * p.per;
    const int64_t blocks = (p.groups + 255) / 256, cap = (int64_t)current_sms() * 32;
    cache4_widen_kernel<<<dim3((unsigned)(blocks < cap ? blocks : cap), 2), 256, 0, (cudaStream_t)stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
