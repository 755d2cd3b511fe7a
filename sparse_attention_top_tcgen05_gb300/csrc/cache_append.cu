// cache_append.cu -- new keys and values into a paged cache of 8-bit numbers.
//
// A page of one head has one scale, a power of two 2^e: the smallest (e >= -40) for which the page's new
// tokens fit in +-448 * 2^e, or the page's old scale if that is larger and the page holds earlier
// tokens.  With powers of two a growing scale only moves the exponents of the earlier codes: they
// stay exact unless they fall among e4m3's subnormals.  Infinities and NaN become NaN codes and do not count for
// the scale; the pass that sorts them out runs only in blocks that have one.
//
// One block per (sequence, page it touches, head, k or v).  It keeps its tokens in registers between
// the maximum and the conversion, so each input byte is read once.
//
// What bounds it: a block waits for start, table and tokens one after the other and the maximum at a barrier, so bytes
// in flight set the rate.  4 x 4097 tokens of 8 heads of 128 (84 MB): 24.5 us, 3.4 TB/s, with inputs that come from memory;
// 17.3 us with the same inputs again, most of which L2 holds.  Five blocks an SM (with L2's help 17.6 us, four 18.5 us, six,
// which spill, 18.3 us).  One token of 64 sequences: 5.4 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "cache.cuh"
#include "kernels.h"
#include "lidx.h"

namespace lidx {

constexpr int kAppThreads = 256;
constexpr int kAppVecs = 128 * (kCacheMaxD / 8) / kAppThreads;  // 16-byte vectors a thread may hold

struct AppendParams {
    const uint16_t* x[2];  // k, v
    int64_t xs[2][3];
    uint8_t* cache[2];
    float* scale[2];
    const int32_t* table;
    const int32_t* start;
    const int32_t* count;
    int64_t num_pages;
    int S, Hkv, D, page, max_pages, J;
};

// Smallest e >= kCacheMinExp with amax <= 448 * 2^e, amax finite.  448 = 1.75 * 2^8.
__device__ __forceinline__ float append_scale(uint32_t amax_bf16) {
    if (amax_bf16 == 0) return exp2f((float)kCacheMinExp);
    int ex;
    const float m = frexpf(__uint_as_float(amax_bf16 << 16), &ex);  // m in [1/2, 1)
    int e = ex - 9 + (m > 0.875f ? 1 : 0);
    e = e < kCacheMinExp ? kCacheMinExp : e;
    return ldexpf(1.f, e);
}

constexpr uint32_t kBf16Inf = 0x7f80;  // |code| of infinity; NaN lies above

// Larger |code| of a pair's finite values; infinities become NaN, which the conversion to e4m3 keeps.
__device__ __forceinline__ uint32_t append_finite(uint32_t& pair) {
    uint32_t lo = pair & 0x7fffu, hi = (pair >> 16) & 0x7fffu;
    if (lo >= kBf16Inf) pair |= 0x7fffu, lo = 0;
    if (hi >= kBf16Inf) pair |= 0x7fff0000u, hi = 0;
    return max(lo, hi);
}

__global__ void __launch_bounds__(kAppThreads, 5) cache_append_kernel(const __grid_constant__ AppendParams p) {
    const int b = blockIdx.x / p.J, j = blockIdx.x % p.J, h = blockIdx.y, which = blockIdx.z;
    const int64_t start = p.start[b];
    int64_t count = p.count ? p.count[b] : p.S;
    count = count < 0 ? 0 : (count > p.S ? p.S : count);
    // page slots are counted from the page of the first position that is not negative
    const int64_t first = start < 0 ? 0 : start;
    const int64_t slot = first / p.page + j;
    const int64_t p0 = slot * p.page;
    const int64_t lo = first > p0 ? first : p0;                  // new tokens: positions [lo, hi)
    int64_t hi = start + count;
    hi = hi < p0 + p.page ? hi : p0 + p.page;
    if (hi <= lo || slot >= p.max_pages) return;
    const int64_t pid = p.table[(int64_t)b * p.max_pages + slot];
    const int C = p.D / 8, n = (int)(hi - lo) * C;
    const uint16_t* x = p.x[which] + b * p.xs[which][0] + (lo - start) * p.xs[which][1] + h * p.xs[which][2];
    uint4 v[kAppVecs];
    uint32_t top = 0;  // packed pairs of |bf16| codes: ordered as integers
    // vector e is chunk c of a token: both step on without a division
    const int step = kAppThreads / C, over = kAppThreads - step * C;
    int c = threadIdx.x % C;
    const uint16_t* row = x + (int64_t)(threadIdx.x / C) * p.xs[which][1];
    const int64_t stride = p.xs[which][1], hop = step * stride;
#pragma unroll
    for (int i = 0; i < kAppVecs; ++i) {
        const int e = threadIdx.x + i * kAppThreads;
        if (e < n) {
            v[i] = *reinterpret_cast<const uint4*>(row + c * 8);
            row += hop;
            c += over;
            if (c >= C) {
                c -= C;
                row += stride;
            }
            top = __vmaxu2(__vmaxu2(top, v[i].x & 0x7fff7fffu), __vmaxu2(v[i].y & 0x7fff7fffu, v[i].z & 0x7fff7fffu));
            top = __vmaxu2(top, v[i].w & 0x7fff7fffu);
        }
    }
    if (pid < 0 || pid >= p.num_pages) return;  // (the loads did not wait for it)
    __shared__ uint32_t s_top[kAppThreads / 32];
    uint32_t m = max(top & 0xffffu, top >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = m;
    const int64_t cell = pid * p.Hkv + h;
    const float old = p.scale[which][cell];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppThreads / 32; ++i) m = max(m, s_top[i]);
    if (m >= kBf16Inf) {  // (the same in all threads)
        // Infinities and NaN are stored as NaN (e4m3 has no infinity), and the scale is that of the finite values.
        uint32_t fin = 0;
#pragma unroll
        for (int i = 0; i < kAppVecs; ++i) {
            if ((int)threadIdx.x + i * kAppThreads < n) {
                fin = max(fin, append_finite(v[i].x));
                fin = max(fin, append_finite(v[i].y));
                fin = max(fin, append_finite(v[i].z));
                fin = max(fin, append_finite(v[i].w));
            }
        }
        fin = __reduce_max_sync(0xffffffffu, fin);
        __syncthreads();  // the maxima above are read
        if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = fin;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < kAppThreads / 32; ++i) m = max(m, s_top[i]);
    }
    const bool kept = p0 < start;
    float now = append_scale(m);
    if (kept) now = fmaxf(now, old);
    const float inv = 1.f / now;  // exact: a power of two (an old scale that is none rounds)
    uint8_t* out = p.cache[which] + cell * p.page * p.D;

    if (kept && now > old) {
        // the earlier tokens' codes move to the new scale
        const float ratio = old / now;
        const int nk = (int)(lo - p0) * p.D / 8;
        for (int e = threadIdx.x; e < nk; e += kAppThreads) {
            uint2 c = reinterpret_cast<const uint2*>(out)[e];
            uint32_t w[2] = {c.x, c.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = e4m3x2_to(w[i]), z = e4m3x2_to(w[i] >> 16);
                w[i] = e4m3x2_from(a.x * ratio, a.y * ratio) | (e4m3x2_from(z.x * ratio, z.y * ratio) << 16);
            }
            reinterpret_cast<uint2*>(out)[e] = make_uint2(w[0], w[1]);
        }
    }
    uint8_t* dst = out + (lo - p0) * p.D;
#pragma unroll
    for (int i = 0; i < kAppVecs; ++i) {
        const int e = threadIdx.x + i * kAppThreads;
        if (e < n) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                q[k] = e4m3x2_from(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xffff0000u) * inv);
            // tokens of a page follow each other in the cache, D codes each
            reinterpret_cast<uint2*>(dst)[e] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        }
    }
    if (threadIdx.x == 0) p.scale[which][cell] = now;
}

}  // namespace lidx

using namespace lidx;

extern "C" int lidx_cache_append(const void* k, const void* v, const int64_t* ks, const int64_t* vs,
                                 const int32_t* block_table, const int32_t* start, const int32_t* count,
                                 int64_t B, int64_t S, int Hkv, int D, int page, int64_t max_pages,
                                 int64_t num_pages, void* k_cache, void* v_cache, float* k_scale,
                                 float* v_scale, void* stream) {
    if (!k || !v || !ks || !vs || !block_table || !start || !k_cache || !v_cache || !k_scale || !v_scale)
        return LIDX_ERR_NULL;
    const int rc = check_cache(B, S, Hkv, D, page, max_pages, num_pages);
    if (rc) return rc;
    const int64_t J = (S + page - 2) / page + 1;  // pages S tokens can touch
    if (B * J > INT_MAX || Hkv > 65535) return LIDX_ERR_SHAPE;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15u) return LIDX_ERR_ALIGN;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)block_table | (uintptr_t)start | (uintptr_t)count) & 3u)
        return LIDX_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if ((ks[i] | vs[i]) & 7) return LIDX_ERR_ALIGN;
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    AppendParams p;
    p.x[0] = (const uint16_t*)k;
    p.x[1] = (const uint16_t*)v;
    for (int i = 0; i < 3; ++i) {
        p.xs[0][i] = ks[i];
        p.xs[1][i] = vs[i];
    }
    p.cache[0] = (uint8_t*)k_cache;
    p.cache[1] = (uint8_t*)v_cache;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
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
    cache_append_kernel<<<dim3((unsigned)(B * J), (unsigned)Hkv, 2), kAppThreads, 0, (cudaStream_t)stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}
