// cache_attn.cu -- attention over a paged cache of 8-bit keys and values.
//
//     o = sum_t p_t v_t,  p = softmax over the row's keys of softmax_scale * q . k_t
// with k_t = code * scale of its page and head, v_t likewise.  One pass over the keys with the running
// maximum m and sum l of the softmax:
//     m' = max(m, max_t s_t);  l = l e^(m - m') + sum_t e^(s_t - m');  o = o e^(m - m') + sum_t e^(s_t - m') v_t
//
// One block per (row, query head): a thread takes one key of a tile of 128, then one output dim.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <climits>

#include "cache.cuh"
#include "kernels.h"
#include "lidx.h"

namespace lidx {

struct AttnParams {
    const uint16_t* q;
    int64_t qs[3];
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_pos;  // nullable
    const int32_t* idx;    // nullable
    int64_t num_pages;
    int B, S, Hq, Hkv, D, page, max_pages, ratio, topk;
    float scale;
    uint16_t* out;
    float* lse;  // nullable
};

// Row (b, s) sees keys [0, end).
__device__ __forceinline__ int attn_end(const AttnParams& p, int b, int s) {
    int n = p.kv_len[b];
    const int cap = p.max_pages * p.page;
    n = n < 0 ? 0 : (n > cap ? cap : n);
    if (p.q_pos) {
        const int64_t seen = (int64_t)p.q_pos[b] + s + 1;
        const int64_t e = seen > 0 ? seen / p.ratio : 0;
        n = e < n ? (int)e : n;
    }
    return n;
}

constexpr int kAttnThreads = 128;

__global__ void __launch_bounds__(kAttnThreads) cache_attn_kernel(const AttnParams p) {
    __shared__ float sq[kCacheMaxD], sw[kAttnThreads], sred[8];
    __shared__ int64_t srow[kAttnThreads];
    const int hq = blockIdx.x % p.Hq, h = hq / (p.Hq / p.Hkv);
    const int64_t row = blockIdx.x / p.Hq;
    const int b = (int)(row / p.S), s = (int)(row % p.S), tid = threadIdx.x;
    const uint16_t* q = p.q + b * p.qs[0] + s * p.qs[1] + hq * p.qs[2];
    if (tid < p.D) sq[tid] = __uint_as_float((uint32_t)q[tid] << 16) * p.scale;
    const int end = attn_end(p, b, s), n = p.idx ? p.topk : end;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int t0 = 0; t0 < n; t0 += kAttnThreads) {
        __syncthreads();
        int t = t0 + tid < n ? t0 + tid : -1;
        if (p.idx && t >= 0) {
            t = p.idx[row * p.topk + t];
            if (t >= end) t = -1;
        }
        float x = -INFINITY, vscale = 0.f;
        srow[tid] = -1;
        if (t >= 0) {
            const int64_t pid = p.table[(int64_t)b * p.max_pages + t / p.page];
            if (pid >= 0 && pid < p.num_pages) {
                const int64_t cell = pid * p.Hkv + h, at = (cell * p.page + t % p.page) * p.D;
                const uint16_t* k = reinterpret_cast<const uint16_t*>(p.kc + at);
                float dot = 0.f;
                for (int d = 0; d < p.D; d += 2) {
                    const float2 kk = e4m3x2_to(k[d / 2]);
                    dot += sq[d] * kk.x + sq[d + 1] * kk.y;
                }
                x = dot * p.ks[cell];
                vscale = p.vs[cell];
                srow[tid] = at;
            }
        }
        float mt = x;
        for (int i = 16; i; i >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, i));
        if ((tid & 31) == 0) sred[tid >> 5] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(sred[0], sred[1]), fmaxf(sred[2], sred[3]));
        const float mn = fmaxf(m, mt);
        if (mn == -INFINITY) continue;  // nothing seen yet (uniform over the block)
        const float w = x == -INFINITY ? 0.f : expf(x - mn), fade = m == -INFINITY ? 0.f : expf(m - mn);
        float ws = w;
        for (int i = 16; i; i >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, i);
        if ((tid & 31) == 0) sred[4 + (tid >> 5)] = ws;
        sw[tid] = w * vscale;
        __syncthreads();
        l = l * fade + (sred[4] + sred[5] + sred[6] + sred[7]);
        m = mn;
        if (tid < p.D) {
            o *= fade;
            for (int i = 0; i < kAttnThreads; ++i)
                if (srow[i] >= 0) o += sw[i] * e4m3x2_to(p.vc[srow[i] + tid]).x;
        }
    }
    if (tid < p.D)
        reinterpret_cast<__nv_bfloat16*>(p.out)[(row * p.Hq + hq) * p.D + tid] =
            __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
    if (p.lse && tid == 0) p.lse[row * p.Hq + hq] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace lidx

using namespace lidx;

extern "C" {

size_t lidx_cache_attn_workspace_bytes(int64_t B, int64_t S, int Hq, int Hkv, int D, int topk) {
    (void)B, (void)S, (void)Hq, (void)Hkv, (void)D, (void)topk;
    return 0;
}

int lidx_cache_attn(const void* q, const int64_t* qs, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    const int32_t* kv_len, const int32_t* q_pos, const int32_t* topk_indices,
                    int64_t B, int64_t S, int Hq, int Hkv, int D, int page, int64_t max_pages,
                    int64_t num_pages, int compress_ratio, int topk, float softmax_scale, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !qs || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_len || !out)
        return LIDX_ERR_NULL;
    const int rc = check_cache(B, S, Hkv, D, page, max_pages, num_pages);
    if (rc) return rc;
    if (Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || B * S > INT_MAX || B * S * Hq > INT_MAX) return LIDX_ERR_SHAPE;
    if (compress_ratio < 1 || !isfinite(softmax_scale) || (topk_indices && (topk < 1 || topk > (1 << 20))))
        return LIDX_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15u) return LIDX_ERR_ALIGN;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)block_table | (uintptr_t)kv_len |
         (uintptr_t)q_pos | (uintptr_t)topk_indices | (uintptr_t)lse) & 3u)
        return LIDX_ERR_ALIGN;
    if ((qs[0] | qs[1] | qs[2]) & 7) return LIDX_ERR_ALIGN;
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    (void)workspace, (void)workspace_bytes;
    AttnParams p;
    p.q = (const uint16_t*)q;
    for (int i = 0; i < 3; ++i) p.qs[i] = qs[i];
    p.kc = (const uint8_t*)k_cache;
    p.vc = (const uint8_t*)v_cache;
    p.ks = k_scale;
    p.vs = v_scale;
    p.table = block_table;
    p.kv_len = kv_len;
    p.q_pos = q_pos;
    p.idx = topk_indices;
    p.num_pages = num_pages;
    p.B = (int)B;
    p.S = (int)S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.page = page;
    p.max_pages = (int)max_pages;
    p.ratio = compress_ratio;
    p.topk = topk;
    p.scale = softmax_scale;
    p.out = (uint16_t*)out;
    p.lse = lse;
    cache_attn_kernel<<<(unsigned)(B * S * Hq), kAttnThreads, 0, (cudaStream_t)stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
