// rope_append.cu -- the entries that write new keys and values with the norm and the rotary positions of the keys on the way
// (rope_append.cuh), and the kernels of the 8-bit cache.
#include "rope_append.cuh"

namespace lidx {

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
    p.page_shift = page == 16 ? 4 : (page == 32 ? 5 : (page == 64 ? 6 : 7));
    // A block of several heads computes its tokens' angles once and loads a head while it converts the one before, so it takes
    // as many as leave four blocks an SM; a few tokens are a chain of latencies, and their blocks take one.
    p.heads = 1;
    if (S >= 16)
        while (p.heads < 8 && p.heads * 2 <= Hkv && B * J * ((Hkv + 2 * p.heads - 1) / (2 * p.heads)) * 2 >= 4 * (int64_t)current_sms())
            p.heads *= 2;
    p.pairs = rope_div(p.r.R / 2);
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = bits == 8 ? ra_launch_bits<8>(p, B, st) : cache4_append_launch(p, B, st);
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

}  // extern "C"
