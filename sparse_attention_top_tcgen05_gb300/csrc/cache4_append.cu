// cache4_append.cu -- new keys and values into the paged 4-bit cache (rope_append.cuh), and that cache as an 8-bit one.
#include "rope_append.cuh"

namespace lidx {

cudaError_t cache4_append_launch(const RopeAppendParams& p, int64_t B, cudaStream_t st) { return ra_launch_bits<4>(p, B, st); }

// Codes and exponents -> e4m3 of number / 32.  Eight threads a slot, one a group of 16 dims.  Of all pages of
// a cache of 4 x 4874 tokens, 8 heads of 128: 12 us behind the append, 61 % of the ALU pipes.
struct WidenParams {
    const uint2* codes[2];
    const int32_t* exps[2];
    uint4* out[2];
    int64_t slots;
    int per;  // groups of a slot
};
__global__ void __launch_bounds__(256) cache4_widen_kernel(const __grid_constant__ WidenParams p) {
    const int which = blockIdx.y, g = threadIdx.x & 7;
    if (g >= p.per) return;
    uint32_t f16 = 16, f65536 = 65536;
    asm volatile("" : "+r"(f16), "+r"(f65536));
#pragma unroll 2
    for (int64_t slot = blockIdx.x * 32ll + (threadIdx.x >> 3); slot < p.slots; slot += gridDim.x * 32ll) {
        const int64_t i = slot * p.per + g;
        const uint2 c = p.codes[which][i];
        const uint32_t x = ((uint32_t)p.exps[which][slot] >> (4 * g)) & 15u;
        uint32_t lo, hi;
        cache4_table(x, lo, hi);
        const uint2 a = cache4_widen_mul(c.x, lo, hi, f16, f65536), b = cache4_widen_mul(c.y, lo, hi, f16, f65536);
        p.out[which][i] = make_uint4(a.x, a.y, b.x, b.y);
    }
}

}  // namespace lidx

using namespace lidx;

extern "C" int lidx_cache4_to_8(const void* k_cache, const void* v_cache, const int32_t* k_exps, const int32_t* v_exps, int Hkv, int D,
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
    p.slots = num_pages * Hkv * page;
    const int64_t blocks = (p.slots + 31) / 32, cap = (int64_t)current_sms() * 32;
    cache4_widen_kernel<<<dim3((unsigned)(blocks < cap ? blocks : cap), 2), 256, 0, (cudaStream_t)stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

