// cache4_attn.cu -- attention over the paged 4-bit cache: the kernels of units of up to 32 rows, and the widening of pages for
// calls of many rows.
//
// code * 2^x is e4m3 times 32 exactly (cache.cuh), so once widened a tile is the 8-bit cache's, and all that follows is
// cache_attn.cu's: k = (32 scale) * e4m3 and v likewise.  Where that happens goes by how often a key is read:
//   - few rows (decode steps): packed tiles come to shared memory, and warps of the kernel widen them there
//   - a key is read by several units of 128 rows, or by several selections: its page is widened once, into the workspace,
//     and the 8-bit kernels read that
//
// What bounds it.  64 ragged sequences to 32768 keys, 64 heads on 8: 339 us (8 bits 337 us), half of the copy rate.  A tile of 128
// keys takes 1650 cycles, of which the widening warps work 1200: 1490 of a tile's 3830 warp instructions widen.  ALU pipes are 52 %
// busy, issue slots 60 %.  Without widening 252 us.  One sequence of 1024 keys: 10.3 us.
#include "cache_attn_narrow.cuh"

namespace lidx {

cudaError_t attn4_launch(int N, const AttnParams& p, int grid, cudaStream_t st) {
    const CUtensorMap none{};
    if (N == 32) return attn_launch<32, 16, 4>(none, none, p, grid, st);
    if (p.TS * p.G <= 8) return attn_launch<16, 8, 4>(none, none, p, grid, st);
    return attn_launch<16, 16, 4>(none, none, p, grid, st);
}

// Block (place in the table, head): the page's keys and values, a thread a group of 16 dims at a time.
__global__ void __launch_bounds__(256) cache4_widen_pages_kernel(const __grid_constant__ AttnParams p,
                                                                 const __grid_constant__ Attn4Copy to) {
    const int at = blockIdx.x, h = blockIdx.y, b = at / p.max_pages, j = at - b * p.max_pages;
    if ((int64_t)j * p.page >= p.kv_len[b]) return;
    const int pid = p.table[at];
    const bool good = pid >= 0 && pid < p.num_pages;
    if (h == 0 && threadIdx.x == 0) to.table[at] = good ? at : -1;
    if (!good) return;
    const int per = p.D / 16, groups = p.page * per, cell = pid * p.Hkv + h;
    const int64_t src = (int64_t)cell * groups, dst = ((int64_t)at * p.Hkv + h) * groups;
    if (threadIdx.x < 2)
        to.scale[threadIdx.x][(int64_t)at * p.Hkv + h] = (threadIdx.x ? p.vs : p.ks)[cell] * kCache4Unit;
#pragma unroll 2
    for (int i = threadIdx.x; i < 2 * groups; i += 256) {
        const int which = i >= groups, g = which ? i - groups : i, slot = g / per;
        const uint2 c = reinterpret_cast<const uint2*>(p.codes[which])[src + g];
        const uint32_t x = ((uint32_t)p.exps[which][(int64_t)cell * p.page + slot] >> (4 * (g - slot * per))) & 15u;
        uint32_t lo, hi;
        cache4_table(x, lo, hi);
        const uint2 a = cache4_widen(c.x, lo, hi), z = cache4_widen(c.y, lo, hi);
        reinterpret_cast<uint4*>(to.cache[which])[dst + g] = make_uint4(a.x, a.y, z.x, z.y);
    }
}

cudaError_t attn4_widen_pages(const AttnParams& p, const Attn4Copy& to, cudaStream_t st) {
    cache4_widen_pages_kernel<<<dim3((unsigned)(p.B * p.max_pages), (unsigned)p.Hkv), 256, 0, st>>>(p, to);
    return cudaGetLastError();
}

LIDX_STATUS_READER(status_cache4_attn)

}  // namespace lidx
