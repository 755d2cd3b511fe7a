// cache4_attn.cu -- the kernels of units of up to 32 rows over the 4-bit cache.
#include "cache_attn_narrow.cuh"

namespace lidx {

cudaError_t attn4_launch(int N, const AttnParams& p, int grid, cudaStream_t st) {
    const CUtensorMap none{};
    if (N == 32) return attn_launch<32, 16, 4>(none, none, p, grid, st);
    if (p.TS * p.G <= 8) return attn_launch<16, 8, 4>(none, none, p, grid, st);
    return attn_launch<16, 16, 4>(none, none, p, grid, st);
}

LIDX_STATUS_READER(status_cache4_attn)

}  // namespace lidx
