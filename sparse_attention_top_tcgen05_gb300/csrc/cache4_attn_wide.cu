// cache4_attn_wide.cu -- the kernels of units of 33 to 128 rows over the 4-bit cache.
#include "cache_attn_wide.cuh"

namespace lidx {

cudaError_t attn4_launch_wide(const AttnParams& p, int grid, cudaStream_t st) {
    const CUtensorMap none{};
    return wide_launch_rows<4>(none, none, p, grid, st);
}

LIDX_STATUS_READER(status_cache4_attn_wide)

}  // namespace lidx
