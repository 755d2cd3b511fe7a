// cache_attn_wide.cu -- the kernels of units of 33 to 128 rows over the 8-bit cache.
#include "cache_attn_wide.cuh"

namespace lidx {

cudaError_t attn_launch_wide(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid, cudaStream_t st) {
    return wide_launch_rows<8>(mk, mv, p, grid, st);
}

LIDX_STATUS_READER(status_cache_attn_wide)

}  // namespace lidx
