// attn_prefix_q8.cu -- the attention over shared prefixes for one cache type (one translation unit
// each: they compile side by side).
#include "attn_prefix.cuh"

namespace wsw {
namespace prefix {

template <>
cudaError_t launch_prefix<WSW_Q8_0>(const Args &a, int row_tiles, cudaStream_t s, int ctas) {
    if (a.dtype == WSW_F32) return WSW_PREFIX_ONE(WSW_Q8_0, 2, 1);
    return row_tiles == 2 ? WSW_PREFIX_ONE(WSW_Q8_0, 1, 2) : WSW_PREFIX_ONE(WSW_Q8_0, 1, 1);
}

}  // namespace prefix
}  // namespace wsw
