// attn_rest_bf16.cu -- the paged decode attention behind a shared prefix, over bf16 pages (one
// translation unit each: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_BF16, false, true)
}  // namespace paged
}  // namespace wsw
