// attn_paged_bf16.cu -- the paged decode attention over bf16 pages (one translation unit per
// cache type: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_BF16, false, false)
}  // namespace paged
}  // namespace wsw
