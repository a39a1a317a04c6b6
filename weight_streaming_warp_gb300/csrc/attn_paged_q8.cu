// attn_paged_q8.cu -- the paged decode attention over q8_0 pages (one translation unit per
// cache type: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_Q8_0, false, false)
}  // namespace paged
}  // namespace wsw
