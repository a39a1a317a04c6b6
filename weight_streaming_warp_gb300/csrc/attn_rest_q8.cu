// attn_rest_q8.cu -- the paged decode attention behind a shared prefix, over q8_0 pages (one
// translation unit each: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_Q8_0, false, true)
}  // namespace paged
}  // namespace wsw
