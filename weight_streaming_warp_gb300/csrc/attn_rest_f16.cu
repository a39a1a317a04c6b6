// attn_rest_f16.cu -- the paged decode attention behind a shared prefix, over binary16 pages (one
// translation unit each: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_F16, false, true)
}  // namespace paged
}  // namespace wsw
