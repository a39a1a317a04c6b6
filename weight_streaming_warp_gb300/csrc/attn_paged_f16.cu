// attn_paged_f16.cu -- the paged decode attention over binary16 pages (one translation unit per
// cache type: they compile side by side).
#include "attn_paged.cuh"

namespace wsw {
namespace paged {
WSW_PAGED_TYPE(WSW_F16, false)
}  // namespace paged
}  // namespace wsw
