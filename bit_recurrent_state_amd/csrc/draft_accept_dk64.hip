// draft_accept_dk64.hip — the accepted path's way into the state for key dimension
// dk = 64 (see draft_accept.h).

#include "draft_accept.h"

namespace qdraft {
hipError_t accept_dk64(const Params& p, hipStream_t s) { return accept<64>(p, s); }
}  // namespace qdraft
