// draft_accept_dk256.hip — the accepted path's way into the state for key dimension
// dk = 256 (see draft_accept.h).

#include "draft_accept.h"

namespace qdraft {
hipError_t accept_dk256(const Params& p, hipStream_t s) { return accept<256>(p, s); }
}  // namespace qdraft
