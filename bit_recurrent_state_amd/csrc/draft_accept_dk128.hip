// draft_accept_dk128.hip — the accepted path's way into the state for key dimension
// dk = 128 (see draft_accept.h).

#include "draft_accept.h"

namespace qdraft {
hipError_t accept_dk128(const Params& p, hipStream_t s) { return accept<128>(p, s); }
}  // namespace qdraft
