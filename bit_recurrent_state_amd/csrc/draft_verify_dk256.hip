// draft_verify_dk256.hip — the readout of drafted tokens for key dimension dk = 256
// (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {
hipError_t verify_dk256(const Params& p, hipStream_t s) { return verify<256>(p, s); }
}  // namespace qdraft
