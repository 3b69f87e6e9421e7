// draft_verify_dk256.hip — the readout of drafted tokens for key dimension dk = 256, one
// gate a token (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {

hipError_t verify_dk256(const Params& p, hipStream_t s) {
  return qs::vector_decay(p.mixer) ? verify_channels_dk256(p, s) : verify_tokens<256>(p, s);
}

}  // namespace qdraft
