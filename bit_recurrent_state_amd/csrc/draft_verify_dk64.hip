// draft_verify_dk64.hip — the readout of drafted tokens for key dimension dk = 64, one
// gate a token (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {

hipError_t verify_dk64(const Params& p, hipStream_t s) {
  return qs::vector_decay(p.mixer) ? verify_channels_dk64(p, s) : verify_tokens<64>(p, s);
}

}  // namespace qdraft
