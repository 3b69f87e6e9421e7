// draft_verify_dk128.hip — the readout of drafted tokens for key dimension dk = 128, one
// gate a token (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {

hipError_t verify_dk128(const Params& p, hipStream_t s) {
  return qs::vector_decay(p.mixer) ? verify_channels_dk128(p, s) : verify_tokens<128>(p, s);
}

}  // namespace qdraft
