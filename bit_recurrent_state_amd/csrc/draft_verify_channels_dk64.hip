// draft_verify_channels_dk64.hip — the readout of drafted tokens for key dimension
// dk = 64, a gate for each key channel (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {

hipError_t verify_channels_dk64(const Params& p, hipStream_t s) { return verify_channels<64>(p, s); }

}  // namespace qdraft
