// draft_verify_channels_dk128.hip — the readout of drafted tokens for key dimension
// dk = 128, a gate for each key channel (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {

hipError_t verify_channels_dk128(const Params& p, hipStream_t s) { return verify_channels<128>(p, s); }

}  // namespace qdraft
