// draft_verify_dk128.hip — the readout of drafted tokens for key dimension dk = 128
// (see draft_verify.h).

#include "draft_verify.h"

namespace qdraft {
hipError_t verify_dk128(const Params& p, hipStream_t s) { return verify<128>(p, s); }
}  // namespace qdraft
