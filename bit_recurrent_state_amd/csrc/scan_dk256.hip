// scan_dk256.hip — the scan's kernels for dk = 256.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk256(const Params& p, hipStream_t s) { return forward<256>(p, s); }
hipError_t backward_dk256(const Params& p, hipStream_t s) { return backward<256>(p, s); }

}  // namespace qscan
