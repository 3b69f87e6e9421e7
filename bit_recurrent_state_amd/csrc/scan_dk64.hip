// scan_dk64.hip — the scan's kernels for dk = 64.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk64(const Params& p, hipStream_t s) { return forward<64>(p, s); }
hipError_t backward_dk64(const Params& p, hipStream_t s) { return backward<64>(p, s); }

}  // namespace qscan
