// scan_dk128.hip — the scan's kernels for dk = 128.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk128(const Params& p, hipStream_t s) { return forward<128>(p, s); }
hipError_t backward_dk128(const Params& p, hipStream_t s) { return backward<128>(p, s); }

}  // namespace qscan
