// scan_dk64.hip — the scan's kernels for dk = 64.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk64(const Params& p, hipStream_t s) { 
  if (p.vblock == 64) return forward<64, 4>(p, s);
  return p.vblock == 16 ? forward<64, 1>(p, s) : forward<64, 2>(p, s);
 }
hipError_t backward_dk64(const Params& p, hipStream_t s) { 
  return p.vblock == 16 ? backward<64, 1>(p, s) : backward<64, 2>(p, s);
 }

}  // namespace qscan
