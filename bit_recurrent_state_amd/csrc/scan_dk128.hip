// scan_dk128.hip — the scan's kernels for dk = 128.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk128(const Params& p, hipStream_t s) { 
  if (p.vblock == 64) return forward<128, 4>(p, s);
  return p.vblock == 16 ? forward<128, 1>(p, s) : forward<128, 2>(p, s);
 }
hipError_t backward_dk128(const Params& p, hipStream_t s) { 
  return p.vblock == 16 ? backward<128, 1>(p, s) : backward<128, 2>(p, s);
 }

}  // namespace qscan
