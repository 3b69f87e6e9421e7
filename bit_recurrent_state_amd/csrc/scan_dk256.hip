// scan_dk256.hip — the scan's kernels for dk = 256.

#include "scan_dk.h"

namespace qscan {

hipError_t forward_dk256(const Params& p, hipStream_t s) { 
  return p.vblock == 16 ? forward<256, 1>(p, s) : forward<256, 2>(p, s);
 }
hipError_t backward_dk256(const Params& p, hipStream_t s) { 
  return p.vblock == 16 ? backward<256, 1>(p, s) : backward<256, 2>(p, s);
 }

}  // namespace qscan
