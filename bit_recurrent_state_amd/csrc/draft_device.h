// draft_device.h — what the kernels of drafted tokens share: which row is a
// node, and its way to the stored state.

#pragma once

#include "draft_launch.h"
#include "qstate_value.h"
#include "scan_device.h"

namespace qdraft {

using qscan::f32x4;
using qscan::Frag;
using qscan::u32x2;
using qscan::u32x4;

// The parent that row t names, or -2 where the row is none by itself.
__device__ __forceinline__ int named_parent(const Params& p, int n, int t) {
  if (t >= p.tokens) return -2;
  const int par = p.parents ? p.parents[(int64_t)n * p.tokens + t] : t - 1;
  return par >= -1 && par < t ? par : -2;
}

// Row (n, t) of [batch][T], as an index into packed rows.
__device__ __forceinline__ int64_t row_of(const Params& p, int n, int t) {
  return (int64_t)n * p.tokens + t;
}

}  // namespace qdraft
