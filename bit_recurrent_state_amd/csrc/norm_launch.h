// norm_launch.h — parameters of the block norm's kernels.

#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace qnorm {

struct Params {
  int64_t rows;   // tokens * groups
  int groups, width, act, each;
  float eps;
  int64_t xs, gs, rs;  // elements between tokens
  const void *x, *gate, *residual, *dr, *dh;
  const float *weight, *scale, *next_weight;
  void *r, *h, *dx, *dgate, *dresidual;
  float *dweight, *dscale, *dnext_weight;
  int has_h;
  // launch plan: teams of `team` threads take rows team, team + teams, ...
  int team;        // threads per row
  int block;       // threads of a workgroup
  int vectors;     // blocks of 8 values per thread
  int wide;        // rows take whole workgroups
  int aligned;     // 16-byte accesses reach every row
  int64_t teams;   // a multiple of groups where weights differ by group
  float* part;     // [3][partials][width]: dweight, dscale, dnext_weight
  int64_t partials;
};

hipError_t forward(const Params& p, int dtype, hipStream_t s);
hipError_t backward(const Params& p, int dtype, hipStream_t s);

}  // namespace qnorm
