// group_norm_launch.h — parameters of the group norm's kernels.

#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace qnorm {

enum { PLAIN = 0, GATE = 1, GATE_FIRST = 2, ACTIVATE = 3 };

struct GroupParams {
  int64_t rows;  // tokens * groups
  int groups, width, act, mode, center, shared;
  float eps;
  int64_t xs, gs;  // elements between tokens
  const void *x, *gate, *dy;
  const float *weight, *bias;
  void *y, *dx, *dgate;
  float *dweight, *dbias;
  // launch plan: teams of `team` threads take rows team, team + teams, ...
  int team;       // threads per row
  int block;      // threads of a workgroup
  int vectors;    // blocks of 8 values per thread
  int wide;       // rows take whole workgroups
  int aligned;    // 16-byte accesses reach every row
  int64_t teams;  // a multiple of groups
  float* part;    // [2][partials][width]: dweight, dbias
  int64_t partials;
};

hipError_t group_forward(const GroupParams& p, int dtype, hipStream_t s);
hipError_t group_backward(const GroupParams& p, int dtype, hipStream_t s);

}  // namespace qnorm
