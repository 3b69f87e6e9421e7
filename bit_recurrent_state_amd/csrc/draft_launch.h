// draft_launch.h — what the host side (draft_api.cpp) hands to the kernels of
// drafted tokens: one parameter block, and one launcher per dk.

#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "qstate_launch.h"

namespace qdraft {

// Nodes of a sequence: what a workgroup's LDS holds.
constexpr int most_tokens(int dk) { return dk > 128 ? 32 : 64; }

// Verify with 64 value columns a workgroup where the LDS does not hold the operands of 128: split rows
// of more than 48 nodes.
constexpr bool narrow(int dk, int tokens, bool split, bool vector) {
  return dk == 128 && tokens > 48 && split && !vector;
}

struct Params {
  int tokens, heads_qk, mixer, dtype, fp32, rounding;
  int64_t qs, ks, vs;  // row strides in elements
  const void *q, *k, *v;
  const float *g, *beta;
  const int32_t *parents, *last;
  void* o;
  const float* writes_in;
  float* writes;
  int direct;     // bfloat16 q and k, rows on 16 bytes: they enter the products as they are
  int pairs;      // two neighbouring values of o and writes are one access
  int vpairs;     // and of v
  int columns;    // verify: value columns of a workgroup, 64 or 128
  int blocks;     // workgroups of a head
  int rows;       // accept: value rows of a workgroup
  qs::KParams s;  // the state: codes, scales, sizes, widths, random bits
};

hipError_t verify_dk64(const Params& p, hipStream_t s);
hipError_t verify_channels_dk64(const Params& p, hipStream_t s);
hipError_t verify_dk128(const Params& p, hipStream_t s);
hipError_t verify_channels_dk128(const Params& p, hipStream_t s);
hipError_t verify_dk256(const Params& p, hipStream_t s);
hipError_t verify_channels_dk256(const Params& p, hipStream_t s);
hipError_t accept_dk64(const Params& p, hipStream_t s);
hipError_t accept_dk128(const Params& p, hipStream_t s);
hipError_t accept_dk256(const Params& p, hipStream_t s);

}  // namespace qdraft
