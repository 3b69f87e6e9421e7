// linear_launch.h — parameters of the kernels of products with 4-bit weights.

#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace qlinear {

constexpr int kOut = 16, kIn = 128;  // a tile of weights: 1 KB of codes

struct Params {
  int inputs, outputs, group, dtype;
  int out_tiles, in_tiles;
  int64_t rows, xs;
  const void* x;
  const uint32_t* packed;
  const float *scales, *bias;
  void* y;
  // laying weights out
  const int8_t* codes;
  const float* group_scales;
  const void* weights;
  uint32_t* packed_out;
  float* scales_out;
};

hipError_t multiply(const Params& p, hipStream_t s);
hipError_t pack(const Params& p, hipStream_t s);
hipError_t quantize(const Params& p, hipStream_t s);

}  // namespace qlinear
