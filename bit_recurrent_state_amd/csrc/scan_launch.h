// scan_launch.h — what the host side (scan_api.cpp) hands to the scan's
// kernels: one parameter block with the caller's arrays and the workspace's
// regions, and one launcher per dk.

#pragma once

#include <hip/hip_runtime_api.h>
#include <hip/hip_vector_types.h>

#include <cstdint>

namespace qscan {

constexpr int kChunk = 64;  // tokens of a chunk
constexpr int kTerms = 3;   // bfloat16 terms of an FP32 operand
// Longest sequence that is taken token by token.  A token costs its own steps
// there, a chunk the same for 1 and for 64 tokens: 96 ragged sequences of up to
// 33 tokens (GLA, 16 heads of 128 x 128, FP32) take 232 us with 8 and 418 us
// with 32.
constexpr int kShort = 8;
constexpr float kFarDecay = 24.0f;  // largest decay of a chunk, as a logarithm, that is divided out

// Workspace operands are bfloat16 terms, a plane per term, in tiles of 16 rows
// x 32 columns (scan_device.h); the sizes below are rows x columns.
// "slot" is a chunk of a sequence: sequence n owns the slots from
// offsets[n] / kChunk + n on, so slots need no prefix sums and never overlap.
struct Params {
  int batch, heads, heads_qk, dk, dv, mixer, dtype;
  int direct;    // q and k enter the products as the caller's bfloat16 rows, one term
  int short_len; // sequences up to this length go to tokens_kernel (forward)
  int some_short, some_long;  // whether there may be sequences up to that length, and beyond
  int nslots;    // upper bound of the slots in use
  int nvb;       // blocks of dv columns of one head
  int vblock;    // dv columns of a block
  int64_t tokens;
  int64_t qs, ks, vs, os;  // row strides in elements
  const void *q, *k, *v, *dO;
  const float *g, *beta;
  const int64_t* offsets;
  const float *s0, *ds1;
  void *o, *dq, *dkk, *dv_out;
  float *s1, *dg, *dbeta, *ds0;
  // workspace
  int4* chunks;              // [slot] sequence (-1: none), chunk of it, tokens, first row
  float* sink;               // [64] where lanes without an output write
  float* rows;               // [slot][head][5][kChunk]: exp(c), exp(c_end - c), beta, c (double)
  float* decay;              // [slot][head][dk] exp(c_end) (per-channel gates)
  uint16_t *qrow, *krow;     // [slot][head|head_qk][term][kChunk][dk]
  uint16_t *knrow;           // per-channel gates: k exp(-c)
  uint32_t* far;             // [slot][head] per-channel gates: a channel decays beyond kFarDecay
  uint16_t *korow;           // per-channel gates, backward: k exp(c_end - c)
  uint16_t *kt, *qt, *ket, *knt;  // [slot][head|head_qk][term][dk][kChunk]
  uint16_t *kt_raw, *qt_raw; // per-channel gates, backward: unscaled, per q/k head
  float *sfx, *pfx;          // per-channel gates, backward: [slot][head][dk][kChunk], decays
                             // from the token to the chunk's end, and from its start (of its
                             // block of 16, where the chunk decays far)
  uint16_t *a, *t;           // [slot][head][kTerms][kChunk][kChunk]
  uint16_t *at, *t2t;        // backward: transposed A, transposed (I + beta L)^-1
  uint16_t* dop;             // [slot][head][term][kChunk][dvp] d_o as planes of plain rows
  float *u, *y;              // [slot][head][kChunk][dvp]
  float *sc, *xc;            // [slot][head][dk][dvp]: states / state gradients
  float* dbpart;             // [nvb][slot][head][kChunk]
  float *dqpart, *dkpart;    // [slot][head][kChunk][dk] when heads share q and k
  int dvp;                   // dv rounded up to 32
  int dop_terms;
};

hipError_t forward_dk64(const Params& p, hipStream_t s);
hipError_t forward_dk128(const Params& p, hipStream_t s);
hipError_t forward_dk256(const Params& p, hipStream_t s);
hipError_t backward_dk64(const Params& p, hipStream_t s);
hipError_t backward_dk128(const Params& p, hipStream_t s);
hipError_t backward_dk256(const Params& p, hipStream_t s);

}  // namespace qscan
