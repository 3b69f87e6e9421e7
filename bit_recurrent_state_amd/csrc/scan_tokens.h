// scan_tokens.h — short sequences, token by token: single new tokens of running
// sequences, and sequences with none.
//
// What a sequence of a few tokens costs is its state, read once and written
// once; the chunks' fixed work would be several times that.  A wave takes 8
// value rows, 8 lanes a row, and keeps them in registers over the tokens: FP32
// throughout, one multiply and two fused multiply-adds per element and token,
// dot products summed over the row's lanes.
// 26 us for one token of 64 sequences, 16 heads of 128 x 128: 137 MB at 5.3 TB/s,
// bound by memory.

#pragma once

#include "scan_prep.h"

namespace qscan {

// Workgroups of it: one per sequence, head and 32 value rows.
__host__ __device__ inline int64_t token_blocks(const Params& p) {
  return p.some_short ? (int64_t)p.batch * p.heads * ((p.dv + 31) / 32) : 0;
}

template <int DK, bool VEC, bool DELTA>
__device__ __forceinline__ void take_tokens(const Params& p, int64_t b) {
  constexpr int Q = DK / 32;  // groups of 4 channels: channel 32 q + 4 (lane & 7)
  const int nb = (p.dv + 31) / 32;
  const int64_t nh = b / nb;
  const int n = (int)(nh / p.heads), h = (int)(nh % p.heads);
  const int64_t o0 = offset_of(p, n), o1 = offset_of(p, n + 1);
  const int64_t left = o1 - o0;
  if (left > p.short_len) return;
  const int len = left > 0 ? (int)left : 0;
  const int lane = threadIdx.x & 63, l = lane & 7;
  const int v = (int)(b % nb) * 32 + (threadIdx.x >> 6) * 8 + (lane >> 3);
  const bool in = v < p.dv;
  const int hq = h / (p.heads / p.heads_qk);
  const bool qeven = p.qs % 4 == 0, keven = p.ks % 4 == 0;
  const int64_t st = (nh * p.dv + (in ? v : p.dv - 1)) * DK + 4 * l;
  f32x4 S[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q)
    S[q] = p.s0 ? *reinterpret_cast<const f32x4*>(p.s0 + st + 32 * q) : f32x4{0, 0, 0, 0};
  // a token's inputs, loaded one token ahead
  u32x4 k[Q], x[Q];
  float ga = 0.0f, beta = 1.0f;
  f32x4 g[VEC ? Q : 1];
  uint32_t vr[1];
  auto load = [&](int i) {
    const int64_t row = o0 + i;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      k[q] = load4(p.k, row * p.ks + (int64_t)hq * DK + 32 * q + 4 * l, p.dtype, keven);
      x[q] = load4(p.q, row * p.qs + (int64_t)hq * DK + 32 * q + 4 * l, p.dtype, qeven);
      if (VEC)
        g[q] = *reinterpret_cast<const f32x4*>(p.g + (row * p.heads + h) * DK + 32 * q + 4 * l);
    }
    if (!VEC) ga = p.g[row * p.heads + h];
    if (p.beta) beta = p.beta[row * p.heads + h];
    const int64_t at[1] = {row * p.vs + (int64_t)h * p.dv + (in ? v : p.dv - 1)};
    load_raw<1>(p.v, at, p.dtype, vr);
  };
  if (len > 0) load(0);
  for (int i = 0; i < len; ++i) {
    float kc[Q][4], xc[Q][4], a[VEC ? Q : 1][4];
    const float bc = beta;
    float w = from_raw(vr[0], p.dtype);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      widen4(k[q], p.dtype, kc[q]);
      widen4(x[q], p.dtype, xc[q]);
      if (VEC) {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[VEC ? q : 0][e] = fast_exp(gate(g[VEC ? q : 0][e]));
      }
    }
    if (!VEC) a[0][0] = fast_exp(gate(ga));
    if (i + 1 < len) load(i + 1);
    float u = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[q][e] *= VEC ? a[VEC ? q : 0][e] : a[0][0];
        if (DELTA) u = fmaf(S[q][e], kc[q][e], u);
      }
    if (DELTA) w -= sum8(u);
    w *= bc;
    float o = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[q][e] = fmaf(w, kc[q][e], S[q][e]);
        o = fmaf(S[q][e], xc[q][e], o);
      }
    o = sum8(o);
    if (p.o && in && l == 0) store_elem(p.o, (o0 + i) * p.os + (int64_t)h * p.dv + v, p.dtype, o);
  }
  if (p.s1 && in) {
#pragma unroll
    for (int q = 0; q < Q; ++q) *reinterpret_cast<f32x4*>(p.s1 + st + 32 * q) = S[q];
  }
}

template <int DK, bool VEC, bool DELTA>
__global__ void __launch_bounds__(256) tokens_kernel(Params p) {
  take_tokens<DK, VEC, DELTA>(p, blockIdx.x);
}

// One gate per token: the operands of longer sequences' chunks are as
// independent and come from the same launch.  One launch less takes 2 to 4 us
// off a call: one token of 64 sequences, 16 heads of 128 x 128, 40.6 -> 39.0 us.
template <int DK, bool DELTA>
__global__ void __launch_bounds__(256) tokens_operands_kernel(Params p) {
  const int64_t tb = token_blocks(p), b = blockIdx.x;
  if (b < tb)
    take_tokens<DK, false, DELTA>(p, b);
  else
    take_operands<DK, false>(p, (int)((b - tb) % p.nslots), (int)((b - tb) / p.nslots));
}

}  // namespace qscan
