// draft_accept.h — the stored state behind the accepted path:
//
//   S' = S e^(c_end) + sum_j w_j (k_j e^(c_end - c_j))^T   over the path's nodes
//
// with the w_j that the readout left.  A workgroup takes up to 128 value rows of
// a head: the path's scaled keys and its writes go to LDS, then waves go over the
// rows with the lanes, the dequantization and the quantizer of the single-token
// step (qstate_device.h, qstate_value.h), so that a state is read and written once.

#pragma once

#include "draft_device.h"

namespace qdraft {

// Columns of a key in LDS: 4 floats of padding behind 16, as loadv_padded reads them.
constexpr int padded(int c) { return c + c / 16 * 4; }

template <int DK, bool VEC, int LEN>
struct alignas(16) PathLds {
  float k[LEN][padded(DK)];
  float w[LEN][128];
  float decay[VEC ? padded(DK) : 4];
  int node[64];    // the path's nodes, the last one first
  float f[64];     // one gate a token: the decay from behind node j to the end
};

// d += w k^T over the path for a lane's E columns of one row.
template <int E, class D>
__device__ __forceinline__ void add_path(const D& lds, int len, int row, int col0, float (&d)[E]) {
  for (int j = 0; j < len; ++j) {
    const float w = lds.w[j][row];
    float k[E];
    qs::loadv_padded(&lds.k[j][padded(col0)], k);
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = fmaf(w, k[e], d[e]);
  }
}

// The rows r0 .. r0 + rows - 1 of a head of one width.
template <int DK, int BITS, int G, int RND, bool VEC, class D>
__device__ __forceinline__ void accept_rows(const Params& p, const D& lds, int n, int h, int len,
                                            int r0, int rows) {
  using Gm = qs::Geo<DK, BITS>;
  constexpr int E = Gm::E, LPR = Gm::LPR, RPW = Gm::RPW;
  constexpr bool two_groups = G < E;
  constexpr int LPG = two_groups ? 0 : G / E;
  constexpr int ngr = DK / G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane % LPR, rsub = lane / LPR, col0 = lr * E;
  const int gcol = two_groups ? col0 / 16 : col0 / G;
  const int64_t head = (int64_t)n * p.s.H + h;
  uint8_t* codes = static_cast<uint8_t*>(p.s.state) + qs::head_code_offset(p.s, n, h);
  float* scales = p.s.scales + head * p.s.dv * ngr;
  const uint32_t key = RND == qs::kSR ? qs::head_key(p.s, (uint32_t)n, (uint32_t)h) : 0u;
  for (int i = wave * RPW; i < rows; i += p.waves * RPW) {
    const int in = min(i + rsub, rows - 1), row = r0 + in;  // rows behind the end repeat the last
    uint8_t* at = codes + (int64_t)row * Gm::ROW_BYTES + lr * 16;
    float* sc = scales + (int64_t)row * ngr + gcol;
    const uint4 raw = qs::ld_stream(reinterpret_cast<const uint4*>(at));
    float s0 = sc[0], s1 = two_groups ? sc[1] : s0;
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float d[E];
    if constexpr (VEC) {
      qs::dequant_lane<BITS, E>(w, s0, s1, d);
      float a[E];
      qs::loadv_padded(&lds.decay[padded(col0)], a);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= a[e];
    } else {
      qs::dequant_lane<BITS, E>(w, s0 * lds.decay[0], s1 * lds.decay[0], d);
    }
    add_path(lds, len, in, col0, d);
    const uint32_t block0 = (uint32_t)((row * DK + col0) >> 4);
    const uint4 packed = qs::quantize_lane<BITS, RND, E, LPG>(d, key, block0, w, s0, s1);
    if (i + rsub >= rows) continue;
    qs::st_stream(reinterpret_cast<uint4*>(at), packed);
    if constexpr (two_groups) {
      sc[0] = s0;
      sc[1] = s1;
    } else if (lr % LPG == 0) {
      sc[0] = s0;
    }
  }
}

// A head whose blocks of 16 columns have different widths.
template <int DK, int G, int RND, bool VEC, class D>
__device__ __forceinline__ void accept_mixed(const Params& p, const D& lds, int n, int h, int len,
                                             int r0, int rows) {
  constexpr int E = 16, LPR = DK / 16, RPW = 64 / LPR, LPG = G / 16, ngr = DK / G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane % LPR, rsub = lane / LPR, col0 = lr * E;
  const qs::MixedLane ml(p.s.int8_blocks[h], lr, LPR);
  const float bias = ml.is8 ? 128.0f : 8.0f;
  const int64_t head = (int64_t)n * p.s.H + h;
  uint8_t* codes = static_cast<uint8_t*>(p.s.state) + qs::head_code_offset(p.s, n, h);
  float* scales = p.s.scales + head * p.s.dv * ngr;
  const uint32_t key = RND == qs::kSR ? qs::head_key(p.s, (uint32_t)n, (uint32_t)h) : 0u;
  for (int i = wave * RPW; i < rows; i += p.waves * RPW) {
    const int in = min(i + rsub, rows - 1), row = r0 + in;
    uint8_t* at = codes + (int64_t)row * ml.row_bytes + ml.lane_off;
    float* sc = scales + (int64_t)row * ngr + col0 / G;
    const uint2 a = *reinterpret_cast<const uint2*>(at);
    const uint2 b = *reinterpret_cast<const uint2*>(at + (ml.is8 ? 8 : 0));
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
    const float s_old = sc[0], sa = VEC ? s_old : s_old * lds.decay[0], nb = -bias * sa;
    float d[E];
    qs::unpack16_rt(w, ml.is8, d);
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = fmaf(d[e], sa, nb);
    if constexpr (VEC) {
      float f[E];
      qs::loadv_padded(&lds.decay[padded(col0)], f);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= f[e];
    }
    add_path(lds, len, in, col0, d);
    float s_new;
    uint32_t out[4];
    qs::quantize_block<RND, LPG>(d, ml.is8, key, (uint32_t)((row * DK + col0) >> 4), w, s_old,
                                 s_new, out);
    if (i + rsub >= rows) continue;
    qs::store_block(at, ml.is8, out);
    if (lr % LPG == 0) sc[0] = s_new;
  }
}

template <int DK, bool VEC, class D>
__device__ __forceinline__ void accept_fp32(const Params& p, const D& lds, int n, int h, int len,
                                            int r0, int rows) {
  constexpr int E = 16, LPR = DK / E, RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane % LPR, rsub = lane / LPR, col0 = lr * E;
  float* S = static_cast<float*>(p.s.state) + ((int64_t)n * p.s.H + h) * p.s.dv * DK;
  for (int i = wave * RPW; i < rows; i += p.waves * RPW) {
    const int in = i + rsub;
    if (in >= rows) continue;
    float* at = S + (int64_t)(r0 + in) * DK + col0;
    float d[E];
    qs::loadv(at, d);
    if constexpr (VEC) {
      float a[E];
      qs::loadv_padded(&lds.decay[padded(col0)], a);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= a[e];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= lds.decay[0];
    }
    add_path(lds, len, in, col0, d);
    qs::storev(at, d);
  }
}

// G = 0: FP32 states.
template <int DK, int G, int RND, bool VEC>
__global__ void __launch_bounds__(256) accept_kernel(Params p) {
  constexpr int LEN = most_tokens(DK);
  __shared__ PathLds<DK, VEC, LEN> lds;
  const int64_t head = blockIdx.x / p.blocks;
  const int n = (int)(head / p.s.H), h = (int)(head % p.s.H);
  const int hq = h / (p.s.H / p.heads_qk);
  const int lane = threadIdx.x & 63, threads = p.waves * 64, dv = p.s.dv;
  const int r0 = (int)(blockIdx.x % p.blocks) * p.rows, rows = min(p.rows, dv - r0);

  // the path, from its end; every wave finds it
  const int parent = named_parent(p, n, lane);
  int t = p.last[n], len = 0, node = 0;
  if (t >= p.tokens) t = -1;
  while (t >= 0) {
    if (lane == len) node = t;
    ++len;
    t = __builtin_amdgcn_readlane(parent, t);
  }
  if (len == 0 || t == -2) return;  // nothing accepted, or no node's path

  if (threadIdx.x < 64) lds.node[lane] = node;
  if (!VEC && threadIdx.x < 64) {
    double c = lane < len ? (double)qscan::gate(p.g[row_of(p, n, node) * p.s.H + h]) : 0.0;
    const double own = c;
    for (int d = 1; d < 64; d *= 2) {
      const double x = __shfl_up(c, d);
      if (lane >= d) c += x;
    }
    lds.f[lane] = qscan::fast_exp((float)(c - own));
    if (lane == 63) lds.decay[0] = qscan::fast_exp((float)c);
  }
  __syncthreads();
  if constexpr (VEC) {
    for (int e = threadIdx.x; e < DK; e += threads) {
      float f = 1.0f;
      for (int j = 0; j < len; ++j) {
        const int64_t row = row_of(p, n, lds.node[j]);
        lds.k[j][padded(e)] = f * qscan::load_elem(p.k, row * p.ks + (int64_t)hq * DK + e, p.dtype);
        f *= qscan::fast_exp(qscan::gate(p.g[(row * p.s.H + h) * DK + e]));
      }
      lds.decay[padded(e)] = f;
    }
  } else {
    const bool four = p.ks % 4 == 0;
    for (int i = threadIdx.x; i < len * (DK / 4); i += threads) {
      const int j = i / (DK / 4), e = i % (DK / 4) * 4;
      const int64_t row = row_of(p, n, lds.node[j]);
      float x[4];
      qscan::widen4(qscan::load4(p.k, row * p.ks + (int64_t)hq * DK + e, p.dtype, four), p.dtype, x);
#pragma unroll
      for (int r = 0; r < 4; ++r) lds.k[j][padded(e) + r] = x[r] * lds.f[j];
    }
  }
  for (int i = threadIdx.x; i < len * 128; i += threads) {
    const int j = i >> 7, r = i & 127;
    const int64_t row = row_of(p, n, lds.node[j]);
    lds.w[j][r] = r < rows ? p.writes_in[(row * p.s.H + h) * dv + r0 + r] : 0.0f;
  }
  __syncthreads();
  if constexpr (G == 0) {
    accept_fp32<DK, VEC>(p, lds, n, h, len, r0, rows);
  } else {
    constexpr uint32_t all = (1u << (DK / 16)) - 1u;
    const uint32_t m = p.s.int8_blocks[h];
    if (m == 0)
      accept_rows<DK, 4, G, RND, VEC>(p, lds, n, h, len, r0, rows);
    else if (m == all)
      accept_rows<DK, 8, G, RND, VEC>(p, lds, n, h, len, r0, rows);
    else
      accept_mixed<DK, G, RND, VEC>(p, lds, n, h, len, r0, rows);
  }
}

template <int DK, int G, int RND>
hipError_t accept_gates(const Params& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.s.B * p.s.H * p.blocks);
  if (qs::vector_decay(p.mixer))
    accept_kernel<DK, G, RND, true><<<grid, p.waves * 64, 0, s>>>(p);
  else
    accept_kernel<DK, G, RND, false><<<grid, p.waves * 64, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK, int G>
hipError_t accept_rounding(const Params& p, hipStream_t s) {
  switch (p.rounding) {
    case qs::kRTN: return accept_gates<DK, G, qs::kRTN>(p, s);
    case qs::kSR: return accept_gates<DK, G, qs::kSR>(p, s);
    case qs::kBDR: return accept_gates<DK, G, qs::kBDR>(p, s);
    default: return hipErrorInvalidValue;
  }
}

template <int DK>
hipError_t accept(const Params& p, hipStream_t s) {
  if (p.fp32) return accept_gates<DK, 0, qs::kRTN>(p, s);
  switch (p.s.G) {
    case 16: return accept_rounding<DK, 16>(p, s);
    case 32: return accept_rounding<DK, 32>(p, s);
    case 64: return accept_rounding<DK, 64>(p, s);
    case 128:
      if constexpr (DK >= 128) return accept_rounding<DK, 128>(p, s);
      return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdraft
