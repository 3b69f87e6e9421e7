// draft_accept.h — the stored state behind the accepted path:
//
//   S' = S e^(c_end) + sum_j w_j (k_j e^(c_end - c_j))^T   over the path's nodes
//
// with the w_j that the readout left.  A workgroup takes up to 128 value rows of
// a head: the path's scaled keys and its writes go to LDS, then waves go over the
// rows with the lanes, the dequantization and the quantizer of the single-token
// step (qstate_device.h, qstate_value.h), so that a state is read and written once.
// The first rows are asked for before the path is looked up.
// Bound by memory and the quantizer's instructions: 128 sequences, 16 heads of 128 x 128, INT8,
// paths of 4 nodes 23 us (78 MB, 3.4 TB/s; 33 us with loads behind the path's); 16 sequences
// of FP32 states, a gate per channel, 10.6 us (34 MB).  256 sequences, 32 heads of INT4, a quarter INT8,
// paths of about 7 nodes 84 to 89 us (245 MB, 2.8 TB/s), with widths per channel 87.

#pragma once

#include "draft_device.h"

namespace qdraft {

constexpr int kWaves = 4;   // of a workgroup
constexpr int kAhead = 4;   // row iterations whose loads are in flight
constexpr int kMostRows = 128;

// Columns of a key in LDS: 4 floats of padding behind 16, as loadv_padded reads them.
constexpr int padded(int c) { return c + c / 16 * 4; }

template <int DK, bool VEC, int LEN>
struct alignas(16) PathLds {
  float k[LEN][padded(DK)];
  float w[LEN][kMostRows];
  float decay[VEC ? padded(DK) : 4];
  int node[64];    // the path's nodes, the last one first
  float f[64];     // one gate a token: the decay from behind node j to the end
};

// A workgroup's part of a head.
struct Part {
  int n, h, r0, rows;
};

// The path to LDS; its length.
template <int DK, bool VEC, class D>
__device__ __forceinline__ int path(const Params& p, D& lds, const Part& w) {
  const int lane = threadIdx.x & 63, threads = kWaves * 64, dv = p.s.dv, n = w.n, h = w.h;
  const int hq = h / (p.s.H / p.heads_qk);
  // from its end; every wave finds it
  const int parent = named_parent(p, n, lane);
  int t = p.last[n], len = 0, node = 0;
  if (t >= p.tokens) t = -1;
  while (t >= 0) {
    if (lane == len) node = t;
    ++len;
    t = __builtin_amdgcn_readlane(parent, t);
  }
  if (len == 0 || t == -2) return 0;  // nothing accepted, or no node's path
  if (threadIdx.x < 64) lds.node[lane] = node;
  if (!VEC && threadIdx.x < 64) {
    // decays from behind each node to the end
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
  for (int i = threadIdx.x; i < len * kMostRows; i += threads) {
    const int j = i / kMostRows, r = i % kMostRows;
    const int64_t row = row_of(p, n, lds.node[j]);
    lds.w[j][r] = r < w.rows ? p.writes_in[(row * p.s.H + h) * dv + w.r0 + r] : 0.0f;
  }
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
  __syncthreads();
  return len;
}

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

// A wave's rows, RPW at a time: load(slot, row) asks for those of an iteration, take(slot, row, stored)
// works on them.  Rows behind the end repeat the last and are not stored.
template <int RPW, class Load, class Ready, class Take>
__device__ __forceinline__ void over_rows(int rows, int rsub, Load load, Ready ready, Take take) {
  const int first = (int)(threadIdx.x >> 6) * RPW, step = kWaves * RPW;
  auto row = [&](int it) { return min(first + it * step + rsub, rows - 1); };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(k, row(k));
  if (!ready()) return;
  for (int it = 0; first + it * step < rows; it += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = first + (it + k) * step;
      if (i >= rows) break;
      take(k, row(it + k), i + rsub < rows);
      load(k, row(it + k + kAhead));
    }
  }
}

// Rows of a head of one width.
template <int DK, int BITS, int G, int RND, bool VEC, class D>
__device__ __forceinline__ void accept_rows(const Params& p, D& lds, const Part& part) {
  using Gm = qs::Geo<DK, BITS>;
  constexpr int E = Gm::E, LPR = Gm::LPR, RPW = Gm::RPW;
  constexpr bool two_groups = G < E;
  constexpr int LPG = two_groups ? 0 : G / E;
  constexpr int ngr = DK / G;
  const int lane = threadIdx.x & 63;
  const int lr = lane % LPR, rsub = lane / LPR, col0 = lr * E;
  const int gcol = two_groups ? col0 / 16 : col0 / G;
  const int64_t head = (int64_t)part.n * p.s.H + part.h;
  uint8_t* codes = static_cast<uint8_t*>(p.s.state) + qs::head_code_offset(p.s, part.n, part.h) +
                   (int64_t)part.r0 * Gm::ROW_BYTES;
  float* scales = p.s.scales + (head * p.s.dv + part.r0) * ngr;
  const uint32_t key = RND == qs::kSR ? qs::head_key(p.s, (uint32_t)part.n, (uint32_t)part.h) : 0u;
  uint4 raw[kAhead];
  float s0[kAhead], s1[kAhead];
  int len = 0;
  over_rows<RPW>(
      part.rows, rsub,
      [&](int k, int row) {
        raw[k] = qs::ld_stream(reinterpret_cast<const uint4*>(codes + row * Gm::ROW_BYTES + lr * 16));
        s0[k] = scales[row * ngr + gcol];
        s1[k] = two_groups ? scales[row * ngr + gcol + 1] : s0[k];
      },
      [&]() { return (len = path<DK, VEC>(p, lds, part)) > 0; },
      [&](int k, int row, bool stored) {
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        float d[E], a = s0[k], b = s1[k];
        if constexpr (VEC) {
          qs::dequant_lane<BITS, E>(w, a, b, d);
          float f[E];
          qs::loadv_padded(&lds.decay[padded(col0)], f);
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] *= f[e];
        } else {
          qs::dequant_lane<BITS, E>(w, a * lds.decay[0], b * lds.decay[0], d);
        }
        add_path(lds, len, row, col0, d);
        const uint32_t block0 = (uint32_t)(((part.r0 + row) * DK + col0) >> 4);
        const uint4 packed = qs::quantize_lane<BITS, RND, E, LPG>(d, key, block0, w, a, b);
        if (!stored) return;
        qs::st_stream(reinterpret_cast<uint4*>(codes + row * Gm::ROW_BYTES + lr * 16), packed);
        if constexpr (two_groups) {
          scales[row * ngr + gcol] = a;
          scales[row * ngr + gcol + 1] = b;
        } else if (lr % LPG == 0) {
          scales[row * ngr + gcol] = a;
        }
      });
}

// Rows of a head whose blocks of 16 columns have different widths.
template <int DK, int G, int RND, bool VEC, class D>
__device__ __forceinline__ void accept_mixed(const Params& p, D& lds, const Part& part) {
  constexpr int E = 16, LPR = DK / 16, RPW = 64 / LPR, LPG = G / 16, ngr = DK / G;
  const int lane = threadIdx.x & 63;
  const int lr = lane % LPR, rsub = lane / LPR, col0 = lr * E;
  const qs::MixedLane ml(p.s.int8_blocks[part.h], lr, LPR);
  const float bias = ml.is8 ? 128.0f : 8.0f;
  const int64_t head = (int64_t)part.n * p.s.H + part.h;
  uint8_t* codes = static_cast<uint8_t*>(p.s.state) + qs::head_code_offset(p.s, part.n, part.h) +
                   (int64_t)part.r0 * ml.row_bytes + ml.lane_off;
  float* scales = p.s.scales + (head * p.s.dv + part.r0) * ngr + col0 / G;
  const uint32_t key = RND == qs::kSR ? qs::head_key(p.s, (uint32_t)part.n, (uint32_t)part.h) : 0u;
  uint2 lo[kAhead], hi[kAhead];
  float s_old[kAhead];
  int len = 0;
  over_rows<RPW>(
      part.rows, rsub,
      [&](int k, int row) {
        const uint8_t* at = codes + row * ml.row_bytes;
        lo[k] = *reinterpret_cast<const uint2*>(at);
        hi[k] = *reinterpret_cast<const uint2*>(at + (ml.is8 ? 8 : 0));
        s_old[k] = scales[row * ngr];
      },
      [&]() { return (len = path<DK, VEC>(p, lds, part)) > 0; },
      [&](int k, int row, bool stored) {
        const uint32_t w[4] = {lo[k].x, lo[k].y, hi[k].x, hi[k].y};
        const float s = s_old[k], sa = VEC ? s : s * lds.decay[0], nb = -bias * sa;
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
        add_path(lds, len, row, col0, d);
        float s_new;
        uint32_t out[4];
        qs::quantize_block<RND, LPG>(d, ml.is8, key, (uint32_t)(((part.r0 + row) * DK + col0) >> 4), w,
                                     s, s_new, out);
        if (!stored) return;
        qs::store_block(codes + row * ml.row_bytes, ml.is8, out);
        if (lr % LPG == 0) scales[row * ngr] = s_new;
      });
}

template <int DK, bool VEC, class D>
__device__ __forceinline__ void accept_fp32(const Params& p, D& lds, const Part& part) {
  // a lane's columns are 4 lr + 4 LPR i .., so that a load reads whole lines
  constexpr int E = 16, LPR = DK / E, RPW = 64 / LPR;
  const int lane = threadIdx.x & 63;
  const int lr = lane % LPR, rsub = lane / LPR;
  float* S = static_cast<float*>(p.s.state) +
             (((int64_t)part.n * p.s.H + part.h) * p.s.dv + part.r0) * DK + 4 * lr;
  f32x4 x[kAhead][4];
  int len = 0;
  over_rows<RPW>(
      part.rows, rsub,
      [&](int k, int row) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[k][i] = *reinterpret_cast<const f32x4*>(S + (int64_t)row * DK + 4 * LPR * i);
      },
      [&]() { return (len = path<DK, VEC>(p, lds, part)) > 0; },
      [&](int k, int row, bool stored) {
        f32x4 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[i] = x[k][i];
          if constexpr (VEC) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&lds.decay[padded(4 * lr + 4 * LPR * i)]);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] *= f[e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] *= lds.decay[0];
          }
        }
        for (int j = 0; j < len; ++j) {
          const float w = lds.w[j][row];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&lds.k[j][padded(4 * lr + 4 * LPR * i)]);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] = fmaf(w, f[e], d[i][e]);
          }
        }
        if (!stored) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(S + (int64_t)row * DK + 4 * LPR * i) = d[i];
      });
}

// G = 0: FP32 states.  LEN: nodes of a path that the LDS holds.
template <int DK, int G, int RND, bool VEC, int LEN>
__global__ void __launch_bounds__(kWaves * 64) accept_kernel(Params p) {
  __shared__ PathLds<DK, VEC, LEN> lds;
  const uint32_t head = blockIdx.x / (uint32_t)p.blocks;
  Part part;
  part.n = (int)(head / (uint32_t)p.s.H);
  part.h = (int)(head - part.n * (uint32_t)p.s.H);
  part.r0 = (int)(blockIdx.x - head * p.blocks) * p.rows;
  part.rows = min(p.rows, p.s.dv - part.r0);
  if constexpr (G == 0) {
    accept_fp32<DK, VEC>(p, lds, part);
  } else {
    constexpr uint32_t all = (1u << (DK / 16)) - 1u;
    const uint32_t m =
        reinterpret_cast<const uint32_t*>(p.s.int8_blocks)[part.h >> 1] >> (part.h & 1) * 16 & 0xFFFFu;
    // beside heads of mixed widths, others need not begin on 16 bytes
    if (p.s.mixed)
      accept_mixed<DK, G, RND, VEC>(p, lds, part);
    else if (m == all)
      accept_rows<DK, 8, G, RND, VEC>(p, lds, part);
    else
      accept_rows<DK, 4, G, RND, VEC>(p, lds, part);
  }
}

template <int DK, int G, int RND, bool VEC>
hipError_t accept_length(const Params& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.s.B * p.s.H * p.blocks);
  if (p.tokens <= 16)
    accept_kernel<DK, G, RND, VEC, 16><<<grid, kWaves * 64, 0, s>>>(p);
  else
    accept_kernel<DK, G, RND, VEC, most_tokens(DK)><<<grid, kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK, int G, int RND>
hipError_t accept_gates(const Params& p, hipStream_t s) {
  return qs::vector_decay(p.mixer) ? accept_length<DK, G, RND, true>(p, s)
                                   : accept_length<DK, G, RND, false>(p, s);
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
