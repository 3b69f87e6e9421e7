// norm.hip — the block norm of include/qstate_norm.h and its gradients.
//
// Every value is read once and written once: a row stays in the registers of
// its team of threads (8 or 16 values each) between the two norms, and the
// backward pass computes n, y and r again from the inputs instead of reading
// them.  Bound by memory.  Teams walk over rows with a fixed stride, so weights
// are loaded, and their gradients summed, once per team: rows up to 512 wide
// take 1 .. 64 lanes of a wave (a readout's 128 values: 16 lanes), wider ones a
// workgroup.  8191 rows of 4096 bfloat16 values with all parts take 74 us forward
// (336 MB, 4.5 TB/s) and 131 us backward (550 MB, 4.2 TB/s); a copy of that size
// runs at 4.6 TB/s.

#include <hip/hip_runtime.h>

#include "norm_device.h"
#include "norm_launch.h"

namespace qnorm {

struct Place {
  int64_t x, gate, residual;
};

__device__ __forceinline__ Place place(const Params& p, int64_t row) {
  if (p.groups == 1) return {row * p.xs, row * p.gs, row * p.rs};
  const int64_t tok = row / p.groups, in = (row - tok * p.groups) * p.width;
  return {tok * p.xs + in, tok * p.gs + in, tok * p.rs + in};
}

template <int DT, int V, bool WIDE, bool VEC, int BLOCK>
__global__ void __launch_bounds__(BLOCK) forward_kernel(Params p) {
  constexpr int N = V * 8;
  __shared__ float lds[BLOCK / 64][2];
  const int team = WIDE ? BLOCK : p.team, t = threadIdx.x & (team - 1);
  const int64_t first = (int64_t)blockIdx.x * (BLOCK / team) + threadIdx.x / team;
  const int width = p.width;
  float w[N], sc[N], w2[N];
  load_weight<V, VEC>(p.weight, p.each ? first % p.groups * width : 0, t, team, width, w);
  load_weight<V, VEC>(p.scale, 0, t, team, width, sc);
  if (p.h) load_weight<V, VEC>(p.next_weight, 0, t, team, width, w2);
  // WIDE teams are whole workgroups, the others stay inside a wave: no barrier is passed by a part
  int64_t row = first < p.teams ? first : p.rows;
  if (row >= p.rows) return;
  Raw<DT, V> rx, rz, ry;
  auto load = [&](int64_t r) {
    const Place at = place(p, r);
    load_raw<DT, V, VEC>(p.x, at.x, t, team, width, rx);
    if (p.gate) load_raw<DT, V, VEC>(p.gate, at.gate, t, team, width, rz);
    if (p.residual) load_raw<DT, V, VEC>(p.residual, at.residual, t, team, width, ry);
  };
  load(row);
  for (; row < p.rows; row += p.teams) {
    const int64_t out = row * width;
    float x[N], z[N], y[N];
    widen<DT, V, VEC>(rx, t, team, width, x);
    if (p.gate) widen<DT, V, VEC>(rz, t, team, width, z);
    if (p.residual) widen<DT, V, VEC>(ry, t, team, width, y);
    if (row + p.teams < p.rows) load(row + p.teams);
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
    team_sum<WIDE>(s, unused, team, lds);
    const float rs = 1.0f / sqrtf(s / (float)width + p.eps);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {  // columns behind the width hold zeros
      float n = x[i] * rs * w[i], slope;
      if (p.gate) n *= activate(z[i], p.act, slope);
      n *= sc[i];
      x[i] = p.residual ? y[i] + n : n;
      s = fmaf(x[i], x[i], s);
    }
    if (p.r) store_row<DT, V, VEC>(p.r, out, t, team, width, x);
    if (!p.h) continue;
    team_sum<WIDE>(s, unused, team, lds);
    const float rs2 = 1.0f / sqrtf(s / (float)width + p.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * rs2 * w2[i];
    store_row<DT, V, VEC>(p.h, out, t, team, width, x);
  }
}

template <int DT, int V, bool WIDE, bool VEC, int BLOCK>
__global__ void __launch_bounds__(BLOCK) backward_kernel(Params p) {
  constexpr int N = V * 8;
  __shared__ float lds[BLOCK / 64][2];
  const int team = WIDE ? BLOCK : p.team, t = threadIdx.x & (team - 1);
  const int64_t first = (int64_t)blockIdx.x * (BLOCK / team) + threadIdx.x / team;
  const int width = p.width;
  const float inv = 1.0f / (float)width;
  float w[N], sc[N], w2[N], dw[N], ds[N], dw2[N];
  load_weight<V, VEC>(p.weight, p.each ? first % p.groups * width : 0, t, team, width, w);
  load_weight<V, VEC>(p.scale, 0, t, team, width, sc);
  if (p.has_h) load_weight<V, VEC>(p.next_weight, 0, t, team, width, w2);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = ds[i] = dw2[i] = 0.0f;
  const bool use_h = p.has_h && p.dh;
  Raw<DT, V> rx, rz, ry, rd, rm;
  auto load = [&](int64_t r) {
    const Place at = place(p, r);
    load_raw<DT, V, VEC>(p.x, at.x, t, team, width, rx);
    if (p.gate) load_raw<DT, V, VEC>(p.gate, at.gate, t, team, width, rz);
    if (p.residual && use_h) load_raw<DT, V, VEC>(p.residual, at.residual, t, team, width, ry);
    if (p.dr) load_raw<DT, V, VEC>(p.dr, r * width, t, team, width, rd);
    if (use_h) load_raw<DT, V, VEC>(p.dh, r * width, t, team, width, rm);
  };
  int64_t row = first < p.teams ? first : p.rows;
  if (row < p.rows) load(row);
  for (; row < p.rows; row += p.teams) {
    const int64_t out = row * width;
    float x[N], z[N], y[N], d[N], m[N], act[N], slope[N];
    widen<DT, V, VEC>(rx, t, team, width, x);
    if (p.gate) {
      widen<DT, V, VEC>(rz, t, team, width, z);
#pragma unroll
      for (int i = 0; i < N; ++i) act[i] = activate(z[i], p.act, slope[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        act[i] = 1.0f;
        slope[i] = 0.0f;
      }
    }
    if (p.residual && use_h) widen<DT, V, VEC>(ry, t, team, width, y);
    if (p.dr) {
      widen<DT, V, VEC>(rd, t, team, width, d);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = 0.0f;
    }
    if (use_h) widen<DT, V, VEC>(rm, t, team, width, m);
    if (row + p.teams < p.rows) load(row + p.teams);
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
    team_sum<WIDE>(s, q, team, lds);
    const float rs = 1.0f / sqrtf(s * inv + p.eps);
    // x becomes n without its weight; y, if needed, r
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= rs;
    if (use_h) {
      float ss = 0.0f, mr = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = x[i] * w[i] * act[i] * sc[i];
        y[i] = p.residual ? y[i] + n : n;
        ss = fmaf(y[i], y[i], ss);
        mr = fmaf(m[i] * w2[i], y[i], mr);
      }
      team_sum<WIDE>(ss, mr, team, lds);
      const float rs2 = 1.0f / sqrtf(ss * inv + p.eps);
      const float k = rs2 * mr * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = y[i] * rs2;  // before rs2 a third time: its cube overflows with a tiny eps
        d[i] += rs2 * (m[i] * w2[i] - k * n);
        dw2[i] = fmaf(m[i], n, dw2[i]);
      }
    }
    if (p.dresidual) store_row<DT, V, VEC>(p.dresidual, out, t, team, width, d);
    float dn = 0.0f;
    q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = act[i], xw = x[i] * w[i], dy = d[i] * sc[i];
      ds[i] = fmaf(d[i], xw * a, ds[i]);
      z[i] = dy * xw * slope[i];
      dw[i] = fmaf(dy * a, x[i], dw[i]);
      d[i] = dy * a * w[i];
      dn = fmaf(d[i], x[i], dn);
    }
    if (p.dgate) store_row<DT, V, VEC>(p.dgate, out, t, team, width, z);
    if (p.dx) {
      team_sum<WIDE>(dn, q, team, lds);
      dn *= inv;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = rs * (d[i] - x[i] * dn);
      store_row<DT, V, VEC>(p.dx, out, t, team, width, d);
    }
  }
  if (!p.part) return;
  int64_t mine = first;  // this team's part
  if (!WIDE && !p.each) {
    // one weight for all rows: the teams of a wave first
#pragma unroll
    for (int i = 0; i < N; ++i)
      for (int o = team; o < 64; o *= 2) {
        dw[i] += __shfl_xor(dw[i], o);
        ds[i] += __shfl_xor(ds[i], o);
        dw2[i] += __shfl_xor(dw2[i], o);
      }
    mine = (int64_t)blockIdx.x * (BLOCK / 64) + (threadIdx.x >> 6);
    if ((int)(threadIdx.x & 63) >= team) return;
  }
  if (mine >= p.partials) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = column<VEC>(i / 8, i % 8, t, team);
    if (c >= width) continue;
    float* o = p.part + mine * width + c;
    const int64_t plane = p.partials * width;
    if (p.dweight) o[0] = dw[i];
    if (p.dscale) o[plane] = ds[i];
    if (p.dnext_weight) o[2 * plane] = dw2[i];
  }
}

// The teams' parts, summed in a fixed order: a workgroup takes 32 columns, its
// 8 rows of threads every 8th part each, in 64 bits.
__global__ void __launch_bounds__(256) parts_kernel(Params p) {
  __shared__ double lds[8][32];
  const int which = blockIdx.z, g = blockIdx.y;
  float* out = which == 0 ? p.dweight : which == 1 ? p.dscale : p.dnext_weight;
  if (!out || (which > 0 && g > 0)) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  const bool each = which == 0 && p.each;
  const int64_t step = each ? p.groups : 1;
  double s = 0.0;
  if (c < p.width)
#pragma unroll 4
    for (int64_t i = (each ? g : 0) + y * step; i < p.partials; i += 8 * step)
      s += p.part[((int64_t)which * p.partials + i) * p.width + c];
  lds[y][threadIdx.x & 31] = s;
  __syncthreads();
  if (y == 0 && c < p.width) {
    for (int k = 1; k < 8; ++k) s += lds[k][threadIdx.x];
    out[(int64_t)g * p.width + c] = (float)s;
  }
}

template <int DT, int V, bool WIDE, int BLOCK>
hipError_t run(const Params& p, bool back, hipStream_t s) {
  const int64_t per = BLOCK / p.team;
  const dim3 grid((unsigned)((p.teams + per - 1) / per));
  if (back) {
    if (p.aligned)
      backward_kernel<DT, V, WIDE, true, BLOCK><<<grid, BLOCK, 0, s>>>(p);
    else
      backward_kernel<DT, V, WIDE, false, BLOCK><<<grid, BLOCK, 0, s>>>(p);
  } else {
    if (p.aligned)
      forward_kernel<DT, V, WIDE, true, BLOCK><<<grid, BLOCK, 0, s>>>(p);
    else
      forward_kernel<DT, V, WIDE, false, BLOCK><<<grid, BLOCK, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const Params& p, bool back, hipStream_t s) {
  if (!p.wide) return run<DT, 1, false, 256>(p, back, s);
  switch (p.block) {
    case 128: return run<DT, 1, true, 128>(p, back, s);
    case 256: return run<DT, 1, true, 256>(p, back, s);
    case 512: return run<DT, 1, true, 512>(p, back, s);
    default: return p.vectors == 1 ? run<DT, 1, true, 1024>(p, back, s) : run<DT, 2, true, 1024>(p, back, s);
  }
}

static hipError_t by_type(const Params& p, int dtype, bool back, hipStream_t s) {
  switch (dtype) {
    case 0: return pick<0>(p, back, s);
    case 1: return pick<1>(p, back, s);
    case 2: return pick<2>(p, back, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t forward(const Params& p, int dtype, hipStream_t s) { return by_type(p, dtype, false, s); }

hipError_t backward(const Params& p, int dtype, hipStream_t s) {
  const hipError_t e = p.teams > 0 ? by_type(p, dtype, true, s) : hipSuccess;
  if (e != hipSuccess || !(p.dweight || p.dscale || p.dnext_weight)) return e;
  parts_kernel<<<dim3((p.width + 31) / 32, p.each ? p.groups : 1, 3), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace qnorm
