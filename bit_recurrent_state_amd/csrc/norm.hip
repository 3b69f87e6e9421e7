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

#include "norm_launch.h"

namespace qnorm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  const f32x2 f = {a, b};
  if (DT == 1) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
}

// Value e of a thread's vector v: VEC, 8 neighbours; else neighbours go to
// neighbouring threads.
template <bool VEC>
__device__ __forceinline__ int column(int v, int e, int t, int team) {
  return VEC ? (v * team + t) * 8 + e : (v * 8 + e) * team + t;
}

// A thread's values of a row as they lie in memory, so that the next row's can
// be on their way while this one is worked on.
template <int DT, int V>
struct Raw {
  u32x4 w[V][DT == 0 ? 2 : 1];
};

template <int DT, int V, bool VEC>
__device__ __forceinline__ void load_raw(const void* p, int64_t at, int t, int team, int width,
                                         Raw<DT, V>& x) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VEC) {
      // columns behind the width repeat the last ones and count as zero later
      const int c = min(column<true>(v, 0, t, team), width - 8);
      const char* s = static_cast<const char*>(p) + (at + c) * (DT == 0 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < (DT == 0 ? 2 : 1); ++i) x.w[v][i] = reinterpret_cast<const u32x4*>(s)[i];
    } else {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = at + min(column<false>(v, i, t, team), width - 1);
        e[i] = DT == 0 ? static_cast<const uint32_t*>(p)[c] : static_cast<const uint16_t*>(p)[c];
      }
      if (DT == 0) {
        x.w[v][0] = u32x4{e[0], e[1], e[2], e[3]};
        x.w[v][DT == 0] = u32x4{e[4], e[5], e[6], e[7]};
      } else {
        x.w[v][0] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
      }
    }
  }
}

template <int DT, int V, bool VEC>
__device__ __forceinline__ void widen(const Raw<DT, V>& r, int t, int team, int width,
                                      float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = DT == 0 ? r.w[v][DT == 0 ? i / 4 : 0][i % 4] : r.w[v][0][i / 2];
      float f;
      if (DT == 0)
        f = __uint_as_float(w);
      else if (DT == 1)
        f = __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
      else
        f = (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
      x[v * 8 + i] = column<VEC>(v, i, t, team) < width ? f : 0.0f;
    }
}

template <int DT, int V, bool VEC>
__device__ __forceinline__ void store_row(void* p, int64_t at, int t, int team, int width,
                                          const float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VEC) {
      const int c = column<true>(v, 0, t, team);
      if (c >= width) continue;
      const float* s = x + v * 8;
      if (DT == 0) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at + c);
        d[0] = f32x4{s[0], s[1], s[2], s[3]};
        d[1] = f32x4{s[4], s[5], s[6], s[7]};
      } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at + c) =
            u32x4{narrow2<DT>(s[0], s[1]), narrow2<DT>(s[2], s[3]), narrow2<DT>(s[4], s[5]),
                  narrow2<DT>(s[6], s[7])};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(v, e, t, team);
        if (c >= width) continue;
        const float f = x[v * 8 + e];
        if (DT == 0)
          static_cast<float*>(p)[at + c] = f;
        else
          static_cast<uint16_t*>(p)[at + c] = (uint16_t)narrow2<DT>(f, 0.0f);
      }
    }
  }
}

template <int V, bool VEC>
__device__ __forceinline__ void load_weight(const float* p, int64_t at, int t, int team, int width,
                                            float (&x)[V * 8]) {
  if (p) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<VEC>(v, e, t, team);
        x[v * 8 + e] = c < width ? p[at + c] : 0.0f;
      }
  } else {
#pragma unroll
    for (int i = 0; i < V * 8; ++i) x[i] = 1.0f;
  }
}

// Sum over the team; every thread gets it.  Two sums at once save a barrier.
template <bool WIDE>
__device__ __forceinline__ void team_sum(float& a, float& b, int team, float (*lds)[2]) {
  const int span = WIDE ? 64 : team;
  for (int d = 1; d < span; d *= 2) {
    a += __shfl_xor(a, d);
    b += __shfl_xor(b, d);
  }
  if (WIDE) {
    const int waves = team >> 6;
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6][0] = a;
      lds[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
    for (int w = 0; w < waves; ++w) {
      a += lds[w][0];
      b += lds[w][1];
    }
  }
}

// act(z) and, for the gradient, its derivative.  exp(-z) is 2^t (1 + r ln 2) with
// t + r = -z log2 e in two parts, the reciprocal is refined once: both hold to
// an ulp or two at a third of the library functions' instructions, which bound
// the backward kernel otherwise.
__device__ __forceinline__ float activate(float z, int act, float& slope) {
  const float hi = -1.44269502f, lo = -1.92596303e-8f;
  const float c = z > 87.0f ? 87.0f : z < -87.0f ? -87.0f : z;  // e stays a normal number; NaN stays
  const float t = c * hi;
  const float r = fmaf(c, lo, fmaf(c, hi, -t));
  float e = __builtin_amdgcn_exp2f(t);
  e = fmaf(e, r * 0.693147182f, e);
  const float d = 1.0f + e;
  float s = __builtin_amdgcn_rcpf(d);
  s = fmaf(fmaf(-d, s, 1.0f), s, s);
  const float q = s * e;  // 1 - s without cancellation
  // s and q stop at e^-87, so what multiplies them has to: z itself would bring z e^-87 instead of
  // nothing where it is a masked gate's lowest value (or, in the slope, the largest)
  slope = act == 0 ? s * fmaf(c, q, 1.0f) : s * q;
  return act == 0 ? (z < c ? c : z) * s : s;
}

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
