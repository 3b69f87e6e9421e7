// norm.hip — the block norm of include/qstate_norm.h and its gradients.
//
// Every value is read once and written once: a row stays in the registers of
// its team of threads (8 or 16 values each) between the two norms, and the
// backward pass computes n, y and r again from the inputs instead of reading
// them.  Bound by memory.  Teams walk over rows with a fixed stride, so weights
// are loaded, and their gradients summed, once per team: rows up to 512 wide
// take 1 .. 64 lanes of a wave (a readout's 128 values: 16 lanes), wider ones a
// workgroup.

#include <hip/hip_runtime.h>

#include "norm_launch.h"

namespace qnorm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ float widen(const void* p, int64_t i) {
  if (DT == 1) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  if (DT == 2) return (float)static_cast<const _Float16*>(p)[i];
  return static_cast<const float*>(p)[i];
}

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

template <int DT, int V, bool VEC>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int t, int team, int width,
                                         float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VEC) {
      const int c = column<true>(v, 0, t, team);
      if (c >= width) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v * 8 + e] = 0.0f;
      } else if (DT == 0) {
        const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at + c);
        const f32x4 a = s[0], b = s[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[v * 8 + e] = a[e];
          x[v * 8 + 4 + e] = b[e];
        }
      } else {
        const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (DT == 1) {
            x[v * 8 + 2 * e] = __uint_as_float(w[e] << 16);
            x[v * 8 + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
          } else {
            const uint32_t two = w[e];  // bit casts take whole values, not vector elements
            const f16x2 h = __builtin_bit_cast(f16x2, two);
            x[v * 8 + 2 * e] = (float)h.x;
            x[v * 8 + 2 * e + 1] = (float)h.y;
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(v, e, t, team);
        x[v * 8 + e] = c < width ? widen<DT>(p, at + c) : 0.0f;
      }
    }
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

// act(z) and, for the gradient, its derivative.
__device__ __forceinline__ float activate(float z, int act, float& slope) {
  const float s = 1.0f / (1.0f + expf(-z));
  slope = act == 0 ? s * (1.0f + z * (1.0f - s)) : s * (1.0f - s);
  return act == 0 ? z * s : s;
}

struct Place {
  int64_t x, gate, residual, out;
};

__device__ __forceinline__ Place place(const Params& p, int64_t row) {
  if (p.groups == 1) return {row * p.xs, row * p.gs, row * p.rs, row * p.width};
  const int64_t tok = row / p.groups, in = (row - tok * p.groups) * p.width;
  return {tok * p.xs + in, tok * p.gs + in, tok * p.rs + in, row * p.width};
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
  for (int64_t row = first < p.teams ? first : p.rows; row < p.rows; row += p.teams) {
    const Place at = place(p, row);
    float x[N], z[N], y[N];
    load_row<DT, V, VEC>(p.x, at.x, t, team, width, x);
    if (p.gate) load_row<DT, V, VEC>(p.gate, at.gate, t, team, width, z);
    if (p.residual) load_row<DT, V, VEC>(p.residual, at.residual, t, team, width, y);
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
    team_sum<WIDE>(s, unused, team, lds);
    const float rs = 1.0f / sqrtf(s / (float)width + p.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float n = x[i] * rs * w[i], slope;
      if (p.gate) n *= activate(z[i], p.act, slope);
      n *= sc[i];
      x[i] = p.residual ? y[i] + n : n;
    }
    if (p.r) store_row<DT, V, VEC>(p.r, at.out, t, team, width, x);
    if (!p.h) continue;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)  // columns behind the width hold zeros
      s = fmaf(x[i], x[i], s);
    team_sum<WIDE>(s, unused, team, lds);
    const float rs2 = 1.0f / sqrtf(s / (float)width + p.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * rs2 * w2[i];
    store_row<DT, V, VEC>(p.h, at.out, t, team, width, x);
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
  for (int64_t row = first < p.teams ? first : p.rows; row < p.rows; row += p.teams) {
    const Place at = place(p, row);
    float x[N], z[N], y[N], d[N], m[N];
    load_row<DT, V, VEC>(p.x, at.x, t, team, width, x);
    if (p.gate) load_row<DT, V, VEC>(p.gate, at.gate, t, team, width, z);
    const bool use_h = p.has_h && p.dh;
    if (p.residual && use_h) load_row<DT, V, VEC>(p.residual, at.residual, t, team, width, y);
    if (p.dr)
      load_row<DT, V, VEC>(p.dr, at.out, t, team, width, d);
    else {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = 0.0f;
    }
    if (use_h) load_row<DT, V, VEC>(p.dh, at.out, t, team, width, m);
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
        float n = x[i] * w[i], slope;
        if (p.gate) n *= activate(z[i], p.act, slope);
        n *= sc[i];
        y[i] = p.residual ? y[i] + n : n;
        ss = fmaf(y[i], y[i], ss);
        mr = fmaf(m[i] * w2[i], y[i], mr);
      }
      team_sum<WIDE>(ss, mr, team, lds);
      const float rs2 = 1.0f / sqrtf(ss * inv + p.eps);
      const float k = rs2 * rs2 * rs2 * mr * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d[i] += m[i] * w2[i] * rs2 - k * y[i];
        dw2[i] = fmaf(m[i], y[i] * rs2, dw2[i]);
      }
    }
    if (p.dresidual) store_row<DT, V, VEC>(p.dresidual, at.out, t, team, width, d);
    float dn = 0.0f;
    q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float slope = 0.0f, a = 1.0f;
      if (p.gate) a = activate(z[i], p.act, slope);
      ds[i] = fmaf(d[i], x[i] * w[i] * a, ds[i]);
      const float dy = d[i] * sc[i];
      z[i] = dy * x[i] * w[i] * slope;
      dw[i] = fmaf(dy * a, x[i], dw[i]);
      d[i] = dy * a * w[i];
      dn = fmaf(d[i], x[i], dn);
    }
    if (p.dgate) store_row<DT, V, VEC>(p.dgate, at.out, t, team, width, z);
    if (p.dx) {
      team_sum<WIDE>(dn, q, team, lds);
      dn *= inv;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = rs * (d[i] - x[i] * dn);
      store_row<DT, V, VEC>(p.dx, at.out, t, team, width, d);
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
  if (p.block == 256) return p.vectors == 1 ? run<DT, 1, true, 256>(p, back, s) : run<DT, 2, true, 256>(p, back, s);
  if (p.block == 512) return run<DT, 2, true, 512>(p, back, s);
  return run<DT, 2, true, 1024>(p, back, s);
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
