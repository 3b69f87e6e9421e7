// group_norm.hip — the group norm of include/qstate_group_norm.h and its gradients.
//
// A row (one group of one token) stays in the registers of its team of threads
// from its load to its store: the mean first, then the variance of the centered
// values, so that no sum of squares cancels.  The backward pass computes the
// normalised values again instead of reading them.  Teams stay in their group: its
// weights are loaded, and their gradients summed, once per team.  8191 rows of 8 groups
// of 512 bfloat16 values with a gate in front take 42 us (201 MB, 4.8 TB/s: memory);
// 8192 x 32 x 128 activated 35 us forward (134 MB, 3.8 TB/s) and 57 backward (201 MB, 3.5
// TB/s), where the activation's instructions take as long as the memory.

#include <hip/hip_runtime.h>

#include "group_norm_launch.h"
#include "norm_device.h"

namespace qnorm {

// Where a team's row lies in x and the gate.  The teams' number is a multiple of the groups: a team
// stays in its group and goes `step` tokens on at a time.
struct GroupPlace {
  int64_t x, gate, xstep, gstep;
  __device__ __forceinline__ GroupPlace(const GroupParams& p, int64_t first) {
    const int64_t tok = first / p.groups, in = (first - tok * p.groups) * p.width;
    const int64_t step = p.teams / p.groups;
    x = tok * p.xs + in;
    gate = tok * p.gs + in;
    xstep = step * p.xs;
    gstep = step * p.gs;
  }
  __device__ __forceinline__ void next() {
    x += xstep;
    gate += gstep;
  }
};

// Sums over the team, by DPP inside 16 lanes: shuffles through LDS cost as much as a quarter of the
// row's own arithmetic.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

template <bool WIDE>
__device__ __forceinline__ void row_sums(float& a, float& b, int team, float (*lds)[2]) {
  if (WIDE) {
    team_sum<true>(a, b, team, lds);
    return;
  }
  auto both = [&](auto step) {
    a += step(a);
    b += step(b);
  };
  if (team > 1) both([](float x) { return dpp<0xB1>(x); });    // quad_perm 1, 0, 3, 2
  if (team > 2) both([](float x) { return dpp<0x4E>(x); });    // quad_perm 2, 3, 0, 1
  if (team > 4) both([](float x) { return dpp<0x141>(x); });   // row_half_mirror
  if (team > 8) both([](float x) { return dpp<0x140>(x); });   // row_mirror
  if (team > 16) both([](float x) { return __shfl_xor(x, 16); });
  if (team > 32) both([](float x) { return __shfl_xor(x, 32); });
}

// 1 / sqrt(v): the instruction's, one Newton step on; the library's where squares would leave the range.
__device__ __forceinline__ float inverse_root(float v) {
  float r = __builtin_amdgcn_rsqf(v);
  const float e = fmaf(-v * r, r, 1.0f);
  r = fmaf(0.5f * r, e, r);
  if (!(v >= 0x1p-100f && v <= 0x1p100f)) r = 1.0f / sqrtf(v);
  return r;
}

// act(z), for the gradient its slope.  What only ends in 16 bits, the forward pass of those types, takes
// exp(-z) as 2^(-z log2 e) without the product's rest (an error of |z| 2^-24 of it, half a step of the
// types being 2^-12 at least).  The backward pass also sums into FP32 gradients of the weights: t = -z
// log2 e rounded is off by -z - t ln 2, a fused multiply-add and exact but for the rest of ln 2 (|z|
// 2.8e-9), and e takes it on, one more.  The reciprocal is the instruction's, to an ulp.  11 and 13
// instead of 20 instructions' time a value, which is what bounds the kernels.
template <int DT, bool SLOPE>
__device__ __forceinline__ float act_of(float z, int act, float& slope) {
  if (DT == 0) return activate(z, act, slope);
  const float c = __builtin_elementwise_maximum(z, -87.0f);  // NaN stays
  float e, s;
  if (SLOPE) {
    const float d = __builtin_elementwise_minimum(c, 87.0f);
    const float t = d * -1.44269502f;
    e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, fmaf(t, -0.693147182f, -d), e);
    s = __builtin_amdgcn_rcpf(1.0f + e);
    const float q = s * e;  // 1 - s without cancellation; with a gate of infinity, nothing of it
    slope = act == 0 ? s * fmaf(d, q, 1.0f) : s * q;
  } else {
    e = __builtin_amdgcn_exp2f(c * -1.44269502f);
    s = __builtin_amdgcn_rcpf(1.0f + e);
  }
  return act == 0 ? c * s : s;
}

// A row's values by type, zeros behind its width.  FULL: every thread's are inside.
template <int DT, int V, bool VEC, bool FULL>
__device__ __forceinline__ void values(const Raw<DT, V>& r, int t, int team, int width,
                                       float (&x)[V * 8]) {
  // (a width that nothing lies behind: the comparisons fall away)
  widen<DT, V, VEC>(r, FULL ? 0 : t, FULL ? 1 : team, FULL ? 1 << 30 : width, x);
}

// x becomes the normalised row (columns behind the width stay zero); returns
// what it was multiplied by.
template <int V, bool WIDE, bool VEC, bool FULL>
__device__ __forceinline__ float normalise(const GroupParams& p, int t, int team,
                                           float (*lds)[2], float (&x)[V * 8]) {
  const float inv = 1.0f / (float)p.width;
  float s = 0.0f, unused = 0.0f;
  if (p.center) {
#pragma unroll
    for (int i = 0; i < V * 8; ++i) s += x[i];
    row_sums<WIDE>(s, unused, team, lds);
    const float mean = s * inv;
#pragma unroll
    for (int i = 0; i < V * 8; ++i)
      x[i] = FULL || column<VEC>(i / 8, i % 8, t, team) < p.width ? x[i] - mean : 0.0f;
    s = unused = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < V * 8; ++i) s = fmaf(x[i], x[i], s);
  row_sums<WIDE>(s, unused, team, lds);
  const float r = inverse_root(s * inv + p.eps);
#pragma unroll
  for (int i = 0; i < V * 8; ++i) x[i] *= r;
  return r;
}

template <int V, bool VEC>
__device__ __forceinline__ void load_affine(const GroupParams& p, int64_t first, int t, int team,
                                            float (&w)[V * 8], float (&b)[V * 8]) {
  const int64_t at = p.shared ? 0 : first % p.groups * p.width;
  load_weight<V, VEC>(p.weight, at, t, team, p.width, w);
  load_weight<V, VEC>(p.bias, at, t, team, p.width, b);
  if (!p.bias) {
#pragma unroll
    for (int i = 0; i < V * 8; ++i) b[i] = 0.0f;
  }
}

template <int DT, int V, bool WIDE, bool VEC, bool FULL, int BLOCK>
__global__ void __launch_bounds__(BLOCK) group_forward_kernel(GroupParams p) {
  constexpr int N = V * 8;
  __shared__ float lds[BLOCK / 64][2];
  const int team = WIDE ? BLOCK : p.team, t = threadIdx.x & (team - 1);
  const int64_t first = (int64_t)blockIdx.x * (BLOCK / team) + threadIdx.x / team;
  const int width = p.width;
  float w[N], b[N];
  load_affine<V, VEC>(p, first, t, team, w, b);
  // WIDE teams are whole workgroups, the others stay inside a wave: no barrier is passed by a part
  int64_t row = first < p.teams ? first : p.rows;
  if (row >= p.rows) return;
  Raw<DT, V> rx, rz;
  GroupPlace at(p, row);
  auto load = [&]() {
    load_raw<DT, V, VEC>(p.x, at.x, t, team, width, rx);
    if (p.gate) load_raw<DT, V, VEC>(p.gate, at.gate, t, team, width, rz);
    at.next();
  };
  load();
  for (; row < p.rows; row += p.teams) {
    float x[N], a[N], slope;
    values<DT, V, VEC, FULL>(rx, t, team, width, x);
    if (p.gate) {
      values<DT, V, VEC, FULL>(rz, t, team, width, a);
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = act_of<DT, false>(a[i], p.act, slope);
    }
    if (row + p.teams < p.rows) load();
    if (p.mode == GATE_FIRST) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= a[i];
    }
    normalise<V, WIDE, VEC, FULL>(p, t, team, lds, x);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(x[i], w[i], b[i]);
    if (p.mode == GATE) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= a[i];
    } else if (p.mode == ACTIVATE) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = act_of<DT, false>(x[i], p.act, slope);
    }
    store_row<DT, V, VEC>(p.y, row * width, t, team, width, x);
  }
}

template <int DT, int V, bool WIDE, bool VEC, bool FULL, int BLOCK>
__global__ void __launch_bounds__(BLOCK) group_backward_kernel(GroupParams p) {
  constexpr int N = V * 8;
  __shared__ float lds[BLOCK / 64][2];
  const int team = WIDE ? BLOCK : p.team, t = threadIdx.x & (team - 1);
  const int64_t first = (int64_t)blockIdx.x * (BLOCK / team) + threadIdx.x / team;
  const int width = p.width;
  const float inv = 1.0f / (float)width;
  float w[N], b[N], dw[N], db[N];
  load_affine<V, VEC>(p, first, t, team, w, b);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.0f;
  Raw<DT, V> rx, rz, rd;
  int64_t row = first < p.teams ? first : p.rows;
  GroupPlace at(p, row);
  auto load = [&](int64_t r) {
    load_raw<DT, V, VEC>(p.x, at.x, t, team, width, rx);
    if (p.gate) load_raw<DT, V, VEC>(p.gate, at.gate, t, team, width, rz);
    load_raw<DT, V, VEC>(p.dy, r * width, t, team, width, rd);
    at.next();
  };
  if (row < p.rows) load(row);
  for (; row < p.rows; row += p.teams) {
    const int64_t out = row * width;
    float x[N], u[N], a[N], slope[N], d[N];
    values<DT, V, VEC, FULL>(rx, t, team, width, x);
    if (p.gate) {
      values<DT, V, VEC, FULL>(rz, t, team, width, a);
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = act_of<DT, true>(a[i], p.act, slope[i]);
    }
    values<DT, V, VEC, FULL>(rd, t, team, width, d);
    if (row + p.teams < p.rows) load(row + p.teams);
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = x[i];
    if (p.mode == GATE_FIRST) {
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] *= a[i];
    }
    const float r = normalise<V, WIDE, VEC, FULL>(p, t, team, lds, u);
    if (p.mode == GATE) {
      float z[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        z[i] = d[i] * fmaf(u[i], w[i], b[i]) * slope[i];
        d[i] *= a[i];
      }
      if (p.dgate) store_row<DT, V, VEC>(p.dgate, out, t, team, width, z);
    } else if (p.mode == ACTIVATE) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float sl;
        act_of<DT, true>(fmaf(u[i], w[i], b[i]), p.act, sl);
        d[i] *= sl;
      }
    }
    float m = 0.0f, mh = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dw[i] = fmaf(d[i], u[i], dw[i]);
      db[i] += d[i];
      d[i] *= w[i];
      m += d[i];
      mh = fmaf(d[i], u[i], mh);
    }
    if (!p.dx && !(p.dgate && p.mode == GATE_FIRST)) continue;
    row_sums<WIDE>(m, mh, team, lds);
    m = p.center ? m * inv : 0.0f;
    mh *= inv;
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = r * (d[i] - fmaf(u[i], mh, m));
    if (p.mode == GATE_FIRST) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u[i] = d[i] * x[i] * slope[i];
        d[i] *= a[i];
      }
    }
    if (p.dx) store_row<DT, V, VEC>(p.dx, out, t, team, width, d);
    if (p.dgate && p.mode == GATE_FIRST) store_row<DT, V, VEC>(p.dgate, out, t, team, width, u);
  }
  if (!p.part) return;
  int64_t mine = first;  // this team's part
  if (!WIDE && p.shared) {
    // one weight for all rows: the teams of a wave first
#pragma unroll
    for (int i = 0; i < N; ++i)
      for (int o = team; o < 64; o *= 2) {
        dw[i] += __shfl_xor(dw[i], o);
        db[i] += __shfl_xor(db[i], o);
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
    if (p.dweight) o[0] = dw[i];
    if (p.dbias) o[p.partials * width] = db[i];
  }
}

// The teams' parts (of a group, where weights differ by group), summed in a fixed order: a workgroup takes 32
// columns, its 8 rows of threads every 8th part each, in 64 bits.
__global__ void __launch_bounds__(256) group_parts_kernel(GroupParams p) {
  __shared__ double lds[8][32];
  const int which = blockIdx.z, g = blockIdx.y;
  float* out = which == 0 ? p.dweight : p.dbias;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  const int64_t step = p.shared ? 1 : p.groups;
  double s = 0.0;
  if (c < p.width)
#pragma unroll 4
    for (int64_t i = g + y * step; i < p.partials; i += 8 * step)
      s += p.part[((int64_t)which * p.partials + i) * p.width + c];
  lds[y][threadIdx.x & 31] = s;
  __syncthreads();
  if (y == 0 && c < p.width) {
    for (int k = 1; k < 8; ++k) s += lds[k][threadIdx.x];
    out[(int64_t)g * p.width + c] = (float)s;
  }
}

template <int DT, int V, bool WIDE, bool VEC, bool FULL, int BLOCK>
static hipError_t launch(const GroupParams& p, bool back, hipStream_t s) {
  const int64_t per = BLOCK / p.team;
  const dim3 grid((unsigned)((p.teams + per - 1) / per));
  if (back)
    group_backward_kernel<DT, V, WIDE, VEC, FULL, BLOCK><<<grid, BLOCK, 0, s>>>(p);
  else
    group_forward_kernel<DT, V, WIDE, VEC, FULL, BLOCK><<<grid, BLOCK, 0, s>>>(p);
  return hipGetLastError();
}

template <int DT, int V, bool WIDE, int BLOCK>
static hipError_t run(const GroupParams& p, bool back, hipStream_t s) {
  if (!p.aligned) return launch<DT, V, WIDE, false, false, BLOCK>(p, back, s);
  return p.width == V * 8 * p.team ? launch<DT, V, WIDE, true, true, BLOCK>(p, back, s)
                                   : launch<DT, V, WIDE, true, false, BLOCK>(p, back, s);
}

template <int DT>
static hipError_t pick(const GroupParams& p, bool back, hipStream_t s) {
  if (!p.wide) return run<DT, 1, false, 256>(p, back, s);
  switch (p.block) {
    case 128: return run<DT, 1, true, 128>(p, back, s);
    case 256: return run<DT, 1, true, 256>(p, back, s);
    case 512: return run<DT, 1, true, 512>(p, back, s);
    default: return p.vectors == 1 ? run<DT, 1, true, 1024>(p, back, s) : run<DT, 2, true, 1024>(p, back, s);
  }
}

static hipError_t by_type(const GroupParams& p, int dtype, bool back, hipStream_t s) {
  switch (dtype) {
    case 0: return pick<0>(p, back, s);
    case 1: return pick<1>(p, back, s);
    case 2: return pick<2>(p, back, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t group_forward(const GroupParams& p, int dtype, hipStream_t s) {
  return by_type(p, dtype, false, s);
}

hipError_t group_backward(const GroupParams& p, int dtype, hipStream_t s) {
  const hipError_t e = p.teams > 0 ? by_type(p, dtype, true, s) : hipSuccess;
  if (e != hipSuccess || !(p.dweight || p.dbias)) return e;
  group_parts_kernel<<<dim3((p.width + 31) / 32, p.shared ? 1 : p.groups, 2), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace qnorm
