// norm_device.h — what the norms' kernels share: a row of values in the registers
// of its team of threads, its loads and stores by type, sums over the team, and the
// gate's activation.

#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

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

}  // namespace qnorm
