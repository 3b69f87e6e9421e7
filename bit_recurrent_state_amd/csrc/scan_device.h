// scan_device.h — what the scan's kernels share: chunk lookup, element access
// by type, splitting FP32 values into bfloat16 terms, and the matrix product of
// split operands.

#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "scan_launch.h"

namespace qscan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int C = kChunk;
constexpr int P = kTerms;
constexpr int CP = C + 8;  // LDS row of kChunk terms; 36 words: 16 rows start in 16 banks

enum { GDN = 0, GLA = 1, SCALAR = 2, KDA = 3 };

// One chunk of a sequence.
struct Chunk {
  int n;        // sequence
  int ci;       // chunk of the sequence
  int len;      // tokens in the chunk
  int64_t row;  // first row
};

__device__ __forceinline__ int64_t offset_of(const Params& p, int n) {
  if (!p.offsets) return p.tokens / p.batch * n;
  const int64_t o = p.offsets[n];
  return o < 0 ? 0 : o > p.tokens ? p.tokens : o;
}

// Which chunk a slot is: sequence n starts at slot offset / C + n, which
// leaves room for its ceil(len / C) chunks and needs no sums over sequences.
// All lanes of a wave search together, 64 probes a step.
__device__ __forceinline__ bool find_chunk(const Params& p, int slot, Chunk& c) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = p.batch;
  int64_t o0, o1;
  for (;;) {
    const int step = (hi - lo + 63) / 64;
    const int64_t at = lo + (int64_t)lane * step;
    // one probe past the end: it is the last sequence's end
    const int64_t o = offset_of(p, (int)(at < p.batch ? at : p.batch));
    const bool le = at < hi && o / C + at <= slot;
    const int count = __popcll(__ballot(le));
    if (count == 0) return false;
    lo += (count - 1) * step;
    if (step == 1) {
      o0 = __shfl(o, count - 1);
      o1 = count < 64 ? __shfl(o, count) : offset_of(p, lo + 1);
      break;
    }
    hi = hi < lo + step ? hi : lo + step;
  }
  const int64_t ci = slot - (o0 / C + lo);
  const int64_t left = o1 - o0 - ci * C;
  if (ci < 0 || left <= 0 || o1 - o0 <= p.short_len) return false;
  c.n = lo;
  c.ci = (int)ci;
  c.len = left < C ? (int)left : C;
  c.row = o0 + ci * C;
  return true;
}

// The first kernel of a call searches and leaves what it found for the others:
// one load instead of a search's two or three that wait for each other.
__device__ __forceinline__ bool find_and_note(const Params& p, int slot, bool note, Chunk& c) {
  const bool found = find_chunk(p, slot, c);
  if (note && threadIdx.x == 0)
    p.chunks[slot] = found ? make_int4(c.n, c.ci, c.len, (int)c.row) : make_int4(-1, 0, 0, 0);
  return found;
}

__device__ __forceinline__ bool noted_chunk(const Params& p, int slot, Chunk& c) {
  const int4 e = p.chunks[slot];
  c.n = e.x;
  c.ci = e.y;
  c.len = e.z;
  c.row = e.w;
  return c.n >= 0;
}

// ---- elements of the caller's arrays -------------------------------------------------------

__device__ __forceinline__ float bf16_to_f(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype) {
  if (dtype == 1) return bf16_to_f(static_cast<const uint16_t*>(p)[i]);
  if (dtype == 2) return (float)static_cast<const _Float16*>(p)[i];
  return static_cast<const float*>(p)[i];
}

// The same in two steps, for many elements at once: load_elem branches on the
// type and converts, so that each load would be waited for before the next.
template <int N, class I>
__device__ __forceinline__ void load_raw(const void* p, const I (&at)[N], int dtype,
                                         uint32_t (&raw)[N]) {
  if (dtype == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = static_cast<const uint32_t*>(p)[at[i]];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = static_cast<const uint16_t*>(p)[at[i]];
  }
}

// Without branches: the type is the same for all, but a branch per element
// would cut the code around it into pieces.
__device__ __forceinline__ float from_raw(uint32_t raw, int dtype) {
  const uint32_t half = dtype == 2 ? ~0u : 0u;
  const uint32_t h = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)raw));
  return __uint_as_float((h & half) | ((raw << (dtype == 1 ? 16 : 0)) & ~half));
}

// Two floats to packed bfloat16, to nearest, ties to even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// Outputs are rounded here, once, to the caller's type.
__device__ __forceinline__ void store_elem(void* p, int64_t i, int dtype, float x) {
  if (dtype == 1)
    static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(x, 0.0f);
  else if (dtype == 2)
    static_cast<_Float16*>(p)[i] = (_Float16)x;
  else
    static_cast<float*>(p)[i] = x;
}

// N outputs, those with `ok`.
template <int N, class I>
__device__ __forceinline__ void store_elems(void* p, const I (&at)[N], const bool (&ok)[N],
                                            int dtype, const float (&x)[N]) {
  if (dtype == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok[i]) static_cast<float*>(p)[at[i]] = x[i];
  } else {
    const uint32_t half = dtype == 2 ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)x[i]);
      if (ok[i])
        static_cast<uint16_t*>(p)[at[i]] = (uint16_t)((h & half) | (pack_bf16(x[i], 0.0f) & ~half));
    }
  }
}

// e^x to an ulp or two for x <= 88 (0 far below): 2^t (1 + r ln 2), x log2 e = t + r.
__device__ __forceinline__ float fast_exp(float x) {
  const float hi = 1.44269502f, lo = 1.92596303e-8f;
  const float t = x * hi;
  const float r = fmaf(x, lo, fmaf(x, hi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147182f, e);
}

// Sums of log decays in fixed point, as powers of two with 25 bits behind the
// point: differences of sums are then exact, and a sum of a chunk that decays by
// up to e^kFarDecay = 2^34.6 is as good at its end as at its start (in FP32 it
// would be held to 2^-20 there).  `fixed` rounds a 64-bit sum to 2^-26 of an
// octave, 1.1e-8; what does not fit wraps round and is not used.
__device__ __forceinline__ int fixed(double s) {
  const double scale = 1.4426950408889634 * 33554432.0, units = 6755399441055744.0;  // 1.5 * 2^52
  return (int)(uint32_t)__double_as_longlong(fma(s, scale, units));
}

// 2^(x 2^-25) to an ulp or two.
__device__ __forceinline__ float fixed_exp(int x) {
  return ldexpf(__builtin_amdgcn_exp2f((float)(x & 0x1FFFFFF) * 0x1p-25f), x >> 25);
}

// Four neighbouring elements as they lie in memory (16-bit ones two to a word),
// and their values; `even`: they are aligned to four.  In two steps for the
// same reason as load_raw.
__device__ __forceinline__ u32x4 load4(const void* p, int64_t at, int dtype, bool even) {
  if (dtype == 0) {
    const uint32_t* s = static_cast<const uint32_t*>(p) + at;
    return even ? *reinterpret_cast<const u32x4*>(s) : u32x4{s[0], s[1], s[2], s[3]};
  }
  const uint16_t* s = static_cast<const uint16_t*>(p) + at;
  u32x2 w;
  if (even)
    w = *reinterpret_cast<const u32x2*>(s);
  else
    w = u32x2{s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16};
  return u32x4{w.x, w.y, 0, 0};
}

__device__ __forceinline__ void widen4(const u32x4& w, int dtype, float (&x)[4]) {
  const uint32_t words = dtype == 0 ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t half = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
    x[i] = from_raw((w[i] & words) | (half & ~words), dtype);
  }
}

// The same without a branch: places that are not `ok` go to the sink.  Loads
// and stores return in order, and a branch around a store would make every
// later wait for a load wait for newer ones too.
template <int N>
__device__ __forceinline__ void store_always(char* p, const uint32_t (&at)[N], const bool (&ok)[N],
                                             int dtype, float* sink, const float (&x)[N]) {
  char* const s = reinterpret_cast<char*>(sink + (threadIdx.x & 63));
  if (dtype == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<float*>(ok[i] ? p + (uint64_t)at[i] * 4 : s) = x[i];
  } else {
    const uint32_t half = dtype == 2 ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)x[i]);
      *reinterpret_cast<uint16_t*>(ok[i] ? p + (uint64_t)at[i] * 2 : s) =
          (uint16_t)((h & half) | (pack_bf16(x[i], 0.0f) & ~half));
    }
  }
}

// Log decays below -87 count as -87; a NaN stays.
__device__ __forceinline__ float gate(float g) { return g < -87.0f ? -87.0f : g; }

// ---- FP32 as a sum of bfloat16 terms --------------------------------------------------------
// x = t0 + t1 + ..., each term the rest rounded to bfloat16: N terms hold x to
// 2^(-8 N) of itself, so three hold an FP32 value (24 bits).

template <int N>
__device__ __forceinline__ void split4(const float (&x)[4], u32x2 (&t)[N]) {
  float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    t[n].x = pack_bf16(r[0], r[1]);
    t[n].y = pack_bf16(r[2], r[3]);
    if (n + 1 < N) {
      r[0] -= __uint_as_float(t[n].x << 16);
      r[1] -= __uint_as_float(t[n].x & 0xFFFF0000u);
      r[2] -= __uint_as_float(t[n].y << 16);
      r[3] -= __uint_as_float(t[n].y & 0xFFFF0000u);
    }
  }
}

template <int N>
struct Frag {  // one operand of a 16 x 16 x 32 product: row lane & 15, columns (lane >> 4) * 8 ..
  u32x4 t[N];
};

template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&x)[8]) {
  Frag<N> f;
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  u32x2 ta[N], tb[N];
  split4<N>(a, ta);
  split4<N>(b, tb);
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = u32x4{ta[n].x, ta[n].y, tb[n].x, tb[n].y};
  return f;
}

template <int N>
__device__ __forceinline__ Frag<N> load_frag(const uint16_t* p, int64_t plane) {
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const u32x4*>(p + n * plane);
  return f;
}

// acc += A B^T over 32 columns.  Of the products of terms i and j those with
// i + j below the number of terms are taken, the smallest first: what is left
// out is below what the terms themselves leave out.  Result: column lane & 15,
// rows (lane >> 4) * 4 + r.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.t[i]),
                                                      __builtin_bit_cast(bf16x8, b.t[j]), acc, 0,
                                                      0, 0);
    }
}

// Four consecutive values of one row into the planes of an LDS array.
template <int N>
__device__ __forceinline__ void put4(uint16_t* dst, int plane, const float (&x)[4]) {
  u32x2 t[N];
  split4<N>(x, t);
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<u32x2*>(dst + n * plane) = t[n];
}

// Operands in the workspace lie in the order in which waves load them: tiles of
// 16 rows x 32 columns, one kilobyte of 64 lanes' 16 bytes, so that a fragment
// load reads eight whole cache lines.  (Rows of 2 DK bytes took 200 cycles a
// load, bound by the lines in flight.)
template <int COLS>
__device__ __forceinline__ int tiled(int row, int col) {
  return ((row >> 4) * (COLS / 32) + (col >> 5)) * 512 + ((row & 15) + ((col & 31) >> 3) * 16) * 8 +
         (col & 7);
}

// Fragment s of row block rb.
template <int N, int COLS>
__device__ __forceinline__ Frag<N> tile_frag(const uint16_t* p, int rb, int s, int64_t plane) {
  return load_frag<N>(p + (rb * (COLS / 32) + s) * 512 + (threadIdx.x & 63) * 8, plane);
}

// q or k of a chunk as the left operand: the caller's bfloat16 rows, or tiles
// in the workspace.  Rows behind the sequence's end repeat its last row: beta is
// zero there, so what they compute reaches neither a state nor an output.
template <int DK, bool DIRECT>
struct Rows {
  const uint16_t* p;
  int64_t stride;
  int last;

  template <int N>
  __device__ __forceinline__ Frag<N> frag(int rb, int s) const {
    const int lane = threadIdx.x & 63;
    if (DIRECT)
      return load_frag<N>(p + min(rb * 16 + (lane & 15), last) * stride + s * 32 + (lane >> 4) * 8, 0);
    return tile_frag<N, DK>(p, rb, s, C * DK);
  }
};

template <int DK, bool DIRECT>
__device__ __forceinline__ Rows<DK, DIRECT> rows_of(const Params& p, const void* user,
                                                    const uint16_t* ws, int64_t stride,
                                                    bool per_head, int slot, int h,
                                                    const Chunk& c) {
  const int group = p.heads / p.heads_qk;
  Rows<DK, DIRECT> r;
  if (DIRECT) {
    r.p = static_cast<const uint16_t*>(user) + c.row * stride + (int64_t)(h / group) * DK;
    r.stride = stride;
    r.last = c.len - 1;
  } else {
    const int64_t sh = per_head ? (int64_t)slot * p.heads + h
                                : (int64_t)slot * p.heads_qk + h / group;
    r.p = ws + sh * P * C * DK;
  }
  return r;
}

__device__ __forceinline__ float* rows_at(const Params& p, int slot, int h) {
  return p.rows + ((int64_t)slot * p.heads + h) * (5 * C);
}

// Sums over the 16 lanes that hold one row of a product, and over 8 lanes, by
// DPP: shuffles go through LDS and were half the time of kernels with many.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float sum16(float x) {
  x += dpp<0x128>(x);  // row_ror 8, 4, 2, 1
  x += dpp<0x124>(x);
  x += dpp<0x122>(x);
  x += dpp<0x121>(x);
  return x;
}

__device__ __forceinline__ float sum8(float x) {
  x += dpp<0xB1>(x);   // quad_perm 1, 0, 3, 2
  x += dpp<0x4E>(x);   // quad_perm 2, 3, 0, 1
  x += dpp<0x141>(x);  // row_half_mirror: the other four of eight
  return x;
}

}  // namespace qscan
