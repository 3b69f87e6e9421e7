// scan_prep.h — the parts of the scan that every chunk computes for itself:
// the operands' transposes and terms, the decays, A and (I + L beta)^-1.

#pragma once

#include "scan_device.h"

namespace qscan {

// ---- transposes and terms of q and k, one gate per token ------------------------------------
// One workgroup per (slot, q/k head).  Threads run over channels, so the
// caller's rows are read whole; each thread turns 8 tokens of its channel into
// 16 bytes of the transposed planes.
template <int DK, bool BWD>
__device__ __forceinline__ void take_operands(const Params& p, int slot, int hq) {
  Chunk c;
  if (!find_and_note(p, slot, hq == 0, c)) return;
  const int64_t sh = (int64_t)slot * p.heads_qk + hq;
  if (p.direct) {
    // bfloat16 is moved as it is: 8 tokens of 2 channels per thread
    for (int which = 0; which <= BWD; ++which) {
      const uint16_t* src = static_cast<const uint16_t*>(which ? p.q : p.k);
      const int64_t stride = which ? p.qs : p.ks;
      uint16_t* tr = which ? p.qt : p.kt;
      for (int u = threadIdx.x; u < DK / 2 * (C / 8); u += 256) {
        const int ch = u % (DK / 2) * 2, t0 = u / (DK / 2) * 8;
        uint32_t x[8];
        const uint16_t* at = src + (int64_t)hq * DK + ch;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = *reinterpret_cast<const uint32_t*>(at + (c.row + min(t0 + i, c.len - 1)) * stride);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t0 + i >= c.len) x[i] = 0;
        u32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = (x[2 * i] & 0xFFFFu) | (x[2 * i + 1] << 16);
          hi[i] = (x[2 * i] >> 16) | (x[2 * i + 1] & 0xFFFF0000u);
        }
        *reinterpret_cast<u32x4*>(tr + sh * DK * C + tiled<C>(ch, t0)) = lo;
        *reinterpret_cast<u32x4*>(tr + sh * DK * C + tiled<C>(ch + 1, t0)) = hi;
      }
    }
    return;
  }
  for (int which = 0; which < 2; ++which) {
    const void* src = which ? p.q : p.k;
    const int64_t stride = which ? p.qs : p.ks;
    uint16_t* tr = which ? p.qt : p.kt;
    uint16_t* rw = which ? p.qrow : p.krow;
    const bool transpose = which == 0 || BWD;
    for (int u = threadIdx.x; transpose && u < DK * (C / 8); u += 256) {
      const int ch = u % DK, t0 = u / DK * 8;
      float x[8];
      int64_t at[8];
      uint32_t raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        at[i] = (c.row + min(t0 + i, c.len - 1)) * stride + (int64_t)hq * DK + ch;
      load_raw<8>(src, at, p.dtype, raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = t0 + i < c.len ? from_raw(raw[i], p.dtype) : 0.0f;
      const Frag<P> f = split8<P>(x);
#pragma unroll
      for (int n = 0; n < P; ++n)
        *reinterpret_cast<u32x4*>(tr + (sh * P + n) * DK * C + tiled<C>(ch, t0)) = f.t[n];
    }
    for (int u = threadIdx.x; u < DK / 8 * C; u += 256) {  // rows: 8 channels of a token
      const int c0 = u % (DK / 8) * 8, tk = u / (DK / 8);
      float x[8];
      int64_t at[8];
      uint32_t raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        at[i] = (c.row + min(tk, c.len - 1)) * stride + (int64_t)hq * DK + c0 + i;
      load_raw<8>(src, at, p.dtype, raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = tk < c.len ? from_raw(raw[i], p.dtype) : 0.0f;
      const Frag<P> f = split8<P>(x);
#pragma unroll
      for (int n = 0; n < P; ++n)
        *reinterpret_cast<u32x4*>(rw + (sh * P + n) * DK * C + tiled<DK>(tk, c0)) = f.t[n];
    }
  }
}

template <int DK>
__global__ void __launch_bounds__(256) operands_kernel(Params p) {
  take_operands<DK, true>(p, blockIdx.x, blockIdx.y);
}

// ---- (I + M)^-1 of a strictly lower triangular M --------------------------------------------
// In LDS, in FP32, stable as forward substitution is: the four diagonal blocks
// of 16 by substitution (a lane per column, a wave per block), then blocks of
// 32 and 64 by X21 = -X22 (M21 X11) on FP32 matrix instructions.  One product's
// result is the next one's right operand without leaving its registers: step r
// of a product takes the columns k = 4 (lane >> 4) + r, as results hold rows.
// 64 steps of substitution by one wave took 20 us a workgroup, this 2 (read from
// the clock inside the kernel).
typedef float Square[C + 4];

// D += A B for one 16 x 16 block: A from LDS rows, B given as four results.
__device__ __forceinline__ f32x4 block_mma(const Square* A, int ra, int ca, const f32x4& b,
                                           f32x4 acc) {
  const int lane = threadIdx.x & 63;
  const f32x4 a = *reinterpret_cast<const f32x4*>(&A[ra * 16 + (lane & 15)][ca * 16 + (lane >> 4) * 4]);
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], acc, 0, 0, 0);
  return acc;
}

__device__ __forceinline__ f32x4 block_load(const Square* X, int rb, int cb) {
  const int lane = threadIdx.x & 63;
  f32x4 b;
#pragma unroll
  for (int r = 0; r < 4; ++r) b[r] = X[rb * 16 + (lane >> 4) * 4 + r][cb * 16 + (lane & 15)];
  return b;
}

__device__ __forceinline__ void block_store(Square* X, int rb, int cb, const f32x4& b, float sign) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    X[rb * 16 + (lane >> 4) * 4 + r][cb * 16 + (lane & 15)] = sign * b[r];
}

// N matrices M (their strict lower triangles set, the rest zero), overwritten
// by the inverses.  All waves (four or eight) call this, with M complete in LDS.
template <int N>
__device__ __forceinline__ void invert(Square* M0, Square* M1) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col = lane & 15, g = lane >> 4;
  {
    const Square* M = N == 2 && (g & 1) ? M1 : M0;
    const int wave = threadIdx.x >> 6 & 3;  // waves beyond four repeat the first four's work
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(&M[wave * 16 + i][wave * 16 + m]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (m + j < i) {
            if (j & 1)
              s1 = fmaf(v[j], x[m + j], s1);
            else
              s0 = fmaf(v[j], x[m + j], s0);
          }
      }
      x[i] = (col == i ? 1.0f : 0.0f) - (s0 + s1);
    }
    __syncthreads();
    if (g < N) {
      Square* X = g ? M1 : M0;
#pragma unroll
      for (int i = 0; i < 16; ++i) X[wave * 16 + i][wave * 16 + col] = x[i];
    }
  }
  __syncthreads();
  const f32x4 zero = {0, 0, 0, 0};
  if (wave < 2 * N) {  // blocks (1, 0) and (3, 2)
    Square* X = wave < 2 ? M0 : M1;
    const int b = (wave & 1) * 2;
    const f32x4 d = block_mma(X, b + 1, b, block_load(X, b, b), zero);
    block_store(X, b + 1, b, block_mma(X, b + 1, b + 1, d, zero), -1.0f);
  }
  __syncthreads();
  f32x4 y2 = zero, y3 = zero;
  Square* X = wave < 2 ? M0 : M1;
  const int b = wave & 1;
  if (wave < 2 * N) {  // column block b of the lower left quarter
    f32x4 d2 = zero, d3 = zero;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (c >= b) {
        const f32x4 x = block_load(X, c, b);
        d2 = block_mma(X, 2, c, x, d2);
        d3 = block_mma(X, 3, c, x, d3);
      }
    y2 = block_mma(X, 2, 2, d2, zero);
    y3 = block_mma(X, 3, 3, d3, block_mma(X, 3, 2, d2, zero));
  }
  __syncthreads();
  if (wave < 2 * N) {
    block_store(X, 2, b, y2, -1.0f);
    block_store(X, 3, b, y3, -1.0f);
  }
  __syncthreads();
}

// What follows once M = L diag(beta) (and, backward, M2 = diag(beta) L) lies in
// LDS: the inverses, the second transposed.
template <bool BWD>
__device__ __forceinline__ void store_inverses(const Params& p, Square* M, Square* M2, int64_t sh) {
  __syncthreads();
  invert<BWD ? 2 : 1>(M, M2);
  uint16_t* t1 = p.t + sh * P * C * C;
  for (int u = threadIdx.x; u < C * C / 4; u += 256) {
    const int r = u / (C / 4), q0 = u % (C / 4) * 4;
    if (r < 32 && q0 >= 32) continue;  // zeros that are not read
    const f32x4 v = *reinterpret_cast<const f32x4*>(&M[r][q0]);
    const float x[4] = {v[0], v[1], v[2], v[3]};
    put4<P>(t1 + tiled<C>(r, q0), C * C, x);
  }
  if (BWD) {
    uint16_t* t2 = p.t2t + sh * P * C * C;
    for (int u = threadIdx.x; u < C * C / 4; u += 256) {
      const int r = u % C, q0 = u / C * 4;
      if (r >= 32 && q0 < 32) continue;
      // rows by lane: LDS columns are then read without conflicts
      const float x[4] = {M2[q0][r], M2[q0 + 1][r], M2[q0 + 2][r], M2[q0 + 3][r]};
      put4<P>(t2 + tiled<C>(r, q0), C * C, x);
    }
  }
}

// d_o as planes of rows, where the backward kernels cannot take the caller's.
__device__ __forceinline__ void store_dop(const Params& p, const Chunk& c, int64_t sh, int h) {
  if (!p.dop) return;
  for (int u = threadIdx.x; u < C * (p.dvp / 8); u += blockDim.x) {
    const int t = u / (p.dvp / 8), v0 = u % (p.dvp / 8) * 8;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = t < c.len && v0 + i < p.dv
                 ? load_elem(p.dO, ((c.row + t) * p.heads + h) * p.dv + v0 + i, p.dtype)
                 : 0.0f;
    const Frag<P> f = split8<P>(x);
    for (int n = 0; n < p.dop_terms; ++n)
      *reinterpret_cast<u32x4*>(p.dop + ((sh * p.dop_terms + n) * C + t) * p.dvp + v0) =
          n == 0 ? f.t[0] : n == 1 ? f.t[1] : f.t[2];
  }
}

// ---- one gate per token ---------------------------------------------------------------------
// One workgroup per (slot, head).  Sums of log decays are kept in 64 bits:
// the differences c_i - c_j of a chunk that decays far are then still exact.
// Forward: A; backward: its transpose (and both inverses).
//
// VEC: a gate per key channel, for chunks over which no channel decays by more
// than e^kFarDecay: A = (q e^c)(k e^-c)^T and L = (k e^c)(k e^-c)^T are then
// plain products.  Sums of log decays are exact in fixed point but for a rounding
// to 1.1e-8 of the token's and of each block's (scan_device.h), and what two tokens
// have in common cancels exactly, so that a quotient holds to that and the two
// exponentials' ulps at any c.  (One channel's values stay far inside FP32's range:
// e^24 = 3e10.)  Other chunks go to chunk_vector_kernel.
template <int DK, int NPQ, bool VEC, bool DELTA, bool BWD>
__global__ void __launch_bounds__(256) chunk_kernel(Params p) {
  __shared__ double cs[C];
  __shared__ float bs[C];
  __shared__ __align__(16) float M[DELTA ? C : 1][C + 4];
  __shared__ __align__(16) float M2[DELTA && BWD ? C : 1][C + 4];
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!noted_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t sh = (int64_t)slot * p.heads + h;
  if (BWD) store_dop(p, c, sh, h);
  if (VEC && p.far[sh]) return;
  constexpr bool D = NPQ == 1;
  const auto q = rows_of<DK, D>(p, p.q, p.qrow, p.qs, VEC, slot, h, c);
  const auto k = rows_of<DK, D>(p, p.k, VEC ? p.knrow : p.krow, p.ks, VEC, slot, h, c);
  const auto ki = rows_of<DK, D>(p, p.k, p.krow, p.ks, VEC, slot, h, c);  // the reading key of L
  const int fr = lane & 15;
  const int own = wave * 16 + fr;  // forward: token i; backward: token j
  Frag<NPQ> fm[DK / 32], fk[DK / 32];
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    fm[s] = BWD ? k.template frag<NPQ>(wave, s) : q.template frag<NPQ>(wave, s);
    if (DELTA) fk[s] = BWD ? fm[s] : ki.template frag<NPQ>(wave, s);
  }
  if (VEC && wave == 0) bs[lane] = rows_at(p, slot, h)[2 * C + lane];
  if (!VEC && wave == 0) {
    const bool in = lane < c.len;
    const int64_t at = (c.row + lane) * p.heads + h;
    double s = in ? (double)gate(p.g[at]) : 0.0;
    const float beta = in ? p.beta[at] : 0.0f;
    for (int d = 1; d < 64; d *= 2) {
      const double o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    const double end = __shfl(s, 63);
    cs[lane] = s;
    bs[lane] = beta;
    float* r = rows_at(p, slot, h);
    r[lane] = expf((float)s);
    r[C + lane] = expf((float)(end - s));
    r[2 * C + lane] = beta;
    reinterpret_cast<double*>(r + 3 * C)[lane] = s;
  }
  __syncthreads();
  // tile (wave, b): columns own (i forward, j backward), rows of block b
  for (int b = 0; b < 4; ++b) {
    f32x4 acc = {0, 0, 0, 0}, acl = {0, 0, 0, 0};
    const bool need = BWD ? b >= wave : b <= wave;
    if (need) {
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const Frag<NPQ> f = BWD ? q.template frag<NPQ>(b, s) : k.template frag<NPQ>(b, s);
        mma(acc, f, fm[s]);
        if (DELTA) mma(acl, BWD ? ki.template frag<NPQ>(b, s) : f, fk[s]);
      }
    }
    float a[4];
    const int r0 = b * 16 + (lane >> 4) * 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = BWD ? r0 + r : own, j = BWD ? own : r0 + r;
      const float e = VEC ? 1.0f : i >= j ? fast_exp((float)(cs[i] - cs[j])) : 0.0f;
      a[r] = i >= j ? acc[r] * e : 0.0f;
      if (DELTA) {
        const float l = i > j ? acl[r] * e : 0.0f;
        M[i][j] = i > j ? l * bs[j] : 0.0f;
        if (BWD) M2[i][j] = i > j ? bs[i] * l : 0.0f;
      }
    }
    // tiles of 32 columns beside the diagonal that hold only zeros are not read
    uint16_t* dst = (BWD ? p.at : p.a) + sh * P * C * C + tiled<C>(own, r0);
    if (BWD ? (b >> 1) >= (wave >> 1) : (b >> 1) <= (wave >> 1)) put4<P>(dst, C * C, a);
  }
  if (DELTA) store_inverses<BWD>(p, M, M2, sh);
}

// ---- a gate per key channel -----------------------------------------------------------------
// Decays between tokens are products of factors of at most 1 and never
// quotients: inside blocks of 16 tokens prefix sums (first token of the block
// .. i) and suffix sums (j + 1 .. last), between them whole blocks.  Nothing
// overflows, and nothing is lost where gates are strong.
//
// One workgroup per (slot, head): the scaled operands q e^c, k e^c,
// k e^(c_end - c) and, unless the chunk decays too far, k e^-c as rows and as
// columns.  A wave writes a whole tile at a time.
template <int DK, bool DELTA, bool BWD>
__global__ void __launch_bounds__(256) operands_vector_kernel(Params p) {
  constexpr int LP = DK + 4;
  // Sums of log decays inside blocks of 16: up to each token in fixed point; where the chunk decays
  // far, in floats, and from each token to its block's end (the block's sum less the token's would
  // cancel there).
  __shared__ __align__(16) float pre[C][LP], suf[C][LP];
  __shared__ __align__(16) float tot[4][DK];
  auto pre_fixed = [&](int t, int ch) -> int& { return reinterpret_cast<int&>(pre[t][ch]); };
  auto tot_fixed = [&](int b, int ch) -> int& { return reinterpret_cast<int&>(tot[b][ch]); };
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!find_and_note(p, slot, h == 0, c)) return;
  const int64_t sh = (int64_t)slot * p.heads + h;
  const int group = p.heads / p.heads_qk, hq = h / group;
  const bool qeven = p.qs % 4 == 0, keven = p.ks % 4 == 0;
  bool over = false;
  auto sums = [&](auto exact) {  // true: fixed point
    for (int u = threadIdx.x; u < DK * 4; u += 256) {
      const int ch = u % DK, t0 = u / DK * 16;
      float g[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        g[i] = p.g[((c.row + min(t0 + i, c.len - 1)) * p.heads + h) * DK + ch];
      std::conditional_t<exact.value, double, float> s = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        g[i] = t0 + i < c.len ? gate(g[i]) : 0.0f;
        s += g[i];
        if constexpr (exact.value)
          pre_fixed(t0 + i, ch) = fixed(s);
        else
          pre[t0 + i][ch] = s;
      }
      if constexpr (exact.value) {
        tot_fixed(u / DK, ch) = fixed(s);
        over = over || !(s >= -kFarDecay && s <= kFarDecay);
      } else {
        tot[u / DK][ch] = s;
        s = 0.0f;
#pragma unroll
        for (int i = 15; i >= 0; --i) {
          suf[t0 + i][ch] = s;
          s += g[i];
        }
      }
    }
  };
  sums(std::true_type());
  if (threadIdx.x < C) {
    const int t = threadIdx.x;
    rows_at(p, slot, h)[2 * C + t] = t < c.len ? (p.beta ? p.beta[(c.row + t) * p.heads + h] : 1.0f) : 0.0f;
  }
  __syncthreads();
  if (threadIdx.x < DK) {  // no block alone is over, so none has wrapped round
    const int ch = threadIdx.x;
    const int64_t all = (int64_t)tot_fixed(0, ch) + tot_fixed(1, ch) + tot_fixed(2, ch) + tot_fixed(3, ch);
    over = over || all < fixed(-kFarDecay) || all > fixed(kFarDecay);
  }
  const bool far = __syncthreads_or(over);
  if (threadIdx.x == 0) p.far[sh] = far;
  if (far) {
    sums(std::false_type());
    __syncthreads();
  }
  if (threadIdx.x < DK) {
    const int ch = threadIdx.x;
    p.decay[sh * DK + ch] =
        far ? fast_exp((tot[0][ch] + tot[1][ch]) + (tot[2][ch] + tot[3][ch]))
            : fixed_exp(tot_fixed(0, ch) + tot_fixed(1, ch) + tot_fixed(2, ch) + tot_fixed(3, ch));
  }

  // rows: 8 channels of a token
  for (int u = threadIdx.x; u < C * DK / 8; u += 256) {
    const int tile = u >> 6, t = tile / (DK / 32) * 16 + (u & 15);
    const int ch = tile % (DK / 32) * 32 + (u >> 4 & 3) * 8, b = t >> 4;
    const int64_t row = c.row + min(t, c.len - 1);
    float qe[8], ke[8], ko[8], kn[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float x[4], y[4];
      widen4(load4(p.q, row * p.qs + (int64_t)hq * DK + ch + 4 * q, p.dtype, qeven), p.dtype, x);
      widen4(load4(p.k, row * p.ks + (int64_t)hq * DK + ch + 4 * q, p.dtype, keven), p.dtype, y);
      float e[4], eo[4], en[4];
      if (far) {
        f32x4 cs = *reinterpret_cast<const f32x4*>(&pre[t][ch + 4 * q]);
        f32x4 se = *reinterpret_cast<const f32x4*>(&suf[t][ch + 4 * q]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(&tot[m][ch + 4 * q]);
          if (m < b) cs += w;
          if (m > b) se += w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = fast_exp(cs[i]);
          eo[i] = fast_exp(se[i]);
          en[i] = 0.0f;
        }
      } else {
        i32x4 cs = *reinterpret_cast<const i32x4*>(&pre[t][ch + 4 * q]), end = {0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const i32x4 w = *reinterpret_cast<const i32x4*>(&tot[m][ch + 4 * q]);
          if (m < b) cs += w;
          end += w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = fixed_exp(cs[i]);
          eo[i] = fixed_exp(end[i] - cs[i]);
          en[i] = fixed_exp(-cs[i]);
        }
      }
      const float in = t < c.len ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qe[4 * q + i] = in * x[i] * e[i];
        ke[4 * q + i] = in * y[i] * e[i];
        if (BWD) ko[4 * q + i] = in * y[i] * eo[i];
        kn[4 * q + i] = in * y[i] * en[i];
      }
    }
    const int64_t at = sh * P * C * DK + u * 8;
    auto put = [&](uint16_t* dst, const float(&x)[8]) {
      const Frag<P> f = split8<P>(x);
#pragma unroll
      for (int n = 0; n < P; ++n) *reinterpret_cast<u32x4*>(dst + at + n * C * DK) = f.t[n];
    };
    put(p.qrow, qe);
    put(p.knrow, kn);
    if (DELTA) put(p.krow, ke);
    if (BWD) put(p.korow, ko);
  }
  // columns: 8 tokens of a channel
  for (int u = threadIdx.x; u < C * DK / 8; u += 256) {
    const int tile = u >> 6, ch = tile / 2 * 16 + (u & 15);
    const int t0 = tile % 2 * 32 + (u >> 4 & 3) * 8, b = t0 >> 4;
    int64_t aq[8], ak[8];
    uint32_t rq[8], rk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = c.row + min(t0 + i, c.len - 1);
      aq[i] = row * p.qs + (int64_t)hq * DK + ch;
      ak[i] = row * p.ks + (int64_t)hq * DK + ch;
    }
    load_raw<8>(p.k, ak, p.dtype, rk);
    if (BWD) load_raw<8>(p.q, aq, p.dtype, rq);
    // decays from the chunk's start to a token (es), from it to the chunk's end (eo), 1 / es (en); for
    // the gradients the first two, or where the chunk decays far those of the token's block (bs, bo)
    float es[8], eo[8], en[8], bs[8], bo[8];
    if (far) {
      float before = 0.0f, after = 0.0f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m < b) before += tot[m][ch];
        if (m > b) after += tot[m][ch];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float cs = pre[t0 + i][ch], se = suf[t0 + i][ch];
        es[i] = fast_exp(cs + before);
        eo[i] = fast_exp(se + after);
        en[i] = 0.0f;
        bs[i] = fast_exp(cs);
        bo[i] = fast_exp(se);
      }
    } else {
      int before = 0, end = 0;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int x = tot_fixed(m, ch);
        if (m < b) before += x;
        end += x;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = pre_fixed(t0 + i, ch) + before;
        bs[i] = es[i] = fixed_exp(x);
        bo[i] = eo[i] = fixed_exp(end - x);
        en[i] = fixed_exp(-x);
      }
    }
    if (BWD && h % group == 0) {  // q and k as they are, once for the heads that share them
      const int terms = p.dtype == 1 ? 1 : P;
      float xk[8], xq[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xk[i] = t0 + i < c.len ? from_raw(rk[i], p.dtype) : 0.0f;
        xq[i] = t0 + i < c.len ? from_raw(rq[i], p.dtype) : 0.0f;
      }
      const Frag<P> fk = split8<P>(xk), fq = split8<P>(xq);
      const int64_t to = ((int64_t)slot * p.heads_qk + hq) * terms * C * DK + u * 8;
#pragma unroll
      for (int n = 0; n < P; ++n)
        if (n < terms) {
          *reinterpret_cast<u32x4*>(p.kt_raw + to + n * C * DK) = fk.t[n];
          *reinterpret_cast<u32x4*>(p.qt_raw + to + n * C * DK) = fq.t[n];
        }
    }
    float qe[8], ke[8], ko[8], kn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float k = t0 + i < c.len ? from_raw(rk[i], p.dtype) : 0.0f;
      ko[i] = k * eo[i];
      if (BWD) {
        const float q = t0 + i < c.len ? from_raw(rq[i], p.dtype) : 0.0f;
        qe[i] = q * es[i];
        ke[i] = k * es[i];
        kn[i] = k * en[i];
      }
    }
    const int64_t at = sh * P * C * DK + u * 8;
    auto put = [&](uint16_t* dst, const float(&x)[8]) {
      const Frag<P> f = split8<P>(x);
#pragma unroll
      for (int n = 0; n < P; ++n) *reinterpret_cast<u32x4*>(dst + at + n * C * DK) = f.t[n];
    };
    put(p.kt, ko);
    if (BWD) {
      put(p.qt, qe);
      put(p.knt, kn);
      if (DELTA) put(p.ket, ke);
      float* dp = p.pfx + (sh * DK + ch) * C + t0;
      float* ds = p.sfx + (sh * DK + ch) * C + t0;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<f32x4*>(dp + i) = f32x4{bs[i], bs[i + 1], bs[i + 2], bs[i + 3]};
        *reinterpret_cast<f32x4*>(ds + i) = f32x4{bo[i], bo[i + 1], bo[i + 2], bo[i + 3]};
      }
    }
  }
}

// A (or its transpose) and the inverses with a gate per channel, for chunks
// that decay far.  Channels go
// by slabs of 64.  Blocks of 16 tokens below the diagonal are matrix products
// of operands scaled towards the boundary between them; the four blocks on the
// diagonal are summed directly, wave b block b: a lane holds one key's 16
// channels, multiplies the decay of each later token into them and takes the
// dot products with that token's q and k.
template <int DK, bool DELTA, bool BWD>
__global__ void __launch_bounds__(256) chunk_vector_kernel(Params p) {
  constexpr int SL = 64, LP = SL + 4;
  __shared__ __align__(16) float qs[C][LP], ks[C][LP], al[C][LP], px[C][LP], sx[C][LP];
  __shared__ float tot[4][SL];
  __shared__ float bs[C];
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!noted_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t sh = (int64_t)slot * p.heads + h;
  if (!p.far[sh]) return;
  const int hq = h / (p.heads / p.heads_qk);
  const int fr = lane & 15, cg = lane >> 4;
  if (threadIdx.x < C)
    bs[threadIdx.x] = threadIdx.x < c.len
                          ? (p.beta ? p.beta[(c.row + threadIdx.x) * p.heads + h] : 1.0f)
                          : 0.0f;
  f32x4 accA[4], accL[4];
  float dA[16], dL[16];
#pragma unroll
  for (int b = 0; b < 4; ++b) accA[b] = accL[b] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) dA[i] = dL[i] = 0.0f;
#pragma unroll 1
  for (int c0 = 0; c0 < DK; c0 += SL) {
    __syncthreads();
    {
      const int ch = threadIdx.x & 63, b = threadIdx.x >> 6;
      float g[16], s = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = b * 16 + i;
        const bool in = t < c.len;
        g[i] = in ? gate(p.g[((c.row + t) * p.heads + h) * DK + c0 + ch]) : 0.0f;
        qs[t][ch] = in ? load_elem(p.q, (c.row + t) * p.qs + (int64_t)hq * DK + c0 + ch, p.dtype) : 0.0f;
        ks[t][ch] = in ? load_elem(p.k, (c.row + t) * p.ks + (int64_t)hq * DK + c0 + ch, p.dtype) : 0.0f;
        al[t][ch] = expf(g[i]);
        s += g[i];
        px[t][ch] = expf(s);
      }
      tot[b][ch] = s;
      s = 0.0f;
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        sx[b * 16 + i][ch] = expf(s);
        s += g[i];
      }
    }
    __syncthreads();
    // below the diagonal: forward wave = block of i, backward = block of j
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool need = BWD ? b > wave : b < wave;
      if (!need) continue;
      const int I = BWD ? b : wave, J = BWD ? wave : b;
#pragma unroll
      for (int s = 0; s < SL / 32; ++s) {
        const int k0 = s * 32 + cg * 8;
        float xq[8], xi[8], xj[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float mid = 0.0f;
          for (int m = J + 1; m < I; ++m) mid += tot[m][k0 + e];
          const float pi = px[I * 16 + fr][k0 + e];
          xq[e] = qs[I * 16 + fr][k0 + e] * pi;
          xi[e] = ks[I * 16 + fr][k0 + e] * pi;
          xj[e] = ks[J * 16 + fr][k0 + e] * (sx[J * 16 + fr][k0 + e] * expf(mid));
        }
        const Frag<P> fq = split8<P>(xq), fj = split8<P>(xj);
        if (BWD)
          mma(accA[b], fq, fj);
        else
          mma(accA[b], fj, fq);
        if (DELTA) {
          const Frag<P> fi = split8<P>(xi);
          if (BWD)
            mma(accL[b], fi, fj);
          else
            mma(accL[b], fj, fi);
        }
      }
    }
    // on the diagonal
    const int t0 = wave * 16;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const int k0 = cg * 16 + part * 8;
      float kj[8], kd[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        kj[e] = ks[t0 + fr][k0 + e];
        kd[e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool first = i == fr;
        asm volatile("" ::: "memory");  // else all tokens' loads come first, and registers spill
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          kd[e] = fmaf(kd[e], al[t0 + i][k0 + e], first ? kj[e] : 0.0f);
          dA[i] = fmaf(qs[t0 + i][k0 + e], kd[e], dA[i]);
          if (DELTA) dL[i] = fmaf(ks[t0 + i][k0 + e], kd[e], dL[i]);
        }
      }
    }
  }
  __syncthreads();
  // the slabs' arrays are free now: M over qs, M2 over ks, A over al
  float(*M)[LP] = qs;
  float(*M2)[LP] = ks;
  float(*A)[LP] = al;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    dA[i] += __shfl_xor(dA[i], 16);
    dA[i] += __shfl_xor(dA[i], 32);
    if (DELTA) {
      dL[i] += __shfl_xor(dL[i], 16);
      dL[i] += __shfl_xor(dL[i], 32);
    }
    if (cg == 0) {
      const int gi = wave * 16 + i, gj = wave * 16 + fr;
      A[gi][gj] = i >= fr ? dA[i] : 0.0f;
      if (DELTA) {
        const float l = i > fr ? dL[i] : 0.0f;
        M[gi][gj] = i > fr ? l * bs[gj] : 0.0f;
        if (BWD) M2[gi][gj] = i > fr ? bs[gi] * l : 0.0f;
      }
    }
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b == wave) continue;
    const bool need = BWD ? b > wave : b < wave;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = b * 16 + cg * 4 + r, col = wave * 16 + fr;
      const int i = BWD ? row : col, j = BWD ? col : row;
      A[i][j] = need ? accA[b][r] : 0.0f;
      if (DELTA) {
        M[i][j] = need ? accL[b][r] * bs[j] : 0.0f;
        if (BWD) M2[i][j] = need ? bs[i] * accL[b][r] : 0.0f;
      }
    }
  }
  __syncthreads();
  uint16_t* dst = (BWD ? p.at : p.a) + sh * P * C * C;
  for (int u = threadIdx.x; u < C * C / 4; u += 256) {
    const int r = u / (C / 4), q0 = u % (C / 4) * 4;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = BWD ? A[q0 + e][r] : A[r][q0 + e];
    put4<P>(dst + tiled<C>(r, q0), C * C, x);
  }
  if (DELTA) store_inverses<BWD>(p, M, M2, sh);
}

}  // namespace qscan
