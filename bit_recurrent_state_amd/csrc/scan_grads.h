// scan_grads.h — the gradients of q, k and the gates inside a chunk, once the
// states at its start (sc), the state gradients at its end (xc), U and Y are
// known.  All chunks at once, one workgroup per (slot, head).
//
//   E_ij = beta_j dO_i . U_j (j <= i),  F_ij = -beta_j Y_i . U_j (j < i)
//   dq_i  =  e^c_i dO_i S + sum_j G_ij E_ij k_j
//   dk+_i = -e^c_i Y_i S + sum_j G_ij F_ij k_j          (k_i reading the state)
//   dk-_j =  e^(c_end - c_j) W_j X + sum_i G_ij (E_ij q_i + F_ij k_i)  (writing)
//   dk = dk+ + dk-
//   dlog_alpha_t = e^c_end <X, S> + sum_{i<t} k_i dk-_i (state part)
//                  + sum_{i>=t} (q_i dq_i + k_i dk+_i - k_i dk-_i (chunk part))
// with the products taken per channel where the gate is.  The last line counts
// each pair of tokens only where t lies between them, so terms that do not
// depend on a gate are not added and taken off again.
//
// Waves split the key channels: the states are then read once per workgroup.

#pragma once

#include "scan_device.h"

namespace qscan {

struct ValueRows {  // [kChunk][dvp] rows of d_o, U or Y
  const uint16_t* p;
  int64_t row, plane;
  int len;
};

__device__ __forceinline__ ValueRows dout_rows(const Params& p, int64_t sh, int h, const Chunk& c) {
  ValueRows r;
  if (p.dop) {
    r.p = p.dop + sh * p.dop_terms * C * p.dvp;
    r.row = p.dvp;
    r.plane = (int64_t)C * p.dvp;
    r.len = C;
  } else {
    r.p = static_cast<const uint16_t*>(p.dO) + (c.row * p.heads + h) * p.dv;
    r.row = (int64_t)p.heads * p.dv;
    r.plane = 0;
    r.len = c.len;
  }
  return r;
}

template <int N>
__device__ __forceinline__ Frag<N> value_frag(const ValueRows& v, int row, int col) {
  return load_frag_if<N>(row < v.len, v.p + row * v.row + col, v.plane);
}

// Eight FP32 values, and their terms.
__device__ __forceinline__ Frag<P> state_frag(const float* s, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(s), b = *reinterpret_cast<const f32x4*>(s + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[4 + e] = b[e];
  }
  return split8<P>(x);
}

template <int DK>
__device__ __forceinline__ void store_qk(const Params& p, const Chunk& c, int64_t sh, int h, int t,
                                         int ch, float dq, float dk) {
  if (t >= c.len) return;
  if (p.heads == p.heads_qk) {
    const int64_t at = ((c.row + t) * p.heads + h) * DK + ch;
    store_elem(p.dq, at, p.dtype, dq);
    store_elem(p.dkk, at, p.dtype, dk);
  } else {
    p.dqpart[(sh * C + t) * DK + ch] = dq;
    p.dkpart[(sh * C + t) * DK + ch] = dk;
  }
}

// dbeta: the column blocks' parts.
__device__ __forceinline__ void store_dbeta(const Params& p, const Chunk& c, int64_t sh, int h) {
  if (!p.dbeta || (int)threadIdx.x >= c.len) return;
  float s = 0.0f;
  for (int b = 0; b < p.nvb; ++b)
    s += p.dbpart[((int64_t)b * p.nslots * p.heads + sh) * C + threadIdx.x];
  p.dbeta[(c.row + threadIdx.x) * p.heads + h] = s;
}

// ---- one gate per token ----------------------------------------------------------------------
template <int DK, int NPQ, int NPO, bool DELTA>
__global__ void __launch_bounds__(256) grads_scalar_kernel(Params p) {
  constexpr int CT = DK / 64, PL = C * CP;
  __shared__ __align__(16) uint16_t E[P][C][CP], Et[P][C][CP];
  __shared__ __align__(16) uint16_t F[DELTA ? P : 1][DELTA ? C : 1][CP];
  __shared__ __align__(16) uint16_t Ft[DELTA ? P : 1][DELTA ? C : 1][CP];
  __shared__ float red[2][4][C];
  __shared__ float redx[4];
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!find_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t sh = (int64_t)slot * p.heads + h;
  const int hq = h / (p.heads / p.heads_qk);
  const float* rows = rows_at(p, slot, h);
  const double* cs = reinterpret_cast<const double*>(rows + 3 * C);
  const ValueRows dO = dout_rows(p, sh, h, c);
  const ValueRows U = {p.u + sh * P * C * p.dvp, p.dvp, (int64_t)C * p.dvp, C};
  const ValueRows Y = {p.y + sh * P * C * p.dvp, p.dvp, (int64_t)C * p.dvp, C};
  const int nvs = p.dvp / 32;

  for (int b = 0; b < 4; ++b) {  // rows of block `wave`, columns of block b
    f32x4 e = {0, 0, 0, 0}, f = {0, 0, 0, 0};
    if (b <= wave)
      for (int s = 0; s < nvs; ++s) {
        const Frag<P> u = value_frag<P>(U, b * 16 + fr, s * 32 + fg * 8);
        mma(e, value_frag<NPO>(dO, wave * 16 + fr, s * 32 + fg * 8), u);
        if (DELTA) mma(f, value_frag<P>(Y, wave * 16 + fr, s * 32 + fg * 8), u);
      }
    const int j = b * 16 + fr, i0 = wave * 16 + fg * 4;
    const float beta = rows[2 * C + j];
    float xe[4], xf[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = i0 + r;
      const float g = i >= j ? beta * expf((float)(cs[i] - cs[j])) : 0.0f;
      xe[r] = i >= j ? e[r] * g : 0.0f;
      xf[r] = i > j ? -f[r] * g : 0.0f;
    }
    u32x2 t[P];
    split4<P>(xe, t);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      *reinterpret_cast<u32x2*>(&Et[q][j][i0]) = t[q];
      E[q][i0][j] = (uint16_t)t[q].x;
      E[q][i0 + 1][j] = (uint16_t)(t[q].x >> 16);
      E[q][i0 + 2][j] = (uint16_t)t[q].y;
      E[q][i0 + 3][j] = (uint16_t)(t[q].y >> 16);
    }
    if (DELTA) {
      split4<P>(xf, t);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        *reinterpret_cast<u32x2*>(&Ft[q][j][i0]) = t[q];
        F[q][i0][j] = (uint16_t)t[q].x;
        F[q][i0 + 1][j] = (uint16_t)(t[q].x >> 16);
        F[q][i0 + 2][j] = (uint16_t)t[q].y;
        F[q][i0 + 3][j] = (uint16_t)(t[q].y >> 16);
      }
    }
  }
  __syncthreads();

  float sS[4][4], sD[4][4], xs = 0.0f;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) sS[m][r] = sD[m][r] = 0.0f;
  const int64_t tq = (int64_t)slot * p.heads_qk + hq;
#pragma unroll 1
  for (int ct = 0; ct < CT; ++ct) {
    const int ch = wave * (DK / 4) + ct * 16 + fr;
    f32x4 aq[4], ap[4], am[4], ai[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) aq[m] = ap[m] = am[m] = ai[m] = f32x4{0, 0, 0, 0};
    for (int s = 0; s < nvs; ++s) {
      const int64_t at = (sh * DK + ch) * p.dvp + s * 32 + fg * 8;
      float x0[8], x1[8];
      const Frag<P> fs = state_frag(p.sc + at, x0), fx = state_frag(p.xc + at, x1);
#pragma unroll
      for (int e = 0; e < 8; ++e) xs = fmaf(x0[e], x1[e], xs);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        mma(aq[m], value_frag<NPO>(dO, m * 16 + fr, s * 32 + fg * 8), fs);
        if (DELTA) mma(ap[m], value_frag<P>(Y, m * 16 + fr, s * 32 + fg * 8), fs);
        mma(am[m], value_frag<P>(U, m * 16 + fr, s * 32 + fg * 8), fx);
      }
    }
    float kx[4][4], qx[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t0 = m * 16 + fg * 4;
      const f32x4 ec = *reinterpret_cast<const f32x4*>(rows + t0);
      const f32x4 eo = *reinterpret_cast<const f32x4*>(rows + C + t0);
      const f32x4 be = *reinterpret_cast<const f32x4*>(rows + 2 * C + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool in = t0 + r < c.len;
        kx[m][r] = in ? load_elem(p.k, (c.row + t0 + r) * p.ks + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        qx[m][r] = in ? load_elem(p.q, (c.row + t0 + r) * p.qs + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        aq[m][r] *= ec[r];
        ap[m][r] *= -ec[r];
        am[m][r] *= eo[r] * be[r];
        sS[m][r] = fmaf(kx[m][r], am[m][r], sS[m][r]);
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t at = (tq * NPQ * DK + ch) * C + s * 32 + fg * 8;
      const Frag<NPQ> fk = load_frag<NPQ>(p.kt + at, DK * C);
      const Frag<NPQ> fq = load_frag<NPQ>(p.qt + at, DK * C);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int row = m * 16 + fr, col = s * 32 + fg * 8;
        if (s <= m / 2) {
          mma(aq[m], load_frag<P>(&E[0][row][col], PL), fk);
          if (DELTA) mma(ap[m], load_frag<P>(&F[0][row][col], PL), fk);
        }
        if (s >= m / 2) {
          mma(ai[m], load_frag<P>(&Et[0][row][col], PL), fq);
          if (DELTA) mma(ai[m], load_frag<P>(&Ft[0][row][col], PL), fk);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        sD[m][r] += qx[m][r] * aq[m][r] + kx[m][r] * (ap[m][r] - ai[m][r]);
        store_qk<DK>(p, c, sh, h, m * 16 + fg * 4 + r, ch, aq[m][r],
                     ap[m][r] + am[m][r] + ai[m][r]);
      }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float a = sum16(sS[m][r]), b = sum16(sD[m][r]);
      if (fr == 0) {
        red[0][wave][m * 16 + fg * 4 + r] = a;
        red[1][wave][m * 16 + fg * 4 + r] = b;
      }
    }
  xs = sum16(xs);
  xs += __shfl_xor(xs, 16);
  xs += __shfl_xor(xs, 32);
  if (lane == 0) redx[wave] = xs;
  __syncthreads();
  if (wave == 0) {
    double s = 0.0, d = 0.0, x = 0.0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      s += red[0][w][lane];
      d += red[1][w][lane];
      x += redx[w];
    }
    double before = s, after = d;
    for (int o = 1; o < 64; o *= 2) {
      const double a = __shfl_up(before, o), b = __shfl_down(after, o);
      if (lane >= o) before += a;
      if (lane + o < 64) after += b;
    }
    if (lane < c.len)
      p.dg[(c.row + lane) * p.heads + h] = (float)(rows[C - 1] * x + (before - s) + after);
    store_dbeta(p, c, sh, h);
  }
}

// ---- a gate per key channel ------------------------------------------------------------------
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The chunk's own part goes by blocks of 16 tokens, as A did: below the
// diagonal by matrix products of operands scaled towards the boundary, on the
// diagonal by one lane per (channel, block) that carries 16 decayed keys
// forward and 16 gradients backward.  NPR: terms of the unscaled q and k.
template <int DK, int NPR, int NPO, bool DELTA>
__global__ void __launch_bounds__(256) grads_vector_kernel(Params p) {
  constexpr int CT = DK / 64, PL = C * CP, FP = C + 4;
  __shared__ __align__(16) uint16_t E[P][C][CP], Et[P][C][CP];
  __shared__ __align__(16) uint16_t F[DELTA ? P : 1][DELTA ? C : 1][CP];
  __shared__ __align__(16) uint16_t Ft[DELTA ? P : 1][DELTA ? C : 1][CP];
  __shared__ __align__(16) float Ed[4][16][16], Fd[4][DELTA ? 16 : 1][16];  // diagonal blocks
  __shared__ __align__(16) float buf[4][16][FP];
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!find_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t sh = (int64_t)slot * p.heads + h;
  const int hq = h / (p.heads / p.heads_qk);
  const float* rows = rows_at(p, slot, h);
  const ValueRows dO = dout_rows(p, sh, h, c);
  const ValueRows U = {p.u + sh * P * C * p.dvp, p.dvp, (int64_t)C * p.dvp, C};
  const ValueRows Y = {p.y + sh * P * C * p.dvp, p.dvp, (int64_t)C * p.dvp, C};
  const int nvs = p.dvp / 32;

  for (int b = 0; b < 4; ++b) {
    f32x4 e = {0, 0, 0, 0}, f = {0, 0, 0, 0};
    if (b <= wave)
      for (int s = 0; s < nvs; ++s) {
        const Frag<P> u = value_frag<P>(U, b * 16 + fr, s * 32 + fg * 8);
        mma(e, value_frag<NPO>(dO, wave * 16 + fr, s * 32 + fg * 8), u);
        if (DELTA) mma(f, value_frag<P>(Y, wave * 16 + fr, s * 32 + fg * 8), u);
      }
    const int j = b * 16 + fr, i0 = wave * 16 + fg * 4;
    const float beta = rows[2 * C + j];
    float xe[4], xf[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      xe[r] = b <= wave ? beta * e[r] : 0.0f;
      xf[r] = b <= wave ? -beta * f[r] : 0.0f;
    }
    if (b == wave) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        Ed[b][fg * 4 + r][fr] = fg * 4 + r >= fr ? xe[r] : 0.0f;
        if (DELTA) Fd[b][fg * 4 + r][fr] = fg * 4 + r > fr ? xf[r] : 0.0f;
        xe[r] = xf[r] = 0.0f;
      }
    }
    u32x2 t[P];
    split4<P>(xe, t);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      *reinterpret_cast<u32x2*>(&Et[q][j][i0]) = t[q];
      E[q][i0][j] = (uint16_t)t[q].x;
      E[q][i0 + 1][j] = (uint16_t)(t[q].x >> 16);
      E[q][i0 + 2][j] = (uint16_t)t[q].y;
      E[q][i0 + 3][j] = (uint16_t)(t[q].y >> 16);
    }
    if (DELTA) {
      split4<P>(xf, t);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        *reinterpret_cast<u32x2*>(&Ft[q][j][i0]) = t[q];
        F[q][i0][j] = (uint16_t)t[q].x;
        F[q][i0 + 1][j] = (uint16_t)(t[q].x >> 16);
        F[q][i0 + 2][j] = (uint16_t)t[q].y;
        F[q][i0 + 3][j] = (uint16_t)(t[q].y >> 16);
      }
    }
  }
  __syncthreads();

  const int64_t tq = (int64_t)slot * p.heads_qk + hq;
#pragma unroll 1
  for (int ct = 0; ct < CT; ++ct) {
    const int ch = wave * (DK / 4) + ct * 16 + fr;
    f32x4 aq[4], ap[4], am[4], ai[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) aq[m] = ap[m] = am[m] = ai[m] = f32x4{0, 0, 0, 0};
    float xs = 0.0f;
    for (int s = 0; s < nvs; ++s) {
      const int64_t at = (sh * DK + ch) * p.dvp + s * 32 + fg * 8;
      float x0[8], x1[8];
      const Frag<P> fs = state_frag(p.sc + at, x0), fx = state_frag(p.xc + at, x1);
#pragma unroll
      for (int e = 0; e < 8; ++e) xs = fmaf(x0[e], x1[e], xs);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        mma(aq[m], value_frag<NPO>(dO, m * 16 + fr, s * 32 + fg * 8), fs);
        if (DELTA) mma(ap[m], value_frag<P>(Y, m * 16 + fr, s * 32 + fg * 8), fs);
        mma(am[m], value_frag<P>(U, m * 16 + fr, s * 32 + fg * 8), fx);
      }
    }
    xs += __shfl_xor(xs, 16);
    xs += __shfl_xor(xs, 32);
    const float* pf = p.pfx + (sh * DK + ch) * C;
    const float* sf = p.sfx + (sh * DK + ch) * C;
    const float tot[4] = {pf[15], pf[31], pf[47], pf[63]};  // decay over each block
    const float bef[4] = {1.0f, tot[0], tot[0] * tot[1], tot[0] * tot[1] * tot[2]};
    const float aft[4] = {tot[1] * tot[2] * tot[3], tot[2] * tot[3], tot[3], 1.0f};
    float sS[4][4];
    f32x4 iq[4], ip[4], im[4];  // below the diagonal
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t0 = m * 16 + fg * 4;
      const f32x4 pe = *reinterpret_cast<const f32x4*>(pf + t0);
      const f32x4 se = *reinterpret_cast<const f32x4*>(sf + t0);
      const f32x4 be = *reinterpret_cast<const f32x4*>(rows + 2 * C + t0);
      iq[m] = ip[m] = im[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float k = t0 + r < c.len
            ? load_elem(p.k, (c.row + t0 + r) * p.ks + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        aq[m][r] *= pe[r] * bef[m];
        ap[m][r] *= -(pe[r] * bef[m]);
        am[m][r] *= se[r] * aft[m] * be[r];
        sS[m][r] = k * am[m][r];
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int t0 = s * 32 + fg * 8, blk = t0 / 16;  // the lane's 8 tokens and their block
      float k[8], q[8], ks[8], qs[8], kp[8];
      const int64_t at = (tq * NPR * DK + ch) * C + t0;
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = q[e] = 0.0f;
#pragma unroll
      for (int n = NPR - 1; n >= 0; --n) {
        const Frag<1> fk = load_frag<1>(p.kt_raw + at + (int64_t)n * DK * C, 0);
        const Frag<1> fq = load_frag<1>(p.qt_raw + at + (int64_t)n * DK * C, 0);
        const uint32_t wk[4] = {fk.t[0].x, fk.t[0].y, fk.t[0].z, fk.t[0].w};
        const uint32_t wq[4] = {fq.t[0].x, fq.t[0].y, fq.t[0].z, fq.t[0].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          k[e] += bf16_to_f((uint16_t)(wk[e / 2] >> (16 * (e & 1))));
          q[e] += bf16_to_f((uint16_t)(wq[e / 2] >> (16 * (e & 1))));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float pe = pf[t0 + e], se = sf[t0 + e];
        ks[e] = k[e] * se;  // towards the end of its block
        kp[e] = k[e] * pe;  // from its block's start
        qs[e] = q[e] * pe;
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int row = m * 16 + fr, col = s * 32 + fg * 8;
        if (s * 32 < m * 16) {  // rows of block m from the blocks before it
          const float mid = blk >= m ? 0.0f : blk + 1 == m ? 1.0f : blk + 2 == m ? tot[blk + 1] : tot[1] * tot[2];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = ks[e] * mid;
          const Frag<P> f = split8<P>(x);
          mma(iq[m], load_frag<P>(&E[0][row][col], PL), f);
          if (DELTA) mma(ip[m], load_frag<P>(&F[0][row][col], PL), f);
        }
        if (s * 32 + 31 >= m * 16 + 16) {  // gradients of block m from the blocks behind it
          const float mid = blk <= m ? 0.0f : blk == m + 1 ? 1.0f : blk == m + 2 ? tot[m + 1] : tot[1] * tot[2];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = qs[e] * mid;
          mma(im[m], load_frag<P>(&Et[0][row][col], PL), split8<P>(x));
          if (DELTA) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = kp[e] * mid;
            mma(im[m], load_frag<P>(&Ft[0][row][col], PL), split8<P>(x));
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t0 = m * 16 + fg * 4;
      const f32x4 pe = *reinterpret_cast<const f32x4*>(pf + t0);
      const f32x4 se = *reinterpret_cast<const f32x4*>(sf + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        aq[m][r] = fmaf(iq[m][r], pe[r], aq[m][r]);
        ap[m][r] = fmaf(ip[m][r], pe[r], ap[m][r]);
        ai[m][r] = im[m][r] * se[r];
      }
    }
    // the diagonal block fg of channel ch
    float x[16], z[16], y[16];
    {
      float q[16], k[16], al[16], kd[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = fg * 16 + i;
        const bool in = t < c.len;
        q[i] = in ? load_elem(p.q, (c.row + t) * p.qs + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        k[i] = in ? load_elem(p.k, (c.row + t) * p.ks + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        al[i] = in ? expf(gate(p.g[((c.row + t) * p.heads + h) * DK + ch])) : 1.0f;
        y[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int j = 0; j < i; ++j) kd[j] *= al[i];
        kd[i] = k[i];
        x[i] = z[i] = 0.0f;
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          x[i] = fmaf(Ed[fg][i][j], kd[j], x[i]);
          if (DELTA && j < i) z[i] = fmaf(Fd[fg][DELTA ? i : 0][j], kd[j], z[i]);
        }
      }
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        y[i] = fmaf(Ed[fg][i][i], q[i], y[i]);
#pragma unroll
        for (int j = 0; j < i; ++j) {
          float s = fmaf(Ed[fg][i][j], q[i], y[j]);
          if (DELTA) s = fmaf(Fd[fg][DELTA ? i : 0][j], k[i], s);
          y[j] = s * al[i];
        }
      }
    }
    // y_j so far holds the decay of token j too where later tokens reach it: see above, the
    // factor of token i is taken on when i is passed, so y_j ends with the decays of j+1 .. i.
    auto exchange = [&](const float(&v)[16], f32x4(&out)[4]) {
      wave_sync();
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(&buf[wave][fr][fg * 16 + i]) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
      wave_sync();
#pragma unroll
      for (int m = 0; m < 4; ++m)
        out[m] = *reinterpret_cast<const f32x4*>(&buf[wave][fr][m * 16 + fg * 4]);
    };
    f32x4 d[4];
    exchange(x, d);
#pragma unroll
    for (int m = 0; m < 4; ++m) aq[m] += d[m];
    if (DELTA) {
      exchange(z, d);
#pragma unroll
      for (int m = 0; m < 4; ++m) ap[m] += d[m];
    }
    exchange(y, d);
#pragma unroll
    for (int m = 0; m < 4; ++m) ai[m] += d[m];
    // gates: token sums per channel, 16 tokens per lane
    f32x4 dc[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = m * 16 + fg * 4 + r;
        const bool in = t < c.len;
        const float q = in ? load_elem(p.q, (c.row + t) * p.qs + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        const float k = in ? load_elem(p.k, (c.row + t) * p.ks + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        dc[m][r] = q * aq[m][r] + k * (ap[m][r] - ai[m][r]);
        store_qk<DK>(p, c, sh, h, t, ch, aq[m][r], ap[m][r] + am[m][r] + ai[m][r]);
      }
    auto gather = [&](const f32x4(&v)[4], float(&out)[16]) {
      wave_sync();
#pragma unroll
      for (int m = 0; m < 4; ++m) *reinterpret_cast<f32x4*>(&buf[wave][fr][m * 16 + fg * 4]) = v[m];
      wave_sync();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(&buf[wave][fr][fg * 16 + i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i + e] = w[e];
      }
    };
    f32x4 ss[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) ss[m] = f32x4{sS[m][0], sS[m][1], sS[m][2], sS[m][3]};
    gather(ss, x);
    gather(dc, y);
    float bx = 0.0f, by = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      bx += x[i];
      by += y[i];
    }
    float pre = 0.0f, post = 0.0f;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const float a = __shfl(bx, fr + 16 * o), b = __shfl(by, fr + 16 * o);
      if (o < fg) pre += a;
      if (o > fg) post += b;
    }
    const float end = p.decay[sh * DK + ch] * xs;
    float z2[16];
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      post += y[i];
      z2[i] = post;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = fg * 16 + i;
      if (t < c.len) p.dg[((c.row + t) * p.heads + h) * DK + ch] = end + pre + z2[i];
      pre += x[i];
    }
  }
  if (wave == 0) store_dbeta(p, c, sh, h);
}

// dq and dk of heads that share them: summed in the order of the heads.
template <int DK>
__global__ void __launch_bounds__(256) share_kernel(Params p) {
  const int slot = blockIdx.x, hq = blockIdx.y;
  Chunk c;
  if (!find_chunk(p, slot, c)) return;
  const int group = p.heads / p.heads_qk;
  for (int u = threadIdx.x; u < c.len * DK; u += 256) {
    float a = 0.0f, b = 0.0f;
    for (int g = 0; g < group; ++g) {
      const int64_t at = ((int64_t)slot * p.heads + hq * group + g) * C * DK + u;
      a += p.dqpart[at];
      b += p.dkpart[at];
    }
    const int64_t to = ((c.row + u / DK) * p.heads_qk + hq) * DK + u % DK;
    store_elem(p.dq, to, p.dtype, a);
    store_elem(p.dkk, to, p.dtype, b);
  }
}

}  // namespace qscan
