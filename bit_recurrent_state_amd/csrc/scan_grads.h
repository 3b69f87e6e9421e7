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
// depend on a gate are not added and taken off again; E's diagonal, which would
// cancel there up to rounding, enters dq and dk beside the products (a single
// token without a state then has a gate's gradient of exactly zero).
//
// Waves split the key channels: the states are then read once per workgroup.
// 104 us for 1024 chunks and heads of 128 x 128 (GDN, bfloat16; 290 MB, 2.8 TB/s;
// matrix instructions 19 % of the time), 115 us for 2048 of 128 x 64 without the
// delta rule (350 MB, 3.1 TB/s): two workgroups a CU, each of which loads a slab,
// splits it and multiplies in turn.

#pragma once

#include "scan_device.h"

namespace qscan {

// [kChunk][dvp] rows of d_o.  Its fragments have p.dop_terms terms: as many planes in the workspace,
// or the caller's bfloat16 rows, which are one term and have no plane to go on to.
struct ValueRows {
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

// Zero behind the end: the caller's rows there are another sequence's.
template <int N>
__device__ __forceinline__ Frag<N> value_frag(const ValueRows& v, int row, int col) {
  Frag<N> f = load_frag<N>(v.p + min(row, v.len - 1) * v.row + col, v.plane);
  if (row >= v.len) {
#pragma unroll
    for (int n = 0; n < N; ++n) f.t[n] = u32x4{0, 0, 0, 0};
  }
  return f;
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

// dq and dk of 4 tokens of a channel.
template <int DK>
__device__ __forceinline__ void store_qk(const Params& p, const Chunk& c, int64_t sh, int h, int t,
                                         int ch, const float (&dq)[4], const float (&dk)[4]) {
  if (p.heads == p.heads_qk) {
    int64_t at[4];
    bool ok[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      at[r] = ((c.row + t + r) * p.heads + h) * DK + ch;
      ok[r] = t + r < c.len;
    }
    store_elems<4>(p.dq, at, ok, p.dtype, dq);
    store_elems<4>(p.dkk, at, ok, p.dtype, dk);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      p.dqpart[(sh * C + t + r) * DK + ch] = dq[r];
      p.dkpart[(sh * C + t + r) * DK + ch] = dk[r];
    }
  }
}

// dbeta: the column blocks' parts, summed in a fixed order; a wave takes every
// NW-th, store_dbeta (the threads of one wave, after a barrier) their sums.
template <int NW>
__device__ __forceinline__ void sum_dbeta(const Params& p, int64_t sh, float (*red)[C]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float s = 0.0f;
  if (p.dbeta)
    for (int b = wave; b < p.nvb; b += NW)
      s += p.dbpart[((int64_t)b * p.nslots * p.heads + sh) * C + lane];
  red[wave][lane] = s;
}

template <int NW>
__device__ __forceinline__ void store_dbeta(const Params& p, const Chunk& c, int h,
                                            const float (*red)[C]) {
  const int t = threadIdx.x & 63;
  if (!p.dbeta || t >= c.len) return;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w][t];
  p.dbeta[(c.row + t) * p.heads + h] = s;
}

// ---- the states' and the chunk's products ----------------------------------------------------
// The value columns pass through LDS in slabs of 64: rows of d_o, U and Y, which
// all waves need.  A wave's own channels of the states come straight from
// memory and are split in its registers.  E and F then take the slabs' place,
// one after the other, as rows and as columns.
//
// One gate per token: E and F carry the decay G.  VEC (chunks that do not decay
// far): G_ij = e^c_i e^-c_j per channel, so sum_j E_ij (k_j e^-c_j) is scaled by
// e^c_i, and sum_i E_ij (q_i e^c_i) by e^-c_j.  NPR: terms of the unscaled q and
// k (VEC).
template <int DK, int NPQ, int NPR, int NPO, bool VEC, bool DELTA>
__global__ void __launch_bounds__(DK >= 128 ? 512 : 256) grads_kernel(Params p) {
  constexpr int NW = DK >= 128 ? 8 : 4, CT = DK / (16 * NW), NE = 16 / NW, VS = 64, VP = VS + 8, NP = NPO + (DELTA ? 2 : 1) * P;
  constexpr int PL = C * CP;
  constexpr int kWords = (NP * C * VP > 2 * P * C * CP ? NP * C * VP : 2 * P * C * CP);
  __shared__ __align__(16) uint16_t lds[kWords];
  __shared__ float red[2][NW][C], redb[NW][C];
  __shared__ __align__(16) float rows[5 * C];
  __shared__ float redx[NW];
  __shared__ __align__(16) float diag[C];  // E's diagonal
  uint16_t* const Ol = lds;
  uint16_t* const Ul = lds + NPO * C * VP;
  uint16_t* const Yl = Ul + P * C * VP;
  uint16_t* const El = lds;           // [P][C][CP]
  uint16_t* const Et = lds + P * PL;  // transposed
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!noted_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t sh = (int64_t)slot * p.heads + h;
  if (VEC && p.far[sh]) return;
  const int hq = h / (p.heads / p.heads_qk);
  if (threadIdx.x >= 64 && threadIdx.x < 64 + 5 * C / 4)
    reinterpret_cast<f32x4*>(rows)[threadIdx.x - 64] =
        reinterpret_cast<const f32x4*>(rows_at(p, slot, h))[threadIdx.x - 64];
  sum_dbeta<NW>(p, sh, redb);
  const ValueRows dO = dout_rows(p, sh, h, c);
  const int ch0 = wave * (DK / NW) + fr;
  // E and F: the wave's row block, and its column blocks b0, b0 + 4 / NE, ..
  const int rb = wave * 4 / NW, b0 = wave % (NW / 4);

  f32x4 e[NE], f[NE], aq[CT][4], ap[DELTA ? CT : 1][4], am[CT][4];
  float xs[CT];
#pragma unroll
  for (int b = 0; b < NE; ++b) e[b] = f[b] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      aq[ct][m] = am[ct][m] = f32x4{0, 0, 0, 0};
      if (DELTA) ap[ct][m] = f32x4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) xs[ct] = 0.0f;

  for (int v0 = 0; v0 < p.dvp; v0 += VS) {
    const int ns = p.dvp - v0 >= VS ? 2 : 1;
    f32x4 sv[CT][2][2], xv[CT][2][2];
    // rows into LDS: 8 vectors of 8 a row
    {
      constexpr int A = DELTA ? 2 : 1;  // U, Y
      const int col = threadIdx.x & 7, row = threadIdx.x >> 3;
      constexpr int R = 8 / NW;  // rows a thread
      u32x4 so[NPO][R];
      f32x4 sf[A][R][2];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = i * 32 + row;
        // columns behind dvp repeat the last ones and are not used
        const int64_t vc = v0 + min(col * 8, p.dvp - v0 - 8);
        const int64_t ro = (int64_t)min(r, dO.len - 1) * dO.row + vc;
#pragma unroll
        for (int n = 0; n < NPO; ++n) {
          so[n][i] = *reinterpret_cast<const u32x4*>(dO.p + n * dO.plane + ro);
          if (r >= c.len) so[n][i] = u32x4{0, 0, 0, 0};
        }
        const int64_t at = (sh * C + r) * p.dvp + vc;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          sf[0][i][q] = *reinterpret_cast<const f32x4*>(p.u + at + q * 4);
          if (DELTA) sf[A - 1][i][q] = *reinterpret_cast<const f32x4*>(p.y + at + q * 4);
        }
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int64_t at = (sh * DK + ch0 + ct * 16) * p.dvp + v0 + min(s, ns - 1) * 32 + fg * 8;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            sv[ct][s][q] = *reinterpret_cast<const f32x4*>(p.sc + at + q * 4);
            xv[ct][s][q] = *reinterpret_cast<const f32x4*>(p.xc + at + q * 4);
          }
        }
      __syncthreads();  // the last slab has been read
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int o = (i * 32 + row) * VP + col * 8;
#pragma unroll
        for (int n = 0; n < NPO; ++n) *reinterpret_cast<u32x4*>(Ol + n * C * VP + o) = so[n][i];
#pragma unroll
        for (int a = 0; a < A; ++a) {
          const float x[8] = {sf[a][i][0][0], sf[a][i][0][1], sf[a][i][0][2], sf[a][i][0][3],
                              sf[a][i][1][0], sf[a][i][1][1], sf[a][i][1][2], sf[a][i][1][3]};
          const Frag<P> f = split8<P>(x);
#pragma unroll
          for (int n = 0; n < P; ++n)
            *reinterpret_cast<u32x4*>((a ? Yl : Ul) + n * C * VP + o) = f.t[n];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s >= ns) break;
      const int at = fr * VP + s * 32 + fg * 8;
      const Frag<NPO> fo = load_frag<NPO>(Ol + rb * 16 * VP + at, C * VP);
      Frag<P> fy;
      if (DELTA) fy = load_frag<P>(Yl + rb * 16 * VP + at, C * VP);
#pragma unroll
      for (int b = 0; b < NE; ++b)
        if (b0 + b * (NW / 4) <= rb) {
          const Frag<P> fu = load_frag<P>(Ul + (b0 + b * (NW / 4)) * 16 * VP + at, C * VP);
          mma(e[b], fo, fu);
          if (DELTA) mma(f[b], fy, fu);
        }
      Frag<P> fs[CT], fx[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float x0[8], x1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x0[i] = sv[ct][s][i / 4][i % 4];
          x1[i] = xv[ct][s][i / 4][i % 4];
          xs[ct] = fmaf(x0[i], x1[i], xs[ct]);
        }
        fs[ct] = split8<P>(x0);
        fx[ct] = split8<P>(x1);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const Frag<NPO> go = load_frag<NPO>(Ol + m * 16 * VP + at, C * VP);
        const Frag<P> gu = load_frag<P>(Ul + m * 16 * VP + at, C * VP);
        Frag<P> gy;
        if (DELTA) gy = load_frag<P>(Yl + m * 16 * VP + at, C * VP);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          mma(aq[ct][m], go, fs[ct]);
          if (DELTA) mma(ap[ct][m], gy, fs[ct]);
          mma(am[ct][m], gu, fx[ct]);
        }
      }
    }
  }

  // E (then F) as planes in LDS
  const double* cs = reinterpret_cast<const double*>(rows + 3 * C);
  auto put_square = [&](f32x4(&x)[NE], float sign) {
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NE; ++b) {
      const int j = (b0 + b * (NW / 4)) * 16 + fr, i0 = rb * 16 + fg * 4;
      const float beta = sign * rows[2 * C + j];
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = i0 + r;
        const bool in = i > j;
        if (sign > 0.0f && i == j) diag[i] = x[b][r] * beta;
        float g = beta;
        if (!VEC) g *= fast_exp(in ? (float)(cs[i] - cs[j]) : 0.0f);
        v[r] = in ? x[b][r] * g : 0.0f;
      }
      u32x2 t[P];
      split4<P>(v, t);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        *reinterpret_cast<u32x2*>(Et + q * PL + j * CP + i0) = t[q];
        uint16_t* d = El + q * PL + i0 * CP + j;
        d[0] = (uint16_t)t[q].x;
        d[CP] = (uint16_t)(t[q].x >> 16);
        d[2 * CP] = (uint16_t)t[q].y;
        d[3 * CP] = (uint16_t)(t[q].y >> 16);
      }
    }
    __syncthreads();
  };
  const int64_t tq = VEC ? sh : (int64_t)slot * p.heads_qk + hq;
  const uint16_t* const kn = (VEC ? p.knt : p.kt) + tq * NPQ * DK * C;  // right operand of E, F
  const uint16_t* const qe = p.qt + tq * NPQ * DK * C;                  // of E transposed
  const uint16_t* const ke = p.ket + tq * NPQ * DK * C;                 // of F transposed (VEC)
  Frag<NPQ> fk[CT][2], fq[CT][2];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fk[ct][s] = tile_frag<NPQ, C>(kn, wave * CT + ct, s, DK * C);
      fq[ct][s] = tile_frag<NPQ, C>(qe, wave * CT + ct, s, DK * C);
    }
  put_square(e, 1.0f);
  f32x4 ai[CT][4];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int ch = ch0 + ct * 16;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t0 = m * 16 + fg * 4;
      const f32x4 be = *reinterpret_cast<const f32x4*>(rows + 2 * C + t0);
      f32x4 ec, eo;
      if (VEC) {
        ec = *reinterpret_cast<const f32x4*>(p.pfx + (sh * DK + ch) * C + t0);
        eo = *reinterpret_cast<const f32x4*>(p.sfx + (sh * DK + ch) * C + t0);
      } else {
        ec = *reinterpret_cast<const f32x4*>(rows + t0);
        eo = *reinterpret_cast<const f32x4*>(rows + C + t0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!VEC) {  // VEC: scaled below, together with the chunk's own part
          aq[ct][m][r] *= ec[r];
          if (DELTA) ap[ct][m][r] *= -ec[r];
        } else if (DELTA) {
          ap[ct][m][r] = -ap[ct][m][r];
        }
        am[ct][m][r] *= eo[r] * be[r];
      }
      ai[ct][m] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int o = (m * 16 + fr) * CP + s * 32 + fg * 8;
        if (s <= m / 2) mma(aq[ct][m], load_frag<P>(El + o, PL), fk[ct][s]);
        if (s >= m / 2) mma(ai[ct][m], load_frag<P>(Et + o, PL), fq[ct][s]);
      }
    }
  }
  // one gate per token: F's right operands are k's columns both times
  if (DELTA && VEC) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int s = 0; s < 2; ++s) fq[ct][s] = tile_frag<NPQ, C>(ke, wave * CT + ct, s, DK * C);
  }
  // the unscaled k and q, for the gates
  const uint16_t* const kr = (VEC ? p.kt_raw : p.kt) + ((int64_t)slot * p.heads_qk + hq) * NPR * DK * C;
  const uint16_t* const qr = (VEC ? p.qt_raw : p.qt) + ((int64_t)slot * p.heads_qk + hq) * NPR * DK * C;
  u32x2 rk[CT][4][NPR], rq[CT][4][NPR];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NPR; ++n) {
        const int at = n * DK * C + tiled<C>(ch0 + ct * 16, m * 16 + fg * 4);
        rk[ct][m][n] = *reinterpret_cast<const u32x2*>(kr + at);
        rq[ct][m][n] = *reinterpret_cast<const u32x2*>(qr + at);
      }
  if (DELTA) {
    put_square(f, -1.0f);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int o = (m * 16 + fr) * CP + s * 32 + fg * 8;
          if (s <= m / 2) mma(ap[ct][m], load_frag<P>(El + o, PL), fk[ct][s]);
          if (s >= m / 2) mma(ai[ct][m], load_frag<P>(Et + o, PL), VEC ? fq[ct][s] : fk[ct][s]);
        }
  }

  // the outputs, and the sums for the gates
  auto sum4 = [&](const u32x2(&w)[NPR], float(&x)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = 0.0f;
#pragma unroll
    for (int n = NPR - 1; n >= 0; --n) {
      x[0] += __uint_as_float(w[n].x << 16);
      x[1] += __uint_as_float(w[n].x & 0xFFFF0000u);
      x[2] += __uint_as_float(w[n].y << 16);
      x[3] += __uint_as_float(w[n].y & 0xFFFF0000u);
    }
  };
  float sS[4][4], sD[4][4];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int ch = ch0 + ct * 16;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t0 = m * 16 + fg * 4;
      float k[4], q[4], dq[4], dk[4];
      sum4(rk[ct][m], k);
      sum4(rq[ct][m], q);
      const f32x4 ed = *reinterpret_cast<const f32x4*>(diag + t0);
      f32x4 ec = {1, 1, 1, 1};
      if (VEC) ec = *reinterpret_cast<const f32x4*>(p.pfx + (sh * DK + ch) * C + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float a = aq[ct][m][r], b = DELTA ? ap[ct][m][r] : 0.0f, i = ai[ct][m][r];
        if (VEC) {
          a *= ec[r];
          b *= ec[r];
          i /= ec[r];
        }
        dq[r] = fmaf(ed[r], k[r], a);
        dk[r] = fmaf(ed[r], q[r], b + am[ct][m][r] + i);
        const float s = k[r] * am[ct][m][r], d = q[r] * a + k[r] * (b - i);
        sS[m][r] = VEC || ct == 0 ? s : sS[m][r] + s;
        sD[m][r] = VEC || ct == 0 ? d : sD[m][r] + d;
      }
      store_qk<DK>(p, c, sh, h, t0, ch, dq, dk);
    }
    if (VEC) {
      // dlog_alpha of the channel: sums over the tokens before and behind
      float x = xs[ct];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      float before[4], after[4], base = p.decay[sh * DK + ch] * x, tail = 0.0f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float a = (sS[m][0] + sS[m][1]) + (sS[m][2] + sS[m][3]);
        before[m] = base;
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          const float y = __shfl(a, fr + 16 * o);
          base += y;
          if (o < fg) before[m] += y;
        }
      }
#pragma unroll
      for (int m = 3; m >= 0; --m) {
        const float a = (sD[m][0] + sD[m][1]) + (sD[m][2] + sD[m][3]);
        after[m] = tail;
#pragma unroll
        for (int o = 3; o >= 0; --o) {
          const float y = __shfl(a, fr + 16 * o);
          tail += y;
          if (o > fg) after[m] += y;
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float b = before[m], a[4], s = after[m];
#pragma unroll
        for (int r = 3; r >= 0; --r) a[r] = s += sD[m][r];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = m * 16 + fg * 4 + r;
          if (t < c.len) p.dg[((c.row + t) * p.heads + h) * DK + ch] = b + a[r];
          b += sS[m][r];
        }
      }
    }
  }
  if (VEC) {
    if (wave == 0) store_dbeta<NW>(p, c, h, redb);
    return;
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
  float x = xs[0];
#pragma unroll
  for (int ct = 1; ct < CT; ++ct) x += xs[ct];
  x = sum16(x);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  if (lane == 0) redx[wave] = x;
  __syncthreads();
  if (wave == 0) {
    double s = 0.0, d = 0.0, sx = 0.0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      s += red[0][w][lane];
      d += red[1][w][lane];
      sx += redx[w];
    }
    double before = s, after = d;
    for (int o = 1; o < 64; o *= 2) {
      const double a = __shfl_up(before, o), b = __shfl_down(after, o);
      if (lane >= o) before += a;
      if (lane + o < 64) after += b;
    }
    if (lane < c.len)
      p.dg[(c.row + lane) * p.heads + h] = (float)(rows[C - 1] * sx + (before - s) + after);
    store_dbeta<NW>(p, c, h, redb);
  }
}

// ---- a gate per key channel, chunks that decay far -------------------------------------------
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
  if (!noted_chunk(p, slot, c)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t sh = (int64_t)slot * p.heads + h;
  if (!p.far[sh]) return;
  const int hq = h / (p.heads / p.heads_qk);
  const float* rows = rows_at(p, slot, h);
  __shared__ float redb[4][C];
  sum_dbeta<4>(p, sh, redb);
  const ValueRows dO = dout_rows(p, sh, h, c);
  auto uy_frag = [&](const float* src, int row, int col) {
    float x[8];
    return state_frag(src + (sh * C + row) * p.dvp + col, x);
  };
  const int nvs = p.dvp / 32;

  for (int b = 0; b < 4; ++b) {
    f32x4 e = {0, 0, 0, 0}, f = {0, 0, 0, 0};
    if (b <= wave)
      for (int s = 0; s < nvs; ++s) {
        const Frag<P> u = uy_frag(p.u, b * 16 + fr, s * 32 + fg * 8);
        mma(e, value_frag<NPO>(dO, wave * 16 + fr, s * 32 + fg * 8), u);
        if (DELTA) mma(f, uy_frag(p.y, wave * 16 + fr, s * 32 + fg * 8), u);
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
        if (DELTA) mma(ap[m], uy_frag(p.y, m * 16 + fr, s * 32 + fg * 8), fs);
        mma(am[m], uy_frag(p.u, m * 16 + fr, s * 32 + fg * 8), fx);
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
      const int64_t at = tq * NPR * DK * C + tiled<C>(ch, t0);
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
        asm volatile("" ::: "memory");  // else all rows' loads come first, and registers spill
#pragma unroll
        for (int j = 0; j < i; ++j) kd[j] *= al[i];
        kd[i] = k[i];
        x[i] = z[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < i; ++j) {
          x[i] = fmaf(Ed[fg][i][j], kd[j], x[i]);
          if (DELTA) z[i] = fmaf(Fd[fg][DELTA ? i : 0][j], kd[j], z[i]);
        }
      }
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        asm volatile("" ::: "memory");
        // token i's decay is taken on as i is passed
#pragma unroll
        for (int j = 0; j < i; ++j) {
          float s = fmaf(Ed[fg][i][j], q[i], y[j]);
          if (DELTA) s = fmaf(Fd[fg][DELTA ? i : 0][j], k[i], s);
          y[j] = s * al[i];
        }
      }
    }
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
    for (int m = 0; m < 4; ++m) {
      float dq[4], dk[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = m * 16 + fg * 4 + r;
        const bool in = t < c.len;
        const float q = in ? load_elem(p.q, (c.row + t) * p.qs + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        const float k = in ? load_elem(p.k, (c.row + t) * p.ks + (int64_t)hq * DK + ch, p.dtype) : 0.0f;
        dc[m][r] = q * aq[m][r] + k * (ap[m][r] - ai[m][r]);
        const float ed = Ed[m][fg * 4 + r][fg * 4 + r];
        dq[r] = fmaf(ed, k, aq[m][r]);
        dk[r] = fmaf(ed, q, ap[m][r] + am[m][r] + ai[m][r]);
      }
      store_qk<DK>(p, c, sh, h, m * 16 + fg * 4, ch, dq, dk);
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
  if (wave == 0) store_dbeta<4>(p, c, h, redb);
}

// dq and dk of heads that share them: summed in the order of the heads, four
// channels a thread.
template <int DK>
__global__ void __launch_bounds__(256) share_kernel(Params p) {
  const int slot = blockIdx.x, hq = blockIdx.y;
  Chunk c;
  if (!noted_chunk(p, slot, c)) return;
  const int group = p.heads / p.heads_qk;
  const int u = (blockIdx.z * 256 + threadIdx.x) * 4;
  if (u >= c.len * DK) return;
  f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  const int64_t from = ((int64_t)slot * p.heads + hq * group) * C * DK + u;
#pragma unroll 4
  for (int g = 0; g < group; ++g) {
    a += *reinterpret_cast<const f32x4*>(p.dqpart + from + (int64_t)g * C * DK);
    b += *reinterpret_cast<const f32x4*>(p.dkpart + from + (int64_t)g * C * DK);
  }
  const int64_t to = ((c.row + u / DK) * p.heads_qk + hq) * DK + u % DK;
  const int64_t at[4] = {to, to + 1, to + 2, to + 3};
  const bool ok[4] = {true, true, true, true};
  const float x[4] = {a[0], a[1], a[2], a[3]}, y[4] = {b[0], b[1], b[2], b[3]};
  store_elems<4>(p.dq, at, ok, p.dtype, x);
  store_elems<4>(p.dkk, at, ok, p.dtype, y);
}

}  // namespace qscan
