// scan_chain.h — the parts of the scan that go from chunk to chunk: the states
// forward and their gradients backward.
//
// One workgroup of four waves per (sequence, head, block of BV value columns).
// The state block stays in FP32 matrix accumulators, transposed: wave w holds
// key channels [w dk/4, (w+1) dk/4) x BV columns.  Its terms are written to LDS
// once a chunk for the products that contract over dk.  The operands that only
// one wave uses (its 16 rows of q, k, A and T, its channels of k^T) come
// straight from memory as matrix fragments; LDS holds what all waves share.

#pragma once

#include "scan_device.h"

namespace qscan {

// Workgroup -> (sequence, head, column block).  The blocks of one head read the
// same operands, so they get numbers that fall on one XCD (blockIdx mod 8).
__device__ __forceinline__ bool chain_block(const Params& p, int& n, int& h, int& vb) {
  const int64_t b = blockIdx.x;
  const int64_t head = b / (8 * p.nvb) * 8 + b % 8;
  vb = (int)(b / 8 % p.nvb);
  if (head >= (int64_t)p.batch * p.heads) return false;
  n = (int)(head / p.heads);
  h = (int)(head % p.heads);
  return true;
}

// Forward.  Per chunk: R = V - e^c K S^T (delta rule), U = T R, W = beta U,
// O = e^c Q S^T + A W, S = e^c_end S + (e^(c_end - c) W)^T K.  Row scales are
// applied to results and to W, so that with one gate per token q and k enter
// the products unrounded.  SAVE (for the backward pass): the states at the
// chunks' starts and U are stored, and no output.
template <int DK, int NT, int NPQ, bool VEC, bool DELTA, bool SAVE>
__global__ void __launch_bounds__(256) states_kernel(Params p) {
  constexpr int BV = 16 * NT, KS = DK / 32, MT = DK / 64, SP = DK + 8;
  __shared__ __align__(16) uint16_t Sl[P][BV][SP];
  __shared__ __align__(16) uint16_t Rt[DELTA ? P : 1][DELTA ? BV : 1][CP];
  __shared__ __align__(16) uint16_t Wt[SAVE ? 1 : P][SAVE ? 1 : BV][CP];
  __shared__ __align__(16) uint16_t Wb[P][BV][CP];  // e^(c_end - c) W (one gate), else W
  int n, h, vb;
  if (!chain_block(p, n, h, vb)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t o0 = offset_of(p, n), o1 = offset_of(p, n + 1);
  const int64_t len = o1 > o0 ? o1 - o0 : 0;
  const int nch = (int)((len + C - 1) / C);
  const int base = (int)(o0 / C) + n;
  const int d0 = wave * (DK / 4) + fg * 4;  // + 16 m: first of the lane's 4 channels
  const int tok = wave * 16 + fg * 4;       // first of the lane's 4 tokens
  const int64_t nh = (int64_t)n * p.heads + h;
  int vcol[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) vcol[t] = vb * BV + t * 16 + fr;

  f32x4 S[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      S[m][t] = f32x4{0, 0, 0, 0};
      if (p.s0 && vcol[t] < p.dv)
        S[m][t] = *reinterpret_cast<const f32x4*>(p.s0 + (nh * p.dv + vcol[t]) * DK + d0 + 16 * m);
    }
  auto put_state = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x[4] = {S[m][t][0], S[m][t][1], S[m][t][2], S[m][t][3]};
        put4<P>(&Sl[0][t * 16 + fr][d0 + 16 * m], BV * SP, x);
      }
  };
  if (DELTA || !SAVE) put_state();
  __syncthreads();

  for (int ci = 0; ci < nch; ++ci) {
    const int slot = base + ci;
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    const int64_t sh = (int64_t)slot * p.heads + h;
    const float* rows = rows_at(p, slot, h);
    if (SAVE) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p.sc[(sh * DK + d0 + 16 * m + r) * p.dvp + vcol[t]] = S[m][t][r];
    }
    // K S^T and Q S^T for the wave's 16 tokens
    f32x4 kS[NT], qS[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) kS[t] = qS[t] = f32x4{0, 0, 0, 0};
    if (DELTA || !SAVE) {
      const Rows qr = rows_of<DK>(p, p.q, p.qrow, p.qs, VEC, slot, h, c);
      const Rows kr = rows_of<DK>(p, p.k, p.krow, p.ks, VEC, slot, h, c);
      const int own = wave * 16 + fr;
      Frag<NPQ> fq[KS], fk[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (DELTA) fk[s] = load_frag_if<NPQ>(own < kr.len, kr.p + own * kr.row + s * 32 + fg * 8, kr.plane);
        if (!SAVE) fq[s] = load_frag_if<NPQ>(own < qr.len, qr.p + own * qr.row + s * 32 + fg * 8, qr.plane);
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const Frag<P> f = load_frag<P>(&Sl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP);
          if (DELTA) mma(kS[t], fk[s], f);
          if (!SAVE) mma(qS[t], fq[s], f);
        }
    }
    const f32x4 beta = *reinterpret_cast<const f32x4*>(rows + 2 * C + tok);
    f32x4 ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1};
    if (!VEC) {
      ec = *reinterpret_cast<const f32x4*>(rows + tok);
      eo = *reinterpret_cast<const f32x4*>(rows + C + tok);
    }
    f32x4 U[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        U[t][r] = tok + r < c.len && vcol[t] < p.dv
                      ? load_elem(p.v, (c.row + tok + r) * p.vs + (int64_t)h * p.dv + vcol[t], p.dtype)
                      : 0.0f;
    if (DELTA) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = fmaf(-ec[r], kS[t][r], U[t][r]);
        put4<P>(&Rt[0][t * 16 + fr][tok], BV * CP, x);
        U[t] = f32x4{0, 0, 0, 0};
      }
      __syncthreads();
      const uint16_t* T = p.t + sh * P * C * C + (wave * 16 + fr) * C + fg * 8;
      for (int s = 0; s <= wave / 2; ++s) {
        const Frag<P> f = load_frag<P>(T + s * 32, C * C);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(U[t], f, load_frag<P>(&Rt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4], wb[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w[r] = beta[r] * U[t][r];
        wb[r] = VEC ? w[r] : w[r] * eo[r];
      }
      if (!SAVE && !VEC) put4<P>(&Wt[0][t * 16 + fr][tok], BV * CP, w);
      put4<P>(&Wb[0][t * 16 + fr][tok], BV * CP, wb);
      if (SAVE) {
        u32x2 uu[P];
        const float x[4] = {U[t][0], U[t][1], U[t][2], U[t][3]};
        split4<P>(x, uu);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint16_t* d = p.u + ((sh * P + q) * C + tok) * p.dvp + vcol[t];
          d[0] = (uint16_t)uu[q].x;
          d[p.dvp] = (uint16_t)(uu[q].x >> 16);
          d[2 * p.dvp] = (uint16_t)uu[q].y;
          d[3 * p.dvp] = (uint16_t)(uu[q].y >> 16);
        }
      }
    }
    __syncthreads();
    if (!SAVE && p.o) {
      const uint16_t* A = p.a + sh * P * C * C + (wave * 16 + fr) * C + fg * 8;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) qS[t][r] *= ec[r];
      for (int s = 0; s <= wave / 2; ++s) {
        const Frag<P> f = load_frag<P>(A + s * 32, C * C);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(qS[t], f,
              load_frag<P>(VEC ? &Wb[0][t * 16 + fr][s * 32 + fg * 8]
                               : &Wt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tok + r < c.len && vcol[t] < p.dv)
            store_elem(p.o, (c.row + tok + r) * p.os + (int64_t)h * p.dv + vcol[t], p.dtype, qS[t][r]);
    }
    // the state at the chunk's end
    {
      const float end = VEC ? 1.0f : rows[C - 1];
      const int64_t th = VEC ? sh : (int64_t)slot * p.heads_qk + h / (p.heads / p.heads_qk);
      const uint16_t* kt = p.kt + th * NPQ * DK * C;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = wave * (DK / 4) + 16 * m;
        f32x4 dec = {end, end, end, end};
        if (VEC) dec = *reinterpret_cast<const f32x4*>(p.decay + sh * DK + d0 + 16 * m);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[m][t][r] *= dec[r];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const Frag<NPQ> f = load_frag<NPQ>(kt + (int64_t)(row + fr) * C + s * 32 + fg * 8, DK * C);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(S[m][t], f, load_frag<P>(&Wb[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
        }
      }
      if (DELTA || !SAVE) put_state();
    }
    __syncthreads();
  }
  if (p.s1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (vcol[t] < p.dv)
          *reinterpret_cast<f32x4*>(p.s1 + (nh * p.dv + vcol[t]) * DK + d0 + 16 * m) = S[m][t];
  }
}

// Backward, chunks in reverse.  X is the gradient of the state at the chunk's
// end: dW = A^T dO + e^(c_end - c) K X^T, Z = (I + beta L)^-T dW (delta rule;
// else dW), dV = Y = beta Z, dbeta = U . Z over the value columns, and
// X = e^c_end X + (e^c dO)^T Q - (e^c Y)^T K (the last with the delta rule).
template <int DK, int NT, int NPQ, int NPO, bool VEC, bool DELTA>
__global__ void __launch_bounds__(256) state_grads_kernel(Params p) {
  constexpr int BV = 16 * NT, KS = DK / 32, MT = DK / 64, SP = DK + 8;
  __shared__ __align__(16) uint16_t Xl[P][BV][SP];
  __shared__ __align__(16) uint16_t Ot[NPO][BV][CP];                            // d_o
  __shared__ __align__(16) uint16_t Oe[VEC ? 1 : P][VEC ? 1 : BV][CP];          // e^c d_o
  __shared__ __align__(16) uint16_t Dt[DELTA ? P : 1][DELTA ? BV : 1][CP];      // dW
  __shared__ __align__(16) uint16_t Yt[DELTA ? P : 1][DELTA ? BV : 1][CP];      // -e^c Y
  int n, h, vb;
  if (!chain_block(p, n, h, vb)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t o0 = offset_of(p, n), o1 = offset_of(p, n + 1);
  const int64_t len = o1 > o0 ? o1 - o0 : 0;
  const int nch = (int)((len + C - 1) / C);
  const int base = (int)(o0 / C) + n;
  const int d0 = wave * (DK / 4) + fg * 4;
  const int tok = wave * 16 + fg * 4;
  const int64_t nh = (int64_t)n * p.heads + h;
  int vcol[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) vcol[t] = vb * BV + t * 16 + fr;
  f32x4 X[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      X[m][t] = f32x4{0, 0, 0, 0};
      if (p.ds1 && vcol[t] < p.dv)
        X[m][t] = *reinterpret_cast<const f32x4*>(p.ds1 + (nh * p.dv + vcol[t]) * DK + d0 + 16 * m);
    }
  auto put_state = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x[4] = {X[m][t][0], X[m][t][1], X[m][t][2], X[m][t][3]};
        put4<P>(&Xl[0][t * 16 + fr][d0 + 16 * m], BV * SP, x);
      }
  };
  put_state();
  __syncthreads();

  for (int ci = nch - 1; ci >= 0; --ci) {
    const int slot = base + ci;
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    const int64_t sh = (int64_t)slot * p.heads + h;
    const float* rows = rows_at(p, slot, h);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p.xc[(sh * DK + d0 + 16 * m + r) * p.dvp + vcol[t]] = X[m][t][r];
    const f32x4 beta = *reinterpret_cast<const f32x4*>(rows + 2 * C + tok);
    f32x4 ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1};
    if (!VEC) {
      ec = *reinterpret_cast<const f32x4*>(rows + tok);
      eo = *reinterpret_cast<const f32x4*>(rows + C + tok);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4], xe[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = tok + r < c.len && vcol[t] < p.dv
                   ? load_elem(p.dO, ((c.row + tok + r) * p.heads + h) * p.dv + vcol[t], p.dtype)
                   : 0.0f;
        xe[r] = x[r] * ec[r];
      }
      put4<NPO>(&Ot[0][t * 16 + fr][tok], BV * CP, x);
      if (!VEC) put4<P>(&Oe[0][t * 16 + fr][tok], BV * CP, xe);
    }
    f32x4 W[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) W[t] = f32x4{0, 0, 0, 0};
    {
      const Rows kr = rows_of<DK>(p, p.k, VEC ? p.korow : p.krow, p.ks, VEC, slot, h, c);
      const int own = wave * 16 + fr;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<NPQ> fk = load_frag_if<NPQ>(own < kr.len, kr.p + own * kr.row + s * 32 + fg * 8, kr.plane);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(W[t], fk, load_frag<P>(&Xl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP));
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) W[t][r] *= eo[r];
    __syncthreads();
    {
      const uint16_t* A = p.at + sh * P * C * C + (wave * 16 + fr) * C + fg * 8;
      for (int s = wave / 2; s < 2; ++s) {
        const Frag<P> f = load_frag<P>(A + s * 32, C * C);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(W[t], f, load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      }
    }
    if (DELTA) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x[4] = {W[t][0], W[t][1], W[t][2], W[t][3]};
        put4<P>(&Dt[0][t * 16 + fr][tok], BV * CP, x);
        W[t] = f32x4{0, 0, 0, 0};
      }
      __syncthreads();
      const uint16_t* T = p.t2t + sh * P * C * C + (wave * 16 + fr) * C + fg * 8;
      for (int s = wave / 2; s < 2; ++s) {
        const Frag<P> f = load_frag<P>(T + s * 32, C * C);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(W[t], f, load_frag<P>(&Dt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      }
    }
    // W holds Z
    float db[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[4], ye[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = beta[r] * W[t][r];
        ye[r] = -ec[r] * y[r];
        const bool in = tok + r < c.len && vcol[t] < p.dv;
        if (in) store_elem(p.dv_out, ((c.row + tok + r) * p.heads + h) * p.dv + vcol[t], p.dtype, y[r]);
        if (p.dbeta) {
          float u = 0.0f;
#pragma unroll
          for (int q = P - 1; q >= 0; --q)
            u += bf16_to_f(p.u[((sh * P + q) * C + tok + r) * p.dvp + vcol[t]]);
          db[r] = fmaf(u, W[t][r], db[r]);
        }
      }
      if (DELTA) {
        put4<P>(&Yt[0][t * 16 + fr][tok], BV * CP, ye);
        u32x2 yy[P];
        split4<P>(y, yy);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint16_t* d = p.y + ((sh * P + q) * C + tok) * p.dvp + vcol[t];
          d[0] = (uint16_t)yy[q].x;
          d[p.dvp] = (uint16_t)(yy[q].x >> 16);
          d[2 * p.dvp] = (uint16_t)yy[q].y;
          d[3 * p.dvp] = (uint16_t)(yy[q].y >> 16);
        }
      }
    }
    if (p.dbeta) {
#pragma unroll
      for (int r = 0; r < 4; ++r) db[r] = sum16(db[r]);
      if (fr == 0)
        *reinterpret_cast<f32x4*>(
            p.dbpart + ((int64_t)vb * p.nslots * p.heads + sh) * C + tok) = f32x4{db[0], db[1], db[2], db[3]};
    }
    if (DELTA) __syncthreads();
    {
      const float end = VEC ? 1.0f : rows[C - 1];
      const int64_t th = VEC ? sh : (int64_t)slot * p.heads_qk + h / (p.heads / p.heads_qk);
      const uint16_t* qt = p.qt + th * NPQ * DK * C;
      const uint16_t* kt = (VEC ? p.ket : p.kt) + th * NPQ * DK * C;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = wave * (DK / 4) + 16 * m;
        f32x4 dec = {end, end, end, end};
        if (VEC) dec = *reinterpret_cast<const f32x4*>(p.decay + sh * DK + d0 + 16 * m);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) X[m][t][r] *= dec[r];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int64_t at = (int64_t)(row + fr) * C + s * 32 + fg * 8;
          const Frag<NPQ> f = load_frag<NPQ>(qt + at, DK * C);
          Frag<NPQ> g;
          if (DELTA) g = load_frag<NPQ>(kt + at, DK * C);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (VEC)
              mma(X[m][t], f, load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
            else
              mma(X[m][t], f, load_frag<P>(&Oe[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
            if (DELTA) mma(X[m][t], g, load_frag<P>(&Yt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
          }
        }
      }
      put_state();
    }
    __syncthreads();
  }
  if (p.ds0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (vcol[t] < p.dv)
          *reinterpret_cast<f32x4*>(p.ds0 + (nh * p.dv + vcol[t]) * DK + d0 + 16 * m) = X[m][t];
  }
}

}  // namespace qscan
