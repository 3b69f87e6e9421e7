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
  __shared__ __align__(16) uint16_t Wt[SAVE || VEC ? 1 : P][SAVE || VEC ? 1 : BV][CP];
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

  // Rows behind a sequence's end repeat its last row: beta is zero there, so
  // what they compute reaches neither the state nor an output.
  // A chunk's operands, each loaded again for the next chunk right after its
  // last use: the loads have most of a chunk's time to arrive and need no
  // second set of registers.
  constexpr bool KQ = DELTA || !SAVE;
  Frag<NPQ> fq[SAVE ? 1 : KS], fk[DELTA ? KS : 1], ft[MT][2];
  Frag<P> fT[DELTA ? 2 : 1], fA[SAVE ? 1 : 2];
  uint32_t v[NT][4];
  f32x4 beta, ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1}, dec[MT];
  const int own = wave * 16 + fr;
  auto chunk = [&](int ci) {
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    return c;
  };
  auto load_kq = [&](int ci) {
    const Chunk c = chunk(ci);
    if (DELTA) {
      const Rows kr = rows_of<DK>(p, p.k, p.krow, p.ks, VEC, base + ci, h, c);
#pragma unroll
      for (int s = 0; s < KS; ++s)
        fk[s] = load_frag<NPQ>(kr.p + min(own, kr.len - 1) * kr.row + s * 32 + fg * 8, kr.plane);
    }
    if (!SAVE) {
      const Rows qr = rows_of<DK>(p, p.q, p.qrow, p.qs, VEC, base + ci, h, c);
#pragma unroll
      for (int s = 0; s < KS; ++s)
        fq[s] = load_frag<NPQ>(qr.p + min(own, qr.len - 1) * qr.row + s * 32 + fg * 8, qr.plane);
    }
  };
  auto load_v = [&](int ci) {
    const Chunk c = chunk(ci);
    const float* rows = rows_at(p, base + ci, h);
    beta = *reinterpret_cast<const f32x4*>(rows + 2 * C + tok);
    if (!VEC) {
      ec = *reinterpret_cast<const f32x4*>(rows + tok);
      eo = *reinterpret_cast<const f32x4*>(rows + C + tok);
    }
    // places outside the sequence or the head read a valid neighbour and count as zero later
    int64_t at[4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        at[r] = (c.row + min(tok + r, c.len - 1)) * p.vs + (int64_t)h * p.dv + min(vcol[t], p.dv - 1);
      load_raw<4>(p.v, at, p.dtype, v[t]);
    }
  };
  auto load_square = [&](const uint16_t* m, int ci, Frag<P>* f) {
    const uint16_t* at = m + ((int64_t)(base + ci) * p.heads + h) * P * C * C + own * C + fg * 8;
    f[0] = load_frag<P>(at, C * C);
    f[1] = load_frag<P>(at + 32, C * C);
  };
  auto load_t = [&](int ci) {
    const int slot = base + ci;
    const int64_t sh = (int64_t)slot * p.heads + h;
    const int64_t th = VEC ? sh : (int64_t)slot * p.heads_qk + h / (p.heads / p.heads_qk);
    const uint16_t* kt = p.kt + th * NPQ * DK * C;
    const float end = VEC ? 1.0f : rows_at(p, slot, h)[C - 1];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ft[m][s] = load_frag<NPQ>(
            kt + (int64_t)(wave * (DK / 4) + 16 * m + fr) * C + s * 32 + fg * 8, DK * C);
      dec[m] = VEC ? *reinterpret_cast<const f32x4*>(p.decay + sh * DK + d0 + 16 * m)
                   : f32x4{end, end, end, end};
    }
  };
  if (nch > 0) {
    load_kq(0);
    load_v(0);
    if (DELTA) load_square(p.t, 0, fT);
    if (!SAVE) load_square(p.a, 0, fA);
    load_t(0);
  }

  for (int ci = 0; ci < nch; ++ci) {
    const Chunk c = chunk(ci);
    const int64_t sh = (int64_t)(base + ci) * p.heads + h;
    const int next = min(ci + 1, nch - 1);  // loads without a branch: the last chunk's again
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
    if (KQ) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const Frag<P> f = load_frag<P>(&Sl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP);
          if (DELTA) mma(kS[t], fk[s], f);
          if (!SAVE) mma(qS[t], fq[s], f);
        }
      load_kq(next);
    }
    f32x4 U[NT], ecur = ec;
    float vf[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vf[t][r] = tok + r < c.len && vcol[t] < p.dv ? from_raw(v[t][r], p.dtype) : 0.0f;
    if (DELTA) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = fmaf(-ec[r], kS[t][r], vf[t][r]);
        put4<P>(&Rt[0][t * 16 + fr][tok], BV * CP, x);
        U[t] = f32x4{0, 0, 0, 0};
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(U[t], fT[s], load_frag<P>(&Rt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      load_square(p.t, next, fT);
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) U[t] = f32x4{vf[t][0], vf[t][1], vf[t][2], vf[t][3]};
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
    load_v(next);
    __syncthreads();
    // the state at the chunk's end
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[m][t][r] *= dec[m][r];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(S[m][t], ft[m][s], load_frag<P>(&Wb[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
    }
    load_t(next);
    if (KQ) put_state();
    if (!SAVE) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) qS[t][r] *= ecur[r];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(qS[t], fA[s],
                load_frag<P>(VEC ? &Wb[0][t * 16 + fr][s * 32 + fg * 8]
                                 : &Wt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      load_square(p.a, next, fA);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        int64_t at[4];
        bool ok[4];
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          at[r] = (c.row + tok + r) * p.os + (int64_t)h * p.dv + vcol[t];
          ok[r] = p.o && tok + r < c.len && vcol[t] < p.dv;
          x[r] = qS[t][r];
        }
        store_elems<4>(p.o, at, ok, p.dtype, x);
      }
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

  // operands are reloaded after their last use, as in states_kernel
  Frag<NPQ> fk[KS], fq[MT][2], ft[DELTA ? MT : 1][2];
  Frag<P> fA[2], fT[DELTA ? 2 : 1];
  uint32_t x[NT][4], u[NT][4][P];
  f32x4 beta, ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1}, dec[MT];
  const int own = wave * 16 + fr;
  auto chunk = [&](int ci) {
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    return c;
  };
  auto load_do = [&](int ci) {
    const Chunk c = chunk(ci);
    const int64_t sh = (int64_t)(base + ci) * p.heads + h;
    const float* rows = rows_at(p, base + ci, h);
    beta = *reinterpret_cast<const f32x4*>(rows + 2 * C + tok);
    if (!VEC) {
      ec = *reinterpret_cast<const f32x4*>(rows + tok);
      eo = *reinterpret_cast<const f32x4*>(rows + C + tok);
    }
    int64_t at[4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        at[r] = ((c.row + min(tok + r, c.len - 1)) * p.heads + h) * p.dv + min(vcol[t], p.dv - 1);
      load_raw<4>(p.dO, at, p.dtype, x[t]);
      if (p.dbeta) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int q = 0; q < P; ++q)
            u[t][r][q] = p.u[((sh * P + q) * C + tok + r) * p.dvp + vcol[t]];
      }
    }
  };
  auto load_k = [&](int ci) {
    const Rows kr = rows_of<DK>(p, p.k, VEC ? p.korow : p.krow, p.ks, VEC, base + ci, h, chunk(ci));
#pragma unroll
    for (int s = 0; s < KS; ++s)
      fk[s] = load_frag<NPQ>(kr.p + min(own, kr.len - 1) * kr.row + s * 32 + fg * 8, kr.plane);
  };
  auto load_square = [&](const uint16_t* m, int ci, Frag<P>* f) {
    const uint16_t* at = m + ((int64_t)(base + ci) * p.heads + h) * P * C * C + own * C + fg * 8;
    f[0] = load_frag<P>(at, C * C);
    f[1] = load_frag<P>(at + 32, C * C);
  };
  auto load_t = [&](int ci) {
    const int slot = base + ci;
    const int64_t sh = (int64_t)slot * p.heads + h;
    const int64_t th = VEC ? sh : (int64_t)slot * p.heads_qk + h / (p.heads / p.heads_qk);
    const uint16_t* qt = p.qt + th * NPQ * DK * C;
    const uint16_t* kt = (VEC ? p.ket : p.kt) + th * NPQ * DK * C;
    const float end = VEC ? 1.0f : rows_at(p, slot, h)[C - 1];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int64_t at = (int64_t)(wave * (DK / 4) + 16 * m + fr) * C + s * 32 + fg * 8;
        fq[m][s] = load_frag<NPQ>(qt + at, DK * C);
        if (DELTA) ft[m][s] = load_frag<NPQ>(kt + at, DK * C);
      }
      dec[m] = VEC ? *reinterpret_cast<const f32x4*>(p.decay + sh * DK + d0 + 16 * m)
                   : f32x4{end, end, end, end};
    }
  };
  if (nch > 0) {
    load_do(nch - 1);
    load_k(nch - 1);
    load_square(p.at, nch - 1, fA);
    if (DELTA) load_square(p.t2t, nch - 1, fT);
    load_t(nch - 1);
  }

  for (int ci = nch - 1; ci >= 0; --ci) {
    const Chunk c = chunk(ci);
    const int64_t sh = (int64_t)(base + ci) * p.heads + h;
    const int next = max(ci - 1, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p.xc[(sh * DK + d0 + 16 * m + r) * p.dvp + vcol[t]] = X[m][t][r];
    const f32x4 bc = beta, ecc = ec, eoc = eo;
    float uc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float xo[4], xe[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        xo[r] = tok + r < c.len && vcol[t] < p.dv ? from_raw(x[t][r], p.dtype) : 0.0f;
        xe[r] = xo[r] * ec[r];
        uc[t][r] = 0.0f;
        if (p.dbeta) {
#pragma unroll
          for (int q = P - 1; q >= 0; --q) uc[t][r] += bf16_to_f((uint16_t)u[t][r][q]);
        }
      }
      put4<NPO>(&Ot[0][t * 16 + fr][tok], BV * CP, xo);
      if (!VEC) put4<P>(&Oe[0][t * 16 + fr][tok], BV * CP, xe);
    }
    load_do(next);
    f32x4 W[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) W[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma(W[t], fk[s], load_frag<P>(&Xl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP));
    load_k(next);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) W[t][r] *= eoc[r];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s >= wave / 2)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(W[t], fA[s], load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
    load_square(p.at, next, fA);
    if (DELTA) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float w[4] = {W[t][0], W[t][1], W[t][2], W[t][3]};
        put4<P>(&Dt[0][t * 16 + fr][tok], BV * CP, w);
        W[t] = f32x4{0, 0, 0, 0};
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s >= wave / 2)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(W[t], fT[s], load_frag<P>(&Dt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      load_square(p.t2t, next, fT);
    }
    // W holds Z
    float db[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[4], ye[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = bc[r] * W[t][r];
        ye[r] = -ecc[r] * y[r];
        if (p.dbeta) db[r] = fmaf(uc[t][r], W[t][r], db[r]);
      }
      if (DELTA) put4<P>(&Yt[0][t * 16 + fr][tok], BV * CP, ye);
      int64_t at[4];
      bool ok[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        at[r] = ((c.row + tok + r) * p.heads + h) * p.dv + vcol[t];
        ok[r] = tok + r < c.len && vcol[t] < p.dv;
      }
      store_elems<4>(p.dv_out, at, ok, p.dtype, y);
      if (DELTA) {
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
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) X[m][t][r] *= dec[m][r];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (VEC)
            mma(X[m][t], fq[m][s], load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
          else
            mma(X[m][t], fq[m][s], load_frag<P>(&Oe[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
          if (DELTA)
            mma(X[m][t], ft[m][s], load_frag<P>(&Yt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
        }
    }
    load_t(next);
    put_state();
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
