// scan_chain.h — the parts of the scan that go from chunk to chunk: the states
// forward and their gradients backward.
//
// One workgroup per (sequence, head, block of BV value columns).
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
// the products unrounded.
//
// What bounds it is the chain from one state to the next, so it has waves of
// its own: waves 0..3 compute R, U and S, waves 4..7 beside them O, which
// nothing waits for.  (All in four waves a chunk took 6400 cycles, O's part of
// them 1900.)  At dk = 128 and 16 columns a chunk takes 2.6 us (GDN, bfloat16,
// 256 workgroups) to 3.1 us (KDA, 128); the matrix instructions are busy for
// 9 to 14 % of it, LDS round trips between the barriers and 100 to 170 KB of
// operands out of L2 for each chunk take the rest.
// Outputs take every term, as the state does, whatever their type: with two terms
// of q, A, S and W a 16-bit output that is small by cancellation would be off by
// more than its own rounding.
//
// SOLVED: U0 = T V and K^ = T K~ are given (scan_prep_vector.h), and U = U0 - K^ S^T.
//
// SAVE (for the backward pass): four waves, no output; the states at the
// chunks' starts and U are stored.
template <int DK, int NT, int NPQ, bool VEC, bool DELTA, bool SAVE, bool SOLVED>
__global__ void __launch_bounds__(SAVE ? 256 : 512) states_kernel(Params p) {
  constexpr int BV = 16 * NT, KS = DK / 32, MT = DK / 64, SP = DK + 8;
  constexpr bool D = NPQ == 1;
  __shared__ __align__(16) uint16_t Sl[P][BV][SP];
  constexpr bool TR = DELTA && !SOLVED;  // U = T R is computed here
  __shared__ __align__(16) uint16_t Rt[TR ? P : 1][TR ? BV : 1][CP];
  __shared__ __align__(16) uint16_t Wt[SAVE || VEC ? 1 : P][SAVE || VEC ? 1 : BV][CP];
  __shared__ __align__(16) uint16_t Wb[P][BV][CP];  // e^(c_end - c) W (one gate), else W
  int n, h, vb;
  if (!chain_block(p, n, h, vb)) return;
  const int wave = (threadIdx.x >> 6) & 3, lane = threadIdx.x & 63;
  const bool reader = !SAVE && threadIdx.x >= 256;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t o0 = offset_of(p, n), o1 = offset_of(p, n + 1);
  const int64_t len = o1 > o0 ? o1 - o0 : 0;
  if (!SAVE && len <= p.short_len) return;
  const int nch = (int)((len + C - 1) / C);
  const int base = (int)(o0 / C) + n;
  const int tok = wave * 16 + fg * 4;  // first of the lane's 4 tokens
  int vcol[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) vcol[t] = vb * BV + t * 16 + fr;
  // Operands are loaded again for the next chunk right after their last use:
  // the loads have most of a chunk's time to arrive and need no second set of
  // registers.  No branch goes around them (the last chunk loads itself again),
  // so that each use waits for its own loads only.
  auto chunk = [&](int ci) {
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    return c;
  };
  auto head_of = [&](int ci) { return (int64_t)(base + ci) * p.heads + h; };

  if (reader) {
    Frag<NPQ> fq[KS];
    Frag<P> fA[2];
    f32x4 ec = {1, 1, 1, 1};
    auto load_q = [&](int ci) {
      const auto q = rows_of<DK, D>(p, p.q, p.qrow, p.qs, VEC, base + ci, h, chunk(ci));
#pragma unroll
      for (int s = 0; s < KS; ++s) fq[s] = q.template frag<NPQ>(wave, s);
      if (!VEC) ec = *reinterpret_cast<const f32x4*>(rows_at(p, base + ci, h) + tok);
    };
    auto load_a = [&](int ci) {
#pragma unroll
      for (int s = 0; s < 2; ++s) fA[s] = tile_frag<P, C>(p.a + head_of(ci) * P * C * C, wave, s, C * C);
    };
    if (nch > 0) {
      load_q(0);
      load_a(0);
    }
    f32x4 O[NT];
    // A chunk's outputs are stored behind the next chunk's first product, while
    // the other waves compute U: right after A W they would hold up the barrier.
    auto store = [&](int ci, const f32x4(&x)[NT]) {
      const Chunk c = chunk(ci);
      const int64_t at = c.row * p.os + (int64_t)h * p.dv;
      char* o = static_cast<char*>(p.o) + at * (p.dtype == 0 ? 4 : 2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t off[4];
        bool ok[4];
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          off[r] = (uint32_t)(tok + r) * (uint32_t)p.os + vcol[t];
          ok[r] = p.o && tok + r < c.len && vcol[t] < p.dv;
          y[r] = x[t][r];
        }
        store_always<4>(o, off, ok, p.dtype, p.sink, y);
      }
    };
    __syncthreads();
    for (int ci = 0; ci < nch; ++ci) {
      const int next = min(ci + 1, nch - 1);
      f32x4 Q[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) Q[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(Q[t], fq[s], load_frag<P>(&Sl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) Q[t][r] *= ec[r];
      load_q(next);
      if (TR) __syncthreads();
      if (ci > 0) store(ci - 1, O);
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NT; ++t) O[t] = Q[t];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(O[t], fA[s],
                load_frag<P>(VEC ? &Wb[0][t * 16 + fr][s * 32 + fg * 8]
                                  : &Wt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      load_a(next);
      __syncthreads();
    }
    store(nch - 1, O);
    return;
  }

  const int d0 = wave * (DK / 4) + fg * 4;  // + 16 m: first of the lane's 4 channels
  const int64_t nh = (int64_t)n * p.heads + h;
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
  Frag<NPQ> fk[DELTA ? KS : 1], ft[MT][2];
  Frag<P> fT[TR ? 2 : 1];
  uint32_t v[NT][4];  // the values, or U0 as floats
  f32x4 beta, ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1}, dec[MT];
  auto load_k = [&](int ci) {
    const auto k = rows_of<DK, D>(p, p.k, p.krow, p.ks, VEC, base + ci, h, chunk(ci));
#pragma unroll
    for (int s = 0; s < KS; ++s) fk[s] = k.template frag<NPQ>(wave, s);
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
    if (SOLVED) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[t][r] = __float_as_uint(p.u[head_of(ci) * C * p.dvp + (uint32_t)((tok + r) * p.dvp + vcol[t])]);
      return;
    }
    const char* src = static_cast<const char*>(p.v) +
                      (c.row * p.vs + (int64_t)h * p.dv) * (p.dtype == 0 ? 4 : 2);
    uint32_t at[4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        at[r] = min((uint32_t)(tok + r) * (uint32_t)p.vs, (uint32_t)(c.len - 1) * (uint32_t)p.vs) +
                min(vcol[t], p.dv - 1);
      load_raw<4>(src, at, p.dtype, v[t]);
    }
  };
  auto load_T = [&](int ci) {
#pragma unroll
    for (int s = 0; s < 2; ++s) fT[s] = tile_frag<P, C>(p.t + head_of(ci) * P * C * C, wave, s, C * C);
  };
  auto load_kt = [&](int ci) {
    const int slot = base + ci;
    const int64_t th = VEC ? head_of(ci) : (int64_t)slot * p.heads_qk + h / (p.heads / p.heads_qk);
    const uint16_t* kt = p.kt + th * NPQ * DK * C;
    const float end = VEC ? 1.0f : rows_at(p, slot, h)[C - 1];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int s = 0; s < 2; ++s) ft[m][s] = tile_frag<NPQ, C>(kt, wave * MT + m, s, DK * C);
      dec[m] = VEC ? *reinterpret_cast<const f32x4*>(p.decay + head_of(ci) * DK + d0 + 16 * m)
                   : f32x4{end, end, end, end};
    }
  };
  if (nch > 0) {
    if (DELTA) load_k(0);
    load_v(0);
    if (TR) load_T(0);
    load_kt(0);
  }
  if (DELTA || !SAVE) put_state();
  __syncthreads();

  for (int ci = 0; ci < nch; ++ci) {
    const Chunk c = chunk(ci);
    const int64_t sh = head_of(ci);
    const int next = min(ci + 1, nch - 1);
    f32x4 U[NT];
    float vf[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vf[t][r] = SOLVED ? __uint_as_float(v[t][r])
                   : tok + r < c.len && vcol[t] < p.dv ? from_raw(v[t][r], p.dtype) : 0.0f;
    if (DELTA) {
      f32x4 kS[NT], kS2[NT];  // two chains of dependent products
#pragma unroll
      for (int t = 0; t < NT; ++t) kS[t] = kS2[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma(s & 1 ? kS2[t] : kS[t], fk[s],
              load_frag<P>(&Sl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP));
#pragma unroll
      for (int t = 0; t < NT; ++t) kS[t] += kS2[t];
      load_k(next);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = fmaf(-ec[r], kS[t][r], vf[t][r]);
        if (TR) put4<P>(&Rt[0][t * 16 + fr][tok], BV * CP, x);
        U[t] = TR ? f32x4{0, 0, 0, 0} : f32x4{x[0], x[1], x[2], x[3]};
      }
    }
    if (TR) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= wave / 2)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma(U[t], fT[s], load_frag<P>(&Rt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
      load_T(next);
    }
    if (!DELTA) {
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
      put4<P>(&Wb[0][t * 16 + fr][tok], BV * CP, wb);
      if (!SAVE && !VEC) put4<P>(&Wt[0][t * 16 + fr][tok], BV * CP, w);
    }
    load_v(next);
    __syncthreads();
    if (SAVE) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p.u[sh * C * p.dvp + (uint32_t)((tok + r) * p.dvp + vcol[t])] = U[t][r];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p.sc[sh * DK * p.dvp + (uint32_t)((d0 + 16 * m + r) * p.dvp + vcol[t])] = S[m][t][r];
    }
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
    load_kt(next);
    if (DELTA || !SAVE) put_state();
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
//
// As forward, the chain has waves of its own (0..3).  What does not wait for X,
// A^T dO and (e^c dO)^T Q, waves 4..7 compute one chunk ahead and hand over in
// LDS.  3.5 us a chunk at dk = 128 and 16 columns (GDN, bfloat16, 256
// workgroups), bound as the forward chain is.
template <int DK, int NT, int NPQ, int NPO, bool VEC, bool DELTA>
__global__ void __launch_bounds__(512) state_grads_kernel(Params p) {
  constexpr bool BETA = DELTA || !VEC;  // GLA has none
  constexpr int BV = 16 * NT, KS = DK / 32, MT = DK / 64, SP = DK + 8, FP = C + 4;
  __shared__ __align__(16) uint16_t Xl[P][BV][SP];
  __shared__ __align__(16) uint16_t Ot[NPO][BV][CP];                        // d_o
  __shared__ __align__(16) uint16_t Oe[VEC ? 1 : P][VEC ? 1 : BV][CP];      // e^c d_o
  __shared__ __align__(16) uint16_t Dt[DELTA ? P : 1][DELTA ? BV : 1][CP];  // dW
  __shared__ __align__(16) uint16_t Yt[DELTA ? P : 1][DELTA ? BV : 1][CP];  // -e^c Y
  __shared__ __align__(16) float Al[BV][FP];                                // A^T dO
  __shared__ __align__(16) float Gl[4][MT * NT][64][4];                     // (e^c dO)^T Q
  int n, h, vb;
  if (!chain_block(p, n, h, vb)) return;
  const int wave = (threadIdx.x >> 6) & 3, lane = threadIdx.x & 63;
  const bool helper = threadIdx.x >= 256;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t o0 = offset_of(p, n), o1 = offset_of(p, n + 1);
  const int64_t len = o1 > o0 ? o1 - o0 : 0;
  const int nch = (int)((len + C - 1) / C);
  const int base = (int)(o0 / C) + n;
  const int tok = wave * 16 + fg * 4;
  const int group = p.heads / p.heads_qk;
  int vcol[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) vcol[t] = vb * BV + t * 16 + fr;
  // operands are reloaded after their last use, without branches, as in states_kernel
  auto chunk = [&](int ci) {
    Chunk c;
    c.n = n;
    c.ci = ci;
    c.row = o0 + (int64_t)ci * C;
    c.len = len - (int64_t)ci * C < C ? (int)(len - (int64_t)ci * C) : C;
    return c;
  };
  auto head_of = [&](int ci) { return (int64_t)(base + ci) * p.heads + h; };
  auto qk_of = [&](int ci) { return VEC ? head_of(ci) : (int64_t)(base + ci) * p.heads_qk + h / group; };

  if (helper) {
    Frag<NPQ> fq[MT][2];
    Frag<P> fA[2];
    uint32_t x[NT][4];
    f32x4 ec = {1, 1, 1, 1}, A[NT], G[MT][NT];
    auto load_do = [&](int ci) {
      const Chunk c = chunk(ci);
      if (!VEC) ec = *reinterpret_cast<const f32x4*>(rows_at(p, base + ci, h) + tok);
      const uint32_t stride = (uint32_t)p.heads * p.dv;
      const char* src = static_cast<const char*>(p.dO) +
                        (c.row * p.heads + h) * p.dv * (p.dtype == 0 ? 4 : 2);
      uint32_t at[4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          at[r] = min((uint32_t)(tok + r) * stride, (uint32_t)(c.len - 1) * stride) + min(vcol[t], p.dv - 1);
        load_raw<4>(src, at, p.dtype, x[t]);
      }
    };
    auto load_mats = [&](int ci) {
#pragma unroll
      for (int s = 0; s < 2; ++s) fA[s] = tile_frag<P, C>(p.at + head_of(ci) * P * C * C, wave, s, C * C);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          fq[m][s] = tile_frag<NPQ, C>(p.qt + qk_of(ci) * NPQ * DK * C, wave * MT + m, s, DK * C);
    };
    auto stage = [&](int ci) {
      const Chunk c = chunk(ci);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float xo[4], xe[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          xo[r] = tok + r < c.len && vcol[t] < p.dv ? from_raw(x[t][r], p.dtype) : 0.0f;
          xe[r] = xo[r] * ec[r];
        }
        put4<NPO>(&Ot[0][t * 16 + fr][tok], BV * CP, xo);
        if (!VEC) put4<P>(&Oe[0][t * 16 + fr][tok], BV * CP, xe);
      }
    };
    auto products = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        A[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (s >= wave / 2)
            mma(A[t], fA[s], load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
        *reinterpret_cast<f32x4*>(&Al[t * 16 + fr][tok]) = A[t];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          G[m][t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (VEC)
              mma(G[m][t], fq[m][s], load_frag<NPO>(&Ot[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
            else
              mma(G[m][t], fq[m][s], load_frag<P>(&Oe[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
        }
    };
    auto hand_over = [&]() {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<f32x4*>(Gl[wave][m * NT + t][lane]) = G[m][t];
    };
    if (nch > 0) {
      load_do(nch - 1);
      load_mats(nch - 1);
      stage(nch - 1);
    }
    __syncthreads();
    if (nch > 0) {
      load_do(max(nch - 2, 0));
      products();
      load_mats(max(nch - 2, 0));
    }
    __syncthreads();
    for (int ci = nch - 1; ci >= 0; --ci) {  // one chunk ahead: ci - 1
      hand_over();
      stage(max(ci - 1, 0));
      load_do(max(ci - 2, 0));
      if (DELTA) __syncthreads();
      __syncthreads();
      products();  // the chain has read this chunk's Al, and reads Gl until the last barrier
      load_mats(max(ci - 2, 0));
      __syncthreads();
    }
    return;
  }

  const int d0 = wave * (DK / 4) + fg * 4;
  const int64_t nh = (int64_t)n * p.heads + h;
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
  Frag<NPQ> fk[KS], ft[DELTA ? MT : 1][2];
  Frag<P> fT[DELTA ? 2 : 1];
  f32x4 beta, ec = {1, 1, 1, 1}, eo = {1, 1, 1, 1}, dec[MT];
  float u[NT][4];
  auto load_k = [&](int ci) {
    const auto k = rows_of<DK, NPQ == 1>(p, p.k, VEC ? p.korow : p.krow, p.ks, VEC, base + ci, h, chunk(ci));
#pragma unroll
    for (int s = 0; s < KS; ++s) fk[s] = k.template frag<NPQ>(wave, s);
    if (!VEC) eo = *reinterpret_cast<const f32x4*>(rows_at(p, base + ci, h) + C + tok);
  };
  auto load_T = [&](int ci) {
#pragma unroll
    for (int s = 0; s < 2; ++s) fT[s] = tile_frag<P, C>(p.t2t + head_of(ci) * P * C * C, wave, s, C * C);
  };
  auto load_u = [&](int ci) {
    const float* rows = rows_at(p, base + ci, h);
    beta = *reinterpret_cast<const f32x4*>(rows + 2 * C + tok);
    if (!VEC) ec = *reinterpret_cast<const f32x4*>(rows + tok);
    if (BETA) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          u[t][r] = p.u[head_of(ci) * C * p.dvp + (uint32_t)((tok + r) * p.dvp + vcol[t])];
    }
  };
  auto load_kt = [&](int ci) {
    const float end = VEC ? 1.0f : rows_at(p, base + ci, h)[C - 1];
    const uint16_t* kt = (VEC ? p.ket : p.kt) + qk_of(ci) * NPQ * DK * C;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (DELTA) {
#pragma unroll
        for (int s = 0; s < 2; ++s) ft[m][s] = tile_frag<NPQ, C>(kt, wave * MT + m, s, DK * C);
      }
      dec[m] = VEC ? *reinterpret_cast<const f32x4*>(p.decay + head_of(ci) * DK + d0 + 16 * m)
                   : f32x4{end, end, end, end};
    }
  };
  if (nch > 0) {
    load_k(nch - 1);
    if (DELTA) load_T(nch - 1);
    load_u(nch - 1);
    load_kt(nch - 1);
  }
  put_state();
  __syncthreads();
  __syncthreads();

  for (int ci = nch - 1; ci >= 0; --ci) {
    const Chunk c = chunk(ci);
    const int64_t sh = head_of(ci);
    const int next = max(ci - 1, 0);
    f32x4 W[NT], W2[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) W[t] = W2[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma(s & 1 ? W2[t] : W[t], fk[s],
            load_frag<P>(&Xl[0][t * 16 + fr][s * 32 + fg * 8], BV * SP));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(&Al[t * 16 + fr][tok]);
#pragma unroll
      for (int r = 0; r < 4; ++r) W[t][r] = fmaf(W[t][r] + W2[t][r], eo[r], a[r]);
    }
    load_k(next);
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
      load_T(next);
    }
    // W holds Z
    float y[NT][4], db[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float ye[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[t][r] = beta[r] * W[t][r];
        ye[r] = -ec[r] * y[t][r];
        if (BETA) db[r] = fmaf(u[t][r], W[t][r], db[r]);
      }
      if (DELTA) put4<P>(&Yt[0][t * 16 + fr][tok], BV * CP, ye);
    }
    load_u(next);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4 g = *reinterpret_cast<const f32x4*>(Gl[wave][m * NT + t][lane]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p.xc[sh * DK * p.dvp + (uint32_t)((d0 + 16 * m + r) * p.dvp + vcol[t])] = X[m][t][r];
          X[m][t][r] = fmaf(X[m][t][r], dec[m][r], g[r]);
        }
        if (DELTA) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
            mma(X[m][t], ft[m][s], load_frag<P>(&Yt[0][t * 16 + fr][s * 32 + fg * 8], BV * CP));
        }
      }
    load_kt(next);
    put_state();
    // stores behind the work that others wait for
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      char* dst = static_cast<char*>(p.dv_out) +
                  (c.row * p.heads + h) * p.dv * (p.dtype == 0 ? 4 : 2);
      uint32_t at[4];
      bool ok[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        at[r] = (uint32_t)(tok + r) * (uint32_t)p.heads * p.dv + vcol[t];
        ok[r] = tok + r < c.len && vcol[t] < p.dv;
        if (DELTA) p.y[sh * C * p.dvp + (uint32_t)((tok + r) * p.dvp + vcol[t])] = y[t][r];
      }
      store_always<4>(dst, at, ok, p.dtype, p.sink, y[t]);
    }
    if (BETA) {
#pragma unroll
      for (int r = 0; r < 4; ++r) db[r] = sum16(db[r]);
      *reinterpret_cast<f32x4*>(p.dbpart + ((int64_t)vb * p.nslots * p.heads + sh) * C + tok) =
          f32x4{db[0], db[1], db[2], db[3]};  // 16 lanes, one value
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
