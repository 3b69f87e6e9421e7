// scan_prep_vector.h — the forward pass's preparation with a gate per key
// channel, dk up to 128: scaled operands, A, and for the delta rule the chunk
// solved in advance.
//
// With R = V - K~ S^T and U = T R, U = U0 - K^ S^T where U0 = T V and K^ = T K~
// do not wait for the state.  The chain then has one product and one barrier
// less a chunk, at the same bytes: K^ takes the place of K~ = k e^c, U0 that of T.
//
// One workgroup of eight waves per (slot, head).  Waves 0..3 take the rows of q
// (block `wave`) and A, waves 4..7 those of k, L and T: the rows they scale are
// the fragments they multiply.  Only k e^-c goes through LDS.  Chunks that decay
// far leave A and L to their own kernel (scan_prep.h) and are solved here after
// it has run (`solve` alone).

#pragma once

#include "scan_prep.h"

namespace qscan {

// V^T of 16 value columns: 8 tokens of a column, both halves of the chunk.
__device__ __forceinline__ void load_columns(const Params& p, const Chunk& c, int h, int b,
                                             uint32_t (&raw)[2][8]) {
  const int lane = threadIdx.x & 63;
  const int v = min(b * 16 + (lane & 15), p.dv - 1);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    int64_t at[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      at[e] = (c.row + min(s * 32 + (lane >> 4) * 8 + e, c.len - 1)) * p.vs + (int64_t)h * p.dv + v;
    load_raw<8>(p.v, at, p.dtype, raw[s]);
  }
}

// K^ and U0 from T's terms in LDS: a wave takes 16 channels (of K~^T, in its
// registers) and 16 value columns at a time.  Results come with four channels or
// columns of a token in a lane.
template <int DK>
__device__ __forceinline__ void solve(const Params& p, const Chunk& c, int64_t sh, int h,
                                      const uint16_t* T, const Frag<P> (&kt)[2],
                                      uint32_t (&raw)[2][8]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int fr = lane & 15, fg = lane >> 4;
  auto t_frag = [&](int rb, int s) { return tile_frag<P, C>(T, rb, s, C * C); };
  const int vb = p.dvp / 16;
  for (int b = wave; b < vb; b += 8) {
    Frag<P> f[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = s * 32 + fg * 8 + e < c.len && b * 16 + fr < p.dv ? from_raw(raw[s][e], p.dtype) : 0.0f;
      f[s] = split8<P>(x);
    }
    if (b + 8 < vb) load_columns(p, c, h, b + 8, raw);
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= rb / 2) mma(acc, f[s], t_frag(rb, s));
      *reinterpret_cast<f32x4*>(p.u + (sh * C + rb * 16 + fr) * p.dvp + b * 16 + fg * 4) = acc;
    }
  }
  if (wave < DK / 16) {
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= rb / 2) mma(acc, kt[s], t_frag(rb, s));
      const float x[4] = {acc[0], acc[1], acc[2], acc[3]};
      put4<P>(p.krow + sh * P * C * DK + tiled<DK>(rb * 16 + fr, wave * 16 + fg * 4), C * DK, x);
    }
  }
}

// FAR: only chunks that decay far, whose T chunk_vector_kernel has left in p.t;
// otherwise everything, but for those chunks no A, L, T and what follows.
template <int DK, bool DELTA, bool FAR>
__global__ void __launch_bounds__(512, DELTA ? 2 : 4) prep_vector_kernel(Params p) {
  // 80 KB for dk = 128, so that without the delta rule a CU holds two workgroups
  // and one computes while the other waits: 64 us with two, 96 us with one (123
  // chunks of 16 heads, three terms).  With it T's steps need more than 128
  // registers; held to that they spill: KDA's prompt of 128 chunks, 16 heads, 696
  // us against 607 us with one workgroup.
  constexpr int KS = DK / 32;
  constexpr int kKn = P * C * DK, kTM = P * C * C + 2 * C * (C + 4);
  // sums of log decays in blocks of 16: fixed point, floats in chunks that decay far
  __shared__ __align__(16) float buf[C * DK];
  __shared__ __align__(16) uint16_t Kn[kKn > kTM ? kKn : kTM];
  // token t's sums, four channels together, turned by t against bank conflicts
  auto pre = [&](int t, int ch) -> float& { return buf[t * DK + (ch ^ ((t & 7) << 2))]; };
  auto pre_fixed = [&](int t, int ch) -> int& { return reinterpret_cast<int&>(pre(t, ch)); };
  auto tot = [&](int b, int ch) -> float& { return pre(b * 16 + 15, ch); };  // a block's
  auto tot_fixed = [&](int b, int ch) -> int& { return pre_fixed(b * 16 + 15, ch); };
  // T's terms, and M behind them, take the place of k e^-c
  Square* const M = reinterpret_cast<Square*>(Kn + P * C * C);
  const int slot = blockIdx.x, h = blockIdx.y;
  Chunk c;
  if (!(FAR ? noted_chunk(p, slot, c) : find_and_note(p, slot, h == 0, c))) return;
  const int64_t sh = (int64_t)slot * p.heads + h;
  if (FAR && !p.far[sh]) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, rb = wave & 3;
  const int fr = lane & 15, fg = lane >> 4;
  const int hq = h / (p.heads / p.heads_qk);
  // what comes from the caller's arrays is on its way before the first sum
  const bool second = wave >= 4, even = (second ? p.ks : p.qs) % 4 == 0;
  const int t = rb * 16 + fr;
  uint32_t rk[2][8], rv[2][8];
  u32x4 rx[KS][2];
  auto load_keys = [&]() {
    if (wave >= DK / 16) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      int64_t at[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        at[i] = (c.row + min(s * 32 + fg * 8 + i, c.len - 1)) * p.ks + (int64_t)hq * DK + wave * 16 + fr;
      load_raw<8>(p.k, at, p.dtype, rk[s]);
    }
  };
  if (FAR || DELTA) load_keys();
  if (!FAR) {
    const int64_t row = c.row + min(t, c.len - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t at = (int64_t)hq * DK + s * 32 + fg * 8 + 4 * q;
        rx[s][q] = load4(second ? p.k : p.q, row * (second ? p.ks : p.qs) + at, p.dtype, even);
      }
  }
  if (DELTA && wave < p.dvp / 16) load_columns(p, c, h, wave, rv);
  bool over = false;
  auto sums = [&](auto exact) {  // true: fixed point
    for (int u = threadIdx.x; u < DK * 4; u += 512) {
      const int ch = u % DK, t0 = u / DK * 16;
      float g[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        g[i] = p.g[((c.row + min(t0 + i, c.len - 1)) * p.heads + h) * DK + ch];
      std::conditional_t<exact.value, double, float> s = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s += t0 + i < c.len ? gate(g[i]) : 0.0f;
        if constexpr (exact.value)
          pre_fixed(t0 + i, ch) = fixed(s);
        else
          pre(t0 + i, ch) = s;
      }
      over = over || !(s >= -kFarDecay && s <= kFarDecay);
    }
  };
  sums(std::bool_constant<!FAR>());
  if (threadIdx.x < C) {
    const int t = threadIdx.x;
    rows_at(p, slot, h)[2 * C + t] =
        t < c.len ? (p.beta ? p.beta[(c.row + t) * p.heads + h] : 1.0f) : 0.0f;
  }
  __syncthreads();
  if (!FAR && threadIdx.x < DK) {  // no block alone is over, so none has wrapped round
    const int ch = threadIdx.x;
    const int64_t all = (int64_t)tot_fixed(0, ch) + tot_fixed(1, ch) + tot_fixed(2, ch) + tot_fixed(3, ch);
    over = over || all < fixed(-kFarDecay) || all > fixed(kFarDecay);
  }
  bool far = FAR;
  if (!FAR) {
    uint32_t* const flag = reinterpret_cast<uint32_t*>(Kn);
    const uint64_t any = __ballot(over);
    if (lane == 0) flag[wave] = any != 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) far = far || flag[w];
    if (threadIdx.x == 0) p.far[sh] = far;
    __syncthreads();
    if (far) {
      sums(std::false_type());
      __syncthreads();
    }
    if (threadIdx.x < DK) {
      const int ch = threadIdx.x;
      p.decay[sh * DK + ch] =
          far ? fast_exp((tot(0, ch) + tot(1, ch)) + (tot(2, ch) + tot(3, ch)))
              : fixed_exp(tot_fixed(0, ch) + tot_fixed(1, ch) + tot_fixed(2, ch) + tot_fixed(3, ch));
    }
  }

  // columns of k: a wave's 16 channels, both halves of the tokens
  Frag<P> kt[2];
  auto columns = [&]() {
    if (wave >= DK / 16) return;
    const int ch = wave * 16 + fr;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int t0 = s * 32 + fg * 8, b = t0 >> 4;
      // decays from the chunk's start to a token, and from the token to the chunk's end
      float ee[8], eo[8];
      if (far) {
        float before = 0.0f, after = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m < b) before += tot(m, ch);
          if (m > b) after += tot(m, ch);
        }
        // to the end of the token's block: summed from there, the block's sum less the token's
        // would cancel
        float sfx = after;
        for (int i = b * 16 + 15; i > t0 + 7; --i)
          sfx += i < c.len ? gate(p.g[((c.row + i) * p.heads + h) * DK + ch]) : 0.0f;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          ee[i] = fast_exp(pre(t0 + i, ch) + before);
          eo[i] = fast_exp(sfx);
          sfx += t0 + i < c.len ? gate(p.g[((c.row + t0 + i) * p.heads + h) * DK + ch]) : 0.0f;
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
          if (DELTA) ee[i] = fixed_exp(x);
          eo[i] = fixed_exp(end - x);
        }
      }
      float ko[8], ke[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float k = t0 + i < c.len ? from_raw(rk[s][i], p.dtype) : 0.0f;
        ko[i] = k * eo[i];
        if (DELTA) ke[i] = k * ee[i];
      }
      if (DELTA) kt[s] = split8<P>(ke);
      if (!FAR) {
        const Frag<P> f = split8<P>(ko);
#pragma unroll
        for (int n = 0; n < P; ++n)
          *reinterpret_cast<u32x4*>(p.kt + (sh * P + n) * C * DK + (wave * 2 + s) * 512 + lane * 8) = f.t[n];
      }
    }
  };
  if (FAR) {
    if (DELTA) {
      columns();
      const uint16_t* from = p.t + sh * P * C * C;
      for (int u = threadIdx.x; u < P * C * C / 8; u += 512)
        reinterpret_cast<u32x4*>(Kn)[u] = reinterpret_cast<const u32x4*>(from)[u];
      __syncthreads();
      solve<DK>(p, c, sh, h, Kn, kt, rv);
    }
    return;
  }

  // rows: block rb of q (waves 0..3) or k (4..7)
  const float in = t < c.len ? 1.0f : 0.0f;
  Frag<P> own[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int ch = s * 32 + fg * 8;
    float xe[8], xn[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float x[4];
      widen4(rx[s][q], p.dtype, x);
      float ex[4];
      if (far) {
        f32x4 cs = *reinterpret_cast<const f32x4*>(&pre(t, ch + 4 * q));
#pragma unroll
        for (int m = 0; m < 3; ++m)
          if (m < rb) cs += *reinterpret_cast<const f32x4*>(&tot(m, ch + 4 * q));
#pragma unroll
        for (int i = 0; i < 4; ++i) ex[i] = fast_exp(cs[i]);
      } else {
        i32x4 cs = *reinterpret_cast<const i32x4*>(&pre(t, ch + 4 * q));
#pragma unroll
        for (int m = 0; m < 3; ++m)
          if (m < rb) cs += *reinterpret_cast<const i32x4*>(&tot(m, ch + 4 * q));
#pragma unroll
        for (int i = 0; i < 4; ++i) ex[i] = fixed_exp(cs[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = ex[i];
        xe[4 * q + i] = in * x[i] * e;
        if (second) {  // 1 / e, refined once
          const float r = __builtin_amdgcn_rcpf(e);
          xn[4 * q + i] = far ? 0.0f : in * x[i] * fmaf(fmaf(-e, r, 1.0f), r, r);
        }
      }
    }
    own[s] = split8<P>(xe);
    if (second) {
      const Frag<P> f = split8<P>(xn);
#pragma unroll
      for (int n = 0; n < P; ++n)
        *reinterpret_cast<u32x4*>(Kn + n * C * DK + (rb * KS + s) * 512 + lane * 8) = f.t[n];
    } else {
#pragma unroll
      for (int n = 0; n < P; ++n)
        *reinterpret_cast<u32x4*>(p.qrow + (sh * P + n) * C * DK + (rb * KS + s) * 512 + lane * 8) =
            own[s].t[n];
    }
  }
  if (!DELTA) load_keys();
  __syncthreads();  // k e^-c is there
  f32x4 all[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) all[b] = f32x4{0, 0, 0, 0};
  if (!far && (DELTA || !second)) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b <= rb) {
          const Frag<P> f = tile_frag<P, DK>(Kn, b, s, C * DK);
          mma(all[b], f, own[s]);
        }
  }
  if (DELTA) __syncthreads();  // M goes where k e^-c was
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (far) break;
    const f32x4 acc = all[b];
    const int i = rb * 16 + fr, j0 = b * 16 + fg * 4;
    f32x4 bj = {0, 0, 0, 0};
    if (DELTA && second) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        bj[r] = j0 + r < c.len ? p.beta[(c.row + j0 + r) * p.heads + h] : 0.0f;
    }
    float x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = j0 + r;
      x[r] = second ? (i > j ? acc[r] * bj[r] : 0.0f) : (i >= j ? acc[r] : 0.0f);
    }
    if (second) {
      if (DELTA) *reinterpret_cast<f32x4*>(&M[i][j0]) = f32x4{x[0], x[1], x[2], x[3]};
    } else if ((b >> 1) <= (rb >> 1)) {
      put4<P>(p.a + sh * P * C * C + tiled<C>(i, j0), C * C, x);
    }
  }
  columns();
  if (far) return;
  if (DELTA) {
    __syncthreads();
    invert<1>(M, M);
    {  // T's terms over k e^-c, as tiles: 8 columns a thread
      const int tile = threadIdx.x >> 6;
      const f32x4* src = reinterpret_cast<const f32x4*>(&M[tile / 2 * 16 + fr][tile % 2 * 32 + fg * 8]);
      const f32x4 a = src[0], b = src[1];
      const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const Frag<P> f = split8<P>(x);
#pragma unroll
      for (int n = 0; n < P; ++n)
        *reinterpret_cast<u32x4*>(Kn + n * C * C + threadIdx.x * 8) = f.t[n];
    }
    __syncthreads();
    solve<DK>(p, c, sh, h, Kn, kt, rv);
  }
}

}  // namespace qscan
