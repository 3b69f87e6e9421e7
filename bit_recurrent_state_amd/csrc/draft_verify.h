// draft_verify.h — the readout of a tree of drafted tokens over the stored
// state, which it reads once and leaves alone.
//
// With M the nodes' ancestors, c the sums of log decays along the paths and
// G_ij = e^(c_i - c_j) for j in M(i) or j = i, the recurrence along all paths is
//
//   A_ij = q_i k_j G_ij      L_ij = k_i k_j G_ij (j in M(i))
//   U = (I + L diag b)^-1 (V - (K e^c) S^T)      delta rule: GDN, KDA; else U = V
//   O = (Q e^c) S^T + A diag b U,   writes diag b U
//
// the chunk of a scan with a tree in the place of the chain: rows are in an
// order in which parents come first, so L stays strictly lower triangular.
// A workgroup takes one head of one sequence and up to 128 value columns, a wave
// 32 of them (two tiles of 16, lanes holding neighbours in pairs, so that a row
// is read and written 128 bytes at a time).  The nodes are tiles of 16.
//
// Products with the state run on 16 x 16 x 32 bfloat16 matrix instructions, the
// state's codes being whole numbers that bfloat16 holds exactly: one term, whose
// sums are multiplied by the group's scale (per value row, so per lane).  What
// is between nodes alone is small and stays in FP32 (16 x 16 x 4 instructions).

#pragma once

#include "draft_device.h"

namespace qdraft {

// Codes of 8 neighbouring columns as an operand.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

__device__ __forceinline__ Frag<1> from_int8(uint32_t lo, uint32_t hi) {
  Frag<1> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? lo : hi;
    const int at = i % 2 * 16;
    f.t[0][i] = top_halves((float)(int8_t)(w >> at), (float)(int8_t)(w >> (at + 8)));
  }
  return f;
}

__device__ __forceinline__ Frag<1> from_int4(uint32_t w) {
  Frag<1> f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f.t[0][i] = top_halves((float)((int32_t)(w << (28 - 8 * i)) >> 28),
                           (float)((int32_t)(w << (24 - 8 * i)) >> 28));
  return f;
}

// A value row of the stored state as the right operand of a product: columns
// 32 s + 8 (lane >> 4) .. of it.
template <int DK, bool F32>
struct StateRow {
  const uint8_t* codes;  // of the row
  const float* scales;
  uint32_t mask;  // INT8 blocks of 16 columns; quantized only

  __device__ __forceinline__ StateRow(const Params& p, int n, int h, int row) {
    const int64_t head = (int64_t)n * p.s.H + h;
    if (F32) {
      codes = static_cast<const uint8_t*>(p.s.state) + (head * p.s.dv + row) * DK * 4;
    } else {
      mask = p.s.int8_blocks[h];
      codes = static_cast<const uint8_t*>(p.s.state) + qs::head_code_offset(p.s, n, h) +
              (int64_t)row * 8 * (DK / 16 + __popc(mask));
      scales = p.s.scales + (head * p.s.dv + row) * (DK / p.s.G);
    }
  }

  __device__ __forceinline__ Frag<F32 ? 3 : 1> frag(int s) const {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (F32) {
      const f32x4* x = reinterpret_cast<const f32x4*>(codes) + s * 8 + g * 2;
      const f32x4 a = x[0], b = x[1];
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      return qscan::split8<3>(v);
    } else {
      if (mask == 0) return from_int4(*reinterpret_cast<const uint32_t*>(codes + s * 16 + g * 4));
      constexpr uint32_t all = (1u << (DK / 16)) - 1u;
      if (mask == all) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(codes + s * 32 + g * 8);
        return from_int8(w.x, w.y);
      }
      const int blk = 2 * s + (g >> 1);
      const bool is8 = (mask >> blk) & 1u;
      const uint8_t* c = codes + 8 * (blk + __popc(mask & ((1u << blk) - 1u))) +
                         (g & 1) * (is8 ? 8 : 4);
      const uint32_t lo = reinterpret_cast<const uint32_t*>(c)[0];
      const uint32_t hi = reinterpret_cast<const uint32_t*>(c)[is8 ? 1 : 0];
      const Frag<1> a = from_int8(lo, hi), b = from_int4(lo);
      Frag<1> f;
#pragma unroll
      for (int i = 0; i < 4; ++i) f.t[0][i] = is8 ? a.t[0][i] : b.t[0][i];
      return f;
    }
  }
};

// (rows of q, k) S^T for one tile of nodes and one of value rows.  op: planes of
// the nodes' rows in LDS, LP terms a row.
template <int DK, int TERMS, int LP, bool DELTA, bool F32>
__device__ __forceinline__ void state_products(const Params& p, const StateRow<DK, F32>& S,
                                               const uint16_t* kop, const uint16_t* qop, int plane,
                                               f32x4& xk, f32x4& xq) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int at = (lane & 15) * LP + g * 8;
  if constexpr (F32) {
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const Frag<3> b = S.frag(s);
      qscan::mma(xq, qscan::load_frag<TERMS>(qop + at + s * 32, plane), b);
      if (DELTA) qscan::mma(xk, qscan::load_frag<TERMS>(kop + at + s * 32, plane), b);
    }
  } else {
    const int G = p.s.G;
    f32x4 pq = {0, 0, 0, 0}, pk = {0, 0, 0, 0};
    auto flush = [&](float scale) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        xq[r] = fmaf(scale, pq[r], xq[r]);
        if (DELTA) xk[r] = fmaf(scale, pk[r], xk[r]);
      }
      pq = pk = f32x4{0, 0, 0, 0};
    };
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const Frag<1> b = S.frag(s);
      const Frag<TERMS> q = qscan::load_frag<TERMS>(qop + at + s * 32, plane);
      const Frag<TERMS> k = DELTA ? qscan::load_frag<TERMS>(kop + at + s * 32, plane) : q;
      if (G == 16) {  // a group is half of a product's columns: the others as zeros
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          Frag<1> c;
#pragma unroll
          for (int i = 0; i < 4; ++i) c.t[0][i] = (g >> 1) == half ? b.t[0][i] : 0u;
          qscan::mma(pq, q, c);
          if (DELTA) qscan::mma(pk, k, c);
          flush(S.scales[2 * s + half]);
        }
      } else {
        qscan::mma(pq, q, b);
        if (DELTA) qscan::mma(pk, k, b);
        if ((s + 1) * 32 % G == 0) flush(S.scales[s * 32 / G]);
      }
    }
  }
}

// acc += A B over 16 of A's columns; A in LDS, row lane & 15, B as a product left
// it in registers (column lane & 15, rows 4 (lane >> 4) + r): step r takes the
// rows 4 g + r of the four lane groups g.
__device__ __forceinline__ void small_mma(f32x4& acc, const float* a, int stride, const f32x4& b) {
  const int lane = threadIdx.x & 63;
  const f32x4 x = *reinterpret_cast<const f32x4*>(a + (lane & 15) * stride + 4 * (lane >> 4));
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], b[r], acc, 0, 0, 0);
}

template <int DK, int MT, int TERMS, bool VEC, bool DELTA>
struct alignas(16) Lds {
  static constexpr int T = MT * 16;
  static constexpr int LP = DK + 8;            // terms of a row: 16 rows start in different banks
  static constexpr int OT = VEC ? 16 : T;      // rows of operands at a time
  static constexpr int MP = T + 4;
  float A[T][MP], L[DELTA ? T : 1][MP];        // A diag b, -L diag b
  float inv[DELTA ? MT : 1][16][20];           // (I + L diag b)^-1 of the tiles on the diagonal
  float ec[T], beta[T];
  double c[T];
  unsigned long long mask[T];                  // node and ancestors; 0: no node
  int parent[T];
  float k[VEC ? T : 1][DK], alpha[VEC ? T : 1][DK];
  alignas(16) uint16_t kop[TERMS][OT][LP], qop[TERMS][OT][LP];
};

// The inverse of the unit triangular tile `tile`, a column a lane.
template <int MT, class M>
__device__ __forceinline__ void invert(const M& L, float (*inv)[16][20], int tile) {
  const int col = threadIdx.x & 15;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = i == col ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < i; ++j) x[i] = fmaf(L[tile * 16 + i][tile * 16 + j], x[j], x[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) inv[tile][i][col] = x[i];
}

template <int DK, int MT, int TERMS, bool VEC, bool DELTA, bool F32>
__global__ void __launch_bounds__(256) verify_kernel(Params p) {
  using D = Lds<DK, MT, TERMS, VEC, DELTA>;
  constexpr int LP = D::LP, MP = D::MP, plane = D::OT * LP;
  __shared__ D lds;
  const int64_t head = blockIdx.x / p.blocks;
  const int n = (int)(head / p.s.H), h = (int)(head % p.s.H);
  const int hq = h / (p.s.H / p.heads_qk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int T = p.tokens, threads = p.waves * 64;

  // the nodes' ways to the stored state, each row's found together with its ancestors': six
  // rounds in which every row takes over what the row it stands at has found
  if (wave == 0) {
    const int t = lane;
    int at = named_parent(p, n, t);
    const int parent = at;
    bool ok = at > -2;
    unsigned long long mask = 1ull << t;
    double c = 0.0;
    if (!VEC && ok) c = (double)qscan::gate(p.g[row_of(p, n, t) * p.s.H + h]);
    for (int r = 0; r < 6; ++r) {
      const int from = at < 0 ? t : at;
      const double c2 = VEC ? 0.0 : __shfl(c, from);
      const unsigned long long m2 = __shfl(mask, from);
      const int ok2 = __shfl((int)ok, from), at2 = __shfl(at, from);
      if (at >= 0) {
        c += c2;
        mask |= m2;
        ok = ok && ok2;
        at = at2;
      }
    }
    if (t < D::T) {
      lds.mask[t] = ok ? mask : 0;
      lds.parent[t] = ok ? parent : -1;
      lds.c[t] = c;
      lds.ec[t] = VEC ? 1.0f : qscan::fast_exp((float)c);
      lds.beta[t] = !ok ? 0.0f : p.beta ? p.beta[row_of(p, n, t) * p.s.H + h] : 1.0f;
    }
  }
  for (int i = threadIdx.x; i < D::T * MP; i += threads) {
    (&lds.A[0][0])[i] = 0.0f;
    if (DELTA) (&lds.L[0][0])[i] = 0.0f;
  }
  const bool kfour = p.ks % 4 == 0, qfour = p.qs % 4 == 0;
  auto load_q = [&](int t, int e) {
    return qscan::load4(p.q, row_of(p, n, t) * p.qs + (int64_t)hq * DK + e, p.dtype, qfour);
  };
  auto load_k = [&](int t, int e) {
    return qscan::load4(p.k, row_of(p, n, t) * p.ks + (int64_t)hq * DK + e, p.dtype, kfour);
  };
  if constexpr (VEC) {
    for (int i = threadIdx.x; i < D::T * (DK / 4); i += threads) {
      const int t = i / (DK / 4), e = i % (DK / 4) * 4;
      f32x4 x = {0, 0, 0, 0}, a = {1, 1, 1, 1};
      if (t < T) {
        float w[4];
        qscan::widen4(load_k(t, e), p.dtype, w);
        a = *reinterpret_cast<const f32x4*>(p.g + (row_of(p, n, t) * p.s.H + h) * DK + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = w[j];
          a[j] = qscan::fast_exp(qscan::gate(a[j]));
        }
      }
      *reinterpret_cast<f32x4*>(&lds.k[t][e]) = x;
      *reinterpret_cast<f32x4*>(&lds.alpha[t][e]) = a;
    }
    __syncthreads();
  } else {
    for (int i = threadIdx.x; i < D::T * (DK / 4); i += threads) {
      const int t = min(i / (DK / 4), T - 1), e = i % (DK / 4) * 4;
      float w[4];
      qscan::widen4(load_k(t, e), p.dtype, w);
      qscan::put4<TERMS>(&lds.kop[0][i / (DK / 4)][e], plane, w);
      qscan::widen4(load_q(t, e), p.dtype, w);
      qscan::put4<TERMS>(&lds.qop[0][i / (DK / 4)][e], plane, w);
    }
    __syncthreads();
    // A and L, tile by tile; what is no ancestor stays zero, whatever its product is
    for (int i = wave; i < MT * MT; i += p.waves) {
      const int it = i / MT, jt = i % MT;
      if (jt > it || it * 16 >= T) continue;
      f32x4 a = {0, 0, 0, 0}, l = {0, 0, 0, 0};
      const int at = (lane & 15) * LP + g * 8;
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const Frag<TERMS> b = qscan::load_frag<TERMS>(&lds.kop[0][jt * 16][0] + at + s * 32, plane);
        qscan::mma(a, qscan::load_frag<TERMS>(&lds.qop[0][it * 16][0] + at + s * 32, plane), b);
        if (DELTA)
          qscan::mma(l, qscan::load_frag<TERMS>(&lds.kop[0][it * 16][0] + at + s * 32, plane), b);
      }
      const int col = jt * 16 + (lane & 15);
      const double cj = lds.c[col];
      const float bj = lds.beta[col];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = it * 16 + 4 * g + r;
        const bool on = (lds.mask[row] >> col) & 1;
        const float f = qscan::fast_exp((float)(lds.c[row] - cj)) * bj;
        lds.A[row][col] = on ? a[r] * f : 0.0f;
        if (DELTA) lds.L[row][col] = on && row != col ? -l[r] * f : 0.0f;
      }
    }
    if constexpr (DELTA) {
      __syncthreads();
      if (wave == 0 && g < MT) invert<MT>(lds.L, lds.inv, g);
    }
    __syncthreads();
  }

  const int dv = p.s.dv;
  const int col0 = (int)(blockIdx.x % p.blocks) * threads / 2 + wave * 32 + 2 * (lane & 15);
  f32x4 u[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt * 16 >= T) break;
    if constexpr (VEC) {
      // each of 16 nodes goes up its path, 16 lanes a node: q and k take the decays on the way
      for (int i = threadIdx.x >> 4; i < 16; i += threads / 16) {
        const int t = mt * 16 + i, sub = threadIdx.x & 15;
        float q[DK / 64][4], k[DK / 64][4];
#pragma unroll
        for (int r = 0; r < DK / 64; ++r) {
          const int e = 64 * r + 4 * sub;
          qscan::widen4(load_q(min(t, T - 1), e), p.dtype, q[r]);
#pragma unroll
          for (int j = 0; j < 4; ++j) k[r][j] = lds.k[t][e + j];
        }
        if (lds.mask[t] != 0) {
          int at = t;
          do {
            float a = 0.0f, l = 0.0f;
#pragma unroll
            for (int r = 0; r < DK / 64; ++r) {
              const f32x4 x = *reinterpret_cast<const f32x4*>(&lds.k[at][64 * r + 4 * sub]);
              const f32x4 d = *reinterpret_cast<const f32x4*>(&lds.alpha[at][64 * r + 4 * sub]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                a = fmaf(q[r][j], x[j], a);
                if (DELTA) l = fmaf(k[r][j], x[j], l);
                q[r][j] *= d[j];
                if (DELTA) k[r][j] *= d[j];
              }
            }
            a = qscan::sum16(a);
            if (DELTA) l = qscan::sum16(l);
            if (sub == 0) {
              lds.A[t][at] = a * lds.beta[at];
              if (DELTA && at != t) lds.L[t][at] = -l * lds.beta[at];
            }
            at = lds.parent[at];
          } while (at >= 0);
        }
#pragma unroll
        for (int r = 0; r < DK / 64; ++r) {
          qscan::put4<TERMS>(&lds.qop[0][i][64 * r + 4 * sub], plane, q[r]);
          if (DELTA) qscan::put4<TERMS>(&lds.kop[0][i][64 * r + 4 * sub], plane, k[r]);
        }
      }
      __syncthreads();
      if constexpr (DELTA) {
        if (wave == 0 && g == 0) invert<MT>(lds.L, lds.inv, mt);
        __syncthreads();
      }
    }
    const int base = VEC ? 0 : mt * 16;
    const f32x4 ec = *reinterpret_cast<const f32x4*>(&lds.ec[mt * 16 + 4 * g]);
    const f32x4 beta = *reinterpret_cast<const f32x4*>(&lds.beta[mt * 16 + 4 * g]);
    uint32_t raw[4][2];
    bool node[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = mt * 16 + 4 * g + r;
      node[r] = lds.mask[t] != 0;
      const int64_t row = row_of(p, n, min(t, T - 1)) * p.vs + (int64_t)h * dv;
      const int64_t at[2] = {row + min(col0, dv - 1), row + min(col0 + 1, dv - 1)};
      qscan::load_raw<2>(p.v, at, p.dtype, raw[r]);
    }
    float out[2][4], wr[2][4];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const StateRow<DK, F32> S(p, n, h, min(col0 + ct, dv - 1));
      f32x4 xk = {0, 0, 0, 0}, xq = {0, 0, 0, 0};
      state_products<DK, TERMS, LP, DELTA, F32>(p, S, &lds.kop[0][base][0], &lds.qop[0][base][0],
                                                plane, xk, xq);
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = qscan::from_raw(raw[r][ct], p.dtype);
        x[r] = node[r] ? (DELTA ? fmaf(-ec[r], xk[r], v) : v) : 0.0f;
        xq[r] *= ec[r];
      }
      if constexpr (DELTA) {
#pragma unroll
        for (int jt = 0; jt < mt; ++jt)
          small_mma(x, &lds.L[mt * 16][jt * 16], MP, u[jt][ct]);
        u[mt][ct] = f32x4{0, 0, 0, 0};
        small_mma(u[mt][ct], &lds.inv[mt][0][0], 20, x);
      } else {
        u[mt][ct] = x;
      }
#pragma unroll
      for (int jt = 0; jt <= mt; ++jt) small_mma(xq, &lds.A[mt * 16][jt * 16], MP, u[jt][ct]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        out[ct][r] = node[r] ? xq[r] : 0.0f;
        wr[ct][r] = node[r] ? u[mt][ct][r] * beta[r] : 0.0f;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = mt * 16 + 4 * g + r;
      if (t >= T) continue;
      const int64_t at = (row_of(p, n, t) * p.s.H + h) * dv + col0;
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        if (col0 + ct >= dv) continue;
        if (p.o) qscan::store_elem(p.o, at + ct, p.dtype, out[ct][r]);
        if (p.writes) p.writes[at + ct] = wr[ct][r];
      }
    }
    if (VEC && MT > 1) __syncthreads();  // the next tile's operands
  }
}

template <int DK, int MT, int TERMS, bool VEC, bool DELTA>
hipError_t verify_state(const Params& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.s.B * p.s.H * p.blocks);
  if (p.fp32)
    verify_kernel<DK, MT, TERMS, VEC, DELTA, true><<<grid, p.waves * 64, 0, s>>>(p);
  else
    verify_kernel<DK, MT, TERMS, VEC, DELTA, false><<<grid, p.waves * 64, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK, int TERMS, bool VEC, bool DELTA>
hipError_t verify_tiles(const Params& p, hipStream_t s) {
  if (p.tokens <= 16) return verify_state<DK, 1, TERMS, VEC, DELTA>(p, s);
  if (p.tokens <= 32) return verify_state<DK, 2, TERMS, VEC, DELTA>(p, s);
  if constexpr (most_tokens(DK) > 32) return verify_state<DK, 4, TERMS, VEC, DELTA>(p, s);
  return hipErrorInvalidValue;
}

template <int DK>
hipError_t verify(const Params& p, hipStream_t s) {
  switch (p.mixer) {
    case qscan::GDN: return p.direct ? verify_tiles<DK, 1, false, true>(p, s)
                                     : verify_tiles<DK, 3, false, true>(p, s);
    case qscan::SCALAR: return p.direct ? verify_tiles<DK, 1, false, false>(p, s)
                                        : verify_tiles<DK, 3, false, false>(p, s);
    case qscan::GLA: return verify_tiles<DK, 3, true, false>(p, s);
    case qscan::KDA: return verify_tiles<DK, 3, true, true>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdraft
