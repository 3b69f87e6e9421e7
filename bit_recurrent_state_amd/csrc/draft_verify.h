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

// A value row of the stored state as the right operand of products: columns
// 32 s + 8 (lane >> 4) .. of it for s = 0, 1, ...  Codes are fetched ahead.
template <int DK, bool F32>
struct StateRow {
  static constexpr int S = DK / 32;
  const uint8_t* at;  // of the row
  const float* scales;
  uint32_t mask;  // INT8 blocks of 16 columns
  uint32_t raw[F32 ? 1 : S][2];
  float scale[F32 ? 1 : S];  // of the group of each 32 columns (groups of 16: read when used)

  __device__ __forceinline__ void fetch(const Params& p, int n, int h, int row) {
    const int64_t head = (int64_t)n * p.s.H + h;
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (F32) {
      at = static_cast<const uint8_t*>(p.s.state) + (head * p.s.dv + row) * DK * 4;
    } else {
      mask = p.s.int8_blocks[h];
      at = static_cast<const uint8_t*>(p.s.state) + qs::head_code_offset(p.s, n, h) +
           (int64_t)row * 8 * (DK / 16 + __popc(mask));
      scales = p.s.scales + (head * p.s.dv + row) * (DK / p.s.G);
      constexpr uint32_t all = (1u << (DK / 16)) - 1u;
      if (mask == 0) {
#pragma unroll
        for (int s = 0; s < S; ++s)
          raw[s][0] = raw[s][1] = *reinterpret_cast<const uint32_t*>(at + s * 16 + g * 4);
      } else if (mask == all) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(at + s * 32 + g * 8);
          raw[s][0] = w.x;
          raw[s][1] = w.y;
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int blk = 2 * s + (g >> 1);
          const bool is8 = (mask >> blk) & 1u;
          const uint32_t* c = reinterpret_cast<const uint32_t*>(
              at + 8 * (blk + __popc(mask & ((1u << blk) - 1u))) + (g & 1) * (is8 ? 8 : 4));
          raw[s][0] = c[0];
          raw[s][1] = c[is8 ? 1 : 0];
        }
      }
      const int per = p.s.G < 32 ? 32 : p.s.G;
#pragma unroll
      for (int s = 0; s < S; ++s) scale[s] = scales[p.s.G < 32 ? 0 : s * 32 / per];
    }
  }

  __device__ __forceinline__ Frag<F32 ? 3 : 1> frag(int s) const {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (F32) {
      const f32x4* x = reinterpret_cast<const f32x4*>(at) + s * 8 + g * 2;
      const f32x4 a = x[0], b = x[1];
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      return qscan::split8<3>(v);
    } else {
      if (mask == 0) return from_int4(raw[s][0]);
      constexpr uint32_t all = (1u << (DK / 16)) - 1u;
      if (mask == all) return from_int8(raw[s][0], raw[s][1]);
      const bool is8 = (mask >> (2 * s + (g >> 1))) & 1u;
      const Frag<1> a = from_int8(raw[s][0], raw[s][1]), b = from_int4(raw[s][0]);
      Frag<1> f;
#pragma unroll
      for (int i = 0; i < 4; ++i) f.t[0][i] = is8 ? a.t[0][i] : b.t[0][i];
      return f;
    }
  }
};

// (rows of q, k) S^T for one tile of nodes and one of value rows.  kop, qop: planes of
// the nodes' rows in LDS, LP terms a row.
template <int DK, int TERMS, int LP, bool DELTA, bool F32>
__device__ __forceinline__ void state_products(int G, const StateRow<DK, F32>& S,
                                               const uint16_t* kop, const uint16_t* qop, int plane,
                                               f32x4& xk, f32x4& xq) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int at = (lane & 15) * LP + g * 8;
  xk = xq = f32x4{0, 0, 0, 0};
  if constexpr (F32) {
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const Frag<3> b = S.frag(s);
      qscan::mma(xq, qscan::load_frag<TERMS>(qop + at + s * 32, plane), b);
      if (DELTA) qscan::mma(xk, qscan::load_frag<TERMS>(kop + at + s * 32, plane), b);
    }
  } else {
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
        if ((s + 1) * 32 % G == 0) flush(S.scale[s]);
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

// A lane's N neighbouring value columns of row t of o and writes.
template <int N>
__device__ __forceinline__ void store_columns(const Params& p, int n, int h, int t, int col,
                                              const float (&o)[N], const float (&w)[N]) {
  if (t >= p.tokens || col >= p.s.dv) return;
  const int64_t at = (row_of(p, n, t) * p.s.H + h) * p.s.dv + col;
  if (N == 2 && p.pairs) {  // dv is even: both or none
    if (p.o) {
      if (p.dtype == 0) {
        *reinterpret_cast<qscan::f32x2*>(static_cast<float*>(p.o) + at) = qscan::f32x2{o[0], o[N - 1]};
      } else {
        const uint32_t half = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)o[0]) |
                              (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)o[N - 1]) << 16;
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at) =
            p.dtype == 2 ? half : qscan::pack_bf16(o[0], o[N - 1]);
      }
    }
    if (p.writes) *reinterpret_cast<qscan::f32x2*>(p.writes + at) = qscan::f32x2{w[0], w[N - 1]};
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (col + i >= p.s.dv) continue;
    if (p.o) qscan::store_elem(p.o, at + i, p.dtype, o[i]);
    if (p.writes) p.writes[at + i] = w[i];
  }
}

constexpr int kThreads = 256;

template <int DK, int MT, int TERMS, bool VEC, bool DELTA>
struct alignas(16) Lds {
  static constexpr int T = MT * 16;
  static constexpr int LP = DK + 8;            // terms of a row: 16 rows start in different banks
  static constexpr int OT = VEC ? 16 : T;      // rows of operands at a time
  static constexpr int MP = T + 4;
  float A[T][MP], L[DELTA ? T : 1][MP];        // A diag b, -L diag b
  float lt[DELTA ? MT : 1][16][20];            // -L diag b of the tiles on the diagonal, transposed
  float inv[DELTA ? MT : 1][16][20];           // (I + L diag b)^-1 of the same tiles
  float ec[T], beta[T];
  double c[T];
  unsigned long long mask[T];                  // node and ancestors; 0: no node
  int parent[T];
  int rows, pad[3];                            // rows up to the last node
  float alpha[VEC ? T : 1][DK];
  alignas(16) uint16_t kop[TERMS][OT][LP], qop[TERMS][OT][LP];
};

// The inverse of the unit triangular tile `tile`, a column a lane: each row that is
// done is taken off all rows below at once, so that nothing waits but for the row before.
__device__ __forceinline__ void invert(const float (*lt)[16][20], float (*inv)[16][20], int tile) {
  const int col = threadIdx.x & 15;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.0f : 0.0f;
#pragma unroll
  for (int j = 0; j < 15; ++j) {
#pragma unroll
    for (int b = (j + 1) / 4; b < 4; ++b) {
      const f32x4 l = *reinterpret_cast<const f32x4*>(&lt[tile][j][4 * b]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * b + i > j) x[4 * b + i] = fmaf(l[i], x[j], x[4 * b + i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) inv[tile][i][col] = x[i];
}

// A workgroup of four waves takes 64 NTW value columns, a wave NTW tiles of 16.
template <int DK, int MT, int TERMS, bool VEC, bool DELTA, bool F32, int NTW>
__global__ void __launch_bounds__(kThreads) verify_kernel(Params p) {
  using D = Lds<DK, MT, TERMS, VEC, DELTA>;
  constexpr int LP = D::LP, MP = D::MP, plane = D::OT * LP;
  constexpr int IT = D::T * DK / 4 / kThreads;  // a thread's groups of four columns of all rows
  __shared__ D lds;
  const int64_t head = blockIdx.x / p.blocks;
  const int n = (int)(head / p.s.H), h = (int)(head % p.s.H);
  const int hq = h / (p.s.H / p.heads_qk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int T = p.tokens, dv = p.s.dv;
  const int col0 = ((int)(blockIdx.x % p.blocks) * 4 + wave) * (16 * NTW) + NTW * (lane & 15);
  const bool idle = col0 - NTW * (lane & 15) >= dv;  // a wave without columns

  // everything that comes from memory is asked for before anything is waited for
  int parent = -2;
  float gate = 0.0f, beta = 1.0f;
  if (wave == 0) {
    parent = named_parent(p, n, lane);
    const int64_t row = row_of(p, n, min(lane, T - 1)) * p.s.H + h;
    if (!VEC) gate = p.g[row];
    if (p.beta) beta = p.beta[row];
  }
  StateRow<DK, F32> S[NTW];
#pragma unroll
  for (int ct = 0; ct < NTW; ++ct) S[ct].fetch(p, n, h, min(col0 + ct, dv - 1));
  const bool kfour = p.ks % 4 == 0, qfour = p.qs % 4 == 0;
  auto load_q = [&](int t, int e) {
    return qscan::load4(p.q, row_of(p, n, min(t, T - 1)) * p.qs + (int64_t)hq * DK + e, p.dtype, qfour);
  };
  auto load_k = [&](int t, int e) {
    return qscan::load4(p.k, row_of(p, n, min(t, T - 1)) * p.ks + (int64_t)hq * DK + e, p.dtype, kfour);
  };
  const int t0 = threadIdx.x / (DK / 4), e0 = threadIdx.x % (DK / 4) * 4;
  constexpr int TS = kThreads / (DK / 4);  // rows between a thread's groups
  if constexpr (VEC) {
    f32x4 a[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i)
      a[i] = *reinterpret_cast<const f32x4*>(
          p.g + (row_of(p, n, min(t0 + i * TS, T - 1)) * p.s.H + h) * DK + e0);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = qscan::fast_exp(qscan::gate(a[i][j]));
      *reinterpret_cast<f32x4*>(&lds.alpha[t0 + i * TS][e0]) = a[i];
    }
  } else {
    u32x4 w[IT];
    auto stage = [&](uint16_t (*op)[D::OT][LP]) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float x[4];
        qscan::widen4(w[i], p.dtype, x);
        qscan::put4<TERMS>(&op[0][t0 + i * TS][e0], plane, x);
      }
    };
#pragma unroll
    for (int i = 0; i < IT; ++i) w[i] = load_k(t0 + i * TS, e0);
    u32x4 w2[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) w2[i] = load_q(t0 + i * TS, e0);
    stage(lds.kop);
#pragma unroll
    for (int i = 0; i < IT; ++i) w[i] = w2[i];
    stage(lds.qop);
  }

  // the nodes' ways to the stored state, each row's found together with its ancestors': six
  // rounds in which every row takes over what the row it stands at has found
  if (wave == 0) {
    const int t = lane;
    int at = parent;
    bool ok = at > -2;
    unsigned long long mask = 1ull << t;
    double c = !VEC && ok ? (double)qscan::gate(gate) : 0.0;
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
    const unsigned long long nodes = __ballot(ok);
    if (lane == 0) lds.rows = nodes ? 64 - __clzll(nodes) : 0;
    if (t < D::T) {
      lds.mask[t] = ok ? mask : 0;
      lds.parent[t] = ok ? parent : -1;
      lds.c[t] = c;
      lds.ec[t] = VEC ? 1.0f : qscan::fast_exp((float)c);
      lds.beta[t] = ok ? beta : 0.0f;
    }
  }
  if constexpr (VEC) {  // the walks below fill in what is an ancestor
    for (int i = threadIdx.x; i < D::T * MP; i += kThreads) {
      (&lds.A[0][0])[i] = 0.0f;
      if (DELTA) (&lds.L[0][0])[i] = 0.0f;
    }
    if (DELTA)
      for (int i = threadIdx.x; i < MT * 320; i += kThreads) (&lds.lt[0][0][0])[i] = 0.0f;
  }
  __syncthreads();
  const int rows = lds.rows;

  if constexpr (!VEC) {
    // A and L, tile by tile; what is no ancestor is zero, whatever its product is
    constexpr int kinds = DELTA ? 2 : 1;
    for (int i = wave; i < MT * MT * kinds; i += 4) {
      const int it = i / kinds / MT, jt = i / kinds % MT;
      const bool is_l = DELTA && i % kinds == 0;
      if (jt > it || it * 16 >= rows) continue;
      f32x4 a = {0, 0, 0, 0};
      const int at = (lane & 15) * LP + g * 8;
      const uint16_t* left = is_l ? &lds.kop[0][it * 16][0] : &lds.qop[0][it * 16][0];
#pragma unroll
      for (int s = 0; s < DK / 32; ++s)
        qscan::mma(a, qscan::load_frag<TERMS>(left + at + s * 32, plane),
                   qscan::load_frag<TERMS>(&lds.kop[0][jt * 16][0] + at + s * 32, plane));
      const int col = jt * 16 + (lane & 15);
      const double cj = lds.c[col];
      const float bj = lds.beta[col];
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = it * 16 + 4 * g + r;
        const bool on = ((lds.mask[row] >> col) & 1) && !(is_l && row == col);
        const float f = qscan::fast_exp((float)(lds.c[row] - cj)) * (is_l ? -bj : bj);
        x[r] = on ? a[r] * f : 0.0f;
        (is_l ? lds.L : lds.A)[row][col] = x[r];
      }
      if (is_l && it == jt) *reinterpret_cast<f32x4*>(&lds.lt[it][lane & 15][4 * g]) = x;
    }
    if constexpr (DELTA) {
      if (MT > 1) __syncthreads();  // with one tile the first wave has all of L
      if (wave == 0 && g < MT) invert(lds.lt, lds.inv, g);
    }
  }

  f32x4 u[MT][NTW];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt * 16 >= rows) break;
    if constexpr (VEC) {
      // each of 16 nodes goes up its path, 16 lanes a node: q and k take the decays on the way
      const int i = threadIdx.x >> 4, t = mt * 16 + i, sub = threadIdx.x & 15;
      float q[DK / 64][4], k[DK / 64][4];
#pragma unroll
      for (int r = 0; r < DK / 64; ++r) {
        qscan::widen4(load_q(t, 64 * r + 4 * sub), p.dtype, q[r]);
        qscan::widen4(load_k(t, 64 * r + 4 * sub), p.dtype, k[r]);
      }
      if (lds.mask[t] != 0) {
        int at = t;
        float x[DK / 64][4];
#pragma unroll
        for (int r = 0; r < DK / 64; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[r][j] = k[r][j];
        for (;;) {
          const int next = lds.parent[at];
          u32x4 w[DK / 64];  // the parent's key, on its way meanwhile
#pragma unroll
          for (int r = 0; r < DK / 64; ++r) w[r] = load_k(max(next, 0), 64 * r + 4 * sub);
          float a = 0.0f, l = 0.0f;
#pragma unroll
          for (int r = 0; r < DK / 64; ++r) {
            const f32x4 d = *reinterpret_cast<const f32x4*>(&lds.alpha[at][64 * r + 4 * sub]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a = fmaf(q[r][j], x[r][j], a);
              if (DELTA) l = fmaf(k[r][j], x[r][j], l);
              q[r][j] *= d[j];
              if (DELTA) k[r][j] *= d[j];
            }
          }
          a = qscan::sum16(a);
          if (DELTA) l = qscan::sum16(l);
          if (sub == 0) {
            lds.A[t][at] = a * lds.beta[at];
            if (DELTA && at != t) {
              lds.L[t][at] = -l * lds.beta[at];
              if (at >= mt * 16) lds.lt[mt][at - mt * 16][i] = -l * lds.beta[at];
            }
          }
          if (next < 0) break;
          at = next;
#pragma unroll
          for (int r = 0; r < DK / 64; ++r) qscan::widen4(w[r], p.dtype, x[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < DK / 64; ++r) {
        qscan::put4<TERMS>(&lds.qop[0][i][64 * r + 4 * sub], plane, q[r]);
        if (DELTA) qscan::put4<TERMS>(&lds.kop[0][i][64 * r + 4 * sub], plane, k[r]);
      }
      __syncthreads();
      if (DELTA && wave == 0 && g == 0) invert(lds.lt, lds.inv, mt);
    }
    const int base = VEC ? 0 : mt * 16;
    uint32_t raw[4][NTW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = row_of(p, n, min(mt * 16 + 4 * g + r, T - 1)) * p.vs + (int64_t)h * dv;
      int64_t at[NTW];
#pragma unroll
      for (int ct = 0; ct < NTW; ++ct) at[ct] = row + min(col0 + ct, dv - 1);
      qscan::load_raw<NTW>(p.v, at, p.dtype, raw[r]);
    }
    f32x4 xk[NTW], xq[NTW];
    if (!idle) {
#pragma unroll
      for (int ct = 0; ct < NTW; ++ct)
        state_products<DK, TERMS, LP, DELTA, F32>(p.s.G, S[ct], &lds.kop[0][base][0],
                                                  &lds.qop[0][base][0], plane, xk[ct], xq[ct]);
    }
    if (VEC || mt == 0) __syncthreads();  // A, L and the inverse are there, this tile's operands read
    if (idle) continue;
    const f32x4 ec = *reinterpret_cast<const f32x4*>(&lds.ec[mt * 16 + 4 * g]);
    const f32x4 bt = *reinterpret_cast<const f32x4*>(&lds.beta[mt * 16 + 4 * g]);
    bool node[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) node[r] = lds.mask[mt * 16 + 4 * g + r] != 0;
    float out[4][NTW], wr[4][NTW];
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct) {
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = qscan::from_raw(raw[r][ct], p.dtype);
        x[r] = node[r] ? (DELTA ? fmaf(-ec[r], xk[ct][r], v) : v) : 0.0f;
        xq[ct][r] *= ec[r];
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
      for (int jt = 0; jt <= mt; ++jt) small_mma(xq[ct], &lds.A[mt * 16][jt * 16], MP, u[jt][ct]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        out[r][ct] = node[r] ? xq[ct][r] : 0.0f;
        wr[r][ct] = node[r] ? u[mt][ct][r] * bt[r] : 0.0f;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      store_columns<NTW>(p, n, h, mt * 16 + 4 * g + r, col0, out[r], wr[r]);
  }
  // rows behind the last node's tile
  const float zero[NTW] = {};
  for (int t = (rows + 15) / 16 * 16 + g; t < T; t += 4)
    store_columns<NTW>(p, n, h, t, col0, zero, zero);
}

template <int DK, int MT, int TERMS, bool VEC, bool DELTA, int NTW>
hipError_t verify_state(const Params& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.s.B * p.s.H * p.blocks);
  if (p.fp32)
    verify_kernel<DK, MT, TERMS, VEC, DELTA, true, NTW><<<grid, kThreads, 0, s>>>(p);
  else
    verify_kernel<DK, MT, TERMS, VEC, DELTA, false, NTW><<<grid, kThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK, int TERMS, bool VEC, bool DELTA, int NTW>
hipError_t verify_tiles(const Params& p, hipStream_t s) {
  if (p.tokens <= 16) return verify_state<DK, 1, TERMS, VEC, DELTA, NTW>(p, s);
  if (p.tokens <= 32) return verify_state<DK, 2, TERMS, VEC, DELTA, NTW>(p, s);
  if constexpr (most_tokens(DK) > 32) {
    if (p.tokens <= 48) return verify_state<DK, 3, TERMS, VEC, DELTA, NTW>(p, s);
    return verify_state<DK, 4, TERMS, VEC, DELTA, NTW>(p, s);
  }
  return hipErrorInvalidValue;
}

template <int DK, int TERMS, bool VEC, bool DELTA>
hipError_t verify_columns(const Params& p, hipStream_t s) {
  return p.columns == 128 ? verify_tiles<DK, TERMS, VEC, DELTA, 2>(p, s)
                          : verify_tiles<DK, TERMS, VEC, DELTA, 1>(p, s);
}

template <int DK>
hipError_t verify(const Params& p, hipStream_t s) {
  switch (p.mixer) {
    case qscan::GDN: return p.direct ? verify_columns<DK, 1, false, true>(p, s)
                                     : verify_columns<DK, 3, false, true>(p, s);
    case qscan::SCALAR: return p.direct ? verify_columns<DK, 1, false, false>(p, s)
                                        : verify_columns<DK, 3, false, false>(p, s);
    case qscan::GLA: return verify_columns<DK, 3, true, false>(p, s);
    case qscan::KDA: return verify_columns<DK, 3, true, true>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdraft
