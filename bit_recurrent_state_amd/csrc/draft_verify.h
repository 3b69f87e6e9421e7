// draft_verify.h — the readout of a tree of drafted tokens over the stored
// state, which it reads once (FP32 states: for every 16 nodes) and leaves alone.
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
// A workgroup takes one head of one sequence and 64 or 128 value columns, each of
// its four waves one or two tiles of 16 (two: lanes hold neighbours in pairs, so
// that a row is read and written in longer pieces).  The nodes are tiles of 16, up
// to the last node of the sequence.
//
// Products with the state run on 16 x 16 x 32 bfloat16 matrix instructions, the
// state's codes being whole numbers that bfloat16 holds exactly: one term, whose
// sums are multiplied by the group's scale (per value row, so per lane).  FP32
// states and rows enter as three terms.  What is between nodes alone is small and
// stays in FP32 (16 x 16 x 4 instructions); U goes from one product to the next
// in the registers that it came out in.
//
// One gate a token: A and L come from products of the rows, decays as
// differences of 64-bit sums.  A gate per channel: each node goes up its path and
// multiplies the decays into its q and k on the way, exact at any decay.
//
// A product over nodes keeps a NaN where its other factor is a zero, the mark of no ancestor.  So each
// tile of U is looked through, and of the inverse; if something is not finite, zeros take its place in
// the products, and what hangs on it is made NaN along the paths: a broken branch changes no bit of
// another (1 to 3 %).
//
// Bound by latency, then by memory: what a workgroup reads is asked for before
// anything is waited for, codes, scales and bfloat16 rows by copies to LDS that
// take no registers, so that four workgroups share a CU.  256 sequences with 16 nodes,
// 32 heads of 128 x 128, GDN, INT4 (a quarter INT8), bfloat16: 75 us, 300 MB at
// 4.0 TB/s (192 us with loads where they are used, 106 with the codes gathered
// into registers).  64 sequences of up to 33 nodes, 16 heads, KDA, INT8: 58 us for
// 53 MB; its workgroups take 80 KB of LDS and 11 of their 30 thousand cycles
// for the walks.  32 sequences of 64 nodes, SCALAR, 32 heads of 64 x 128, INT4: 24 us
// for 40 MB.  The first batch with float16 rows (three terms) takes 110 us, with FP32 rows 125, over
// states with widths per channel, whose codes lanes gather for themselves, 100.

#pragma once

#include "draft_device.h"

namespace qdraft {

// The upper halves of two floats: two bfloat16 numbers where the lower halves are zeros.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Codes of 8 neighbouring columns as an operand.
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

typedef const __attribute__((address_space(1))) void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;

// 16 (4) bytes a lane from memory to LDS, lane after lane from `to` on, without registers in between;
// there once vmcnt says so.  All lanes take part: an unused one repeats what another loads.
__device__ __forceinline__ void copy16(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 4, 0, 0);
}
__device__ __forceinline__ void copies_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// How a wave's 16 N value rows of BITS-bit codes lie in LDS.  A copy takes 1 KB of neighbouring rows,
// so that memory is read in whole lines; which lane takes which 16 bytes of it is chosen so that what
// the lanes of an operand read at a time (one 16-byte chunk of every N-th row) lies in different banks.
// (Each lane loading its own 4 or 8 bytes instead touched 16 lines a load; the address unit's time for
// that was a third of the kernel's.)  Row N c + t, chunk j is in copy c / CC, at lane
// 16 (o / COPIES) + CC ((c / CC + o) % COPIES) + c % CC with o = N j + t.
template <int DK, int BITS, int N>
struct CodeTile {
  static constexpr int ROW = DK * BITS / 8;
  static constexpr int PER = 1024 / ROW < 16 * N ? 1024 / ROW : 16 * N;  // rows of a copy
  static constexpr int CC = PER / N, COPIES = 16 / CC, ORDERS = ROW / 16 * N;

  static __device__ __forceinline__ void copy(const uint8_t* head, int row0, int dv, uint8_t* to) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int o = (COPIES * (lane >> 4) + (((lane & 15) / CC - i) & (COPIES - 1))) & (ORDERS - 1);
      const int row = min(row0 + N * (i * CC + (lane & 15) % CC) + o % N, dv - 1);
      copy16(head + (uint32_t)(row * ROW + o / N * 16), to + i * 1024);
    }
  }

  // where chunk j of row N c + t begins
  static __device__ __forceinline__ int at(int c, int t, int j) {
    const int i = c / CC, o = N * j + t;
    return i * 1024 + (16 * (o / COPIES) + CC * ((i + o) & (COPIES - 1)) + c % CC) * 16;
  }
};

// The wave's value rows of the stored state, N tiles of 16, as right operands of products.
template <int DK, bool F32, int N>
struct StateRows {
  static constexpr int S = DK / 32;
  static constexpr int CODES = F32 ? 16 : 16 * N * DK < 1024 ? 1024 : 16 * N * DK;  // bytes of LDS
  static constexpr int SCALES = F32 ? 4 : 16 * N * S < 64 ? 64 : 16 * N * S;        // floats of LDS
  const uint8_t* head;  // FP32 states, codes
  const float* scales;  // of the head
  uint32_t mask;        // INT8 blocks of 16 columns
  int row0, dv, G, groups;
  bool apart;           // heads of mixed widths: lanes load for themselves
  const uint8_t* codes;
  const float* near;    // scales in LDS

  // asks for all of it
  __device__ __forceinline__ void fetch(const Params& p, int n, int h, int row0_, uint8_t* to,
                                        float* scales_to) {
    const int64_t at = (int64_t)n * p.s.H + h;
    row0 = row0_;
    dv = p.s.dv;
    if constexpr (F32) {
      head = static_cast<const uint8_t*>(p.s.state) + at * dv * DK * 4;
    } else {
      // a scalar load, so that branches on it are the wave's: there are none of 16 bits
      mask = reinterpret_cast<const uint32_t*>(p.s.int8_blocks)[h >> 1] >> (h & 1) * 16 & 0xFFFFu;
      head = static_cast<const uint8_t*>(p.s.state) + qs::head_code_offset(p.s, n, h);
      G = p.s.G;
      groups = DK >> (31 - __clz(G));
      scales = p.s.scales + at * dv * groups;
      apart = p.s.mixed;
      codes = to;
      near = scales_to;
      if (!apart) {
        if (mask == 0)
          CodeTile<DK, 4, N>::copy(head, row0, dv, to);
        else
          CodeTile<DK, 8, N>::copy(head, row0, dv, to);
      }
      if (G >= 32) {
        const int lane = threadIdx.x & 63, last = dv * groups - 1;
        for (int i = 0; i < 16 * N * groups; i += 64)
          copy4(scales + min(row0 * groups + i + lane, last), scales_to + i);
      }
    }
  }

  __device__ __forceinline__ int row(int t) const { return min(row0 + N * ((int)threadIdx.x & 15) + t, dv - 1); }

  // FP32: columns 32 s .. of tile t as an operand.  Loaded and split again for every tile of nodes: three
  // terms of all columns would take 3 DK / 8 registers more a tile of value rows (64 sequences, 32 heads of
  // 128 x 128: 34 us with 16 nodes, 139 with 64)
  __device__ __forceinline__ Frag<3> values(int t, int s) const {
    const f32x4* x = reinterpret_cast<const f32x4*>(head + (int64_t)row(t) * DK * 4) + s * 8 +
                     ((threadIdx.x & 63) >> 4) * 2;
    const f32x4 a = x[0], b = x[1];
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return qscan::split8<3>(v);
  }

  // The codes of tile t as operands.
  __device__ __forceinline__ void operands(int t, Frag<1> (&f)[S]) const {
    const int c = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if (apart) {
      const uint8_t* const from = head + (uint32_t)(row(t) * 8 * (DK / 16 + __popc(mask)));
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int blk = 2 * s + (g >> 1);
        const bool is8 = (mask >> blk) & 1u;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(
            from + 8 * (blk + __popc(mask & ((1u << blk) - 1u))) + (g & 1) * (is8 ? 8 : 4));
        const uint32_t lo = w[0], hi = w[is8 ? 1 : 0];
        const Frag<1> a = from_int8(lo, hi), b = from_int4(lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[s].t[0][i] = is8 ? a.t[0][i] : b.t[0][i];
      }
    } else if (mask == 0) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        f[s] = from_int4(*reinterpret_cast<const uint32_t*>(codes + CodeTile<DK, 4, N>::at(c, t, s) + g * 4));
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(
            codes + CodeTile<DK, 8, N>::at(c, t, 2 * s + (g >> 1)) + (g & 1) * 8);
        f[s] = from_int8(w.x, w.y);
      }
    }
  }

  // The scale of columns 32 s .. of the lane's row of tile t (groups of 16: of their half).
  __device__ __forceinline__ float scale(int t, int s, int half) const {
    if (G < 32) return scales[row(t) * groups + 2 * s + half];
    return near[(N * ((int)threadIdx.x & 15) + t) * groups + (s * 32 >> (31 - __clz(G)))];
  }
};

// Rows of q and k as left operands.  One term: rows of DK values, whose 16-byte chunks are exchanged
// within the row by its number, so that 16 rows' are in different banks; else planes of rows with 8
// terms of padding.
template <int DK, int TERMS>
struct Operands {
  static constexpr int LP = TERMS == 1 ? DK : DK + 8;
  static constexpr int CH = DK / 8;  // chunks of a row
  static __device__ __forceinline__ int exchanged(int row, int chunk) {
    return chunk ^ (CH >= 16 ? row & 15 : (row >> 1) & 7);
  }
  static __device__ __forceinline__ Frag<TERMS> frag(const uint16_t* op, int row, int s, int plane) {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (TERMS == 1)
      return qscan::load_frag<1>(op + row * DK + exchanged(row, 4 * s + g) * 8, 0);
    else
      return qscan::load_frag<TERMS>(op + row * LP + s * 32 + g * 8, plane);
  }
};

// (rows of q, k) S^T for nodes row0 .. + 15 of the operands and tile t of value rows.
template <int DK, int TERMS, bool DELTA, bool F32, int N>
__device__ __forceinline__ void state_products(const StateRows<DK, F32, N>& S, int t,
                                               const Frag<1> (&b)[DK / 32], const uint16_t* kop, const uint16_t* qop, int row0,
                                               int plane, f32x4& xk, f32x4& xq) {
  using Op = Operands<DK, TERMS>;
  const int g = (threadIdx.x & 63) >> 4, row = row0 + (threadIdx.x & 15);
  xk = xq = f32x4{0, 0, 0, 0};
  if constexpr (F32) {
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const Frag<3> b = S.values(t, s);
      qscan::mma(xq, Op::frag(qop, row, s, plane), b);
      if (DELTA) qscan::mma(xk, Op::frag(kop, row, s, plane), b);
    }
  } else {
    // a product's sums are multiplied by the scale of its columns
    auto scaled = [&](f32x4& acc, const Frag<TERMS>& a, const Frag<1>& b, float scale) {
      f32x4 part = {0, 0, 0, 0};
      qscan::mma(part, a, b);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale, part[r], acc[r]);
    };
    if (S.G >= 32) {
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const float f = S.scale(t, s, 0);
        scaled(xq, Op::frag(qop, row, s, plane), b[s], f);
        if (DELTA) scaled(xk, Op::frag(kop, row, s, plane), b[s], f);
      }
    } else {  // a group is half of a product's columns: the others as zeros
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const Frag<TERMS> q = Op::frag(qop, row, s, plane);
        const Frag<TERMS> k = DELTA ? Op::frag(kop, row, s, plane) : q;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          Frag<1> c;
#pragma unroll
          for (int i = 0; i < 4; ++i) c.t[0][i] = (g >> 1) == half ? b[s].t[0][i] : 0u;
          scaled(xq, q, c, S.scale(t, s, half));
          if (DELTA) scaled(xk, k, c, S.scale(t, s, half));
        }
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

// Products with zeros keep a NaN, so what is not finite would spoil nodes that do not hang on it.
__device__ __forceinline__ bool broken(float x) { return __builtin_amdgcn_classf(x, 0x207); }

// Zeros in the place of a tile's values that are not finite; their rows, in the lane's column.
__device__ __forceinline__ uint32_t take_out(f32x4& x) {
  uint32_t rows = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    rows |= (uint32_t)broken(x[r]) << r;
    x[r] = broken(x[r]) ? 0.0f : x[r];
  }
  rows <<= (threadIdx.x & 63) >> 4 << 2;
  rows |= __shfl_xor(rows, 16);
  return rows | __shfl_xor(rows, 32);
}

// Rows of a sequence, from a base address that is the same for the workgroup.
struct Rows {
  const char* base;
  uint32_t stride;  // in 32 bits without a sign: an access is the base and an offset register
  int dtype;
  __device__ __forceinline__ Rows(const void* p, int64_t at, int stride_, int dtype_)
      : base(static_cast<const char*>(p) + at * (dtype_ == 0 ? 4 : 2)), stride((uint32_t)stride_), dtype(dtype_) {}

  template <class W>
  __device__ __forceinline__ W word(uint32_t byte) const {
    return *reinterpret_cast<const W*>(base + byte);
  }

  // 16-bit values: where column e of row t is
  __device__ __forceinline__ const void* at(uint32_t t, uint32_t e) const {
    return base + (t * stride + e) * 2;
  }

  // columns e .. e + 3 as they lie in memory
  __device__ __forceinline__ u32x4 four(uint32_t t, uint32_t e, bool even) const {
    const uint32_t at = t * stride + e;
    if (!even) return qscan::load4(base, at, dtype, false);
    if (dtype == 0) return word<u32x4>(at * 4);
    const u32x2 w = word<u32x2>(at * 2);
    return u32x4{w.x, w.y, 0, 0};
  }

  // columns col .. col + N - 1; behind the last, the last again.  pairs: two are one access.
  // WORDS < N: two 16-bit values in a word
  template <int N, int WORDS>
  __device__ __forceinline__ void columns(uint32_t t, int col, int width, bool pairs,
                                          uint32_t (&raw)[WORDS]) const {
    if (N == 2 && pairs && dtype != 0) {
      const uint32_t w = word<uint32_t>((t * stride + min(col, width - 2)) * 2);
      raw[0] = WORDS < N ? w : w & 0xFFFFu;
      if (WORDS == N) raw[WORDS - 1] = w >> 16;
      return;
    }
    uint32_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t at = t * stride + min(col + i, width - 1);
      x[i] = dtype == 0 ? word<uint32_t>(at * 4) : word<uint16_t>(at * 2);
    }
    raw[0] = x[0];
    if (N > 1) raw[WORDS - 1] = WORDS < N ? x[0] | x[N - 1] << 16 : x[N - 1];
  }
};

// Where a lane's N neighbouring value columns of o and writes go.
template <int N>
struct Columns {
  char* o;
  float* writes;
  uint32_t row;
  int col, dv, dtype;
  bool pairs;
  __device__ __forceinline__ Columns(const Params& p, int n, int h, int col_, int dtype_)
      : row((uint32_t)(p.s.H * p.s.dv)), col(col_), dv(p.s.dv), dtype(dtype_), pairs(p.pairs) {
    const int64_t base = row_of(p, n, 0) * row + (int64_t)h * dv;
    o = p.o ? static_cast<char*>(p.o) + base * (dtype == 0 ? 4 : 2) : nullptr;
    writes = p.writes ? p.writes + base : nullptr;
  }

  __device__ __forceinline__ void store(uint32_t t, const float (&x)[N], const float (&w)[N]) const {
    if (col >= dv) return;
    const uint32_t at = t * row + col;
    if (N == 2 && pairs) {  // dv is even: both or none
      if (o) {
        if (dtype == 0) {
          *reinterpret_cast<qscan::f32x2*>(o + at * 4) = qscan::f32x2{x[0], x[N - 1]};
        } else {
          const uint32_t half = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[0]) |
                                (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[N - 1]) << 16;
          *reinterpret_cast<uint32_t*>(o + at * 2) =
              dtype == 2 ? half : qscan::pack_bf16(x[0], x[N - 1]);
        }
      }
      if (writes)
        *reinterpret_cast<qscan::f32x2*>(reinterpret_cast<char*>(writes) + at * 4) =
            qscan::f32x2{w[0], w[N - 1]};
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (col + i >= dv) continue;
      if (o) qscan::store_elem(o, at + i, dtype, x[i]);
      if (writes) writes[at + i] = w[i];
    }
  }
};

constexpr int kThreads = 256;

template <int DK, int MT, int TERMS, bool VEC, bool DELTA, bool F32, int NTW>
struct alignas(16) Lds {
  using State = StateRows<DK, F32, NTW>;
  static constexpr int T = MT * 16;
  static constexpr int LP = Operands<DK, TERMS>::LP;
  // with a gate per channel a tile of nodes is worked out at a time
  static constexpr int OT = VEC ? 16 : T, OM = VEC ? 1 : MT;
  static constexpr int MP = T + 4;
  // (without the delta rule and with a gate per channel no product takes k)
  uint16_t kop[VEC && !DELTA ? 1 : TERMS][VEC && !DELTA ? 1 : OT][LP], qop[TERMS][OT][LP];
  uint8_t codes[4][State::CODES];              // of each wave
  float scales[4][State::SCALES];
  float A[OT][MP], L[DELTA ? OT : 1][MP];      // A diag b, -L diag b
  float lt[DELTA ? OM : 1][16][20];            // -L diag b of the tiles on the diagonal, transposed
  float inv[DELTA ? OM : 1][16][20];           // (I + L diag b)^-1 of the same tiles
  float ec[T], beta[T];
  float alpha[VEC ? T : 1][DK];
  double c[T];
  unsigned long long mask[T];                  // node and ancestors; 0: no node
  unsigned long long nodes;                    // which rows are nodes
  unsigned long long gone[4][NTW][16];         // of a wave's columns: the nodes whose U is not finite
  int parent[T];
};

// The inverse of the unit triangular tile `tile`, a column a lane: each row that is
// done is taken off all rows below at once, so that nothing waits but for the row before.
// Finite factors may still have a product beyond the range, which a zero, the mark of no ancestor, would
// hand to rows beside the branch: such a column is done again without the products of zeros, and its
// infinite rows, zeros in the inverse, are spoilt by their e^c (of the tile's rows).
__device__ __forceinline__ void invert(const float (*lt)[16][20], float (*inv)[16][20], int tile, float* ec) {
  const int col = threadIdx.x & 15;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.0f : 0.0f;
  int from = tile * 80;  // 16-byte words in front of the tile's
#pragma unroll
  for (int j = 0; j < 15; ++j) {
    // three rows' loads wait for row j: all rows at once would take every register there is
    if (j % 3 == 0) asm volatile("" : "+v"(from), "+v"(x[j]));
#pragma unroll
    for (int b = (j + 1) / 4; b < 4; ++b) {
      const f32x4 f = reinterpret_cast<const f32x4*>(lt)[from + j * 5 + b];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * b + i > j) x[4 * b + i] = fmaf(f[i], x[j], x[4 * b + i]);
    }
  }
  float none = 0.0f;  // NaN once something is not finite
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    inv[tile][i][col] = x[i];
    none = fmaf(x[i], 0.0f, none);
  }
  if (none == 0.0f) return;
  // (rolled: unrolled, what hardly ever runs cost every call of KDA 9 %)
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    float y = i == col ? 1.0f : 0.0f;
#pragma unroll 1
    for (int j = 0; j < i; ++j) {
      const float f = lt[tile][j][i];
      if (f != 0.0f) y = fmaf(f, inv[tile][j][col], y);
    }
    if (broken(y)) ec[i] = NAN;
    inv[tile][i][col] = broken(y) ? 0.0f : y;
  }
}

// Workgroups of a CU that the registers have to leave room for: with a gate per channel two where the
// LDS holds two (64 sequences of up to 33 nodes, KDA: 58 us; 84 with one workgroup, six registers more).
template <int DK, int MT, int TERMS, bool VEC, bool DELTA, bool F32, int NTW>
constexpr int kResident = TERMS == 1 && MT == 1 && DK <= 128 ? 4
                          : VEC && sizeof(Lds<DK, MT, TERMS, VEC, DELTA, F32, NTW>) <= 80 << 10 ? 2 : 1;

// A workgroup of four waves takes 64 NTW value columns, a wave NTW tiles of 16.
template <int DK, int MT, int TERMS, bool VEC, bool DELTA, bool F32, int NTW>
__global__ void __launch_bounds__(kThreads, (kResident<DK, MT, TERMS, VEC, DELTA, F32, NTW>))
verify_kernel(Params p) {
  using D = Lds<DK, MT, TERMS, VEC, DELTA, F32, NTW>;
  using Op = Operands<DK, TERMS>;
  constexpr int LP = D::LP, MP = D::MP, plane = D::OT * LP;
  __shared__ D lds;
  // TERMS = 1: bfloat16 throughout
  const int dtype = TERMS == 1 ? 1 : p.dtype;
  const uint32_t head = blockIdx.x / (uint32_t)p.blocks;
  const int n = (int)(head / (uint32_t)p.s.H), h = (int)(head - n * (uint32_t)p.s.H);
  const int hq = (int)((uint32_t)h * (uint32_t)p.heads_qk / (uint32_t)p.s.H);
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = p.tokens, dv = p.s.dv;
  const int first = ((int)(blockIdx.x - head * p.blocks) * 4 + wave) * (16 * NTW);
  const int col0 = first + NTW * (lane & 15);
  const bool idle = first >= dv;  // a wave without columns

  // everything that comes from memory is asked for before anything is waited for
  int parent = -2;
  float gate = 0.0f, beta = 1.0f;
  if (wave == 0) {
    parent = named_parent(p, n, lane);
    const int64_t base = row_of(p, n, 0) * p.s.H + h;
    const int row = min(lane, T - 1) * p.s.H;
    if (!VEC) gate = (p.g + base)[row];
    if (p.beta) beta = (p.beta + base)[row];
  }
  const bool kfour = p.ks % 4 == 0, qfour = p.qs % 4 == 0;
  // what is the same for a workgroup goes into base addresses; 64 rows lie within 32 bits of them
  const Rows qrows(p.q, row_of(p, n, 0) * p.qs + (int64_t)hq * DK, (int)p.qs, dtype);
  const Rows krows(p.k, row_of(p, n, 0) * p.ks + (int64_t)hq * DK, (int)p.ks, dtype);
  const Rows vrows(p.v, row_of(p, n, 0) * p.vs + (int64_t)h * dv, (int)p.vs, dtype);
  auto load_q = [&](int t, int e) { return qrows.four(min(t, T - 1), e, qfour); };
  auto load_k = [&](int t, int e) { return krows.four(min(t, T - 1), e, kfour); };
  constexpr int VW = TERMS == 1 ? 1 : NTW;
  uint32_t raw[4][VW];  // of a tile's v
  auto load_v = [&](int mt) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      vrows.columns<NTW, VW>(min(mt * 16 + 4 * g + r, T - 1), col0, dv, p.vpairs, raw[r]);
  };
  StateRows<DK, F32, NTW> S;
  if constexpr (TERMS == 1) {  // rows of q and k go to LDS as they are
    constexpr int copies = D::T * Op::CH / 64;
#pragma unroll
    for (int i = 0; i < (2 * copies + 3) / 4; ++i) {
      const int at = wave + 4 * i;
      if (at >= 2 * copies) break;
      const bool is_k = at < copies;
      const int slot = (is_k ? at : at - copies) * 64 + lane, t = slot / Op::CH;
      const int chunk = Op::exchanged(t, slot % Op::CH);
      copy16((is_k ? krows : qrows).at(min(t, T - 1), chunk * 8),
             (is_k ? &lds.kop[0][0][0] : &lds.qop[0][0][0]) + (slot - lane) * 8);
    }
    S.fetch(p, n, h, first, lds.codes[wave], lds.scales[wave]);
    load_v(0);
  } else {
    // a thread's groups of four columns of all rows, from row t0 on, TS rows apart
    constexpr int IT = D::T * DK / 4 / kThreads, TS = kThreads / (DK / 4);
    const int t0 = threadIdx.x / (DK / 4), e0 = threadIdx.x % (DK / 4) * 4;
    if constexpr (VEC) {
      f32x4 a[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i)
        a[i] = *reinterpret_cast<const f32x4*>(p.g + (row_of(p, n, 0) * p.s.H + h) * DK +
                                               min(t0 + i * TS, T - 1) * p.s.H * DK + e0);
      S.fetch(p, n, h, first, lds.codes[wave], lds.scales[wave]);
      load_v(0);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i][j] = qscan::fast_exp(qscan::gate(a[i][j]));
        *reinterpret_cast<f32x4*>(&lds.alpha[t0 + i * TS][e0]) = a[i];
      }
    } else {
      u32x4 w[IT], w2[IT];
      auto stage = [&](const u32x4 (&w)[IT], uint16_t (*op)[D::OT][LP]) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          float x[4];
          qscan::widen4(w[i], dtype, x);
          qscan::put4<TERMS>(&op[0][t0 + i * TS][e0], plane, x);
        }
      };
#pragma unroll
      for (int i = 0; i < IT; ++i) w[i] = load_k(t0 + i * TS, e0);
#pragma unroll
      for (int i = 0; i < IT; ++i) w2[i] = load_q(t0 + i * TS, e0);
      S.fetch(p, n, h, first, lds.codes[wave], lds.scales[wave]);
      load_v(0);
      stage(w, lds.kop);
      stage(w2, lds.qop);
    }
  }

  f32x4 xk[NTW], xq[NTW];
  // the state's codes as operands: kept where several tiles of nodes use them and registers are left
  constexpr bool hold = MT > 1 && !VEC && !F32 && DK <= 128 && (NTW == 1 || !DELTA);
  Frag<1> codes[hold ? NTW : 1][DK / 32];
  auto products = [&](int mt) {
    if (idle) return;
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct) {
      if (!F32 && (!hold || mt == 0)) S.operands(ct, codes[hold ? ct : 0]);
      state_products<DK, TERMS, DELTA, F32, NTW>(S, ct, codes[hold ? ct : 0], &lds.kop[0][0][0], &lds.qop[0][0][0],
                                                 VEC ? 0 : mt * 16, plane, xk[ct], xq[ct]);
      asm volatile("" ::: "memory");  // one tile's operands in registers at a time
    }
  };

  // the nodes' ways to the stored state, each row's found together with its ancestors': in every
  // round a row takes over what the row it stands at has found
  auto paths = [&]() {
    int at = parent;
    unsigned long long mask = 1ull << lane;
    double c = !VEC && parent > -2 ? (double)qscan::gate(gate) : 0.0;
    while (__ballot(at >= 0)) {
      const int from = at < 0 ? lane : at;
      const double c2 = VEC ? 0.0 : __shfl(c, from);
      const unsigned long long m2 = __shfl(mask, from);
      const int at2 = __shfl(at, from);
      if (at >= 0) {
        c += c2;
        mask |= m2;
        at = at2;  // -2: the row hangs on one that is none
      }
    }
    const bool ok = at == -1;
    const unsigned long long nodes = __ballot(ok);
    if (lane == 0) lds.nodes = nodes;
    if (lane < D::T) {
      lds.mask[lane] = ok ? mask : 0;
      lds.parent[lane] = ok ? parent : -1;
      lds.c[lane] = c;
      lds.ec[lane] = VEC ? 1.0f : qscan::fast_exp((float)c);
      lds.beta[lane] = ok ? beta : 0.0f;
    }
  };
  // A and L by tiles, shared out to the waves behind the first; what is no ancestor is zero,
  // whatever its product is
  auto between = [&](int rows) {
    constexpr int kinds = DELTA ? 2 : 1;
    for (int i = wave - 1; i < MT * MT * kinds; i += 3) {
      const int it = i / kinds / MT, jt = i / kinds % MT;
      const bool is_l = DELTA && i % kinds == 0;
      if (jt > it || it * 16 >= rows) continue;
      f32x4 a = {0, 0, 0, 0};
      const uint16_t* left = is_l ? &lds.kop[0][0][0] : &lds.qop[0][0][0];
#pragma unroll
      for (int s = 0; s < DK / 32; ++s)
        qscan::mma(a, Op::frag(left, it * 16 + (lane & 15), s, plane),
                   Op::frag(&lds.kop[0][0][0], jt * 16 + (lane & 15), s, plane));
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
      if (is_l && it == jt) {
        // not into the inverse: the node's U is spoilt by its e^c instead
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (broken(x[r])) lds.ec[it * 16 + 4 * g + r] = NAN;
          x[r] = broken(x[r]) ? 0.0f : x[r];
        }
        *reinterpret_cast<f32x4*>(&lds.lt[it][lane & 15][4 * g]) = x;
      }
    }
  };

  unsigned long long nodes;
  if constexpr (VEC) {
    copies_done();
    if (wave == 0) paths();
    __syncthreads();
    nodes = lds.nodes;
  } else {
    // the first wave finds the paths while the others multiply the first tile by the state, and
    // does that while they do what is between nodes
    copies_done();
    __syncthreads();
    if (wave == 0)
      paths();
    else
      products(0);
    __syncthreads();
    nodes = lds.nodes;
    if (wave == 0)
      products(0);
    else
      between(nodes ? 64 - __clzll(nodes) : 0);
    if (DELTA) {
      if (MT > 1) __syncthreads();  // with one tile the second wave has all of L
      if (wave == 1 && g < MT) invert(lds.lt, lds.inv, g, &lds.ec[g * 16]);
    }
  }
  const int rows = nodes ? 64 - __clzll(nodes) : 0;  // up to the last node

  const Columns<NTW> to(p, n, h, col0, dtype);
  f32x4 u[MT][NTW];
  bool spoilt = false;  // something in the wave's part of U is not finite: zeros stand in its place
  if (lane < 16)
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct) lds.gone[wave][ct][lane] = 0;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt * 16 >= rows) break;
    if constexpr (VEC) {
      if (mt > 0) __syncthreads();  // the last tile's A and L are done with
      // each of 16 nodes goes up its path, 16 lanes a node: q and k take the decays on the way
      const int i = threadIdx.x >> 4, t = mt * 16 + i, sub = threadIdx.x & 15;
      constexpr int R = DK / 64;
      u32x4 wq[R], wk[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        wq[r] = load_q(t, 64 * r + 4 * sub);
        wk[r] = load_k(t, 64 * r + 4 * sub);
      }
      // what is no ancestor is zero
      for (int j = sub; j < MP; j += 16) {
        lds.A[i][j] = 0.0f;
        if (DELTA) lds.L[i][j] = 0.0f;
      }
      if (DELTA) lds.lt[0][sub][i] = 0.0f;
      const bool on = lds.mask[t] != 0;
      // nodes and keys of the next steps, fetched three ahead
      int ahead[3];
      u32x4 kw[3][R];
      ahead[0] = on ? lds.parent[t] : -1;
#pragma unroll
      for (int d = 1; d < 3; ++d) ahead[d] = ahead[d - 1] < 0 ? -1 : lds.parent[ahead[d - 1]];
#pragma unroll
      for (int d = 0; d < 3; ++d)
#pragma unroll
        for (int r = 0; r < R; ++r) kw[d][r] = load_k(max(ahead[d], 0), 64 * r + 4 * sub);
      float q[R][4], k[R][4], x[R][4];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        qscan::widen4(wq[r], dtype, q[r]);
        qscan::widen4(wk[r], dtype, k[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[r][j] = k[r][j];
      }
      int at = on ? t : -1;
      while (at >= 0) {
#pragma unroll
        for (int d = 0; d < 3; ++d) {  // in turns, so that what was fetched is not moved
          if (at < 0) break;
          float a = 0.0f, l = 0.0f;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&lds.alpha[at][64 * r + 4 * sub]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a = fmaf(q[r][j], x[r][j], a);
              if (DELTA) l = fmaf(k[r][j], x[r][j], l);
              q[r][j] *= f[j];
              if (DELTA) k[r][j] *= f[j];
            }
          }
          a = qscan::sum16(a);
          if (DELTA) l = qscan::sum16(l);
          if (sub == 0) {
            const float b = lds.beta[at];
            lds.A[i][at] = a * b;
            if (DELTA && at != t) {
              lds.L[i][at] = -l * b;
              if (at >= mt * 16) lds.lt[0][at - mt * 16][i] = broken(l * b) ? 0.0f : -l * b;
              if (broken(l * b)) lds.ec[t] = NAN;  // not into the inverse
            }
          }
          at = ahead[d];
          ahead[d] = ahead[(d + 2) % 3] < 0 ? -1 : lds.parent[ahead[(d + 2) % 3]];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            qscan::widen4(kw[d][r], dtype, x[r]);
            kw[d][r] = load_k(max(ahead[d], 0), 64 * r + 4 * sub);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        qscan::put4<TERMS>(&lds.qop[0][i][64 * r + 4 * sub], plane, q[r]);
        if (DELTA) qscan::put4<TERMS>(&lds.kop[0][i][64 * r + 4 * sub], plane, k[r]);
      }
      __syncthreads();
      if (DELTA && wave == 0 && g == 0) invert(lds.lt, lds.inv, 0, &lds.ec[mt * 16]);
    }
    if (mt > 0) load_v(mt);
    if (VEC || mt > 0) products(mt);
    if (VEC || mt == 0) __syncthreads();  // A, L and the inverse are there, this tile's operands read
    if (idle) continue;
    const f32x4 ec = *reinterpret_cast<const f32x4*>(&lds.ec[mt * 16 + 4 * g]);
    const f32x4 bt = *reinterpret_cast<const f32x4*>(&lds.beta[mt * 16 + 4 * g]);
    bool node[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) node[r] = (uint32_t)(nodes >> (mt * 16)) & (1u << (4 * g + r));
    f32x4 x[NTW];
    bool bad = false;
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = VW < NTW ? __uint_as_float(ct ? raw[r][0] & 0xFFFF0000u : raw[r][0] << 16)
                                 : qscan::from_raw(raw[r][VW == 1 ? 0 : ct], dtype);
        x[ct][r] = node[r] ? (DELTA ? fmaf(-ec[r], xk[ct][r], v) : v) : 0.0f;
        xq[ct][r] *= ec[r];
      }
      if constexpr (DELTA) {
#pragma unroll
        for (int jt = 0; jt < mt; ++jt)
          small_mma(x[ct], &lds.L[VEC ? 0 : mt * 16][jt * 16], MP, u[jt][ct]);
        u[mt][ct] = f32x4{0, 0, 0, 0};
        small_mma(u[mt][ct], &lds.inv[VEC ? 0 : mt][0][0], 20, x[ct]);
      } else {
        u[mt][ct] = x[ct];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) bad |= broken(u[mt][ct][r]);
    }
    spoilt |= __ballot(bad) != 0;
    if (spoilt) {
#pragma unroll
      for (int ct = 0; ct < NTW; ++ct) {
        unsigned long long gone = lds.gone[wave][ct][lane & 15];
        gone |= (unsigned long long)take_out(x[ct]) << (mt * 16);
        if (DELTA) {
          f32x4 below;
#pragma unroll
          for (int r = 0; r < 4; ++r) below[r] = lds.mask[mt * 16 + 4 * g + r] & gone ? NAN : 0.0f;
          gone |= (unsigned long long)take_out(below) << (mt * 16);
          u[mt][ct] = f32x4{0, 0, 0, 0};
          small_mma(u[mt][ct], &lds.inv[VEC ? 0 : mt][0][0], 20, x[ct]);
        } else {
          u[mt][ct] = x[ct];
        }
        gone |= (unsigned long long)take_out(u[mt][ct]) << (mt * 16);
        lds.gone[wave][ct][lane & 15] = gone;  // the four lanes of a column have the same
      }
    }
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct) {
#pragma unroll
      for (int jt = 0; jt <= mt; ++jt)
        small_mma(xq[ct], &lds.A[VEC ? 0 : mt * 16][jt * 16], MP, u[jt][ct]);
    }
    float out[4][NTW], wr[4][NTW];
#pragma unroll
    for (int ct = 0; ct < NTW; ++ct)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        out[r][ct] = node[r] ? xq[ct][r] : 0.0f;
        wr[r][ct] = node[r] ? u[mt][ct][r] * bt[r] : 0.0f;
      }
    if (spoilt) {
#pragma unroll
      for (int ct = 0; ct < NTW; ++ct) {
        const unsigned long long gone = lds.gone[wave][ct][lane & 15];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = mt * 16 + 4 * g + r;
          if (lds.mask[row] & gone) out[r][ct] = NAN;
          if (gone >> row & 1) wr[r][ct] = NAN;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = mt * 16 + 4 * g + r;
      if (t < T) to.store(t, out[r], wr[r]);
    }
  }
  // rows behind the last node's tile
  const float zero[NTW] = {};
  for (int t = (rows + 15) / 16 * 16 + g; t < T; t += 4) to.store(t, zero, zero);
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
    if constexpr (NTW == 1 || !narrow(DK, 64, TERMS > 1, VEC))
      return verify_state<DK, 4, TERMS, VEC, DELTA, NTW>(p, s);
  }
  return hipErrorInvalidValue;
}

template <int DK, int TERMS, bool VEC, bool DELTA>
hipError_t verify_columns(const Params& p, hipStream_t s) {
  return p.columns == 128 ? verify_tiles<DK, TERMS, VEC, DELTA, 2>(p, s)
                          : verify_tiles<DK, TERMS, VEC, DELTA, 1>(p, s);
}

// One gate a token: bfloat16 q and k enter the products as they are.
template <int DK>
hipError_t verify_tokens(const Params& p, hipStream_t s) {
  if (p.mixer == qscan::GDN)
    return p.direct ? verify_columns<DK, 1, false, true>(p, s) : verify_columns<DK, 3, false, true>(p, s);
  return p.direct ? verify_columns<DK, 1, false, false>(p, s) : verify_columns<DK, 3, false, false>(p, s);
}

template <int DK>
hipError_t verify_channels(const Params& p, hipStream_t s) {
  return p.mixer == qscan::KDA ? verify_columns<DK, 3, true, true>(p, s)
                               : verify_columns<DK, 3, true, false>(p, s);
}

}  // namespace qdraft
