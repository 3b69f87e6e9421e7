// linear.hip — products with 4-bit weights and group scales (include/qstate_linear.h).
//
// Few rows of x: every weight is read once, and its bytes bound the call.  A tile
// of 16 outputs x 128 inputs is one 16-byte load a lane, whose four words are the
// right operands of four 16 x 16 x 32 matrix instructions; the left ones are rows
// of x, 16 at a time.  A nibble of sign and size becomes an E4M3 byte by moving
// its sign bit (size * 2^-9), which one packed conversion scales to the whole
// number in 16 bits: five instructions for four codes.  Sums of whole numbers times
// x are multiplied by a group's scale, one per lane.  Waves of a workgroup share out
// the inputs and add their sums up in LDS, in a fixed order.  4096 x 4096 weights times
// one row take 4.6 us (9.5 MB; an empty launch 2 to 3), 12288 x 4096 times 16 rows
// 9.4 us (27 MB, 2.9 TB/s): the rows' way from L2, 64 bytes a cycle and CU, comes on top.

#include <hip/hip_runtime.h>

#include "linear_launch.h"
#include "qstate_value.h"
#include "scan_device.h"

namespace qlinear {

using qscan::f32x4;
using qscan::Frag;
using qscan::u32x2;
using qscan::u32x4;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The eight codes of a word as an operand of bfloat16 (F16: float16) numbers.
template <bool F16>
__device__ __forceinline__ u32x4 widen(uint32_t w) {
  const uint32_t lo = (w & 0x07070707u) | ((w & 0x08080808u) << 4);
  const uint32_t hi = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
  u32x4 f;
  if constexpr (F16) {
    f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 512.0f, false));
    f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 512.0f, true));
    f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 512.0f, false));
    f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 512.0f, true));
  } else {
    f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.0f, false));
    f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.0f, true));
    f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.0f, false));
    f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.0f, true));
  }
  return f;
}

// Eight neighbouring values of a row of x as they lie in memory.
template <int DT>
struct RawX {
  u32x4 w[DT == 0 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ void product(f32x4& acc, const RawX<DT>& x, const u32x4& w) {
  if constexpr (DT == 0) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x.w[i / 4][i % 4]);
    Frag<1> b;
    b.t[0] = w;
    qscan::mma(acc, qscan::split8<3>(v), b);
  } else if constexpr (DT == 1) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(qscan::bf16x8, x.w[0]),
                                                  __builtin_bit_cast(qscan::bf16x8, w), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x.w[0]),
                                                 __builtin_bit_cast(f16x8, w), acc, 0, 0, 0);
  }
}

constexpr int kWaves = 8, kAhead = 2;  // of a workgroup; of a wave's tiles of inputs in flight

// 16 rows of x, NT tiles of 16 outputs.
template <int DT, int G, int NT>
__global__ void __launch_bounds__(kWaves * 64) linear_kernel(Params p) {
  constexpr int S = kIn / G;  // groups of a tile
  __shared__ float sums[kWaves][NT][256];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = (int64_t)blockIdx.y * 16;
  const int ot0 = blockIdx.x * NT;
  // rows behind the last repeat it: a row of y depends on its own only
  const char* x = static_cast<const char*>(p.x) +
                  ((row0 + c < p.rows ? row0 + c : p.rows - 1) * p.xs + g * 8) * (DT == 0 ? 4 : 2);
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0, 0, 0, 0};
  u32x4 w[kAhead][NT];
  float s[kAhead][NT][S];
  RawX<DT> xr[kAhead][4];
  auto load = [&](int d, int kt) {
    if (kt >= p.in_tiles) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t tile = (int64_t)min(ot0 + n, p.out_tiles - 1) * p.in_tiles + kt;
      w[d][n] = reinterpret_cast<const u32x4*>(p.packed)[tile * 64 + lane];
#pragma unroll
      for (int j = 0; j < S; ++j) s[d][n][j] = p.scales[(tile * 16 + c) * S + j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = kt * kIn + i * 32;  // inputs behind the last count as zeros
      const u32x4* at = reinterpret_cast<const u32x4*>(x + (col < p.inputs ? col : 0) * (DT == 0 ? 4 : 2));
#pragma unroll
      for (int h = 0; h < (DT == 0 ? 2 : 1); ++h)
        xr[d][i].w[h] = col < p.inputs ? at[h] : u32x4{0, 0, 0, 0};
    }
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load(d, wave + d * kWaves);
  for (int kt = wave; kt < p.in_tiles; kt += kAhead * kWaves) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      if (kt + d * kWaves >= p.in_tiles) break;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 part;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i * 32 % G == 0) part = f32x4{0, 0, 0, 0};
          product<DT>(part, xr[d][i], widen<DT == 2>(w[d][n][i]));
          if ((i + 1) * 32 % G == 0) {
            const float f = s[d][n][i * 32 / G];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[n][r] = fmaf(f, part[r], acc[n][r]);
          }
        }
      }
      load(d, kt + (d + kAhead) * kWaves);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(&sums[wave][n][lane * 4]) = acc[n];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 256; e += kWaves * 64) {
    // element e: row (e / 16) % 16 of its tile, output e % 16, in the lane that holds them
    const int tile = e >> 8, r = (e >> 4) & 15, o = e & 15;
    const int at = ((r >> 2) * 16 + o) * 4 + (r & 3);
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) y += sums[i][tile][at];
    const int64_t row = row0 + r;
    const int out = (ot0 + tile) * 16 + o;
    if (row >= p.rows || out >= p.outputs) continue;
    if (p.bias) y += p.bias[out];
    qscan::store_elem(p.y, row * p.outputs + out, DT, y);
  }
}

// A nibble of sign and size.
__device__ __forceinline__ uint32_t nibble(int c) {
  const int m = min(c < 0 ? -c : c, 7);
  return (uint32_t)(m | (c < 0 ? 8 : 0));
}

// The word of lane l, number i, from the eight codes it holds.
template <class F>
__device__ __forceinline__ uint32_t word_of(F code) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= nibble(code(j)) << (j < 4 ? 8 * j : 8 * (j - 4) + 4);
  return w;
}

// A thread for each word: tile, lane, word of it.
__global__ void __launch_bounds__(256) pack_kernel(Params p) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tile = at >> 8;
  if (tile >= (int64_t)p.out_tiles * p.in_tiles) return;
  const int l = (at >> 2) & 63, i = at & 3;
  const int out = (int)(tile / p.in_tiles) * kOut + (l & 15);
  const int in = (int)(tile % p.in_tiles) * kIn + 32 * i + 8 * (l >> 4);
  const bool ok = out < p.outputs && in < p.inputs;
  const int8_t* src = p.codes + (ok ? (int64_t)out * p.inputs + in : 0);
  p.packed_out[at] = ok ? word_of([&](int j) { return (int)src[j]; }) : 0u;
  const int S = kIn / p.group;
  if (l < 16 && i < S) {
    const int col = (int)(tile % p.in_tiles) * S + i;
    p.scales_out[(tile * 16 + l) * S + i] =
        out < p.outputs && col < p.inputs / p.group
            ? p.group_scales[(int64_t)out * (p.inputs / p.group) + col]
            : 0.0f;
  }
}

// A wave for each 16 outputs and group: lane l quantizes an output's columns
// 8 (l / 16) .. of each 32 of the group.
__global__ void __launch_bounds__(64) quantize_kernel(Params p) {
  const int l = threadIdx.x, o = l & 15, g = l >> 4;
  const int groups = p.in_tiles * (kIn / p.group), S = kIn / p.group;
  const int64_t ot = blockIdx.x / groups;
  const int gr = (int)(blockIdx.x % groups), out = (int)ot * kOut + o;
  const int col0 = gr * p.group;
  const bool ok = out < p.outputs && col0 < p.inputs;
  const int64_t row = (int64_t)(ok ? out : 0) * p.inputs + (ok ? col0 : 0);
  float m = 0.0f;
  for (int i = 0; i < p.group / 32; ++i)
    for (int j = 0; j < 8; ++j) {
      const float x = ok ? fabsf(qscan::load_elem(p.weights, row + i * 32 + g * 8 + j, p.dtype)) : 0.0f;
      m = x > m || x != x ? x : m;
    }
  for (int d = 16; d < 64; d *= 2) {
    const float x = __shfl_xor(m, d);
    m = x > m || x != x ? x : m;
  }
  float s, inv;
  qs::group_scale<7>(m, s, inv);
  const int64_t tile = ot * p.in_tiles + gr / S;
  if (g == 0) p.scales_out[(tile * 16 + o) * S + gr % S] = s;
  for (int i = 0; i < p.group / 32; ++i) {
    const uint32_t w = word_of([&](int j) {
      const float x = ok ? qscan::load_elem(p.weights, row + i * 32 + g * 8 + j, p.dtype) : 0.0f;
      return (int)(__float_as_uint(fmaf(x, inv, qs::kMagic)) - 0x4B400000u);  // of the exact product
    });
    p.packed_out[tile * 256 + l * 4 + gr % S * (p.group / 32) + i] = w;
  }
}

template <int DT, int G, int NT>
static hipError_t run(const Params& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.out_tiles + NT - 1) / NT), (unsigned)((p.rows + 15) / 16));
  linear_kernel<DT, G, NT><<<grid, kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

// How many tiles of outputs a workgroup takes.  Each of them reads the 16 rows of x once, which costs
// its CU what four tiles of weights do; workgroups are shared out to 256 CUs.  Bfloat16, 16 rows of
// 4096, us with 1 / 2 / 3 / 4 tiles: 4096 outputs 6.3 / 7.5 / 8.3 / 9.2, 6144 10.2 / 7.3 / 8.4 / 9.3,
// 12288 14.2 / 10.9 / 8.2 / 8.9, 32768 36 / 23 / 22 / 21; 64 rows, 12288 outputs 48 / 27 / 22 / 19 (with
// more rows a workgroup instead, 32 and 64: 21 at best).
static int tiles_of(const Params& p) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= 4; ++n) {
    const int64_t groups = (int64_t)((p.out_tiles + n - 1) / n) * ((p.rows + 15) / 16);
    const int64_t cost = (groups + 255) / 256 * (4 + n);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

template <int DT, int G>
static hipError_t by_tiles(const Params& p, hipStream_t s) {
  switch (tiles_of(p)) {
    case 1: return run<DT, G, 1>(p, s);
    case 2: return run<DT, G, 2>(p, s);
    case 3: return run<DT, G, 3>(p, s);
    default: return run<DT, G, 4>(p, s);
  }
}

template <int DT>
static hipError_t by_group(const Params& p, hipStream_t s) {
  switch (p.group) {
    case 32: return by_tiles<DT, 32>(p, s);
    case 64: return by_tiles<DT, 64>(p, s);
    case 128: return by_tiles<DT, 128>(p, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t multiply(const Params& p, hipStream_t s) {
  switch (p.dtype) {
    case 0: return by_group<0>(p, s);
    case 1: return by_group<1>(p, s);
    case 2: return by_group<2>(p, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t pack(const Params& p, hipStream_t s) {
  pack_kernel<<<(unsigned)((int64_t)p.out_tiles * p.in_tiles), 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t quantize(const Params& p, hipStream_t s) {
  const int64_t groups = (int64_t)p.in_tiles * (kIn / p.group);
  quantize_kernel<<<(unsigned)(p.out_tiles * groups), 64, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace qlinear
