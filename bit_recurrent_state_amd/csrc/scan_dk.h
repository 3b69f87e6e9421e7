// scan_dk.h — launches of the scan's kernels for one dk (one translation unit
// each).

#pragma once

#include "scan_chain.h"
#include "scan_grads.h"
#include "scan_prep.h"
#include "scan_prep_vector.h"
#include "scan_tokens.h"

namespace qscan {

inline dim3 chain_grid(const Params& p) {
  const int64_t heads = ((int64_t)p.batch * p.heads + 7) / 8 * 8;
  return dim3((unsigned)(heads * p.nvb));
}

template <int DK, int NT, int NPQ, bool VEC, bool DELTA>
hipError_t forward_tail(const Params& p, hipStream_t s) {
  const dim3 slots(p.nslots, p.heads);
  const int64_t short_ones = token_blocks(p);
  if (short_ones && (VEC || !p.some_long))
    tokens_kernel<DK, VEC, DELTA><<<dim3((unsigned)short_ones), 256, 0, s>>>(p);
  if (!p.some_long) return hipGetLastError();
  constexpr bool SOLVED = VEC && DELTA && DK <= 128;
  if constexpr (VEC && DK <= 128) {
    prep_vector_kernel<DK, DELTA, false><<<slots, 512, 0, s>>>(p);
    chunk_vector_kernel<DK, DELTA, false><<<slots, 256, 0, s>>>(p);
    if (DELTA) prep_vector_kernel<DK, DELTA, true><<<slots, 512, 0, s>>>(p);
  } else if constexpr (VEC) {
    operands_vector_kernel<DK, DELTA, false><<<slots, 256, 0, s>>>(p);
    chunk_kernel<DK, P, true, DELTA, false><<<slots, 256, 0, s>>>(p);
    chunk_vector_kernel<DK, DELTA, false><<<slots, 256, 0, s>>>(p);
  } else {
    const dim3 blocks((unsigned)(short_ones + (int64_t)p.nslots * p.heads_qk));
    tokens_operands_kernel<DK, DELTA><<<blocks, 256, 0, s>>>(p);
    chunk_kernel<DK, NPQ, false, DELTA, false><<<slots, 256, 0, s>>>(p);
  }
  states_kernel<DK, NT, NPQ, VEC, DELTA, false, SOLVED><<<chain_grid(p), 512, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK, int NT, int NPQ, int NPO, bool VEC, bool DELTA>
hipError_t backward_tail(const Params& p, hipStream_t s) {
  const dim3 slots(p.nslots, p.heads);
  if (VEC) {
    operands_vector_kernel<DK, DELTA, true><<<slots, 256, 0, s>>>(p);
    chunk_kernel<DK, P, true, DELTA, true><<<slots, 256, 0, s>>>(p);
    chunk_vector_kernel<DK, DELTA, true><<<slots, 256, 0, s>>>(p);
  } else {
    operands_kernel<DK><<<dim3(p.nslots, p.heads_qk), 256, 0, s>>>(p);
    chunk_kernel<DK, NPQ, false, DELTA, true><<<slots, 256, 0, s>>>(p);
  }
  states_kernel<DK, NT, NPQ, VEC, DELTA, true, false><<<chain_grid(p), 256, 0, s>>>(p);
  state_grads_kernel<DK, NT, NPQ, NPO, VEC, DELTA><<<chain_grid(p), 512, 0, s>>>(p);
  grads_kernel<DK, NPQ, VEC ? NPO : NPQ, NPO, VEC, DELTA>
      <<<slots, DK >= 128 ? 512 : 256, 0, s>>>(p);
  if (VEC) grads_vector_kernel<DK, NPO, NPO, DELTA><<<slots, 256, 0, s>>>(p);
  if (p.heads != p.heads_qk)
    share_kernel<DK><<<dim3(p.nslots, p.heads_qk, kChunk * DK / 1024), 256, 0, s>>>(p);
  return hipGetLastError();
}

// Column blocks as the host's rule has them (scan_api.cpp).
template <int DK, int NPQ, bool VEC, bool DELTA>
hipError_t forward_width(const Params& p, hipStream_t s) {
  if constexpr (DK <= 128 && !(DELTA && NPQ > 1))
    if (p.vblock == 64) return forward_tail<DK, 4, NPQ, VEC, DELTA>(p, s);
  return p.vblock == 16 ? forward_tail<DK, 1, NPQ, VEC, DELTA>(p, s)
                        : forward_tail<DK, 2, NPQ, VEC, DELTA>(p, s);
}

template <int DK, int NPQ, int NPO, bool VEC, bool DELTA>
hipError_t backward_width(const Params& p, hipStream_t s) {
  if constexpr (!(DELTA && NPQ > 1))
    if (p.vblock == 32) return backward_tail<DK, 2, NPQ, NPO, VEC, DELTA>(p, s);
  return backward_tail<DK, 1, NPQ, NPO, VEC, DELTA>(p, s);
}

// Operand kinds: the caller's bfloat16 rows (one term); rows split into terms
// (FP32, FP16, unaligned bfloat16); rows scaled per channel (always split).
template <int DK>
hipError_t forward(const Params& p, hipStream_t s) {
  switch (p.mixer) {
    case GDN: return p.direct ? forward_width<DK, 1, false, true>(p, s)
                              : forward_width<DK, P, false, true>(p, s);
    case SCALAR: return p.direct ? forward_width<DK, 1, false, false>(p, s)
                                 : forward_width<DK, P, false, false>(p, s);
    case GLA: return forward_width<DK, P, true, false>(p, s);
    case KDA: return forward_width<DK, P, true, true>(p, s);
    default: return hipErrorInvalidValue;
  }
}

// d_o's terms (NPO) are those of the workspace's layout, whether or not q and k are split: bfloat16
// rows off 16 bytes have split q and k and a d_o of one term.
template <int DK>
hipError_t backward(const Params& p, hipStream_t s) {
  const bool one = p.dop_terms == 1;
  switch (p.mixer) {
    case GDN: return p.direct ? backward_width<DK, 1, 1, false, true>(p, s)
                     : one    ? backward_width<DK, P, 1, false, true>(p, s)
                              : backward_width<DK, P, P, false, true>(p, s);
    case SCALAR: return p.direct ? backward_width<DK, 1, 1, false, false>(p, s)
                        : one    ? backward_width<DK, P, 1, false, false>(p, s)
                                 : backward_width<DK, P, P, false, false>(p, s);
    case GLA: return one ? backward_width<DK, P, 1, true, false>(p, s)
                         : backward_width<DK, P, P, true, false>(p, s);
    case KDA: return one ? backward_width<DK, P, 1, true, true>(p, s)
                         : backward_width<DK, P, P, true, true>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qscan
