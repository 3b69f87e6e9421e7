// draft_api.cpp — the C ABI declared in include/qstate_draft.h: argument checks
// and the launch plan.  Host code only.

#include "qstate_draft.h"

#include <hip/hip_runtime_api.h>

#include <cstring>

#include "draft_launch.h"
#include "qstate_scan.h"

namespace {

using qdraft::Params;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool vector_gate(int mixer) { return mixer == QSTATE_GLA || mixer == QSTATE_KDA; }

int check_config(const qstate_config* c, const qstate_draft_config* d) {
  size_t codes, scales;
  const int rc = qstate_state_bytes(c, &codes, &scales);  // checks the state's part
  if (rc != QSTATE_OK) return rc;
  if (!d || d->tokens < 1 || d->heads_qk < 1 || d->pad != 0) return QSTATE_E_INVALID;
  if (d->dtype < QSTATE_FP32 || d->dtype > QSTATE_FP16) return QSTATE_E_INVALID;
  if (c->heads % d->heads_qk != 0) return QSTATE_E_INVALID;
  const int64_t qk = (int64_t)d->heads_qk * c->dk, hv = (int64_t)c->heads * c->dv;
  if ((d->q_stride && d->q_stride < qk) || (d->k_stride && d->k_stride < qk) ||
      (d->v_stride && d->v_stride < hv))
    return QSTATE_E_INVALID;
  if (d->tokens > qdraft::most_tokens(c->dk)) return QSTATE_E_UNSUPPORTED;
  if (!c->fp32_state && (c->group_axis != QSTATE_VALUE_AXIS || c->window != 0))
    return QSTATE_E_UNSUPPORTED;
  const int64_t far = (int64_t)1 << 22;
  if (d->q_stride > far || d->k_stride > far || d->v_stride > far) return QSTATE_E_UNSUPPORTED;
  // the grids, a workgroup of up to 256 threads per head and 32 value rows, stay below 2^32 threads
  if ((int64_t)c->batch * c->heads * ((c->dv + 31) / 32) > 16777215) return QSTATE_E_UNSUPPORTED;
  return QSTATE_OK;
}

int block_width(const qstate_config* c, int h, int q) {
  if (c->channel_bits) return c->channel_bits[(size_t)h * (c->dk / 16) + q];
  return c->head_bits ? c->head_bits[h] : 8;
}

void set_state(const qstate_config* c, const qstate_draft_config* d, void* codes, float* scales,
               Params& p) {
  std::memset(&p, 0, sizeof(p));
  p.s.state = codes;
  p.s.scales = scales;
  p.s.B = c->batch;
  p.s.H = c->heads;
  p.s.dv = c->dv;
  p.s.G = c->fp32_state ? 16 : c->group;
  p.s.seed = c->seed;
  p.s.layer = c->layer;
  if (!c->fp32_state) {
    // as qstate_create lays heads out: 8 bytes per INT4 and 16 per INT8 block of 16 columns
    const int blocks = c->dk / 16;
    uint32_t units = 0;
    for (int h = 0; h < c->heads; ++h) {
      uint16_t m = 0;
      for (int q = 0; q < blocks; ++q)
        if (block_width(c, h, q) == 8) m = (uint16_t)(m | (1u << q));
      p.s.int8_blocks[h] = m;
      p.s.head_units[h] = units;
      units += (uint32_t)(blocks + __builtin_popcount(m));
      if (m != 0 && m != (uint16_t)((1u << blocks) - 1u)) p.s.mixed = 1;
    }
    p.s.bytes_per_b = (uint64_t)8 * c->dv * units;
  }
  p.fp32 = c->fp32_state;
  p.rounding = c->fp32_state ? 0 : c->rounding;
  p.mixer = c->mixer;
  p.tokens = d->tokens;
  p.heads_qk = d->heads_qk;
  p.dtype = d->dtype;
  p.qs = d->q_stride ? d->q_stride : (int64_t)d->heads_qk * c->dk;
  p.ks = d->k_stride ? d->k_stride : (int64_t)d->heads_qk * c->dk;
  p.vs = d->v_stride ? d->v_stride : (int64_t)c->heads * c->dv;
}

bool state_ok(const qstate_config* c, const void* codes, const float* scales) {
  return codes && aligned(codes, 16) &&
         (c->fp32_state || (scales && aligned(scales, 16)));
}

int status(hipError_t e) { return e == hipSuccess ? QSTATE_OK : QSTATE_E_LAUNCH; }

}  // namespace

extern "C" {

int qstate_verify(const qstate_config* state, const qstate_draft_config* draft,
                  const void* codes, const float* scales, const void* q, const void* k,
                  const void* v, const float* log_alpha, const float* beta,
                  const int32_t* parents, void* o, float* writes, void* stream) {
  const int rc = check_config(state, draft);
  if (rc != QSTATE_OK) return rc;
  const size_t e = draft->dtype == QSTATE_FP32 ? 4 : 2;
  if (!state_ok(state, codes, scales)) return QSTATE_E_INVALID;
  if (!q || !k || !v || !log_alpha || (state->mixer != QSTATE_GLA && !beta) || (!o && !writes))
    return QSTATE_E_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, e) || !aligned(log_alpha, 16) ||
      !aligned(beta, 4) || !aligned(parents, 4) || !aligned(o, e) || !aligned(writes, 16))
    return QSTATE_E_INVALID;
  Params p;
  set_state(state, draft, const_cast<void*>(codes), const_cast<float*>(scales), p);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = log_alpha;
  p.beta = state->mixer == QSTATE_GLA ? nullptr : beta;
  p.parents = parents;
  p.o = o;
  p.writes = writes;
  p.direct = !vector_gate(state->mixer) && draft->dtype == QSTATE_BF16 && p.qs % 8 == 0 && p.ks % 8 == 0;
  p.pairs = state->dv % 2 == 0 && aligned(o, 2 * e);
  p.vpairs = state->dv % 2 == 0 && p.vs % 2 == 0 && aligned(v, 2 * e);
  const bool narrow =
      qdraft::narrow(state->dk, draft->tokens, !p.direct, vector_gate(state->mixer));
  p.columns = state->dv > 64 && !narrow ? 128 : 64;
  p.blocks = (state->dv + p.columns - 1) / p.columns;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (state->dk) {
    case 64: return status(qdraft::verify_dk64(p, s));
    case 128: return status(qdraft::verify_dk128(p, s));
    default: return status(qdraft::verify_dk256(p, s));
  }
}

int qstate_accept(const qstate_config* state, const qstate_draft_config* draft, uint64_t step,
                  void* codes, float* scales, const void* k, const float* log_alpha,
                  const int32_t* parents, const float* writes, const int32_t* last, void* stream) {
  const int rc = check_config(state, draft);
  if (rc != QSTATE_OK) return rc;
  if (!state_ok(state, codes, scales)) return QSTATE_E_INVALID;
  if (!k || !log_alpha || !writes || !last) return QSTATE_E_INVALID;
  if (!aligned(k, 16) || !aligned(log_alpha, 16) || !aligned(parents, 4) || !aligned(writes, 16) ||
      !aligned(last, 4))
    return QSTATE_E_INVALID;
  Params p;
  set_state(state, draft, codes, scales, p);
  p.s.step = step;
  p.k = k;
  p.g = log_alpha;
  p.parents = parents;
  p.writes_in = writes;
  p.last = last;
  // 128 value rows a workgroup (the most its LDS has writes for), fewer while there are not enough
  // workgroups for the chip: 1024, four a CU
  p.rows = 128;
  while (p.rows > 32 && (int64_t)state->batch * state->heads * ((state->dv + p.rows - 1) / p.rows) < 1024)
    p.rows /= 2;
  p.blocks = (state->dv + p.rows - 1) / p.rows;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (state->dk) {
    case 64: return status(qdraft::accept_dk64(p, s));
    case 128: return status(qdraft::accept_dk128(p, s));
    default: return status(qdraft::accept_dk256(p, s));
  }
}

}  // extern "C"
