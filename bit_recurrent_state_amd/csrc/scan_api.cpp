// scan_api.cpp — the C ABI declared in include/qstate_scan.h: argument checks,
// the workspace's layout and the launches.  Host code only.

#include "qstate_scan.h"

#include <hip/hip_runtime_api.h>

#include <cstring>

#include "qstate.h"
#include "scan_launch.h"

namespace {

using qscan::kChunk;
using qscan::kTerms;
using qscan::Params;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool vector_gate(int mixer) { return mixer == QSTATE_GLA || mixer == QSTATE_KDA; }
bool delta_rule(int mixer) { return mixer == QSTATE_GDN || mixer == QSTATE_KDA; }

int check_config(const qstate_scan_config* c) {
  if (!c) return QSTATE_E_INVALID;
  if (c->batch < 1 || c->heads < 1 || c->heads_qk < 1 || c->dk < 1 || c->dv < 1)
    return QSTATE_E_INVALID;
  if (c->mixer < QSTATE_GDN || c->mixer > QSTATE_KDA) return QSTATE_E_INVALID;
  if (c->dtype < QSTATE_FP32 || c->dtype > QSTATE_FP16) return QSTATE_E_INVALID;
  if (c->heads % c->heads_qk != 0 || c->pad != 0) return QSTATE_E_INVALID;
  if (c->tokens < 0) return QSTATE_E_INVALID;
  const int64_t qk = (int64_t)c->heads_qk * c->dk, hv = (int64_t)c->heads * c->dv;
  if ((c->q_stride && c->q_stride < qk) || (c->k_stride && c->k_stride < qk) ||
      (c->v_stride && c->v_stride < hv) || (c->o_stride && c->o_stride < hv))
    return QSTATE_E_INVALID;
  if (c->dk != 64 && c->dk != 128 && c->dk != 256) return QSTATE_E_UNSUPPORTED;
  if (c->heads > 256 || c->dv > 4096 || c->tokens > 2147483647) return QSTATE_E_UNSUPPORTED;
  const int64_t far = (int64_t)1 << 22;  // offsets inside a chunk take 32 bits
  if (c->q_stride > far || c->k_stride > far || c->v_stride > far || c->o_stride > far)
    return QSTATE_E_UNSUPPORTED;
  // the grids stay below 2^32 threads: chunks of all sequences, or a workgroup per
  // head and 16 columns, of up to 512 threads; a workgroup per chunk and q/k head
  // and per head and 32 columns, of 256
  const int64_t most = 8388607, chunks = c->tokens / kChunk + c->batch;
  if (chunks > most || ((int64_t)c->batch * c->heads + 8) * ((c->dv + 31) / 32 * 2) > most ||
      chunks * c->heads_qk > most / 2 * 3)
    return QSTATE_E_UNSUPPORTED;
  return QSTATE_OK;
}

// Hands out the workspace's regions; with a null base it only counts.
struct Area {
  char* base;
  size_t used;
  template <class T>
  void take(T*& p, uint64_t n, bool want) {
    p = nullptr;
    if (!want) return;
    if (base) p = reinterpret_cast<T*>(base + used);
    used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
  }
};

size_t layout(const qstate_scan_config* c, bool backward, void* workspace, Params& p) {
  const bool vec = vector_gate(c->mixer), delta = delta_rule(c->mixer), bf16 = c->dtype == QSTATE_BF16;
  std::memset(&p, 0, sizeof(p));
  p.batch = c->batch;
  p.heads = c->heads;
  p.heads_qk = c->heads_qk;
  p.dk = c->dk;
  p.dv = c->dv;
  p.mixer = c->mixer;
  p.dtype = c->dtype;
  p.tokens = c->tokens;
  p.qs = c->q_stride ? c->q_stride : (int64_t)c->heads_qk * c->dk;
  p.ks = c->k_stride ? c->k_stride : (int64_t)c->heads_qk * c->dk;
  p.vs = c->v_stride ? c->v_stride : (int64_t)c->heads * c->dv;
  p.os = c->o_stride ? c->o_stride : (int64_t)c->heads * c->dv;
  // bfloat16 rows enter the products as they are where 16-byte loads reach them
  p.direct = !vec && bf16 && p.qs % 8 == 0 && p.ks % 8 == 0;
  p.nslots = (int)(c->tokens / kChunk + c->batch);
  p.dvp = (c->dv + 31) / 32 * 32;
  // Value columns of a chain workgroup, of which a CU (256) holds one at a time: eight waves of 132 to
  // 256 registers a lane (SCALAR's of 16 columns take 112, two of them share a CU and what it brings
  // out of L2).  16 or 32 by the fewest rounds, each as long as its width makes it: narrow blocks
  // shorten the chain from chunk to chunk, wide ones share its fixed work; 10 for 16 columns and 15
  // forward, 16 backward for 32.  64, forward, beyond 256 blocks of 32.  Whole calls in us, 1024 tokens
  // a sequence (1536: 512), dk 128:
  //   blocks of 32        128  256  384  512  768 1536
  //   GDN, 16 columns      64  110  158  209  336  355   backward  167  334  500  660  980  987
  //   32                   73   87  144  159  249  260             200  317  494  570  847  855
  //   64                  103  115  129  145  260  231
  // SCALAR, 16 / 32 / 64 columns: 63 / 59 / 84 at 256, 89 / 98 / 91 at 384, 110 / 107 / 99 at 512;
  // GLA: 118 / 103 / 121, 186 / 175 / 161 and 260 / 211 / 192.  Equal lengths at 768 are the exception
  // (SCALAR 166 with 32, 188 with 64); ragged ones are not (GDN, six prompts of up to 2900 tokens: 410
  // with 32, 374 with 64).
  // With the delta rule on split q and k a workgroup has no registers left for 64 columns forward and 32
  // backward: KDA at 512 446 / 370 / 377 and 1123 / 1216, FP32 GDN 454 / 380 / 483 and 1039 / 1135.
  const int64_t blocks = (int64_t)c->batch * c->heads * (p.dvp / 32);
  const bool heavy = delta && !p.direct;
  const int64_t narrow = (2 * blocks + 255) / 256 * 10, wide = (blocks + 255) / 256 * (backward ? 16 : 15);
  p.vblock = narrow < wide || (backward && heavy) ? 16 : 32;
  if (!backward && !heavy && blocks > 256 && p.dvp % 64 == 0 && c->dk <= 128) p.vblock = 64;
  p.nvb = p.dvp / p.vblock;
  p.dop_terms = bf16 ? 1 : kTerms;

  Area w = {static_cast<char*>(workspace), 0};
  const uint64_t sh = (uint64_t)p.nslots * p.heads, sq = (uint64_t)p.nslots * p.heads_qk;
  const uint64_t tile = (uint64_t)kChunk * p.dk, ops = (vec ? sh : sq) * (p.direct ? 1 : kTerms) * tile;
  const uint64_t square = sh * kTerms * kChunk * kChunk;
  w.take(p.chunks, p.nslots, true);
  w.take(p.sink, 64, true);
  w.take(p.rows, sh * 5 * kChunk, true);
  w.take(p.decay, sh * p.dk, vec);
  w.take(p.far, sh, vec);
  const bool fused = vec && !backward && c->dk <= 128;  // scan_prep_vector.h
  w.take(p.knrow, ops, vec && !fused);
  w.take(p.qrow, ops, !p.direct);
  w.take(p.krow, ops, !p.direct && (!vec || delta));
  w.take(p.kt, ops, true);
  w.take(p.a, square, !backward);
  w.take(p.t, square, delta);
  w.take(p.u, sh * kChunk * p.dvp, backward || (fused && delta));
  if (backward) {
    const uint64_t raw = sq * (bf16 ? 1 : kTerms) * tile;
    w.take(p.korow, ops, vec);
    w.take(p.qt, ops, true);
    w.take(p.ket, ops, vec && delta);
    w.take(p.knt, ops, vec);
    w.take(p.kt_raw, raw, vec);
    w.take(p.qt_raw, raw, vec);
    w.take(p.pfx, sh * tile, vec);
    w.take(p.sfx, sh * tile, vec);
    w.take(p.at, square, true);
    w.take(p.t2t, square, delta);
    // d_o's rows serve as they are where they are bfloat16 and fill whole blocks
    w.take(p.dop, sh * p.dop_terms * kChunk * p.dvp, !(bf16 && c->dv % 32 == 0));
    w.take(p.y, sh * kChunk * p.dvp, delta);
    w.take(p.sc, sh * p.dk * p.dvp, true);
    w.take(p.xc, sh * p.dk * p.dvp, true);
    w.take(p.dbpart, (uint64_t)p.nvb * sh * kChunk, c->mixer != QSTATE_GLA);
    w.take(p.dqpart, sh * tile, p.heads != p.heads_qk);
    w.take(p.dkpart, sh * tile, p.heads != p.heads_qk);
  }
  return w.used;
}

// The arrays that both directions read.
int check_inputs(const qstate_scan_config* c, const void* q, const void* k, const void* v,
                 const float* log_alpha, const float* beta, const int64_t* offsets,
                 const float* initial_state) {
  const size_t e = c->dtype == QSTATE_FP32 ? 4 : 2;
  const bool beta_needed = c->mixer != QSTATE_GLA;
  if (c->tokens > 0 && (!q || !k || !v || !log_alpha || (beta_needed && !beta)))
    return QSTATE_E_INVALID;
  if (!offsets && c->tokens % c->batch != 0) return QSTATE_E_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, e) || !aligned(log_alpha, 16) ||
      !aligned(beta, 16) || !aligned(offsets, 8) || !aligned(initial_state, 16))
    return QSTATE_E_INVALID;
  return QSTATE_OK;
}

void set_inputs(Params& p, const void* q, const void* k, const void* v, const float* log_alpha,
                const float* beta, const int64_t* offsets, const float* initial_state) {
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = log_alpha;
  p.beta = p.mixer == QSTATE_GLA ? nullptr : beta;
  p.offsets = offsets;
  p.s0 = initial_state;
}

int status(hipError_t e) { return e == hipSuccess ? QSTATE_OK : QSTATE_E_LAUNCH; }

}  // namespace

extern "C" {

int qstate_scan_workspace(const qstate_scan_config* cfg, int backward, size_t* bytes) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!bytes || (backward != 0 && backward != 1)) return QSTATE_E_INVALID;
  Params p;
  *bytes = layout(cfg, backward == 1, nullptr, p);
  return QSTATE_OK;
}

int qstate_scan(const qstate_scan_config* cfg, const void* q, const void* k, const void* v,
                const float* log_alpha, const float* beta, const int64_t* offsets,
                const float* initial_state, void* o, float* final_state, void* workspace,
                size_t workspace_bytes, void* stream) {
  int rc = check_config(cfg);
  if (rc == QSTATE_OK) rc = check_inputs(cfg, q, k, v, log_alpha, beta, offsets, initial_state);
  if (rc != QSTATE_OK) return rc;
  if (!o && !final_state) return QSTATE_E_INVALID;
  if (!aligned(o, cfg->dtype == QSTATE_FP32 ? 4 : 2) || !aligned(final_state, 16))
    return QSTATE_E_INVALID;
  Params p;
  if (!workspace || !aligned(workspace, 256) || layout(cfg, false, workspace, p) > workspace_bytes)
    return QSTATE_E_INVALID;
  set_inputs(p, q, k, v, log_alpha, beta, offsets, initial_state);
  p.o = o;
  p.s1 = final_state;
  // The lengths are on the device.  Without offsets they are known here.
  const int64_t most = offsets ? cfg->tokens : cfg->tokens / cfg->batch;
  p.short_len = qscan::kShort;
  p.some_short = offsets || most <= qscan::kShort;
  p.some_long = most > qscan::kShort;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (cfg->dk) {
    case 64: return status(qscan::forward_dk64(p, s));
    case 128: return status(qscan::forward_dk128(p, s));
    default: return status(qscan::forward_dk256(p, s));
  }
}

int qstate_scan_backward(const qstate_scan_config* cfg, const void* q, const void* k,
                         const void* v, const float* log_alpha, const float* beta,
                         const int64_t* offsets, const float* initial_state, const void* d_o,
                         const float* d_final_state, void* dq, void* dk, void* dv,
                         float* dlog_alpha, float* dbeta, float* d_initial_state,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_config(cfg);
  if (rc == QSTATE_OK) rc = check_inputs(cfg, q, k, v, log_alpha, beta, offsets, initial_state);
  if (rc != QSTATE_OK) return rc;
  const size_t e = cfg->dtype == QSTATE_FP32 ? 4 : 2;
  const bool beta_needed = cfg->mixer != QSTATE_GLA;
  if (cfg->tokens > 0 && (!d_o || !dq || !dk || !dv || !dlog_alpha || (beta_needed && !dbeta)))
    return QSTATE_E_INVALID;
  if (!aligned(d_o, 16) || !aligned(d_final_state, 16) || !aligned(dq, e) || !aligned(dk, e) ||
      !aligned(dv, e) || !aligned(dlog_alpha, 4) || !aligned(dbeta, 4) ||
      !aligned(d_initial_state, 16))
    return QSTATE_E_INVALID;
  Params p;
  if (!workspace || !aligned(workspace, 256) || layout(cfg, true, workspace, p) > workspace_bytes)
    return QSTATE_E_INVALID;
  set_inputs(p, q, k, v, log_alpha, beta, offsets, initial_state);
  p.dO = d_o;
  p.ds1 = d_final_state;
  p.dq = dq;
  p.dkk = dk;
  p.dv_out = dv;
  p.dg = dlog_alpha;
  p.dbeta = beta_needed ? dbeta : nullptr;
  p.ds0 = d_initial_state;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (cfg->dk) {
    case 64: return status(qscan::backward_dk64(p, s));
    case 128: return status(qscan::backward_dk128(p, s));
    default: return status(qscan::backward_dk256(p, s));
  }
}

}  // extern "C"
