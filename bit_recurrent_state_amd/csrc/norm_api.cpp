// norm_api.cpp — the C ABI declared in include/qstate_norm.h: argument checks
// and the launch plan.  Host code only.

#include "qstate_norm.h"

#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cstring>

#include "norm_launch.h"
#include "qstate.h"
#include "qstate_scan.h"

namespace {

using qnorm::Params;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem(int dtype) { return dtype == QSTATE_FP32 ? 4 : 2; }

int check_config(const qstate_norm_config* c) {
  if (!c) return QSTATE_E_INVALID;
  if (c->tokens < 0 || c->groups < 1 || c->width < 1) return QSTATE_E_INVALID;
  if (c->dtype < QSTATE_FP32 || c->dtype > QSTATE_FP16) return QSTATE_E_INVALID;
  if (c->act != QSTATE_SILU && c->act != QSTATE_SIGMOID) return QSTATE_E_INVALID;
  if (c->weight_groups != 0 && c->weight_groups != 1) return QSTATE_E_INVALID;
  if (!(c->eps > 0.0f && c->eps <= FLT_MAX)) return QSTATE_E_INVALID;
  const int64_t row = (int64_t)c->groups * c->width, far = (int64_t)1 << 40;
  if ((c->x_stride && c->x_stride < row) || (c->gate_stride && c->gate_stride < row) ||
      (c->residual_stride && c->residual_stride < row))
    return QSTATE_E_INVALID;
  if (c->groups > 65535 || c->width > 16384 || c->tokens > 2147483647 || c->x_stride > far ||
      c->gate_stride > far || c->residual_stride > far)
    return QSTATE_E_UNSUPPORTED;
  return QSTATE_OK;
}

// Teams: rows of up to 512 values take 1 .. 64 lanes of a wave, 8 values a
// lane; wider ones a workgroup, 8 values a thread (16 above 8192).  As many
// teams as fill the card (256 CUs, 16 waves each forward, 8 backward, as the
// registers allow), or one per row if there are fewer rows.  With a
// weight for each group their number is a multiple of the groups, so that a
// team meets one group only.
void plan(const qstate_norm_config* c, bool backward, Params& p) {
  std::memset(&p, 0, sizeof(p));
  p.rows = c->tokens * c->groups;
  p.groups = c->groups;
  p.width = c->width;
  p.act = c->act;
  p.each = c->weight_groups;
  p.eps = c->eps;
  const int64_t row = (int64_t)c->groups * c->width;
  p.xs = c->x_stride ? c->x_stride : row;
  p.gs = c->gate_stride ? c->gate_stride : row;
  p.rs = c->residual_stride ? c->residual_stride : row;
  p.wide = c->width > 512;
  p.vectors = c->width > 8192 ? 2 : 1;
  if (p.wide) {
    p.block = 128;
    while (p.block * 8 < c->width && p.block < 1024) p.block *= 2;
    p.team = p.block;
  } else {
    p.block = 256;
    p.team = 1;
    while (p.team * 8 < c->width) p.team *= 2;
  }
  int64_t teams = (int64_t)256 * (backward ? 512 : 1024) / p.team;
  if (teams > p.rows) teams = p.rows;
  if (p.each) teams = (teams + p.groups - 1) / p.groups * p.groups;
  p.teams = teams;
  // parts of the weights' gradients: a team's, or a wave's where its teams share the weight
  const int64_t per = p.block / p.team;
  p.partials = p.each || p.wide ? teams : (teams + per - 1) / per * (p.block / 64);
}

bool rows_aligned(const void* q, int64_t stride, size_t e) {
  return aligned(q, 16) && (stride * (int64_t)e) % 16 == 0;
}

}  // namespace

extern "C" {

int qstate_norm(const qstate_norm_config* cfg, const void* x, const float* weight,
                const void* gate, const void* residual, const float* scale,
                const float* next_weight, void* r, void* h, void* stream) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  const size_t e = elem(cfg->dtype);
  if (cfg->tokens > 0 && (!x || (!r && !h) || (next_weight && !h))) return QSTATE_E_INVALID;
  if (!aligned(x, e) || !aligned(gate, e) || !aligned(residual, e) || !aligned(r, e) ||
      !aligned(h, e) || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(next_weight, 4))
    return QSTATE_E_INVALID;
  Params p;
  plan(cfg, false, p);
  if (p.rows == 0) return QSTATE_OK;
  p.x = x;
  p.weight = weight;
  p.gate = gate;
  p.residual = residual;
  p.scale = scale;
  p.next_weight = next_weight;
  p.r = r;
  p.h = h;
  p.has_h = h != nullptr;
  p.aligned = cfg->width % 8 == 0 && rows_aligned(x, p.xs, e) && rows_aligned(gate, p.gs, e) &&
              rows_aligned(residual, p.rs, e) && aligned(r, 16) && aligned(h, 16);
  return qnorm::forward(p, cfg->dtype, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QSTATE_OK
             : QSTATE_E_LAUNCH;
}

int qstate_norm_workspace(const qstate_norm_config* cfg, size_t* bytes) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!bytes) return QSTATE_E_INVALID;
  Params p;
  plan(cfg, true, p);
  *bytes = (size_t)p.partials * p.width * 3 * sizeof(float);
  return QSTATE_OK;
}

int qstate_norm_backward(const qstate_norm_config* cfg, const void* x, const float* weight,
                         const void* gate, const void* residual, const float* scale,
                         const float* next_weight, int has_h, const void* dr, const void* dh,
                         void* dx, void* dgate, void* dresidual, float* dweight, float* dscale,
                         float* dnext_weight, void* workspace, size_t workspace_bytes,
                         void* stream) {
  size_t need = 0;
  const int rc = qstate_norm_workspace(cfg, &need);
  if (rc != QSTATE_OK) return rc;
  const size_t e = elem(cfg->dtype);
  if (has_h != 0 && has_h != 1) return QSTATE_E_INVALID;
  if ((cfg->tokens > 0 && !x) || (dgate && !gate) || (!has_h && (dh || next_weight || dnext_weight)))
    return QSTATE_E_INVALID;
  const bool sums = dweight || dscale || dnext_weight;
  if (sums && need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return QSTATE_E_INVALID;
  const void* rows[] = {x, gate, residual, dr, dh, dx, dgate, dresidual};
  const void* floats[] = {weight, scale, next_weight, dweight, dscale, dnext_weight};
  for (const void* q : rows)
    if (!aligned(q, e)) return QSTATE_E_INVALID;
  for (const void* q : floats)
    if (!aligned(q, 4)) return QSTATE_E_INVALID;
  Params p;
  plan(cfg, true, p);
  p.x = x;
  p.weight = weight;
  p.gate = gate;
  p.residual = residual;
  p.scale = scale;
  p.next_weight = next_weight;
  p.has_h = has_h;
  p.dr = dr;
  p.dh = dh;
  p.dx = dx;
  p.dgate = dgate;
  p.dresidual = dresidual;
  p.dweight = dweight;
  p.dscale = dscale;
  p.dnext_weight = dnext_weight;
  if (!sums && p.rows == 0) return QSTATE_OK;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.aligned = cfg->width % 8 == 0 && rows_aligned(x, p.xs, e) && rows_aligned(gate, p.gs, e) &&
              rows_aligned(residual, p.rs, e);
  for (int i = 3; i < 8; ++i) p.aligned = p.aligned && aligned(rows[i], 16);
  return qnorm::backward(p, cfg->dtype, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QSTATE_OK
             : QSTATE_E_LAUNCH;
}

}  // extern "C"
