// group_norm_api.cpp — the C ABI declared in include/qstate_group_norm.h: argument
// checks and the launch plan.  Host code only.

#include "qstate_group_norm.h"

#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cstring>

#include "group_norm_launch.h"
#include "qstate.h"
#include "qstate_norm.h"
#include "qstate_scan.h"

namespace {

using qnorm::GroupParams;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem(int dtype) { return dtype == QSTATE_FP32 ? 4 : 2; }

int check_config(const qstate_group_norm_config* c) {
  if (!c || (c->shared != 0 && c->shared != 1)) return QSTATE_E_INVALID;
  if (c->tokens < 0 || c->groups < 1 || c->width < 1) return QSTATE_E_INVALID;
  if (c->dtype < QSTATE_FP32 || c->dtype > QSTATE_FP16) return QSTATE_E_INVALID;
  if (c->act != QSTATE_SILU && c->act != QSTATE_SIGMOID) return QSTATE_E_INVALID;
  if (c->mode < QSTATE_NORM_PLAIN || c->mode > QSTATE_NORM_ACTIVATE) return QSTATE_E_INVALID;
  if (c->center != 0 && c->center != 1) return QSTATE_E_INVALID;
  if (!(c->eps > 0.0f && c->eps <= FLT_MAX)) return QSTATE_E_INVALID;
  const int64_t row = (int64_t)c->groups * c->width, far = (int64_t)1 << 40;
  if ((c->x_stride && c->x_stride < row) || (c->gate_stride && c->gate_stride < row))
    return QSTATE_E_INVALID;
  if (c->groups > 65535 || c->width > 16384 || c->tokens > 2147483647 || c->x_stride > far ||
      c->gate_stride > far)
    return QSTATE_E_UNSUPPORTED;
  return QSTATE_OK;
}

bool gated(const qstate_group_norm_config* c) {
  return c->mode == QSTATE_NORM_GATE || c->mode == QSTATE_NORM_GATE_FIRST;
}

// Teams: rows of up to 512 values take 1 .. 64 lanes of a wave, 8 values a lane;
// wider ones a workgroup, 8 values a thread (16 above 8192).  As many teams as fill
// the card (256 CUs, 16 waves each; 8 waves in the backward pass left it at 64
// instead of 56 us), or one per row if there are fewer rows; a multiple of the
// groups, so that a team meets one group.
void plan(const qstate_group_norm_config* c, GroupParams& p) {
  std::memset(&p, 0, sizeof(p));
  p.rows = c->tokens * c->groups;
  p.groups = c->groups;
  p.width = c->width;
  p.act = c->act;
  p.mode = c->mode;
  p.center = c->center;
  p.shared = c->shared || c->groups == 1;
  p.eps = c->eps;
  const int64_t row = (int64_t)c->groups * c->width;
  p.xs = c->x_stride ? c->x_stride : row;
  p.gs = c->gate_stride ? c->gate_stride : row;
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
  int64_t teams = (int64_t)256 * 1024 / p.team;
  if (teams > p.rows) teams = p.rows;
  p.teams = (teams + p.groups - 1) / p.groups * p.groups;
  // parts of the weights' gradients: a team's, or a wave's where its teams share the weight
  const int64_t per = p.block / p.team;
  p.partials = !p.shared || p.wide ? p.teams : (p.teams + per - 1) / per * (p.block / 64);
}

bool rows_aligned(const void* q, int64_t stride, size_t e) {
  return aligned(q, 16) && (stride * (int64_t)e) % 16 == 0;
}

int status(hipError_t e) { return e == hipSuccess ? QSTATE_OK : QSTATE_E_LAUNCH; }

}  // namespace

extern "C" {

int qstate_group_norm(const qstate_group_norm_config* cfg, const void* x, const float* weight,
                      const float* bias, const void* gate, void* y, void* stream) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  const size_t e = elem(cfg->dtype);
  if (!aligned(x, e) || !aligned(gate, e) || !aligned(y, e) || !aligned(weight, 4) ||
      !aligned(bias, 4))
    return QSTATE_E_INVALID;
  if (!gated(cfg) && gate) return QSTATE_E_INVALID;
  if (cfg->tokens == 0) return QSTATE_OK;
  if (!x || !y || (gated(cfg) && !gate)) return QSTATE_E_INVALID;
  GroupParams p;
  plan(cfg, p);
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.gate = gate;
  p.y = y;
  p.aligned = cfg->width % 8 == 0 && rows_aligned(x, p.xs, e) && rows_aligned(gate, p.gs, e) &&
              aligned(y, 16);
  return status(qnorm::group_forward(p, cfg->dtype, reinterpret_cast<hipStream_t>(stream)));
}

int qstate_group_norm_workspace(const qstate_group_norm_config* cfg, size_t* bytes) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!bytes) return QSTATE_E_INVALID;
  GroupParams p;
  plan(cfg, p);
  *bytes = (size_t)p.partials * p.width * 2 * sizeof(float);
  return QSTATE_OK;
}

int qstate_group_norm_backward(const qstate_group_norm_config* cfg, const void* x,
                               const float* weight, const float* bias, const void* gate,
                               const void* dy, void* dx, void* dgate, float* dweight,
                               float* dbias, void* workspace, size_t workspace_bytes,
                               void* stream) {
  size_t need = 0;
  const int rc = qstate_group_norm_workspace(cfg, &need);
  if (rc != QSTATE_OK) return rc;
  const size_t e = elem(cfg->dtype);
  const void* rows[] = {x, gate, dy, dx, dgate};
  const void* floats[] = {weight, bias, dweight, dbias};
  for (const void* q : rows)
    if (!aligned(q, e)) return QSTATE_E_INVALID;
  for (const void* q : floats)
    if (!aligned(q, 4)) return QSTATE_E_INVALID;
  if (!gated(cfg) && (gate || dgate)) return QSTATE_E_INVALID;
  if (cfg->tokens > 0 && (!x || !dy || (gated(cfg) && !gate))) return QSTATE_E_INVALID;
  const bool sums = dweight || dbias;
  if (sums && need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return QSTATE_E_INVALID;
  GroupParams p;
  plan(cfg, p);
  if (!sums && p.rows == 0) return QSTATE_OK;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.gate = gate;
  p.dy = dy;
  p.dx = dx;
  p.dgate = dgate;
  p.dweight = dweight;
  p.dbias = dbias;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.aligned = cfg->width % 8 == 0 && rows_aligned(x, p.xs, e) && rows_aligned(gate, p.gs, e) &&
              aligned(dy, 16) && aligned(dx, 16) && aligned(dgate, 16);
  return status(qnorm::group_backward(p, cfg->dtype, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
