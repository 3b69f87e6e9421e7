// linear_api.cpp — the C ABI declared in include/qstate_linear.h: argument checks.
// Host code only.

#include "qstate_linear.h"

#include <hip/hip_runtime_api.h>

#include <cstring>

#include "linear_launch.h"
#include "qstate.h"
#include "qstate_scan.h"

namespace {

using qlinear::Params;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_config(const qstate_linear_config* c) {
  if (!c || c->inputs < 1 || c->outputs < 1 || c->rows < 0) return QSTATE_E_INVALID;
  if (c->dtype < QSTATE_FP32 || c->dtype > QSTATE_FP16) return QSTATE_E_INVALID;
  if (c->group < 1 || c->inputs % c->group != 0) return QSTATE_E_INVALID;
  if (c->x_stride && c->x_stride < c->inputs) return QSTATE_E_INVALID;
  const int64_t most = (int64_t)1 << 20, far = (int64_t)1 << 40;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->inputs > most ||
      c->outputs > most || c->rows > most / 2 || c->x_stride > far)
    return QSTATE_E_UNSUPPORTED;
  // grids of 256 threads a tile, and of 64 a group of 16 outputs, stay below 2^32 threads
  const int64_t tiles = ((int64_t)c->outputs + 15) / 16 * ((c->inputs + 127) / 128);
  if (tiles > 16777215) return QSTATE_E_UNSUPPORTED;
  return QSTATE_OK;
}

void plan(const qstate_linear_config* c, Params& p) {
  std::memset(&p, 0, sizeof(p));
  p.inputs = c->inputs;
  p.outputs = c->outputs;
  p.group = c->group;
  p.dtype = c->dtype;
  p.out_tiles = (c->outputs + qlinear::kOut - 1) / qlinear::kOut;
  p.in_tiles = (c->inputs + qlinear::kIn - 1) / qlinear::kIn;
  p.rows = c->rows;
  p.xs = c->x_stride ? c->x_stride : c->inputs;
}

int status(hipError_t e) { return e == hipSuccess ? QSTATE_OK : QSTATE_E_LAUNCH; }

}  // namespace

extern "C" {

int qstate_linear_bytes(const qstate_linear_config* cfg, size_t* packed_bytes,
                        size_t* scales_bytes) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!packed_bytes || !scales_bytes) return QSTATE_E_INVALID;
  Params p;
  plan(cfg, p);
  const size_t tiles = (size_t)p.out_tiles * p.in_tiles;
  *packed_bytes = tiles * (qlinear::kOut * qlinear::kIn / 2);
  *scales_bytes = tiles * qlinear::kOut * (qlinear::kIn / cfg->group) * sizeof(float);
  return QSTATE_OK;
}

int qstate_linear_pack(const qstate_linear_config* cfg, const int8_t* codes,
                       const float* group_scales, void* packed, float* scales, void* stream) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!codes || !group_scales || !packed || !scales || !aligned(group_scales, 4) ||
      !aligned(packed, 16) || !aligned(scales, 16))
    return QSTATE_E_INVALID;
  Params p;
  plan(cfg, p);
  p.codes = codes;
  p.group_scales = group_scales;
  p.packed_out = static_cast<uint32_t*>(packed);
  p.scales_out = scales;
  return status(qlinear::pack(p, reinterpret_cast<hipStream_t>(stream)));
}

int qstate_linear_quantize(const qstate_linear_config* cfg, const void* weights, void* packed,
                           float* scales, void* stream) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  if (!weights || !packed || !scales || !aligned(weights, cfg->dtype == QSTATE_FP32 ? 4 : 2) ||
      !aligned(packed, 16) || !aligned(scales, 16))
    return QSTATE_E_INVALID;
  Params p;
  plan(cfg, p);
  p.weights = weights;
  p.packed_out = static_cast<uint32_t*>(packed);
  p.scales_out = scales;
  return status(qlinear::quantize(p, reinterpret_cast<hipStream_t>(stream)));
}

int qstate_linear(const qstate_linear_config* cfg, const void* x, const void* packed,
                  const float* scales, const float* bias, void* y, void* stream) {
  const int rc = check_config(cfg);
  if (rc != QSTATE_OK) return rc;
  const size_t e = cfg->dtype == QSTATE_FP32 ? 4 : 2;
  if (!packed || !scales || !aligned(packed, 16) || !aligned(scales, 16) || !aligned(bias, 4))
    return QSTATE_E_INVALID;
  if (!aligned(x, 16) || (cfg->x_stride * (int64_t)e) % 16 != 0 || !aligned(y, e))
    return QSTATE_E_INVALID;
  if (cfg->rows == 0) return QSTATE_OK;
  if (!x || !y) return QSTATE_E_INVALID;
  Params p;
  plan(cfg, p);
  p.x = x;
  p.packed = static_cast<const uint32_t*>(packed);
  p.scales = scales;
  p.bias = bias;
  p.y = y;
  return status(qlinear::multiply(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
