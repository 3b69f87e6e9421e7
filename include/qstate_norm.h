/*
 * qstate_norm.h — C ABI of the norms around the mixer block and their
 * gradients (gfx950).
 *
 * What a layer does with the readout o of qstate_step / qstate_scan and at the
 * block's end, in one pass over the rows.  For each row x of `width` values:
 *
 *   n = x rsqrt(mean(x^2) + eps) weight        norm after the block
 *   y = n act(gate)                            its gate: silu or sigmoid
 *   r = residual + scale y                     the residual
 *   h = r rsqrt(mean(r^2) + eps) next_weight   norm before the next block
 *
 * Every part but the first norm is left out by a null pointer: gate (y = n),
 * residual (r = scale y), scale (1), next_weight (no h).  Everything between
 * the inputs and the outputs r and h is FP32, rounded once at the end (h is
 * taken from r before r is rounded); squares of values beyond 1e19 overflow.
 * silu goes to zero below (to 2e-36, at minus infinity too) and to the gate above.
 *
 * Layout: rows are [tokens][groups]; a readout has groups = heads and
 * width = dv, a block's end groups = 1 and width the model's.
 *   x, gate, residual, r, h   dtype [tokens][groups][width]; x, gate and
 *              residual tokens x_stride / gate_stride / residual_stride
 *              elements apart (0: groups * width)
 *   weight     float [width], or [groups][width] with weight_groups = 1
 *   scale, next_weight  float [width]
 * r may be the residual's own array, and r or h may be x's own, if rows are
 * packed; otherwise outputs must not overlap inputs.  weight, scale, next_weight may be
 * NULL (1).  Row pointers are aligned to their type (16-byte aligned rows are
 * read fastest).
 *
 * Workspace (backward only): qstate_norm_workspace bytes, 256-byte aligned;
 * its contents have no meaning between calls; calls that may run at the same
 * time need one each.  Calls are asynchronous on the stream, allocate nothing
 * and can be captured into a graph; results do not depend on the order in
 * which workgroups run.  Errors: as in qstate.h.
 */
#ifndef QSTATE_NORM_H
#define QSTATE_NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QSTATE_SILU = 0, QSTATE_SIGMOID = 1 } qstate_activation;

typedef struct {
  int64_t tokens;        /* >= 0                                            */
  int32_t groups;        /* rows of a token, 1..65535                       */
  int32_t width;         /* 1..16384                                        */
  int32_t dtype;         /* qstate_dtype                                    */
  int32_t act;           /* qstate_activation of the gate                   */
  int32_t weight_groups; /* 1: weight is [groups][width]                    */
  float eps;             /* > 0, finite                                     */
  int64_t x_stride, gate_stride, residual_stride; /* elements; 0: packed    */
} qstate_norm_config;

/* r is needed unless next_weight's h is the only output wanted. */
int qstate_norm(const qstate_norm_config* cfg, const void* x, const float* weight,
                const void* gate, const void* residual, const float* scale,
                const float* next_weight, void* r, void* h, void* stream);

int qstate_norm_workspace(const qstate_norm_config* cfg, size_t* bytes);

/* Gradients from dr and dh (either may be NULL; dh only with h).  has_h says
 * that the forward call made h (next_weight may be NULL even so).  Outputs are
 * packed; any may be NULL: dx, dgate, dresidual (dtype), dweight (as weight),
 * dscale, dnext_weight (float [width]).  dgate needs gate. */
int qstate_norm_backward(const qstate_norm_config* cfg, const void* x, const float* weight,
                         const void* gate, const void* residual, const float* scale,
                         const float* next_weight, int has_h, const void* dr, const void* dh,
                         void* dx, void* dgate, void* dresidual, float* dweight, float* dscale,
                         float* dnext_weight, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSTATE_NORM_H */
