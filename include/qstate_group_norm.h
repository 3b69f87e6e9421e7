/*
 * qstate_group_norm.h — C ABI of the group norm of a mixer's readout, with its
 * activation or gate, and of its gradients (gfx950).
 *
 * Channels are last: a token has groups * width of them, and every group of
 * `width` neighbouring channels of a token is normalised by itself (statistics
 * never reach over tokens, which would let a token see later ones):
 *
 *   u = x act(gate)                        gate before the norm, else u = x
 *   c = (u - mean(u)) rsqrt(var(u) + eps)  centered, else u rsqrt(mean(u^2) + eps)
 *   n = c weight + bias
 *   y = n act(gate)                        gate after the norm
 *       n act(n) / n, i.e. silu(n) or sigmoid(n)   activated
 *       n                                  otherwise
 *
 * which is the readout of a retention layer (centered, a gate after), of a
 * Mamba2 block (not centered, the gate before), and a norm with its activation.
 * Everything between x, gate and y is FP32, rounded once at the end (an
 * activation at z that goes into a 16-bit y is off by up to |z| 2^-23 of its
 * value before that); dweight and dbias hold to FP32 whatever x's type; the
 * variance is taken from the centered values.  Squares of values beyond 1e19
 * overflow.  silu goes to zero below (to 2e-36, at minus infinity too) and to its
 * argument above.  A NaN or an infinity spoils its group of its token (and the sums of
 * dweight and dbias that it enters).
 *
 * Layout: x, gate, y  dtype [tokens][groups * width], x and gate tokens
 * x_stride / gate_stride elements apart (0: packed); weight, bias  float
 * [groups * width], or [width] with shared = 1; NULL: 1 and 0.  y may be x's or the gate's own array if rows
 * are packed; otherwise outputs must not overlap inputs.  Pointers are aligned
 * to their type (16-byte aligned rows are read fastest).
 *
 * Workspace (backward only): qstate_group_norm_workspace bytes, 256-byte aligned;
 * its contents have no meaning between calls; calls that may run at the same
 * time need one each.  Calls are asynchronous on the stream, allocate nothing
 * and can be captured into a graph; the same call gives the same bits.
 * Errors: as in qstate.h.
 */
#ifndef QSTATE_GROUP_NORM_H
#define QSTATE_GROUP_NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QSTATE_NORM_PLAIN = 0,      /* no gate, no activation       */
  QSTATE_NORM_GATE = 1,       /* y = n act(gate)              */
  QSTATE_NORM_GATE_FIRST = 2, /* the norm of x act(gate)      */
  QSTATE_NORM_ACTIVATE = 3    /* y = silu(n) or sigmoid(n)    */
} qstate_norm_mode;

typedef struct {
  int64_t tokens;        /* >= 0                                            */
  int32_t groups;        /* 1..65535                                        */
  int32_t width;         /* channels of a group, 1..16384                   */
  int32_t dtype;         /* qstate_dtype                                    */
  int32_t act;           /* qstate_activation                               */
  int32_t mode;          /* qstate_norm_mode                                */
  int32_t center;        /* 1: centered                                     */
  float eps;             /* > 0, finite                                     */
  int32_t shared;        /* 1: weight and bias are [width], the same for all groups */
  int64_t x_stride, gate_stride; /* elements; 0: packed                     */
} qstate_group_norm_config;

int qstate_group_norm(const qstate_group_norm_config* cfg, const void* x, const float* weight,
                      const float* bias, const void* gate, void* y, void* stream);

int qstate_group_norm_workspace(const qstate_group_norm_config* cfg, size_t* bytes);

/* Gradients from dy (dtype, packed).  Outputs are packed; any may be NULL: dx,
 * dgate (dtype; dgate needs a gate), dweight, dbias (as weight and bias). */
int qstate_group_norm_backward(const qstate_group_norm_config* cfg, const void* x,
                               const float* weight, const float* bias, const void* gate,
                               const void* dy, void* dx, void* dgate, float* dweight,
                               float* dbias, void* workspace, size_t workspace_bytes,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSTATE_GROUP_NORM_H */
