/*
 * qstate_scan.h — C ABI of the sequence forms of the recurrences in qstate.h:
 * the scan over whole sequences and its gradients (gfx950).
 *
 * qstate_step takes one token per sequence; qstate_scan takes any number of
 * them: a prompt before decoding, chunks of new tokens of running sequences,
 * or a training step.  For every sequence and head, from S_0,
 *
 *   d_t = S_{t-1} diag(exp(log_alpha_t))         (one gate, or one per channel)
 *   w_t = beta_t (v_t - d_t k_t)   GDN, KDA
 *         v_t                      GLA
 *         beta_t v_t               SCALAR
 *   S_t = d_t + w_t k_t^T,   o_t = S_t q_t
 *
 * with S [dv][dk] as in qstate.h.  Decays are given as their logarithms, at
 * most 0; minus infinity drops the state.  Anything below -87 counts as -87
 * (a factor of 1.6e-38); a value above 0 or a NaN is the caller's error and
 * only spoils its own sequence and head.
 *
 * Arithmetic: FP32 state and sums.  Matrix products run on bfloat16 matrix
 * instructions with every FP32 operand split into bfloat16 terms (hi + lo
 * ...), so that results hold to FP32 and not to bfloat16; outputs are rounded
 * once, to the type of v.  Results do not depend on the order in which the
 * device runs the workgroups: the same call gives the same bits.  A NaN or an
 * infinity in a token's inputs spoils its head of its sequence, from the start
 * of the 64-token chunk that holds it; no other head or sequence.
 *
 * Layout (device memory, caller-owned).  Sequences are packed behind each
 * other, rows are tokens:
 *   q, k       dtype [tokens][heads_qk][dk], rows q_stride / k_stride
 *              elements apart (0: heads_qk * dk; at most 2^22); head h uses q/k head
 *              h / (heads / heads_qk)
 *   v, o       dtype [tokens][heads][dv], rows v_stride / o_stride apart
 *   log_alpha  float [tokens][heads] (GDN, SCALAR) or [tokens][heads][dk]
 *   beta       float [tokens][heads] (not for GLA)
 *   offsets    int64 [batch + 1]: sequence n is rows offsets[n] ..
 *              offsets[n+1]-1; ascending, within 0 .. tokens.  NULL: batch
 *              equal sequences of tokens / batch rows.  Rows of no sequence
 *              are neither read nor written.  Offsets outside the rule are
 *              clamped: the results are then meaningless, but nothing outside
 *              the arrays is touched.
 *   initial_state, final_state  float [batch][heads][dv][dk]; NULL: zeros, or
 *              not wanted.  They may be the same array.  A sequence of no
 *              rows copies one into the other.
 * o must not overlap an input.  Aligned to 16 bytes: q, k, d_o, the gates, beta,
 * the initial and final states and their gradients; to their type: v, o and the
 * other gradients.  (Row strides of q and k that keep rows on 16 bytes are read
 * fastest.)
 *
 * Workspace: qstate_scan_workspace bytes of device memory, 256-byte aligned;
 * what it holds before and after a call is of no meaning.  Calls that may run
 * at the same time, captured graphs among them, need one each.  It grows with
 * the chunks, tokens / 64 + batch, times the heads: 40 to 230 KB for each
 * forward at dk = dv = 128, and 220 to 860 KB backward.
 *
 * Calls are asynchronous on the given HIP stream, make no allocation, no copy
 * from host memory and no synchronisation, and can be captured into a graph.
 * The current device has to be the stream's and the arrays'.
 * Errors: as in qstate.h; checks come before any launch.
 */
#ifndef QSTATE_SCAN_H
#define QSTATE_SCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QSTATE_FP32 = 0,
  QSTATE_BF16 = 1,
  QSTATE_FP16 = 2
} qstate_dtype;

typedef struct {
  int32_t batch;    /* sequences, >= 1                                        */
  int32_t heads;    /* H, 1..256: heads of v, o, the gates and the state      */
  int32_t heads_qk; /* heads of q and k; divides heads                        */
  int32_t dk;       /* 64, 128 or 256                                         */
  int32_t dv;       /* 1..4096                                                */
  int32_t mixer;    /* qstate_mixer                                           */
  int32_t dtype;    /* qstate_dtype of q, k, v, o and their gradients         */
  int32_t pad;      /* 0                                                      */
  int64_t tokens;   /* rows in all; without offsets a multiple of batch.
                       tokens / 64 + batch and (batch * heads + 8) * dv / 16
                       (dv rounded up to 32) are at most 8388607, and
                       (tokens / 64 + batch) * heads_qk at most 12582909      */
  int64_t q_stride, k_stride, v_stride, o_stride; /* elements; 0: packed      */
} qstate_scan_config;

/* Bytes of workspace for qstate_scan (backward = 0) or qstate_scan_backward
 * (backward = 1). */
int qstate_scan_workspace(const qstate_scan_config* cfg, int backward, size_t* bytes);

/* The scan.  o may be NULL (only the final state is wanted). */
int qstate_scan(const qstate_scan_config* cfg, const void* q, const void* k, const void* v,
                const float* log_alpha, const float* beta, const int64_t* offsets,
                const float* initial_state, void* o, float* final_state, void* workspace,
                size_t workspace_bytes, void* stream);

/* Gradients of a scalar of o and final_state, from d_o (dtype [tokens][heads][dv],
 * packed: o_stride is not used here) and d_final_state (NULL: zeros).  The states
 * are computed again from the inputs.  Written, each packed without row strides:
 *   dq, dk  dtype [tokens][heads_qk][dk], summed over the heads that share them
 *   dv      dtype [tokens][heads][dv]
 *   dlog_alpha  float, laid out as log_alpha;  dbeta  float (not for GLA)
 *   d_initial_state  float, or NULL
 * Gradients must not overlap the inputs or each other. */
int qstate_scan_backward(const qstate_scan_config* cfg, const void* q, const void* k,
                         const void* v, const float* log_alpha, const float* beta,
                         const int64_t* offsets, const float* initial_state, const void* d_o,
                         const float* d_final_state, void* dq, void* dk, void* dv,
                         float* dlog_alpha, float* dbeta, float* d_initial_state,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSTATE_SCAN_H */
