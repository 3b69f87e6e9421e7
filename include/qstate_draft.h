/*
 * qstate_draft.h — C ABI of drafted tokens over the stored recurrent state of
 * qstate.h (gfx950): a tree of them is read out without touching the state
 * (qstate_verify), and the path that was accepted enters it (qstate_accept).
 *
 * Every sequence of the batch has T rows of drafted tokens.  Row t is a node
 * with a parent: an earlier row of the same sequence, or -1, the stored state.
 * With S_p the state behind the parent, for every node and head,
 *
 *   d = S_p diag(exp(log_alpha_t))               (one gate, or one per channel)
 *   w_t = beta_t (v_t - d k_t)   GDN, KDA
 *         v_t                    GLA
 *         beta_t v_t             SCALAR
 *   S_t = d + w_t k_t^T,   o_t = S_t q_t
 *
 * with S [dv][dk] as in qstate.h: what qstate_step does token by token along
 * the node's path, without the quantization after each.  qstate_verify gives
 * o_t and w_t ("writes") of all nodes; qstate_accept replaces each sequence's
 * stored state by the one behind its last accepted node, in one quantization
 * event (as in qstate.h: rounding, scales, random bits of the given step).
 *
 * Arithmetic: FP32 state and sums; matrix products on bfloat16 matrix
 * instructions with every FP32 operand split into three bfloat16 terms (codes,
 * and bfloat16 q and k with one gate a token, need one), so that results hold
 * to FP32; o is rounded once.  Log decays are at most 0; anything below -87
 * counts as -87.  A NaN or an infinity in a node's inputs, or products of them
 * that leave FP32's range, spoil what depends on it, in that node and the nodes
 * that hang on it, and change no bit of the others; what rows of no node hold is
 * of no matter.  The same call gives the same bits.
 *
 * Layout (device memory, caller-owned); rows are [batch][T]:
 *   q, k       dtype [batch][T][heads_qk][dk], rows q_stride / k_stride
 *              elements apart (0: packed; at most 2^22); head h uses q/k head
 *              h / (heads / heads_qk)
 *   v          dtype [batch][T][heads][dv], rows v_stride apart
 *   log_alpha  float [batch][T][heads] (GDN, SCALAR) or [batch][T][heads][dk]
 *   beta       float [batch][T][heads] (not for GLA)
 *   parents    int32 [batch][T], -1 or a smaller row; any other value marks a
 *              row of no node (padding), and so are rows that hang on one.
 *              NULL: a chain, row t hangs on row t - 1
 *   o          dtype [batch][T][heads][dv], zero in rows of no node
 *   writes     float [batch][T][heads][dv], zero in rows of no node
 *   last       int32 [batch]: the last accepted node; its path is accepted.  -1
 *              (or no node): the sequence's stored state stays bit for bit
 *   codes, scales   the state as qstate_create takes it (FP32 state: codes is
 *              the state, scales is NULL)
 * Aligned to 16 bytes: q, k, log_alpha, codes, scales, writes; to their type:
 * the others.  Outputs must not overlap inputs.
 *
 * States: FP32, or quantized with value-axis groups, INT8, INT4 or both; key-axis
 * groups and pair windows are QSTATE_E_UNSUPPORTED.  Of `state` fp32_state,
 * rounding, head_bits, channel_bits, seed and layer mean what they mean in
 * qstate_create; `step` is the event's counter, which a handle of the same state
 * has (qstate_get_step) and which its user sets one higher after the call
 * (qstate_set_step).
 *
 * Calls are asynchronous on the given HIP stream, need no workspace, make no
 * allocation and no synchronisation, and can be captured into a graph (every
 * replay of an accept has the step of the capture).  The current device has to
 * be the stream's and the arrays'.  Errors: as in qstate.h; checks come before
 * any launch.
 */
#ifndef QSTATE_DRAFT_H
#define QSTATE_DRAFT_H

#include <stddef.h>
#include <stdint.h>

#include "qstate.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t tokens;   /* T: rows of a sequence, 1..64 (1..32 with dk = 256)     */
  int32_t heads_qk; /* heads of q and k; divides heads                        */
  int32_t dtype;    /* qstate_dtype of q, k, v and o                          */
  int32_t pad;      /* 0                                                      */
  int64_t q_stride, k_stride, v_stride; /* elements; 0: packed                */
} qstate_draft_config;

/* Either of o and writes may be NULL. */
int qstate_verify(const qstate_config* state, const qstate_draft_config* draft,
                  const void* codes, const float* scales, const void* q, const void* k,
                  const void* v, const float* log_alpha, const float* beta,
                  const int32_t* parents, void* o, float* writes, void* stream);

/* k, log_alpha, parents as verify had them, writes as it left them. */
int qstate_accept(const qstate_config* state, const qstate_draft_config* draft, uint64_t step,
                  void* codes, float* scales, const void* k, const float* log_alpha,
                  const int32_t* parents, const float* writes, const int32_t* last, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSTATE_DRAFT_H */
