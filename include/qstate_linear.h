/*
 * qstate_linear.h — C ABI of products with 4-bit weights and group scales, for the
 * projections around the mixer while a few tokens are decoded (gfx950).
 *
 *   y = x W^T + bias,   W_nk = code_nk * scale_n,k/group
 *
 * with the state's INT4 format: codes -7 .. 7, one FP32 scale for each output and
 * `group` neighbouring inputs.  Products run on 16-bit matrix instructions, whose
 * operands hold the codes exactly; 16-bit inputs enter as they are, FP32 ones
 * split into three bfloat16 terms; sums are FP32, y is rounded once.  The same call
 * gives the same bits.  A NaN or an infinity in a row of x spoils that row of y.
 *
 * Weights are laid out once, by qstate_linear_pack or qstate_linear_quantize, into
 * two arrays of qstate_linear_bytes: tiles of 16 outputs x 128 inputs (1 KB), a
 * lane of a wave after the other: lane l holds output l % 16 and, in word i of its
 * four, inputs 32 i + 8 (l / 16) .. + 7 of the tile, input j < 4 of the eight in
 * the low nibble of byte j, j >= 4 in the high nibble of byte j - 4; a nibble is
 * the code's sign (bit 3) and size.  Scales: for each tile [16][128 / group].
 * Outputs and inputs behind the last are zeros.
 *
 * Layout: x  dtype [rows][inputs], rows x_stride elements apart (0: packed);
 * y  dtype [rows][outputs], packed; bias  float [outputs] or NULL.  Aligned to 16
 * bytes: x (each row), packed, scales; to their type: the others.  y must not
 * overlap an input.
 *
 * Calls are asynchronous on the given HIP stream, need no workspace, make no
 * allocation and no synchronisation, and can be captured into a graph.  The
 * current device has to be the stream's and the arrays'.  Errors: as in qstate.h;
 * checks come before any launch.
 */
#ifndef QSTATE_LINEAR_H
#define QSTATE_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t inputs;   /* a multiple of group, at most 2^20                       */
  int32_t outputs;  /* 1 .. 2^20                                               */
  int32_t group;    /* 32, 64 or 128                                           */
  int32_t dtype;    /* qstate_dtype of x and y                                 */
  int64_t rows;     /* of x; >= 0, at most 2^19.  Meant for few: every 16 rows read
                       the weights again, from the caches as far as they hold, and
                       widen them again: beyond about 100 rows a dense bfloat16
                       product takes less time (4096 rows times 4096 x 4096: 496 us,
                       dense 94)                                                */
  int64_t x_stride; /* elements; 0: packed                                     */
} qstate_linear_config;

/* Sizes of the packed codes and of the packed scales. */
int qstate_linear_bytes(const qstate_linear_config* cfg, size_t* packed_bytes,
                        size_t* scales_bytes);

/* codes int8 [outputs][inputs] (beyond -7 .. 7: cut), group_scales float
 * [outputs][inputs / group]; cfg's dtype, rows and x_stride do not matter. */
int qstate_linear_pack(const qstate_linear_config* cfg, const int8_t* codes,
                       const float* group_scales, void* packed, float* scales, void* stream);

/* Quantizes weights (dtype [outputs][inputs], packed) as the state is: scale = the
 * group's largest magnitude / 7, codes to nearest, ties to even. */
int qstate_linear_quantize(const qstate_linear_config* cfg, const void* weights, void* packed,
                           float* scales, void* stream);

int qstate_linear(const qstate_linear_config* cfg, const void* x, const void* packed,
                  const float* scales, const float* bias, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSTATE_LINEAR_H */
