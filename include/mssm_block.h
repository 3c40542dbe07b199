/*
 * mssm_block.h -- C ABI of the operators that serve a Mamba block around its
 * scan, in the same library (libmssm.so) as mssm.h: the residual addition with
 * its root-mean-square norm, the projections with their epilogue, and one
 * beam-search step over the logits with the reordering of the recurrent and
 * convolution states.  Forward only: these are the operators of serving.
 *
 * Conventions are those of mssm.h: row-major contiguous tensors, 16-byte
 * aligned device pointers owned by the caller, caller-owned workspace, work
 * enqueued on `hip_stream`, argument errors found on the host before anything
 * is enqueued, no allocation, no state kept between calls, no exception across
 * the ABI.  No call uses atomics; repeated calls give bitwise equal results.
 * Arithmetic is float32 (products of 8-bit and bfloat16 operands are summed in
 * float32 on the matrix cores; 8-bit operands with a bfloat16 output are the
 * exception that mssm_linear names); every output is rounded once, to nearest
 * even.
 */
#ifndef MSSM_BLOCK_H
#define MSSM_BLOCK_H

#include "mssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit element type of mssm_linear's operands and of mssm_add_rmsnorm_q8's
 * output, next to MSSM_F32 and MSSM_BF16: OCP e4m3 (torch.float8_e4m3fn; 4
 * exponent bits, 3 mantissa bits, largest value 448, no infinities). */
#define MSSM_F8 2

/*
 * Residual addition and root-mean-square norm of every row:
 *
 *     h = x + residual                       (h = x without a residual)
 *     residual_out = h
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *
 *   x, y                    (rows, dim) in p->dtype (MSSM_F32 or MSSM_BF16)
 *   residual, residual_out  (rows, dim) in p->residual_dtype (either type)
 *   weight                  (dim) float32
 * The norm is taken of the float32 sum, not of its rounded copy, and the squares
 * are float32: a row with |h| beyond about 1e19 gives 0, and with eps = 0 a row
 * of magnitudes below 1e-19 is not normalised (a row of zeros is 0 / 0, NaN);
 * 8-bit rows take h * weight within float32's range as well.  Required: x,
 * weight, y.  Optional (NULL): residual; residual_out -> not written.
 * residual_out may be the residual's own buffer, and y may be x's.
 */
typedef struct {
    int64_t rows;           /* >= 1, below 2^31 */
    int64_t dim;            /* >= 1, below 2^24 */
    int32_t dtype;          /* mssm_dtype of x and y */
    int32_t residual_dtype; /* mssm_dtype of residual and residual_out */
    float eps;              /* >= 0 */
} mssm_norm_problem;

mssm_status mssm_add_rmsnorm(const mssm_norm_problem* p, const void* x, const void* residual, const float* weight,
                             void* y, void* residual_out, void* hip_stream);

/*
 * The same with y in 8 bits and one scale a row, as mssm_linear takes it:
 *
 *     scale[row] = max(max |y|, 1e-30) / 448,   q = e4m3(y / scale[row])
 *
 *   q (rows, dim) bytes, scale (rows) float32, both required.
 * A row of zeros gives q = 0 and the scale 1e-30 / 448, with eps = 0 too.  A row that holds a NaN
 * or an infinity gives NaN in all of q and in its scale.
 */
mssm_status mssm_add_rmsnorm_q8(const mssm_norm_problem* p, const void* x, const void* residual,
                                const float* weight, void* q, float* scale, void* residual_out, void* hip_stream);

/*
 * Projection with its epilogue (the weight laid out as torch.nn.Linear's):
 *
 *     y[m,n] = act(sum_k x[m,k] w[n,k] * x_scale[m] * w_scale[n] + bias[n]) + residual[m,n]
 *
 *   x (rows, in_dim), w (out_dim, in_dim)  in p->dtype: MSSM_F32, MSSM_BF16 or MSSM_F8
 *   x_scale (rows), w_scale (out_dim)      float32, required with MSSM_F8, NULL otherwise
 *   bias (out_dim) float32                 NULL -> 0
 *   residual (rows, out_dim)               in p->out_dtype, NULL -> 0
 *   y (rows, out_dim)                      in p->out_dtype: MSSM_F32, or MSSM_BF16 (not with
 *                                          MSSM_F32 operands)
 * 8-bit operands with a bfloat16 output go through the 8-bit matrix
 * instructions, twice as fast as bfloat16's, which cut each product towards zero
 * at about 2^-13 of the largest of the eight that they add first: the sum is
 * within 2^-10 sum |x w| (typically 1.5e-5 of the sum itself, up to 1e-4 where
 * wide channels of x and w meet), which a bfloat16 rounding hides unless the sum
 * cancels or the residual cancels it.  For such sums ask for MSSM_F32: the
 * operands are then widened, which is exact, and summed in float32.
 * y may be the residual's own buffer, and no other input's.  Few output tiles
 * and a long in_dim are cut along in_dim: the workspace then holds the partial
 * sums (float32), which a second pass adds in a fixed order.
 */
typedef enum {
    MSSM_ACT_NONE = 0,
    MSSM_ACT_RELU = 1,
    MSSM_ACT_SILU = 2, /* v / (1 + exp(-v)) */
    MSSM_ACT_GELU = 3  /* v / 2 (1 + erf(v / sqrt 2)) */
} mssm_activation;

typedef struct {
    int64_t rows;       /* >= 1, below 2^31 */
    int64_t in_dim;     /* >= 1, below 2^20 */
    int64_t out_dim;    /* >= 1, below 2^31 */
    int32_t dtype;      /* type of x and w */
    int32_t out_dtype;  /* type of y and residual */
    int32_t activation; /* mssm_activation */
} mssm_linear_problem;

/* Bytes of device scratch mssm_linear needs on the current device (0: none, or an invalid problem). */
size_t mssm_linear_workspace_bytes(const mssm_linear_problem* p);

mssm_status mssm_linear(const mssm_linear_problem* p, const void* x, const float* x_scale, const void* w,
                        const float* w_scale, const float* bias, const void* residual, void* y,
                        void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * One selection of beam search: of the beams * vocab continuations of every
 * batch row,
 *
 *     value[k,v] = scores[k] + ((x - max x) - log(sum exp(x - max x))),   x = logits[k, v],
 *
 * the `beams` best, in descending order; equal values go to the lowest
 * k * vocab + v.  (Where rounding makes the values of one beam equal, its
 * logits are compared first when the beam's own best are taken.)
 *   logits (batch, beams, vocab) in p->dtype;  scores, scores_out (batch, beams) float32
 *   finished, finished_out (batch, beams) bytes, 0 or 1
 *   parent, token (batch, beams) int32: the beam that is continued, and its next token
 * A logit of -infinity bans its token (value -infinity, and so has every token
 * of a beam whose logits are all banned); NaN bans it too; +infinity counts as
 * the largest finite float32.  A score that is NaN or +infinity counts as
 * -infinity (a beam that is not in use).  A finished beam has one
 * continuation, p->end_token at its unchanged score.
 * finished_out = finished of the parent, or token == end_token.
 * Required: logits, scores, scores_out, parent, token, workspace.  Optional
 * (NULL): finished -> none is; finished_out -> not written.  scores_out may be
 * scores, and finished_out may be finished.
 */
#define MSSM_MAX_BEAMS 16

typedef struct {
    int64_t batch;     /* >= 1, batch * beams below 2^31 */
    int64_t beams;     /* 1 .. MSSM_MAX_BEAMS (else MSSM_ERR_UNSUPPORTED) */
    int64_t vocab;     /* >= 1, below 2^27 */
    int32_t dtype;     /* MSSM_F32 or MSSM_BF16 */
    int32_t end_token; /* 0 .. vocab - 1; -1: none (then finished must be NULL) */
} mssm_beam_problem;

size_t mssm_beam_select_workspace_bytes(const mssm_beam_problem* p);

mssm_status mssm_beam_select(const mssm_beam_problem* p, const void* logits, const float* scores,
                             const uint8_t* finished, float* scores_out, int32_t* parent, int32_t* token,
                             uint8_t* finished_out, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * The beams' states follow their parents, in place and in one launch for up to
 * MSSM_MAX_BEAM_STATES tensors: for every layer l, batch row b and beam k
 *
 *     data[l][b * beams + k] = data[l][b * beams + parent[b][k]]   (the old contents)
 *
 * Beams that stay where they are (parent[b][k] == k) are neither read nor
 * written for themselves.  data: (layers, batch * beams, bytes), e.g. the
 * recurrent states (layers, batch * beams, D, N) float32 and the convolution
 * states (layers, batch * beams, d_conv - 1, D) of mssm_conv_step; 16-byte
 * aligned, bytes any number.  The tensors may not overlap.  A parent outside
 * 0 .. beams - 1 leaves its beam as it is.
 */
#define MSSM_MAX_BEAM_STATES 16

typedef struct {
    void* data;
    int64_t layers; /* >= 1 */
    int64_t bytes;  /* of one beam's state in one layer, >= 1, below 2^31 */
} mssm_beam_state;

mssm_status mssm_beam_reorder(int64_t batch, int64_t beams, const int32_t* parent, int32_t count,
                              const mssm_beam_state* states, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MSSM_BLOCK_H */
