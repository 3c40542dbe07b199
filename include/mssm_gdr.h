/*
 * mssm_gdr.h -- C ABI of the gated delta rule, in the same library (libmssm.so)
 * as mssm.h: a recurrence next to the selective scan and the SSD layer whose
 * state is corrected towards each value instead of only added to.  For every
 * sequence and head, with the state S (V, K), S before the first token given or
 * zero, and the decay exp(g_t):
 *
 *     e_t = v_t - exp(g_t) S_{t-1} k_t            what the state misses of v_t
 *     S_t = exp(g_t) S_{t-1} + beta_t e_t k_tᵀ
 *     y_t = scale S_t q_t
 *
 * and, with norm_qk, q_t / sqrt(|q_t|^2 + 1e-6) and k_t / sqrt(|k_t|^2 + 1e-6) in
 * the places of q_t and k_t.  The heads of q and k may be fewer than those of v:
 * head h of v, g, beta and the state goes with head h / (heads / qk_heads) of q
 * and k.
 *
 * Conventions are those of mssm.h: row-major contiguous tensors, 16-byte
 * aligned device pointers owned by the caller, caller-owned workspace, work
 * enqueued on `hip_stream`, argument errors found on the host before anything is
 * enqueued, no allocation, no state kept between calls, no exception across the
 * ABI.  No call uses atomics; repeated calls give bitwise equal results.
 * Arithmetic is float32 or better (matrix products by exact splits of their
 * float32 operands); every output is rounded once, to nearest even.
 *
 *   q, k          (tokens, qk_heads, key_dim)    in p->dtype
 *   v, y          (tokens, heads, value_dim)     in p->dtype
 *   g, beta       (tokens, heads)                float32
 *   h0, h_final   (seqs, heads, value_dim, key_dim) float32
 *   offsets       (seqs + 1) int32: sequence n is tokens offsets[n] ..
 *                 offsets[n+1] - 1, possibly none (then h_final = h0).  NULL:
 *                 all sequences have tokens / seqs tokens.
 * g is a log decay, g <= 0: values below -200 count as -200 (exp is 0 there).
 * The products of decays are taken of differences of their float64 sums, so that
 * long sums cost no accuracy.
 * Sums of products and of squares of q and k (with norm_qk too) have to stay in
 * float32's range: lengths below 1e19.
 * Offsets have to be in ascending order within 0 .. tokens.  They are read on
 * the device, clamped to that range: others give wrong results, but no access
 * out of bounds.  Tokens that belong to no sequence are neither read nor
 * written (y and the gradients stay as they were there).
 */
#ifndef MSSM_GDR_H
#define MSSM_GDR_H

#include "mssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest key_dim and value_dim; both have to be multiples of 16. */
#define MSSM_GDR_MAX_KEY_DIM 128
#define MSSM_GDR_MAX_VALUE_DIM 512

typedef struct {
    int64_t tokens;    /* of all sequences together (mssm_gdr_step: rows), 1 .. 2^31 - 1 */
    int64_t seqs;      /* sequences (mssm_gdr_step: states in the pool), 1 .. 2^31 - 1 */
    int64_t qk_heads;  /* >= 1 */
    int64_t heads;     /* a multiple of qk_heads */
    int64_t key_dim;   /* multiple of 16, up to MSSM_GDR_MAX_KEY_DIM (else MSSM_ERR_UNSUPPORTED) */
    int64_t value_dim; /* multiple of 16, up to MSSM_GDR_MAX_VALUE_DIM (else MSSM_ERR_UNSUPPORTED) */
    int32_t dtype;     /* mssm_dtype of q, k, v, y and their gradients */
    int32_t norm_qk;   /* nonzero: q and k are divided by their lengths */
    float scale;       /* of y; finite */
} mssm_gdr_problem;

/*
 * Whole sequences, in chunks of 64 tokens as dense products on the matrix
 * cores.  Required: p, q, k, v, g, beta, y, workspace.  Optional (NULL): h0 ->
 * zeros; offsets; h_final -> not written (it may be h0's own buffer).  Without
 * offsets tokens has to be a multiple of seqs (else MSSM_ERR_SHAPE).  heads *
 * (tokens / 64 + seqs) has to be below 2^23, heads * seqs at most 2^20, heads *
 * value_dim and qk_heads * key_dim at most 2^22 (MSSM_ERR_SHAPE).  A NaN or an
 * infinity in a token spoils its chunk of 64 tokens and what follows it in its
 * sequence, in the heads that read it, and nothing else (as NaN: an infinity is cut
 * into operands, which leaves none).
 */
size_t mssm_gdr_fwd_workspace_bytes(const mssm_gdr_problem* p);

mssm_status mssm_gdr_fwd(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* offsets, void* y, float* h_final,
                         void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Training: the forward that keeps what its backward starts from in the
 * caller-owned ctx (at least mssm_gdr_ctx_bytes; contents are the library's: the
 * state before every chunk, what the state missed of every value and the chunks'
 * 64 x 64 matrices), and the gradients of sum(dy y) + sum(dh_final h_final).
 * y and h_final are those of mssm_gdr_fwd bit for bit.
 *   dq, dk (as q, k), dv (as v) in p->dtype;  dg, dbeta (as g, beta) float32;
 *   dh0 (as h0) float32, NULL -> not written;  dh_final NULL -> zeros.
 * Gradients are overwritten; those of shared heads of q and k are summed in a
 * fixed order.  mssm_gdr_bwd takes the forward's inputs (h0 among them) instead
 * of a ctx and recomputes what it would hold in its workspace.
 */
size_t mssm_gdr_ctx_bytes(const mssm_gdr_problem* p);

mssm_status mssm_gdr_fwd_train(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* h0, const int32_t* offsets, void* y, float* h_final,
                               void* ctx, size_t ctx_bytes, void* hip_stream);

size_t mssm_gdr_bwd_saved_workspace_bytes(const mssm_gdr_problem* p);

mssm_status mssm_gdr_bwd_saved(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const int32_t* offsets, const void* ctx, size_t ctx_bytes,
                               const void* dy, const float* dh_final, void* dq, void* dk, void* dv, float* dg,
                               float* dbeta, float* dh0, void* workspace, size_t workspace_bytes, void* hip_stream);

size_t mssm_gdr_bwd_workspace_bytes(const mssm_gdr_problem* p);

mssm_status mssm_gdr_bwd(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* offsets, const void* dy,
                         const float* dh_final, void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0,
                         void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * One token of every row, the recurrent form for decoding: tokens = rows, seqs =
 * states in the pool.  q, k (rows, qk_heads, key_dim), v, y (rows, heads,
 * value_dim), g, beta (rows, heads), state (seqs, heads, value_dim, key_dim) read
 * and overwritten in place.
 *   slots (rows) int32: the state of every row; NULL: row r has state r (rows <=
 *   seqs, else MSSM_ERR_SHAPE).  A row whose slot is not in 0 .. seqs - 1 is not
 *   in use: its y is 0 and no state changes.  Rows with the same slot are tokens
 *   of one sequence and go through its state in the order of the rows.
 * rows * heads has to be below 2^31, heads at most 2^20 (MSSM_ERR_SHAPE).
 */
mssm_status mssm_gdr_step(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const int32_t* slots, float* state, void* y, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MSSM_GDR_H */
