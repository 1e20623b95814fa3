/*
 * r2l_mixer.h -- C ABI of libr2l_mixer.so (B200, sm_100a): a linear-attention mixer beside the selective
 * scans of r2l.h.  It has two operators:
 *
 *   linear attention with a fixed decay for each head -- the selective scan's recurrence with a matrix
 *   state per head, so that prompts run on the tensor cores in chunks -- over prompts and blocks
 *   (r2l_linattn), over one token of every sequence (r2l_linattn_step), and its gradients
 *   (r2l_linattn_bwd);
 *
 *   the RMS norm of each query and key head together with the rotary position embedding
 *   (r2l_qk_norm_rope), and its gradients (r2l_qk_norm_rope_bwd).
 *
 * The conventions are those of r2l.h: device pointers owned by the caller, no device memory allocated,
 * work enqueued asynchronously on `stream` of the current device, host-side argument checks before any
 * CUDA call, empty problems are no-ops, no CPU fallback, thread-safe entry points.
 */
#ifndef R2L_MIXER_H
#define R2L_MIXER_H

#include <stddef.h>

#include "r2l.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay per head.  For every sequence and every head h = 0 .. n_heads - 1, with
 * gamma = exp(log_decay[h]) and a state S [d_k][d_v] held in fp32,
 *
 *   S_t = gamma * S_(t-1) + k_t v_t^T        (forward; S_(-1) = h0, or zero)
 *   S_t = gamma * S_(t+1) + k_t v_t^T        (reverse: right to left, as r2l_scan_block)
 *   y_t = scale * q_t . S_t
 *
 *   q : [batch][seqlen][q_heads][d_k]   k : [batch][seqlen][k_heads][d_k]
 *   v : [batch][seqlen][v_heads][d_v]   y : [batch][seqlen][n_heads][d_v], dense    (all of dtype)
 *   log_decay : [n_heads] fp32, at most 0 for a decay; -inf forgets every earlier token (gamma = 0).
 *   h0, h_last: [batch][n_heads][d_k][d_v] fp32.
 *
 * q_heads, k_heads and v_heads divide n_heads; head h uses q head h / (n_heads / q_heads), and so on.
 * The head and channel dimensions are dense; q_stride, k_stride and v_stride are the elements from one
 * token to the next (0: dense), so that q, k and v may lie in one fused projection's output; a batch row
 * is seqlen such strides.
 *
 * block_len: reverse runs restart from a zero state at the right edge of every block of block_len tokens
 *   (it must divide seqlen); ignored by forward runs.
 * seq_lens: NULL, or [batch] int32 on the device: row b holds seq_lens[b] tokens (clamped to
 *   0 .. seqlen); what stands behind them is not used, y is zero there, and h_last is the state after the
 *   row's own tokens.  Reverse runs start at token seq_lens[b] - 1.  Not with blocks (block_len must be
 *   seqlen in reverse runs).
 *
 * Infinities: one in a state stays there, unless its decay over a run's tokens vanishes in fp32, and reaches the outputs as
 * the formulas say.  What an infinite k or v token leaves in a state is not finite, but bf16 runs may leave NaN where the
 * formulas give an infinity.
 *
 * Sums over nothing are zero: with n_heads, d_k or d_v 0, those outputs that are not empty all the same (y and dv
 * without key channels, dq and dk without value channels) are set to zero, or may be NULL.
 *
 * Requirements: dtype R2L_F32 or R2L_BF16; d_k and d_v at most 128 and multiples of 8 (bf16) or 4 (fp32);
 * strides multiples of 8 (bf16) or 4 (fp32) and no smaller than the token's heads; batch * seqlen less than
 * 2^31 - 256 tokens; q, k, v, y and the states 16-byte aligned.
 */
typedef struct {
    int batch, seqlen, block_len;
    int n_heads, q_heads, k_heads, v_heads;
    int d_k, d_v;
    int reverse;
    r2l_dtype dtype;
    float scale;
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const float *log_decay;
    const int *seq_lens;
} r2l_linattn_args;

/* Bytes of device workspace r2l_linattn needs (0 for many shapes). */
R2L_API size_t r2l_linattn_workspace_size(const r2l_linattn_args *a);

/*
 * Linear attention over whole sequences or blocks.
 *   h0     : cached state before the first token (in scan order), NULL = zeros.
 *   h_last : state after the last token, NULL = not written.  May be h0 itself.
 *   y      : must not overlap any input.
 * h0 and h_last need one block per row (forward, or block_len == seqlen).  `workspace`: caller-owned,
 * r2l_linattn_workspace_size bytes, 256-byte aligned (NULL when that is 0).  seqlen 0 copies h0 (or
 * zeros) to h_last.
 */
R2L_API r2l_status r2l_linattn(const r2l_linattn_args *a, const float *h0, float *h_last, void *y, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/*
 * One token of every sequence (a->seqlen 1, a->reverse 0, a->seq_lens NULL): reads the state h, writes
 * the updated one to h_out (h_out == h: in place) and y [batch][n_heads][d_v].
 */
R2L_API r2l_status r2l_linattn_step(const r2l_linattn_args *a, const float *h, float *h_out, void *y, cudaStream_t stream);

/* Bytes of device workspace r2l_linattn_bwd needs. */
R2L_API size_t r2l_linattn_bwd_workspace_size(const r2l_linattn_args *a);

/*
 * Gradients of r2l_linattn given dy = dL/dy (dtype, laid out as y) and, where the final state was used,
 * dh_last = dL/dh_last (fp32, NULL = zero).  Writes dq, dk, dv (dtype, dense, shaped as q, k, v; the
 * gradients of shared heads are summed in fp32 before they are rounded) and, unless it is NULL,
 * dh0 = dL/dh0 (fp32).  Tokens past seq_lens get zero gradients.  log_decay is a fixed schedule and
 * gets none.  Every output is overwritten and must overlap no input and no other output (dh0 being h0 or
 * dh_last is refused); no atomics, so results are the same from run to run.
 */
R2L_API r2l_status r2l_linattn_bwd(const r2l_linattn_args *a, const void *dy, const float *h0, const float *dh_last,
                                   void *dq, void *dk, void *dv, float *dh0, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream);

/*
 * Per-head RMS norm of queries and keys with the rotary position embedding, one pass:
 *
 *   z = x * rsqrt(mean(x^2) + eps) * weight             over the head's `head_dim` channels
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t)    t = positions[token] * inv_freq[i]
 *
 * for the rot_dim / 2 pairs (a, b) = channels (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved;
 * channels from rot_dim on are only normalised.  Angles are formed in fp64, so far positions keep their
 * precision; the result is rounded to dtype once.  Squares are summed in fp32: a head whose squares pass 3e38 in sum (values
 * of some 1e19) comes out as zeros.
 *
 *   q : [tokens][q_heads][head_dim], k : [tokens][k_heads][head_dim] of dtype; q_stride and k_stride as in
 *       r2l_linattn_args.  Either may have zero heads.
 *   q_weight, k_weight : [head_dim] fp32, NULL = ones.
 *   positions : [tokens], int64 when position_64 is set, else int32.   inv_freq : [rot_dim / 2] fp32.
 *       Both may be NULL when rot_dim is 0.
 * Requirements: head_dim at most 256 and even, rot_dim even and at most head_dim; q and k aligned to their
 * type.  (16-byte aligned heads whose rotated halves are whole 16-byte pieces run the wide path.)
 */
typedef struct {
    int tokens, q_heads, k_heads, head_dim, rot_dim;
    int interleaved, position_64;
    r2l_dtype dtype;
    float eps;
    const void *q, *k;
    long long q_stride, k_stride;
    const float *q_weight, *k_weight;
    const void *positions;
    const float *inv_freq;
} r2l_qk_norm_rope_args;

/*
 * q_out, k_out: dtype, with q_out_stride / k_out_stride elements from token to token (0: dense).  In place
 * (q_out == q with the same stride) is allowed; any other overlap is not.
 */
R2L_API r2l_status r2l_qk_norm_rope(const r2l_qk_norm_rope_args *a, void *q_out, long long q_out_stride, void *k_out,
                                    long long k_out_stride, cudaStream_t stream);

/* Bytes of device workspace r2l_qk_norm_rope_bwd needs (partial sums of the weight gradients). */
R2L_API size_t r2l_qk_norm_rope_bwd_workspace_size(const r2l_qk_norm_rope_args *a);

/*
 * Gradients given dq_out, dk_out (dtype, dense): dq, dk (dtype, dense, the gradients of the inputs before the
 * norm) and dq_weight, dk_weight ([head_dim] fp32, summed over tokens and heads in a fixed order; NULL = not
 * wanted).  a->q and a->k are the inputs of the forward call.  workspace: caller-owned, 256-byte aligned.
 */
R2L_API r2l_status r2l_qk_norm_rope_bwd(const r2l_qk_norm_rope_args *a, const void *dq_out, const void *dk_out, void *dq,
                                        void *dk, float *dq_weight, float *dk_weight, void *workspace,
                                        size_t workspace_bytes, cudaStream_t stream);

/* As r2l_device_status and r2l_last_error, for the kernels and calls of this library. */
R2L_API r2l_status r2l_mixer_device_status(cudaStream_t stream);
R2L_API const char *r2l_mixer_last_error(void);

/* ABI version of this header (major * 100 + minor): 100. */
R2L_API int r2l_mixer_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* R2L_MIXER_H */
