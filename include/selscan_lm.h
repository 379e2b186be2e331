/*
 * selscan_lm.h - C ABI of libselscan_lm: the operators that stand next to the scan of
 * selscan.h when Mamba layers serve and train a language model, as hand-written HIP kernels
 * for MI355X (gfx950):
 *   - the short causal convolution and the selective scan on packed prompts of different
 *     lengths, with each prompt's state kept in a cache, and on one token per sequence;
 *   - residual addition + root-mean-square norm, with an 8-bit output, and its gradients;
 *   - log probability of a token, entropy and top alternatives from logits, and their gradient;
 *   - a few rows times a 4-bit weight matrix with group scales;
 *   - linear attention with a decay for each head, on packed prompts and on one token per sequence;
 *   - the next token drawn from logits; entries of a cache copied, moved and freed.
 *
 * Conventions: those of selscan.h (status codes, device pointers owned by the caller, work only
 * enqueued on `stream`, nothing allocated or kept by the library, host validation before any HIP
 * call), and further:
 *  - Row-major; a `*_stride` argument is the distance between consecutive rows of that array in
 *    elements (at least the row length, SELSCAN_E_SHAPE otherwise); the elements of a row are
 *    adjacent.  Arrays without a stride argument are contiguous.
 *  - Index arrays (cu_seqlens, slots, targets) live in device memory and are read by the kernels
 *    alone.  What they hold cannot be checked on the host: a kernel never follows an index out of
 *    its array, as each call says below.
 *  - No output may overlap an input or another output unless a call says so (SELSCAN_E_ALIAS).
 *  - All sums are in a fixed order: results are the same from run to run.
 *  - A launch holds 2^32 - 1 threads along an axis, 16,777,215 workgroups of 256; calls that take more are refused
 *    (SELSCAN_E_UNSUPPORTED, before any launch).  Workgroups of 256 are: of the packed scan, 64 channels of a sequence or of one of
 *    its segments; of the packed convolution, 2,048 channels of at least 4 tokens; of the log probabilities, a row of up to 8,192
 *    logits or 4,096 and more of a longer one's; of the norm, four rows up to width 1,024, one up to 8,192 (beyond, 1,024
 *    threads each: 4,194,303 rows); of the 4-bit product, 64 rows of the matrix; of linear attention, 64 columns of a head's values of a
 *    sequence or of one of its segments, and of its step of a row (16 or 32 columns of heads that are no wider).  Sampling takes
 *    4,194,303 rows; a move of entries is counted in pieces of 16 bytes to 1 KB of an entry, of 256 to 1,024 threads.
 */
#ifndef SELSCAN_LM_H
#define SELSCAN_LM_H

#include "selscan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SELSCAN_LM_ABI_VERSION 1

/* output kinds of add_rms_norm_fwd */
typedef enum { SELSCAN_LM_OUT_IO = 0, SELSCAN_LM_OUT_INT8 = 1, SELSCAN_LM_OUT_FP8 = 2 } selscan_lm_out;

/*
 * Packed prompts.  The tokens of nseq sequences lie one after another in arrays of `tokens` rows;
 * sequence s has rows cu_seqlens[s] <= t < cu_seqlens[s+1] (int32 [nseq+1], rising, from 0 to
 * tokens; a sequence may be empty).  Offsets are clamped to [0, tokens], and a pair that falls
 * counts as an empty sequence; then, and for rows that no sequence holds, outputs are unspecified.  At most 2^31 - 2^17
 * tokens, or rows of a token step (SELSCAN_E_UNSUPPORTED).
 *
 * The cache has nslots entries.  slots[s] (int32 [nseq], NULL: slots[s] = s, which needs
 * nslots >= nseq) is the entry of sequence s; a value outside [0, nslots) means none: the sequence
 * starts from zeros and its state is not kept.  The entries of one call must differ from one
 * another (if two sequences name one, its content is unspecified).  carry[s] != 0 (uint8 [nseq],
 * NULL: all 0): the sequence continues from what its entry holds; else it starts from zeros.
 * Either way the entry then receives the state after the sequence's last token (an empty
 * sequence's: the state it starts from).
 */

/*
 * causal_conv1d_packed_fwd - causal_conv1d_fwd on packed prompts: for token t of a sequence
 *     out = act(bias[d] + sum_{i<width} weight[d][i] * x[t-(width-1)+i][d]),
 * rows before the sequence's first being its cached rows (carry) or zeros.
 *   x          : [tokens][dim] io_dtype, row stride x_stride;  out : [tokens][dim]
 *   weight     : [dim][width] fp32, width 1..4;  bias : [dim] fp32, nullable
 *   conv_state : [nslots][width-1][dim] io_dtype, nullable (no cache: slots and carry are ignored);
 *                oldest row first.  Read and written in place.
 *   flags      : SELSCAN_FLAG_SILU or 0
 */
int causal_conv1d_packed_fwd(const void *x, int64_t x_stride, const float *weight, const float *bias,
                             const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry, void *conv_state,
                             unsigned flags, void *out, int64_t tokens, int64_t nseq, int64_t nslots, int64_t dim,
                             int64_t width, int io_dtype, void *stream);

/*
 * selscan_packed_fwd - selscan_fwd on packed prompts: every sequence is scanned by itself.
 *   x, delta, z, y : [tokens][dim] io_dtype; z (nullable) has row stride z_stride
 *   B, C           : [tokens][dstate] io_dtype, both with row stride bc_stride
 *   A [dim][dstate], D, delta_bias [dim], flags : as for selscan_fwd (dstate must be 16)
 *   h_state        : [nslots][dim][dstate] fp32, 16-byte aligned, nullable (no cache); in place
 *   dim, bc_stride, z_stride : at most 2^26 (SELSCAN_E_UNSUPPORTED)
 *   max_seqlen     : the longest sequence's length, or any bound on it (tokens if unknown).  It
 *                    only chooses how the work is split and never changes what is computed.
 *   workspace      : selscan_packed_workspace_bytes(...) bytes, 16-byte aligned (0 where the
 *                    sequences alone fill the chip: NULL will do).  Where it is not 0, a sequence is
 *                    scanned in segments side by side: each segment's end state from zero, the
 *                    segments' states joined in order, then each segment from its true start.
 */
int selscan_packed_fwd(const void *x, const void *delta, const float *A, const void *B, const void *C,
                       int64_t bc_stride, const float *D, const void *z, int64_t z_stride, const float *delta_bias,
                       unsigned flags, const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry,
                       float *h_state, void *y, int64_t tokens, int64_t nseq, int64_t nslots, int64_t max_seqlen,
                       int64_t dim, int64_t dstate, int io_dtype, void *workspace, size_t workspace_bytes,
                       void *stream);
size_t selscan_packed_workspace_bytes(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t dim, int64_t dstate);

/*
 * causal_conv1d_step, selscan_step - one token for each of `rows` running sequences: the two calls
 * above with every sequence one token long, carried, and row r on cache entry slots[r] (NULL: r,
 * which needs nslots >= rows).  A row whose slot is outside [0, nslots) starts from zeros and keeps
 * nothing.
 *   x, out, delta, z, y : [rows][dim] io_dtype (x of the convolution and z with a row stride)
 *   B, C                : [rows][dstate] io_dtype, row stride bc_stride
 */
int causal_conv1d_step(const void *x, int64_t x_stride, const float *weight, const float *bias, const int32_t *slots,
                       void *conv_state, unsigned flags, void *out, int64_t rows, int64_t nslots, int64_t dim,
                       int64_t width, int io_dtype, void *stream);
int selscan_step(const void *x, const void *delta, const float *A, const void *B, const void *C, int64_t bc_stride,
                 const float *D, const void *z, int64_t z_stride, const float *delta_bias, unsigned flags,
                 const int32_t *slots, float *h_state, void *y, int64_t rows, int64_t nslots, int64_t dim,
                 int64_t dstate, int io_dtype, void *stream);

/*
 * add_rms_norm_fwd - residual addition and root-mean-square norm of each row:
 *     s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * weight
 *   x            : [rows][width] io_dtype, row stride x_stride
 *   residual     : [rows][width] residual_dtype (SELSCAN_F32, or io_dtype), nullable (s = x)
 *   residual_out : [rows][width] residual_dtype, nullable; written with s, and may be `residual`
 *                  itself.  y is formed from s before it is rounded to residual_dtype.
 *   weight       : [width] fp32
 *   out_kind, y  : SELSCAN_LM_OUT_IO: [rows][width] io_dtype; SELSCAN_LM_OUT_INT8: int8,
 *                  SELSCAN_LM_OUT_FP8: 8-bit floats (e4m3, largest value 448)
 *   scale        : [rows] fp32, written for the 8-bit outputs and required then: y stands for
 *                  scale[r] * y[r][c], scale = max|row| / 127 (/ 448), each element rounded to
 *                  nearest even.  A row of zeros (or smaller than 1e-32) has scale 0 and zeros; a row whose
 *                  mean square is not finite in fp32 has scale NaN and zeros (values past 1.8e19, which
 *                  SELSCAN_LM_OUT_IO norms as any other), and so has one whose normed row holds a NaN or an
 *                  infinity (a weight's, or a product's past fp32's range).
 *   rstd         : [rows] fp32, nullable
 *   eps          : >= 0, finite (SELSCAN_E_UNSUPPORTED); width at most 32768 (SELSCAN_E_UNSUPPORTED)
 */
int add_rms_norm_fwd(const void *x, int64_t x_stride, const void *residual, const float *weight, float eps,
                     int out_kind, void *y, void *residual_out, float *scale, float *rstd, int64_t rows, int64_t width,
                     int io_dtype, int residual_dtype, void *stream);

/*
 * add_rms_norm_bwd - gradients of add_rms_norm_fwd (SELSCAN_LM_OUT_IO).  With xhat = s * rstd and
 * g = dy * weight:
 *     ds = rstd * (g - xhat * mean(g * xhat)) + dresidual_out,  dx = dresidual = ds,
 *     dweight[c] = sum_rows dy * xhat
 *   dy             : [rows][width] io_dtype
 *   s              : [rows][width] residual_dtype, the forward's residual_out;  rstd : its rstd
 *   x              : [rows][width] io_dtype, row stride x_stride, nullable.  Given, the sum is formed anew as
 *                    x + s, with s the forward's residual instead: for a residual_out rounded to 16 bits, which is
 *                    not the sum that was normed (its rounding, up to 2^-8 of a value, would go into dweight)
 *   dresidual_out  : [rows][width] residual_dtype, nullable (no gradient through residual_out)
 *   dx             : [rows][width] io_dtype, nullable;  dresidual : [rows][width] residual_dtype,
 *                    nullable (both are ds, each in its type)
 *   dweight        : [width] fp32, nullable (written with zeros when rows == 0)
 *   workspace      : add_rms_norm_bwd_workspace_bytes(...) bytes, 16-byte aligned (per-workgroup
 *                    sums of dweight); required with dweight
 */
int add_rms_norm_bwd(const void *dy, const void *s, const void *x, int64_t x_stride, const float *weight,
                     const float *rstd, const void *dresidual_out, void *dx, void *dresidual, float *dweight,
                     int64_t rows, int64_t width, int io_dtype, int residual_dtype, void *workspace,
                     size_t workspace_bytes, void *stream);
size_t add_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t width);

/*
 * token_logprobs_fwd - from the logits of a row, with v = scale * logits and p = softmax(v):
 *     logprob = v[target] - log sum exp(v),  entropy = -sum p log p  (0 log 0 = 0),
 *     and the `top` largest logits as (log probability, index), largest first, equal ones by index
 *   logits      : [rows][vocab] io_dtype, row stride logits_stride
 *   targets     : [rows] int64; a target outside [0, vocab) gives logprob 0 (an ignored token)
 *   logprob, entropy : [rows] fp32
 *   stats       : [rows][2] fp32: the largest logit x, and log sum exp(v - scale * x); their sum, scale * x +
 *                 log sum, is the log of the softmax's denominator.  Apart, they lose nothing to the logits' size
 *                 (the gradient takes them).
 *   top         : 0..32 (SELSCAN_E_UNSUPPORTED above; no more than vocab, SELSCAN_E_SHAPE)
 *   top_logprob : [rows][top] fp32, top_index : [rows][top] int64; entries without probability
 *                 (a logit of -inf) are (-inf, -1)
 *   scale       : > 0 and at most 2.35e38 (times log2 e it is finite); vocab at most 2^21 (SELSCAN_E_UNSUPPORTED)
 * A logit of -inf has probability 0.  A row of nothing but -inf has stats -inf, logprob -inf and
 * entropy 0.  A row with a NaN or +inf has NaN for its log sum, logprob, entropy and alternatives (index -1).
 *   workspace   : token_logprobs_workspace_bytes(...) bytes, 16-byte aligned (0, and NULL will do, where a workgroup holds
 *                 a whole row: vocab at most 8192)
 */
int token_logprobs_fwd(const void *logits, int64_t logits_stride, const int64_t *targets, float scale, int top,
                       float *logprob, float *entropy, float *stats, float *top_logprob, int64_t *top_index, int64_t rows,
                       int64_t vocab, int io_dtype, void *workspace, size_t workspace_bytes, void *stream);
size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top);

/*
 * token_logprobs_bwd - gradient of sum(dlogprob * logprob + dentropy * entropy) for the logits:
 *     dlogits = scale * (dlogprob * (1[target] - p) - dentropy * p * (log p + entropy))
 *   stats, entropy : the forward's;  dlogprob, dentropy : [rows] fp32, nullable (0), not both
 *                  (SELSCAN_E_NULL)
 *   dlogits      : [rows][vocab] io_dtype, contiguous
 * The alternatives carry no gradient; an ignored target's logprob carries none.  A row of nothing
 * but -inf has gradient 0.
 */
int token_logprobs_bwd(const void *logits, int64_t logits_stride, const int64_t *targets, const float *stats,
                       const float *entropy, const float *dlogprob, const float *dentropy, float scale, void *dlogits,
                       int64_t rows, int64_t vocab, int io_dtype, void *stream);

/*
 * w4_matvec - y[r][j] = bias[j] + sum_k x[r][k] * (q[j][k] - zero[j][k / group]) * scale[j][k / group]
 *   x       : [rows][k] io_dtype, row stride x_stride
 *   qweight : [n][k / 2] bytes, 16-byte aligned: q[j][2i] in the low, q[j][2i+1] in the high 4 bits
 *             of byte i, unsigned (0..15)
 *   scales  : [n][k / group] bf16;  zeros : [n][k / group] bytes, the low 4 bits count, nullable (8)
 *   bias    : [n] fp32, nullable;  y : [rows][n] io_dtype
 *   group   : 32, 64 or 128 (SELSCAN_E_UNSUPPORTED), dividing k (SELSCAN_E_SHAPE)
 *   k at most 2^24 and x_stride at most 2^26 (SELSCAN_E_UNSUPPORTED)
 * The products and sums of a group are exact up to fp32 accumulation; fp32 x is not rounded.  An output whose sums pass
 * fp32's range on the way (an infinite x, or one above 1e37) is formed anew in 64 bits, with the infinities and NaN of the
 * formula.
 * Meant for few rows; any number is computed, 32 at a time per pass over the weights.
 */
int w4_matvec(const void *x, int64_t x_stride, const void *qweight, const void *scales, const void *zeros,
              const float *bias, void *y, int64_t rows, int64_t n, int64_t k, int64_t group, int io_dtype,
              void *stream);

/*
 * linear_attn_packed_fwd - linear attention with a decay for each head, on packed prompts (cu_seqlens, slots and carry as
 * above).  Each head has a state S [dk][dv]; for token t of a sequence
 *     S_t = exp(log_decay[t][h]) S_{t-1} + k_t v_t^T,   out[t][h] = scale * q_t^T S_t,
 * with q and k of the head's group: heads / groups heads one after another share them.
 *   q, k       : [tokens][groups][dk] io_dtype, row strides q_stride and k_stride (of a token)
 *   v          : [tokens][heads][dv] io_dtype, row stride v_stride;  out : [tokens][heads][dv], contiguous
 *   log_decay  : [tokens][heads] fp32, row stride decay_stride; decay_stride 0: one row for all tokens (a fixed decay for
 *                each head).  Usually <= 0; -infinity clears the state before the token's own product is added (the
 *                number is taken as -16384, whose exponential is 0 too).  Values above 0 make the state grow (up to 16384; beyond
 *                are taken as that): a state of 0 stays 0 however large they are, others come out as the numbers that they grow to,
 *                infinities where fp32 ends.  Where those of a block of 64 tokens (fp32: 32) add up to more than 44 it is read
 *                token by token.  (A product formed on the way, of q and k or of a value and its power, that passes fp32 comes
 *                out as an infinity or as NaN; of a state nothing is left by a power below 2^-149 within a block.)
 *                An infinity in q, k, v or a state comes out as an infinity or as NaN, from its token on.
 *   state      : [nslots][heads][dk][dv] fp32, 16-byte aligned, nullable (no cache); in place
 *   dk         : 1..256, dv : 1..1024, heads a multiple of groups (SELSCAN_E_UNSUPPORTED, SELSCAN_E_SHAPE); row strides at
 *                most 2^23 (SELSCAN_E_UNSUPPORTED)
 *   max_seqlen : the longest sequence's length, or any bound on it (tokens if unknown); speed only
 *   workspace  : linear_attn_packed_workspace_bytes(...) bytes, 16-byte aligned (0 where the heads of the sequences fill
 *                the chip: NULL will do).  Where it is not 0, a long sequence is read in segments side by side.
 */
int linear_attn_packed_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const float *log_decay, int64_t decay_stride, float scale,
                           const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry, float *state, void *out,
                           int64_t tokens, int64_t nseq, int64_t nslots, int64_t max_seqlen, int64_t heads, int64_t groups,
                           int64_t dk, int64_t dv, int io_dtype, void *workspace, size_t workspace_bytes, void *stream);
size_t linear_attn_packed_workspace_bytes(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t heads, int64_t dk,
                                          int64_t dv, int io_dtype);

/*
 * linear_attn_step - one token for each of `rows` running sequences: the call above with every sequence one token long,
 * carried, and row r on cache entry slots[r] (NULL: r, which needs nslots >= rows).  A row whose slot is outside
 * [0, nslots) starts from zeros and keeps nothing.
 */
int linear_attn_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const float *log_decay, int64_t decay_stride, float scale, const int32_t *slots, float *state,
                     void *out, int64_t rows, int64_t nslots, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                     int io_dtype, void *stream);

/*
 * token_sample - draws a token from each row of logits x, given a number u in [0, 1) for each.  With T the temperature and m
 * the row's largest logit, a token has weight exp((x - m) / T).  Of the tokens (largest logit first, equal ones by index) stay
 *     the first top_k (0: all);  of these the fewest whose weights reach top_p of their sum (1: all; at least one);
 *     and only those of weight min_p and more (the largest has weight 1).
 * The token drawn is the first of those that stay, in the order of their indices, at which the sum of weights passes u
 * times the whole.  T = 0: the largest logit.
 *   logits  : [rows][vocab] io_dtype, row stride logits_stride;  uniform : [rows] fp32
 *   temperature, top_p, min_p : [rows] fp32, top_k : [rows] int32, for each row; or NULL, and the value after it is every
 *             row's: temperature >= 0 and finite, top_k >= 0, top_p and min_p in [0, 1] (SELSCAN_E_UNSUPPORTED).  In the
 *             arrays, which the host does not see, a temperature that is not > 0 counts as 0, a top_k below 0 as 0, a top_p
 *             or min_p outside [0, 1] as the nearer end, a NaN of them as no limit.  A u outside [0, 1) counts as the nearer
 *             end, a NaN as 0.
 *   token   : [rows] int64
 *   logprob : [rows] fp32, the log of the token's weight over the weights of all that stay
 *   kept    : [rows] int32, how many tokens stay
 *   vocab   : 1..2^21 (SELSCAN_E_SHAPE, SELSCAN_E_UNSUPPORTED)
 * Weights are whole multiples of 2^-45 (for a vocab of 2^17; of 2^-62 times the vocab rounded up to a power of 2, and of 2^-51 at
 * least), summed as whole numbers: what is drawn does not depend on how a row is split.  A logit of -infinity never stays.  A
 * row of nothing else has token -1, logprob -infinity and kept 0; a row with a NaN or +infinity has token -1, logprob NaN and kept
 * 0.
 */
int token_sample(const void *logits, int64_t logits_stride, const float *uniform, const float *temperature,
                 float temperature_all, const int32_t *top_k, int top_k_all, const float *top_p, float top_p_all,
                 const float *min_p, float min_p_all, int64_t *token, float *logprob, int32_t *kept, int64_t rows,
                 int64_t vocab, int io_dtype, void *stream);

/*
 * cache_entries_copy - entry dst[i] of every one of `ncaches` caches becomes what entry src[i] was before the call, for all i
 * at once: entries are forked (one src for several dst), moved and exchanged.  A src outside [0, nslots) stands for zeros
 * (the entry is freed); a dst outside [0, nslots) is passed over.  The dst of one call must differ from one another (if two
 * are alike, that entry's content is unspecified).
 *   caches, entry_bytes : host arrays of ncaches device addresses (any alignment) and of the bytes of an entry of each; a
 *              cache is nslots entries one after another.  The caches may not overlap one another.
 *   src, dst : [n] int32, n at most 16384 (SELSCAN_E_UNSUPPORTED)
 *   entry_bytes at most 2^32; entries of all caches together within one launch (SELSCAN_E_UNSUPPORTED)
 */
int cache_entries_copy(void *const *caches, const int64_t *entry_bytes, int64_t ncaches, const int32_t *src,
                       const int32_t *dst, int64_t n, int64_t nslots, void *stream);

int selscan_lm_abi_version(void);
/* text of the calling thread's most recent launch that the HIP runtime rejected */
const char *selscan_lm_last_hip_error(void);

#ifdef __cplusplus
}
#endif
#endif
