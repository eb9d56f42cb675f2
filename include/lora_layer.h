/*
 * lora_layer.h -- C ABI of the operators between the LoRA projections of a decoder layer: masked
 * attention between Q/K/V and O, the residual add with the norms before and after a block, and
 * the log probabilities of given tokens.  Forward and backward, in the same library and under the
 * same conventions as lora_mlp.h (device pointers, caller-owned buffers, asynchronous on the given
 * stream, lm_status errors found on the host before anything is enqueued, no allocation, T == 0 is
 * a no-op).  Every result is the same bits from run to run: no sum depends on an order of arrival.
 *
 * What differs from lora_mlp.h: a buffer whose rows may be strided needs 16-byte alignment where
 * that is said below (32 bytes elsewhere), and head sizes are multiples of 8.
 */
#ifndef LORA_LAYER_H
#define LORA_LAYER_H

#include "lora_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lm_dtype { LM_BF16 = 0, LM_F32 = 1 } lm_dtype;
typedef enum lm_index { LM_I32 = 0, LM_I64 = 1 } lm_index;

/* ---- attention over packed documents -----------------------------------------------------
 * For token i, head h (key/value head g = h / (hq / hk)):
 *   z_ij = scale q_i . k_j            u_ij = cap tanh(z_ij / cap)   (cap > 0; u = z for cap == 0)
 *   s_ij = u_ij - slopes[h] |i - j|   (slopes != NULL)
 *   O_i  = sum_j P_ij v_j,  P = softmax of s over the keys j that i sees,  lse_i = log sum_j exp(s_ij).
 * Token i sees token j when both are in the same document, and
 *   j <= i, or causal == 0, or j is one of the document's first prefix[] tokens, and
 *   |i - j| < window (window > 0; 0 is no window).
 * Document m holds the tokens [cu_docs[m], cu_docs[m + 1]) (cu_docs == NULL: one document, all T
 * tokens).  Tokens outside [cu_docs[0], cu_docs[n_docs]) are padding: they see nothing and nothing
 * sees them, whatever values they hold, NaN included.  A token that sees nothing has O = 0,
 * lse = -inf and adds nothing to any gradient.  cu_docs must not decrease; offsets are clamped to
 * [0, T] and a prefix to its document.  (They are device values: the host cannot check them.  With
 * other contents results are unspecified, and no access leaves its buffer.)  A NaN score makes its
 * query's weights, O and lse NaN, as does one of +inf (but capped); what they reach by the formulas is NaN.
 * A value that is not finite can besides reach tokens that see nothing of it, of its own document and of
 * documents that have a token in the same 128 (128 n to 128 n + 127): it is a factor of hidden weights too.
 *
 * q (T x hq x d), k and v (T x hk x d) bf16, hk divides hq, d a multiple of 8, at most 128.  Their
 * tokens and heads may be strided (slices of one QKV buffer, head-major layouts): strides in
 * elements, multiples of 8 and at least d, base 16-byte aligned, last dimension contiguous.
 * T <= 2^20.  O (T x hq x d) bf16 and lse (hq x T, natural logarithm) fp32 are contiguous.
 * O_lo (T x hq x d16 int8, d16 = d rounded up to 16, or NULL where no backward follows) takes the
 * next eight bits of O's fp32 pattern: fp32 bits of O = (bits of the bf16 << 16) + (O_lo << 8), to the
 * nearest, O_lo in [-128, 127].
 * The backward takes O, O_lo and lse as the forward left them and writes dQ (T x hq x d), dK and dV
 * (T x hk x d) bf16, contiguous; a key/value head's gradients are summed over its hq / hk query
 * heads in fp32.  The slopes are constants (no gradient).  P and the score gradients are rounded
 * to bf16 for the second products, as are the outputs; every sum is fp32.  dO_i . O_i cancels most of
 * dO_i . v_j where few keys matter, which is why the backward takes O with O_lo's bits (O_lo may be
 * NULL there too: the first tokens of a document then have gradients good to a per cent or two).
 * The workspace begins with the error word (lm_workspace_reset, lm_workspace_check); the same one
 * serves both calls.  Kernel families in its reports: 5 forward, 6 dK and dV, 7 dQ.
 * attn_debug_inject is a test hook like lm_debug_inject, for this thread's following calls: the
 * loaders of the masked kernels (1 forward, 2 dK and dV, 4 dQ) ask for nothing, so their waits run out
 * after wait_ns (0: the default); attn_debug_inject(0, 0) restores normal operation. */
typedef struct lm_heads {
    const uint16_t* p;
    int64_t token_stride;
    int64_t head_stride;
} lm_heads;

typedef struct lm_attn {
    float scale;            /* finite */
    float cap;              /* 0, or in [2^-14, 2^12]: a capped score's absolute error is up to 2^-21 cap */
    const float* slopes;    /* hq floats (4-byte aligned), or NULL */
    int32_t causal;
    int32_t window;         /* 0, or positive */
    const int32_t* cu_docs; /* n_docs + 1 offsets (4-byte aligned), or NULL */
    const int32_t* prefix;  /* n_docs lengths (4-byte aligned), or NULL; needs cu_docs */
    int32_t n_docs;
    int32_t reserved;
} lm_attn;

LM_API lm_status attn_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t d, size_t* bytes);
LM_API lm_status attn_debug_inject(int32_t kernel_mask, uint64_t wait_ns);
LM_API lm_status attn_fwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                          const lm_heads* v, const lm_attn* a, uint16_t* O, int8_t* O_lo, float* lse, void* ws,
                          size_t ws_bytes, lm_stream stream);
LM_API lm_status attn_bwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                          const lm_heads* v, const lm_heads* dO, const uint16_t* O, const int8_t* O_lo,
                          const float* lse, const lm_attn* a, uint16_t* dQ, uint16_t* dK, uint16_t* dV, void* ws,
                          size_t ws_bytes, lm_stream stream);

/* ---- residual add with the norms before and after a block ----------------------------------
 *   N(a; w) = a * rsqrt(mean(a^2) + eps) * (w + w_offset)     (over a row's d values)
 *   h_out = h + alpha * gate * N(y; w_post)      x = N(h_out; w_in)
 * h is the residual stream (T x d, bf16 or fp32 by h_dtype), y the block's output and x the next
 * block's input (T x d bf16); w_in, w_post and gate are d values each (bf16 or fp32 by w_dtype).
 * y == NULL: no add (h_out is not written, x = N(h; w_in); w_post and gate must be NULL).
 * w_post == NULL: y is added as it is.  gate == NULL: 1.  w_in == NULL: only the add (x is not
 * written).  rstd_y and rstd_h (T fp32) are the reciprocal roots, for the backward (each NULL when
 * its norm is missing).  d is a multiple of 32, at most 16384.
 * The backward takes the gradients dh_out (T x d, h's type; NULL: zero) and dx (T x d bf16; NULL
 * with w_in), the forward's h and y (h_out is formed again in fp32, never read back rounded) and
 * writes dh (h's type), dy (bf16; with y) and, where wanted (not NULL), the fp32 sums over the
 * tokens dw_in, dw_post and dgate (d each; of a missing vector: NULL).  eps > 0. */
typedef struct lm_addnorm {
    const void* w_in;
    const void* w_post;
    const void* gate;
    float alpha;
    float eps;
    float w_offset;
    int32_t h_dtype; /* lm_dtype */
    int32_t w_dtype; /* lm_dtype */
    int32_t reserved;
} lm_addnorm;

LM_API lm_status addnorm_workspace_size(int64_t T, int64_t d, size_t* bytes);
LM_API lm_status addnorm_fwd(int64_t T, int64_t d, const void* h, const uint16_t* y, const lm_addnorm* n, void* h_out,
                             uint16_t* x, float* rstd_y, float* rstd_h, lm_stream stream);
LM_API lm_status addnorm_bwd(int64_t T, int64_t d, const void* h, const uint16_t* y, const void* dh_out,
                             const uint16_t* dx, const float* rstd_y, const float* rstd_h, const lm_addnorm* n,
                             void* dh, uint16_t* dy, float* dw_in, float* dw_post, float* dgate, void* ws,
                             size_t ws_bytes, lm_stream stream);

/* ---- log probabilities of given tokens ------------------------------------------------------
 *   x = scale * logits   lse = log sum_j exp(x_j)   logp = x_target - lse
 *   entropy = lse - sum_j p_j x_j,  p = exp(x - lse)
 * logits (T x V, bf16 or fp32, element-aligned, row stride ld >= V), targets (T int32 or int64; a
 * target outside [0, V) is none: logp = 0 and dlogp is not used), scale > 0 (inverse temperature).
 * logp, lse and entropy (T fp32; entropy may be NULL).  k > 0 (at most 32 and at most V): top_ids
 * (T x k int32) and top_logp (T x k fp32), the row's k largest logits from the largest down, equal
 * ones by the lower index first, and their log probabilities (k == 0: both NULL).  A NaN logit
 * counts as the largest.  Logits of -inf have p = 0 and count nothing in the entropy; a row of
 * nothing else has lse = logp = top_logp = -inf, entropy 0 and gradient 0.  logp and p are formed with
 * lse as fp32 holds it: log p is off by up to 2^-24 |lse|.
 * The backward: dlogits_j = scale (dlogp (1[j = target] - p_j) - dentropy p_j (log p_j + entropy)),
 * in the logits' type (T x V, row stride ld_out >= V), from the forward's lse and entropy; dlogp and
 * dentropy T fp32, each may be NULL (zero; entropy is needed with dentropy).  dlogits may be the
 * logits themselves (ld_out == ld).  Rows that lie alike in both, modulo 16 bytes (the same stride does), are read
 * and written in vectors, others element by element, about seven times as long: a slice of a padded buffer's
 * rows wants its gradient in place, or in a buffer padded alike. */
LM_API lm_status logprob_fwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                             int32_t index, float scale, int32_t k, float* logp, float* entropy, float* lse,
                             int32_t* top_ids, float* top_logp, lm_stream stream);
LM_API lm_status logprob_bwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                             int32_t index, float scale, const float* lse, const float* entropy, const float* dlogp,
                             const float* dentropy, void* dlogits, int64_t ld_out, lm_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_LAYER_H */
