/*
 * gptq_run.h -- C ABI for running and scoring a layer stored at 8 bits per
 * row, in libgptq_mi355x.so next to the calls of gptq.h (whose conventions
 * on pointers, streams, workspaces and errors hold here too).
 *
 * A layer quantized by gptq_quantize_layer on the affine grid with one group
 * per row (group = cols, bits 2..8) has codes c, one float scale w and one
 * zero point z per output row.  Activations are quantized per token when
 * they reach it, so the product runs in 8-bit integers:
 *
 *   gptq_norm_block          the residual stream: the norms after and before
 *                            a block, its gate and scales, in one pass, with
 *                            the next block's input in float or as codes
 *   gptq_quantize_tokens,    a layer's input, or silu(g) u of a gated MLP,
 *   gptq_silu_mul_quantize   as 8-bit codes with a scale per token
 *   gptq_w8a8_gemm,          the product on codes, or on float activations
 *   gptq_w8a8_linear         (quantized on the way)
 *   gptq_gated_mlp_forward   a gated MLP block made of these, in one call
 *   gptq_token_logprobs      log probabilities of given tokens from logits,
 *                            whose mean is minus the log of the perplexity
 *                            the pages quote for quantized models ("GPTQ",
 *                            section Zlozonosc obliczeniowa)
 *
 * Token-major layout: activations are tokens x features, row-major, with a
 * row stride (ld) in elements.  Unless stated, a float buffer needs only its
 * element's alignment, and any stride of at least the row's length.
 * Token counts of zero are no-ops; they go up to 2^21 where nothing else is
 * stated.  Everything is asynchronous on `stream`.
 * Each result depends on its own row's inputs alone and comes out as the
 * same bits on every call with the same sizes.
 */
#ifndef GPTQ_RUN_MI355X_H
#define GPTQ_RUN_MI355X_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation types here: GPTQ_DT_F32, GPTQ_DT_BF16 and this one. */
#define GPTQ_DT_F16 2

/* ------------------------------------------------------------ token codes
 * Row t of x becomes codes and a scale, in float32 arithmetic:
 *   a = max_k |x[t][k]|,  scale[t] = a / 127,
 *   codes[t][k] = clamp(rint(x[t][k] / scale[t]), -127, 127), half to even,
 *   sum[t] = sum_k codes[t][k].
 * A row of zeros (or one whose scale is 0 in float32) has codes 0.  A row
 * that holds a NaN or an infinity has scale NaN and codes 0, so that every
 * output the product makes of it is NaN.
 *
 *  codes   tokens x ld_codes bytes, 16-byte aligned; ld_codes >=
 *          gptq_tokens_ld(cols), a multiple of 16.  Bytes cols ..
 *          gptq_tokens_ld(cols) - 1 of each row are written as 0.
 *  scale, sum  tokens float / int32.
 */

/* Bytes of a row of codes: cols rounded up to 128 (0 unless 1 <= cols <=
 * 65536, the widest row whose products with 8-bit weights fit in int32). */
int64_t gptq_tokens_ld(int64_t cols);

gptq_status gptq_quantize_tokens(const void *x, int32_t x_dtype, int64_t tokens,
                                 int64_t cols, int64_t ld_x, int8_t *codes,
                                 int64_t ld_codes, float *scale, int32_t *sum,
                                 void *stream);

/* The same of x = silu(g) * u, silu(g) = g / (1 + e^-g) (NaN for g =
 * -infinity), which is not rounded in between.  g and u have dtype `dtype` and
 * row stride ld (they may be the two halves of one matrix). */
gptq_status gptq_silu_mul_quantize(const void *g, const void *u, int32_t dtype,
                                   int64_t tokens, int64_t cols, int64_t ld,
                                   int8_t *codes, int64_t ld_codes,
                                   float *scale, int32_t *sum, void *stream);

/* ---------------------------------------------------------- 8-bit product */

/* Host-side description of a prepared layer, filled by gptq_w8a8_prepare.
 * The caller owns the struct and `mem`; treat the fields as read-only. */
typedef struct {
  int64_t rows;      /* out features                                         */
  int64_t cols;      /* in features                                          */
  int64_t rows_pad;  /* rows rounded up to 16                                */
  int64_t k_pad;     /* cols rounded up to 128                               */
  void *mem;         /* device buffer given to gptq_w8a8_prepare             */
  size_t mem_bytes;
} gptq_w8a8_layer;

/* Bytes of device memory a prepared layer needs (0 on invalid sizes: rows in
 * [1, 2^24], cols in [1, 65536], rows_pad * k_pad <= 2^35). */
size_t gptq_w8a8_layer_bytes(int64_t rows, int64_t cols);

/*
 * Lay a per-row layer out for the product (asynchronous).
 *
 *  q      rows x cols bytes: codes in original column order.
 *  scale  rows float;  zero  rows bytes.  w^[r][c] = scale[r] (q[r][c] -
 *         zero[r]).
 *  mem    device buffer, 256-byte aligned, >= gptq_w8a8_layer_bytes;
 *         read-only for the products, which may run concurrently.
 */
gptq_status gptq_w8a8_prepare(const uint8_t *q, const float *scale,
                              const uint8_t *zero, int64_t rows, int64_t cols,
                              void *mem, size_t mem_bytes,
                              gptq_w8a8_layer *layer, void *stream);

/* Scratch bytes of gptq_w8a8_gemm and of gptq_w8a8_linear (0: none). */
size_t gptq_w8a8_gemm_ws_bytes(const gptq_w8a8_layer *layer, int64_t tokens);
size_t gptq_w8a8_linear_ws_bytes(const gptq_w8a8_layer *layer, int64_t tokens);

/*
 * y[t][r] = scale[t] * w[r] * sum_k codes[t][k] (q[r][k] - zero[r]): the sum
 * exact in int32, then one float32 product of it with scale[t] * w[r], then
 * one rounding to y's type (nearest, ties to even).
 *
 *  codes, ld_codes, scale, sum  as above, ld_codes <= 2^22, tokens <= 2^20.
 *         Bytes cols .. k_pad - 1 of a row of codes are read but do not
 *         matter.
 *  y      tokens x rows of y_dtype, row stride ld_y.
 *  ws     scratch, 256-byte aligned, >= gptq_w8a8_gemm_ws_bytes.
 */
gptq_status gptq_w8a8_gemm(const gptq_w8a8_layer *layer, const int8_t *codes,
                           int64_t ld_codes, const float *scale,
                           const int32_t *sum, int64_t tokens, void *y,
                           int32_t y_dtype, int64_t ld_y, void *ws,
                           size_t ws_bytes, void *stream);

/* The same on float activations: the outputs are those of
 * gptq_quantize_tokens followed by gptq_w8a8_gemm, bit for bit. */
gptq_status gptq_w8a8_linear(const gptq_w8a8_layer *layer, const void *x,
                             int32_t x_dtype, int64_t ld_x, int64_t tokens,
                             void *y, int32_t y_dtype, int64_t ld_y, void *ws,
                             size_t ws_bytes, void *stream);

/* -------------------------------------------------------------- norm block
 * Between two blocks of a residual network, per token (row) of width d:
 *
 *   p  = N_post(b)                    b: the output of the block before
 *   r' = residual_scale r + block_scale g . p
 *   h  = N_pre(r')                    h: the input of the block after
 *
 *   RMS:    N(v) = v / sqrt(mean(v^2) + eps) . (weight_offset + weight) + bias
 *   LAYER:  the same of v - mean(v)
 *   NONE:   N(v) = v
 *
 * in float32; r' is rounded to the stream's type where it is stored, h is
 * made from r' before that rounding.  Without b (the first block), r' =
 * residual_scale r.
 */
typedef enum {
  GPTQ_NORM_NONE = 0,
  GPTQ_NORM_RMS = 1,
  GPTQ_NORM_LAYER = 2
} gptq_norm_kind;

/* Host-side description of the two norms; the vectors are d values on the
 * device, or NULL (weight: weight_offset + weight is taken as 1; bias: 0). */
typedef struct {
  int32_t post, pre;      /* gptq_norm_kind                                  */
  int32_t w_dtype;        /* type of the four vectors                        */
  float eps;              /* >= 0                                            */
  float weight_offset;    /* 0, or 1 for weights stored as w - 1             */
  float residual_scale;
  float block_scale;
  const void *post_weight, *post_bias, *pre_weight, *pre_bias;
} gptq_norm_params;

/*
 *  dtype    type of r, b, gate, r_out and h.  1 <= d <= 32768.
 *  b        block output, or NULL (then post, gate and block_scale are not
 *           used).
 *  gate     NULL (ones), or rows of d: token t takes row t / gate_tokens
 *           (gate_tokens = tokens: one row for all; 1: one per token).
 *  r_out    r', or NULL.
 *  h        h in dtype, or NULL.
 *           Either may be r, b or gate itself (one row per token, the same
 *           stride); otherwise its rows may not overlap any of those, nor each
 *           other's: such calls are refused.
 *  codes, ld_codes, scale, sum  h as token codes, or codes NULL.
 * At least one of r_out, h and codes is given.
 */
gptq_status gptq_norm_block(const gptq_norm_params *p, int32_t dtype,
                            int64_t tokens, int64_t d, const void *r,
                            int64_t ld_r, const void *b, int64_t ld_b,
                            const void *gate, int64_t ld_gate,
                            int64_t gate_tokens, void *r_out, int64_t ld_r_out,
                            void *h, int64_t ld_h, int8_t *codes,
                            int64_t ld_codes, float *scale, int32_t *sum,
                            void *stream);

/* --------------------------------------------------------- gated MLP block
 * With an input r of the residual stream (tokens x d):
 *
 *   x = codes(N_pre(r))             enter (its pre norm, of r scaled by its
 *                                   residual_scale; leave takes r as it is)
 *   g, u = the halves of x W_gu^T   gate_up, 2 inner x d, rounded to dtype
 *   b = codes(silu(g) u) W_d^T      down, d x inner, rounded to dtype
 *   r', h                           leave, of r and b
 *
 * bit for bit what the calls above give one after the other.
 */
typedef struct {
  gptq_norm_params enter, leave;
  gptq_w8a8_layer gate_up, down;
} gptq_gated_mlp;

/* Scratch bytes (0 on invalid arguments). */
size_t gptq_gated_mlp_ws_bytes(const gptq_gated_mlp *mlp, int32_t dtype,
                               int64_t tokens);

/*
 *  dtype     type of r, gate, r_out, h and the stored intermediates.  tokens
 *            <= 2^20, d <= 32768.
 *  gate      of leave, as in gptq_norm_block.
 *  r_out, h  as there; either may be r.  At least one is given.
 *  ws        scratch, 256-byte aligned, >= gptq_gated_mlp_ws_bytes.
 * On an error r_out and h are as before; ws may have been written.
 */
gptq_status gptq_gated_mlp_forward(const gptq_gated_mlp *mlp, int32_t dtype,
                                   int64_t tokens, const void *r, int64_t ld_r,
                                   const void *gate, int64_t ld_gate,
                                   int64_t gate_tokens, void *r_out,
                                   int64_t ld_r_out, void *h, int64_t ld_h,
                                   void *ws, size_t ws_bytes, void *stream);

/* ----------------------------------------------------------------- scoring
 * Per row of logits l (with z = scale l, p = softmax(z), in float32):
 *
 *   logprob = ln p[id]     log probability of the row's given token
 *   rank    = how many entries come before the given token in the order by
 *             value, largest first, ties by lower index (0: it is the top)
 *   entropy = -sum_v p_v ln p_v
 *   top_ids, top_logprobs  the first top_k entries of that order and their
 *             log probabilities
 *
 * Entries of -infinity have probability 0 and are no alternatives: past the
 * last finite entry a row's top_ids are -1 and its top_logprobs -infinity.  A
 * row of nothing but -infinity has logprob -infinity and entropy 0.  A row
 * that holds a NaN or +infinity has NaN for every float and -1 for every
 * integer output.  id < 0 means no token is given: logprob 0, rank -1.  An
 * id >= vocab gives logprob NaN and rank -1 (nothing is read for it).
 */

/* Scratch bytes (0: none). */
size_t gptq_token_logprobs_ws_bytes(int64_t rows, int64_t vocab, int32_t top_k);

/*
 *  logits  rows x vocab of dtype, row stride ld.  1 <= vocab <= 2^24, rows <=
 *          2^23.
 *  ids     rows int64, or NULL (then logprob and rank are not written).
 *  scale   the inverse temperature, in [1e-30, 1e30].
 *  top_k   0..64 and at most vocab.
 *  logprob, rank, entropy  rows float / int32 / float, each may be NULL.
 *  top_ids, top_logprobs   rows x top_k int32 / float, not NULL for top_k >
 *          0.
 *  ws      scratch, 256-byte aligned, >= gptq_token_logprobs_ws_bytes.
 */
gptq_status gptq_token_logprobs(const void *logits, int32_t dtype, int64_t rows,
                                int64_t vocab, int64_t ld, const int64_t *ids,
                                float scale, int32_t top_k, float *logprob,
                                int32_t *rank, float *entropy, int32_t *top_ids,
                                float *top_logprobs, void *ws, size_t ws_bytes,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_RUN_MI355X_H */
