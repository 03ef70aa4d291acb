/*
 * gs_head.h -- the feature-head calls of libgs_splat_gb300.so: what follows a
 * render of feature channels (gs_rasterize_fwd with up to GS_MAX_CHANNELS
 * channels) in a network that is trained through it.
 *   gs_layer_norm_fwd / _bwd       layer norm over the channels of each row
 *   gs_expert_sort                 (token, choice) pairs sorted by expert
 *   gs_expert_dispatch             rows copied into expert order
 *   gs_expert_combine / _bwd       rows summed back with their weights
 *   gs_expert_linear_fwd / _bwd    every expert's matrix product
 *   gs_expert_route_fwd / _bwd     the choice of experts, its weights, the
 *                                  experts' counts and the balance loss
 *   gs_rows_pack8 / gs_rows_unpack8  rows kept in 8 bits, and back
 *   gs_expert_linear8_fwd / _bwd   the experts' products of 8-bit rows
 * A row is one pixel's (token's) channels.  No counterpart on the pages of
 * gs_splat.h; the formulas stand at each call.
 *
 * The conventions of gs_splat.h hold (device pointers, stream, workspace,
 * status codes, nothing allocated).  In addition:
 *   - `dtype` names the element type of the `void*` arrays.  Sums, statistics
 *     and products are accumulated in float32 whatever the type, and each
 *     output is rounded to its type once.
 *   - `ld...` is the distance in elements between the starts of two rows
 *     (>= channels): a channel slice of a wider image is read or written in
 *     place.  Arrays without one are contiguous.
 *   - Outputs do not overlap inputs, and no row of an output another row.
 *   - Results do not depend on the run: no floating-point atomics.
 *   - d_status receives GS_ERR_TIMEOUT from a product whose wait ran out (two
 *     seconds on what takes microseconds; part of its output is then
 *     unwritten).  With NULL nothing tells.
 *   - An index read from a device array (a slot, an offset) that lies outside
 *     its array is treated as -1 or clamped; the range-checking build also
 *     reports GS_ERR_OUT_OF_BOUNDS in d_status.
 */
#ifndef GS_HEAD_H
#define GS_HEAD_H

#include "gs_splat.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gs_dtype {
    GS_F32 = 0,
    GS_F16 = 1,
    GS_BF16 = 2
} gs_dtype;

/* Most channels of a normalised row, and most experts and choices a token. */
#define GS_MAX_NORM_CHANNELS 16384
#define GS_MAX_EXPERTS 1024
#define GS_MAX_TOPK 64
/* Most rows of the experts' products: the kernels number rows in 32 bits, to
 * the end of a tile of 256. */
#define GS_MAX_EXPERT_ROWS 2147483392

/* 8-bit rows: an element is q * 2^(byte - 127), q in e4m3 (1.4.3 bits, no
 * infinity, largest 448) and one byte (e8m0; 255 is a NaN) for each
 * GS_SCALE_BLOCK channels.  A row's elements take GS_ROW8_BYTES bytes, zeros
 * behind the last channel, its scale bytes GS_ROW8_SCALES, zeros behind the
 * last block; rows follow each other.  The elements begin on a 16-byte
 * boundary, the scale bytes on a 4-byte one. */
#define GS_SCALE_BLOCK 128
#define GS_ROW8_BYTES(channels) (((channels) + 15) / 16 * 16)
#define GS_ROW8_SCALES(channels) (((channels) + 511) / 512 * 4)

/*
 * gs_layer_norm_fwd -- per row of x (rows, channels):
 *   mean = sum(x) / channels,  var = sum((x - mean)^2) / channels,
 *   rstd = 1 / sqrt(var + eps),  y = (x - mean) * rstd * weight + bias.
 * weight, bias (channels), of param_dtype: GS_F32 or dtype; NULL = 1 and 0.
 * mean, rstd float32 (rows): outputs for the backward, or both NULL.
 * y (rows, channels) of dtype, row distance ldy.
 * Limits: rows >= 0, 1 <= channels <= GS_MAX_NORM_CHANNELS, eps >= 0.
 */
int gs_layer_norm_fwd(const void* x, int64_t ldx, const void* weight, const void* bias,
                      int64_t rows, int channels, int dtype, int param_dtype, float eps,
                      void* y, int64_t ldy, float* mean, float* rstd, void* stream);

/* Bytes of workspace gs_layer_norm_bwd needs for the gradients of weight and
 * bias (0 when neither is asked for). */
size_t gs_layer_norm_bwd_workspace_size(int64_t rows, int channels);

/*
 * gs_layer_norm_bwd -- with xh = (x - mean) * rstd and g = grad_y * weight:
 *   grad_x = rstd * (g - sum(g) / channels - xh * sum(g * xh) / channels)
 *   grad_weight = sum over rows of grad_y * xh,  grad_bias = that of grad_y
 * mean, rstd: as gs_layer_norm_fwd wrote them.  Each of grad_x (dtype, row
 * distance ldgx), grad_weight and grad_bias (param_dtype) may be NULL; the
 * workspace is needed with one of the last two.  rows = 0 gives zero
 * grad_weight and grad_bias.
 */
int gs_layer_norm_bwd(const void* grad_y, int64_t ldgy, const void* x, int64_t ldx,
                      const void* weight, const float* mean, const float* rstd, int64_t rows,
                      int channels, int dtype, int param_dtype, void* grad_x, int64_t ldgx,
                      void* grad_weight, void* grad_bias, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Bytes of workspace gs_expert_sort needs (0 for a few thousand pairs). */
size_t gs_expert_sort_workspace_size(int64_t tokens, int topk, int experts);

/*
 * gs_expert_sort -- the (token, choice) pairs i = t * topk + j sorted by
 * expert, equal experts in order of i.
 * expert_ids int32 (tokens, topk); an id outside [0, experts) drops its pair.
 * Outputs (n = tokens * topk):
 *   offsets int32 (experts + 1): expert e has the sorted rows
 *       [offsets[e], offsets[e + 1]); offsets[experts] pairs are kept
 *   order   int32 (n): the pair at each sorted row, -1 from offsets[experts] on
 *   slots   int32 (tokens, topk): the sorted row of each pair, -1 if dropped
 * Limits: tokens >= 0, 1 <= topk <= GS_MAX_TOPK, 1 <= experts <=
 * GS_MAX_EXPERTS, n < 2^31.
 */
int gs_expert_sort(const int32_t* expert_ids, int64_t tokens, int topk, int experts,
                   int32_t* offsets, int32_t* order, int32_t* slots, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * gs_expert_dispatch -- sorted rows of x (tokens, channels):
 *   xs[slots[t, j]] = x[t],  xs[r] = 0 for r >= offsets[experts].
 * xs (tokens * topk, channels) of dtype.  Its gradient in x is
 * gs_expert_combine of the gradient of xs without weights.
 */
int gs_expert_dispatch(const void* x, int64_t ldx, const int32_t* slots, const int32_t* offsets,
                       int64_t tokens, int topk, int experts, int channels, int dtype, void* xs,
                       int32_t* d_status, void* stream);

/*
 * gs_expert_combine -- y[t] = sum over j with slots[t, j] >= 0 of
 * weights[t, j] * ys[slots[t, j]] (j ascending; 0 if there is none; the
 * weight of a dropped pair is not used).  weights float32 (tokens, topk) or
 * NULL for ones; y (tokens, channels), row distance ldy.
 */
int gs_expert_combine(const void* ys, const int32_t* slots, const float* weights,
                      int64_t tokens, int topk, int channels, int dtype, void* y, int64_t ldy,
                      int32_t* d_status, void* stream);

/*
 * gs_expert_combine_bwd -- for every pair with a slot s = slots[t, j]:
 *   grad_ys[s] = weights[t, j] * grad_y[t]
 *   grad_weights[t, j] = sum over channels of grad_y[t] * ys[s]
 * grad_ys rows from offsets[experts] on and grad_weights of dropped pairs
 * are 0.  grad_weights float32 (tokens, topk) may be NULL (ys then too).
 */
int gs_expert_combine_bwd(const void* grad_y, int64_t ldgy, const void* ys,
                          const int32_t* slots, const float* weights, const int32_t* offsets,
                          int64_t tokens, int topk, int experts, int channels, int dtype,
                          void* grad_ys, float* grad_weights, int32_t* d_status, void* stream);

/* Bytes of workspace gs_expert_linear_fwd and _bwd need.  aligned != 0: every
 * array read begins on a 16-byte boundary; 0: the size serves whichever do not.
 * float32 operands, and rows that are not whole 16-byte vectors, are laid out
 * there for the tensor cores; the backward keeps partial sums there. */
size_t gs_expert_linear_fwd_workspace_size(int64_t rows, int experts, int in_features,
                                           int out_features, int dtype, int aligned);
size_t gs_expert_linear_bwd_workspace_size(int64_t rows, int experts, int in_features,
                                           int out_features, int dtype, int aligned);

/*
 * gs_expert_linear_fwd -- for the rows r of expert e (offsets as
 * gs_expert_sort wrote them):
 *   ys[r] = weight[e] xs[r] + bias[e];  rows of no expert are 0.
 * xs (rows, in_features), weight (experts, out_features, in_features), bias
 * (experts, out_features) or NULL, ys (rows, out_features), all of dtype.
 * workspace (16-byte aligned): as the size call says, or NULL where that is 0.
 * A float32 product is off by at most 2^-24 of it (operands from 2^-110 on) and
 * sums of them are float32 sums; a factor below 2^-133 counts as 0.
 * Limits: 0 <= rows <= GS_MAX_EXPERT_ROWS (a third of it for float32),
 * 1 <= in_features, out_features <= 65536.
 */
int gs_expert_linear_fwd(const void* xs, const int32_t* offsets, const void* weight,
                         const void* bias, int64_t rows, int experts, int in_features,
                         int out_features, int dtype, void* ys, void* workspace,
                         size_t workspace_bytes, int32_t* d_status, void* stream);

/*
 * gs_expert_linear_bwd -- gradients of gs_expert_linear_fwd:
 *   grad_xs[r] = weight[e]^T grad_ys[r]   (rows of no expert 0)
 *   grad_weight[e] = sum over the expert's rows of grad_ys[r] xs[r]^T
 *   grad_bias[e] = sum over the expert's rows of grad_ys[r]
 * (0 for an expert without rows).  grad_xs may be NULL (weight is then not
 * read), grad_bias may be NULL, and grad_weight where grad_bias is (xs is then
 * not read).
 */
int gs_expert_linear_bwd(const void* grad_ys, const void* xs, const int32_t* offsets,
                         const void* weight, int64_t rows, int experts, int in_features,
                         int out_features, int dtype, void* grad_xs, void* grad_weight,
                         void* grad_bias, void* workspace, size_t workspace_bytes,
                         int32_t* d_status, void* stream);

/* Bytes of workspace gs_expert_route_fwd needs where counts are asked for. */
size_t gs_expert_route_workspace_size(int64_t tokens, int experts);

/*
 * gs_expert_route_fwd -- with p the softmax of a row of logits (tokens,
 * experts):
 *   ids[t, j]  the expert of the j-th largest logit (equal ones: the lowest
 *              expert first; a NaN before every number); a logit of minus
 *              infinity is not chosen
 *   weights[t, j] = p[ids[t, j]], divided by their sum over j if renormalise
 *   counts[e] = how many ids are e;  counts[experts] = tokens that take part
 *   loss = experts * sum over e of counts[e] / (all counts[e]) * (mean of p[e]
 *          over the tokens that take part);  0 where none does
 * keep (tokens bytes, or NULL): a token whose byte is 0 does not take part and
 * its logits are not looked at; nor does one without a logit above minus
 * infinity.  What is not chosen has ids -1 (gs_expert_sort drops it) and
 * weight 0.  Logits of dtype, row distance ldl; ids int32 and weights float32
 * (tokens, topk).  counts int32 (experts + 1) may be NULL (loss then too, and
 * no workspace is needed), loss (one float32) may be NULL.
 * Limits: tokens, topk and experts as gs_expert_sort, topk <= experts.
 */
int gs_expert_route_fwd(const void* logits, int64_t ldl, const uint8_t* keep, int64_t tokens,
                        int topk, int experts, int dtype, int renormalise, int32_t* ids,
                        float* weights, int32_t* counts, float* loss, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * gs_expert_route_bwd -- the gradient of weights and loss in the logits, for
 * the choice made (the counts do not change with the logits): with g the
 * gradient of weights, h[e] = *grad_loss * experts * counts[e] / (all
 * counts[e]) / counts[experts], sums over the choices j and all experts i
 *   grad_logits[e] = p[e] (h[e] - sum p[i] h[i])
 *     + (renormalise)  for e = ids[j]: w[j] (g[j] - sum w g), w the weights
 *     + (otherwise)    p[e] ((g[j] for e = ids[j]) - sum p[ids[j]] g[j])
 * and 0 for a token whose first id is -1.  ids, counts: as gs_expert_route_fwd
 * wrote them.  grad_weights (tokens, topk) and grad_loss (one float32 on the
 * device) may each be NULL for zeros (counts with grad_loss).
 */
int gs_expert_route_bwd(const void* logits, int64_t ldl, const int32_t* ids,
                        const int32_t* counts, const float* grad_weights, const float* grad_loss,
                        int64_t tokens, int topk, int experts, int dtype, int renormalise,
                        void* grad_logits, int64_t ldg, int32_t* d_status, void* stream);

/*
 * gs_rows_pack8 -- x (rows, channels) of dtype, row distance ldx, as 8-bit
 * rows: a block's byte is the smallest (at least 0) with |x| <= 448 * 2^(byte
 * - 127) for its finite elements, q the e4m3 nearest to x * 2^(127 - byte),
 * ties to even; what is not finite becomes a NaN.
 * gs_rows_unpack8 -- the values back, rounded to dtype (a finite q beyond the
 * type becomes its largest finite value).
 * Limits: rows >= 0, 1 <= channels <= 65536.
 */
int gs_rows_pack8(const void* x, int64_t ldx, int64_t rows, int channels, int dtype, uint8_t* q,
                  uint8_t* scales, void* stream);
int gs_rows_unpack8(const uint8_t* q, const uint8_t* scales, int64_t rows, int channels,
                    int dtype, void* y, int64_t ldy, void* stream);

/* Bytes of workspace gs_expert_linear8_bwd needs.  aligned != 0: grad_ys begins
 * on a 16-byte boundary. */
size_t gs_expert_linear8_bwd_workspace_size(int64_t rows, int experts, int in_features,
                                            int out_features, int dtype, int aligned);

/*
 * gs_expert_linear8_fwd -- gs_expert_linear_fwd of 8-bit rows:
 *   ys[r] = weight[e] xs[r] + bias[e];  rows of no expert are 0,
 * xs (rows, in_features) and weight (experts * out_features, in_features) 8-bit
 * rows with their scales; bias and ys of dtype.  Limits as there.
 */
int gs_expert_linear8_fwd(const uint8_t* xs, const uint8_t* xs_scales, const int32_t* offsets,
                          const uint8_t* weight, const uint8_t* weight_scales, const void* bias,
                          int64_t rows, int experts, int in_features, int out_features, int dtype,
                          void* ys, int32_t* d_status, void* stream);

/*
 * gs_expert_linear8_bwd -- gradients of gs_expert_linear8_fwd in the values of
 * xs, weight and bias, from rows kept in 8 bits since the forward:
 *   grad_xs[r] = weight[e]^T grad_ys[r]   (rows of no expert 0)
 *   grad_weight[e] = sum over the expert's rows of grad_ys[r] xs[r]^T
 *   grad_bias[e] = sum over the expert's rows of grad_ys[r]
 * grad_ys and the gradients of dtype.  With float32 and bfloat16 a value of xs or
 * weight is taken as bfloat16 holds it: exactly where its block's byte is 3 to
 * 246, as the type's largest, 255 * 2^120, from 2^128 on, and in steps of 2^-133
 * below 2^-126.  With float16 a value of xs (of weight) is taken exactly where
 * its block's byte is at most 22 below the largest of the experts' rows (of the
 * weights of experts that have rows), else to within 2^-39 of the largest value.
 * grad_xs may be NULL (weight is then not read), grad_bias may be NULL, and
 * grad_weight where grad_bias is (xs is then not read).
 */
int gs_expert_linear8_bwd(const void* grad_ys, const uint8_t* xs, const uint8_t* xs_scales,
                          const int32_t* offsets, const uint8_t* weight,
                          const uint8_t* weight_scales, int64_t rows, int experts,
                          int in_features, int out_features, int dtype, void* grad_xs,
                          void* grad_weight, void* grad_bias, void* workspace,
                          size_t workspace_bytes, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GS_HEAD_H */
