/*
 * gs_head.h -- the feature-head calls of libgs_splat_gb300.so: what follows a
 * render of feature channels (gs_rasterize_fwd with up to GS_MAX_CHANNELS
 * channels) in a network that is trained through it.
 *   gs_layer_norm_fwd / _bwd       layer norm over the channels of each row
 *   gs_expert_sort                 (token, choice) pairs sorted by expert
 *   gs_expert_dispatch             rows copied into expert order
 *   gs_expert_combine / _bwd       rows summed back with their weights
 *   gs_expert_linear_fwd / _bwd    every expert's matrix product
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

#ifdef __cplusplus
}
#endif

#endif /* GS_HEAD_H */
