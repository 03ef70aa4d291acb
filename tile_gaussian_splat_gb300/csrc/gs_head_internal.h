// Host-side launchers of the feature-head calls (gs_head.h), shared between
// their translation units.  Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gs {

// ---- norm.cu
struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* weight;
    int64_t rows;
    int channels, dtype, param_dtype;
};
void launch_norm_fwd(const NormArgs& a, const void* bias, float eps, void* y, int64_t ldy,
                     float* mean, float* rstd, cudaStream_t s);
// Row slices the gradients of weight and bias are summed over (each gives one
// row of partial sums).
int norm_bwd_slices(int64_t rows, int channels);
// partial: 2 * norm_bwd_slices * channels floats.
void launch_norm_bwd(const NormArgs& a, const void* grad_y, int64_t ldgy, const float* mean,
                     const float* rstd, void* grad_x, int64_t ldgx, void* grad_weight,
                     void* grad_bias, float* partial, cudaStream_t s);

// ---- experts.cu
// Contiguous ranges of pairs that gs_expert_sort counts and places one warp
// each; 0 when one block sorts them all and needs no workspace.
int sort_units(int64_t n);
// counts: sort_units * experts words; totals: experts words.
void launch_expert_sort(const int32_t* ids, int64_t n, int experts, int32_t* offsets,
                        int32_t* order, int32_t* slots, int32_t* counts, int32_t* totals,
                        cudaStream_t s);
struct RowArgs {
    int64_t tokens;
    int topk, experts, channels, dtype;
    int32_t* d_status;
};
void launch_dispatch(const RowArgs& a, const void* x, int64_t ldx, const int32_t* slots,
                     const int32_t* offsets, void* xs, cudaStream_t s);
void launch_combine(const RowArgs& a, const void* ys, const int32_t* slots, const float* weights,
                    void* y, int64_t ldy, cudaStream_t s);
void launch_combine_bwd(const RowArgs& a, const void* grad_y, int64_t ldgy, const void* ys,
                        const int32_t* slots, const float* weights, const int32_t* offsets,
                        void* grad_ys, float* grad_weights, cudaStream_t s);

// ---- route.cu
struct RouteArgs {
    const void* logits;
    int64_t ld, tokens;
    int topk, experts, dtype, renormalise;
};
constexpr int kMaxRouteBlocks = 152 * 8;  // blocks that leave partial sums
size_t route_workspace(int64_t tokens, int experts);
// counts and loss may be null (loss where counts is).
void launch_route_fwd(const RouteArgs& a, const uint8_t* keep, int32_t* ids, float* weights,
                      int32_t* counts, float* loss, void* workspace, cudaStream_t s);
void launch_route_bwd(const RouteArgs& a, const int32_t* ids, const int32_t* counts,
                      const float* grad_weights, const float* grad_loss, void* grad, int64_t ldg,
                      int32_t* d_status, cudaStream_t s);

// ---- rows8.cu: rows of GS_ROW8_BYTES and scales of GS_ROW8_SCALES bytes
void launch_pack8(const void* x, int64_t ldx, int64_t rows, int channels, int dtype, uint8_t* q,
                  uint8_t* scales, cudaStream_t s);
// With offsets: `rows` rows for each of the experts, of which those without rows
// of their own are left out.  With tops (float16): as multiples of 2^(top_of - 134).
// (Either: y aligned and its rows whole 16-byte vectors.)
void launch_unpack8(const uint8_t* q, const uint8_t* scales, int64_t rows, int channels,
                    int dtype, void* y, int64_t ldy, cudaStream_t s,
                    const int32_t* offsets = nullptr, int experts = 0,
                    const int32_t* tops = nullptr);

// ---- the experts' products; the launchers of expert_mma.cu return a gs_status
struct LinearArgs {
    const int32_t* offsets;
    int64_t rows;
    int experts, in, out, dtype;
    int32_t* d_status;
    bool packed = false;  // xs and weight are 8-bit rows
};
struct Rows8 {
    const uint8_t *q, *scales;
};
// ---- rows8.cu: the largest scale byte of the rows' blocks, then of the weights',
// of those that the products use and that are numbers (0 for a null), as the
// largest of kTopParts words each
constexpr int kTopParts = 128;
void launch_top_bytes(const LinearArgs& a, const uint8_t* xs, const uint8_t* weight,
                      int32_t* tops, cudaStream_t s);
// ---- expert_few.cu: the products of few rows, bound by reading the weights.
// as_they_lie: the tensor cores could read the weights in place.
bool few_rows(const LinearArgs& a, bool as_they_lie);
void launch_few_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                    void* ys, cudaStream_t s);
void launch_few8_fwd(const LinearArgs& a, Rows8 xs, Rows8 weight, const void* bias, void* ys,
                     cudaStream_t s);
void launch_few_dx(const LinearArgs& a, const void* grad_ys, const void* weight, void* grad_xs,
                   cudaStream_t s);
// ---- expert_mma.cu
size_t linear_fwd_workspace(const LinearArgs& a, const void* xs, const void* weight);
int launch_linear_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                      void* ys, void* workspace, cudaStream_t s);
size_t linear_bwd_workspace(const LinearArgs& a, const void* grad_ys, const void* xs,
                            const void* weight);
// grad_xs, or grad_weight and with it grad_bias, may be null.
int launch_linear_bwd(const LinearArgs& a, const void* grad_ys, const void* xs,
                      const void* weight, void* grad_xs, void* grad_weight, void* grad_bias,
                      void* workspace, cudaStream_t s);
// The same of 8-bit rows (a.packed).
// ---- expert_mma8.cu
int launch_linear8_fwd(const LinearArgs& a, Rows8 xs, Rows8 weight, const void* bias, void* ys,
                       cudaStream_t s);
// ---- expert_mma.cu
size_t linear8_bwd_workspace(const LinearArgs& a, const void* grad_ys);
int launch_linear8_bwd(const LinearArgs& a, const void* grad_ys, Rows8 xs, Rows8 weight,
                       void* grad_xs, void* grad_weight, void* grad_bias, void* workspace,
                       cudaStream_t s);

}  // namespace gs
