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

// ---- the experts' products; the launchers of expert_mma.cu return a gs_status
struct LinearArgs {
    const int32_t* offsets;
    int64_t rows;
    int experts, in, out, dtype;
    int32_t* d_status;
};
// ---- expert_few.cu: the products of few rows, bound by reading the weights.
// as_they_lie: the tensor cores could read the weights in place.
bool few_rows(const LinearArgs& a, bool as_they_lie);
void launch_few_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                    void* ys, cudaStream_t s);
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

}  // namespace gs
