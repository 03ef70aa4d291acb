// C ABI of the feature-head calls (declared in include/gs_head.h): argument
// checks, workspace layout and launches.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/gs_head.h"
#include "gs_head_internal.h"

namespace {

using namespace gs;

constexpr size_t kAlign = 256;
constexpr int kMaxFeatures = 65536;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int check_launch() { return cudaGetLastError() == cudaSuccess ? GS_OK : GS_ERR_CUDA; }

bool dtype_ok(int dtype) { return dtype == GS_F32 || dtype == GS_F16 || dtype == GS_BF16; }

// A pointer to elements of `dtype`: not null and aligned to them.
bool array_ok(const void* p, int dtype) {
    return p && (reinterpret_cast<uintptr_t>(p) & (dtype == GS_F32 ? 3u : 1u)) == 0;
}

bool words_ok(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool norm_args_ok(const void* x, int64_t ldx, int64_t rows, int channels, int dtype,
                  int param_dtype) {
    if (rows < 0 || channels < 1 || channels > GS_MAX_NORM_CHANNELS) return false;
    if (!dtype_ok(dtype) || (param_dtype != dtype && param_dtype != GS_F32)) return false;
    return rows == 0 || (array_ok(x, dtype) && ldx >= channels);
}

bool pairs_ok(int64_t tokens, int topk, int experts) {
    if (tokens < 0 || topk < 1 || topk > GS_MAX_TOPK) return false;
    if (experts < 1 || experts > GS_MAX_EXPERTS) return false;
    return tokens < ((int64_t)1 << 31) && tokens * topk < ((int64_t)1 << 31);
}

bool rows_ok(int64_t tokens, int topk, int experts, int channels, int dtype) {
    return pairs_ok(tokens, topk, experts) && channels >= 1 && channels <= kMaxFeatures &&
           dtype_ok(dtype);
}

bool linear_ok(const int32_t* offsets, int64_t rows, int experts, int in, int out, int dtype) {
    if (rows < 0 || rows > GS_MAX_EXPERT_ROWS || experts < 1 || experts > GS_MAX_EXPERTS)
        return false;
    if (in < 1 || in > kMaxFeatures || out < 1 || out > kMaxFeatures || !dtype_ok(dtype))
        return false;
    // the three planes of float32 rows are numbered on end
    if (dtype == GS_F32 && 3 * rows > GS_MAX_EXPERT_ROWS) return false;
    return words_ok(offsets);
}

const int32_t kSomeOffsets = 0;  // stands for the offsets where only sizes are checked

size_t dtype_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

bool workspace_ok(const void* p, size_t bytes, size_t need) {
    return need == 0 || (p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && bytes >= need);
}

// Stands for an array that is read, where only sizes are checked.
const void* some_array(bool aligned) {
    return reinterpret_cast<const void*>((uintptr_t)(aligned ? 16 : 2));
}

size_t sort_counts_bytes(int64_t n, int experts) {
    return align_up((size_t)sort_units(n) * experts * sizeof(int32_t));
}

}  // namespace

extern "C" {

int gs_layer_norm_fwd(const void* x, int64_t ldx, const void* weight, const void* bias,
                      int64_t rows, int channels, int dtype, int param_dtype, float eps, void* y,
                      int64_t ldy, float* mean, float* rstd, void* stream) {
    if (!norm_args_ok(x, ldx, rows, channels, dtype, param_dtype) || !(eps >= 0.0f))
        return GS_ERR_INVALID_ARG;
    if ((weight && !array_ok(weight, param_dtype)) || (bias && !array_ok(bias, param_dtype)))
        return GS_ERR_INVALID_ARG;
    if (rows > 0 && (!array_ok(y, dtype) || ldy < channels)) return GS_ERR_INVALID_ARG;
    if (rows > 0 && ((mean == nullptr) != (rstd == nullptr) ||
                     (mean && (!words_ok(mean) || !words_ok(rstd)))))
        return GS_ERR_INVALID_ARG;
    if (rows == 0) return GS_OK;
    launch_norm_fwd(NormArgs{x, ldx, weight, rows, channels, dtype, param_dtype}, bias, eps, y,
                    ldy, mean, rstd, static_cast<cudaStream_t>(stream));
    return check_launch();
}

size_t gs_layer_norm_bwd_workspace_size(int64_t rows, int channels) {
    if (rows < 0 || channels < 1 || channels > GS_MAX_NORM_CHANNELS) return 0;
    return align_up((size_t)norm_bwd_slices(rows, channels) * 2 * channels * sizeof(float));
}

int gs_layer_norm_bwd(const void* grad_y, int64_t ldgy, const void* x, int64_t ldx,
                      const void* weight, const float* mean, const float* rstd, int64_t rows,
                      int channels, int dtype, int param_dtype, void* grad_x, int64_t ldgx,
                      void* grad_weight, void* grad_bias, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (!norm_args_ok(x, ldx, rows, channels, dtype, param_dtype)) return GS_ERR_INVALID_ARG;
    if (weight && !array_ok(weight, param_dtype)) return GS_ERR_INVALID_ARG;
    if (rows > 0 && (!array_ok(grad_y, dtype) || ldgy < channels || !words_ok(mean) ||
                     !words_ok(rstd)))
        return GS_ERR_INVALID_ARG;
    if (rows > 0 && grad_x && (!array_ok(grad_x, dtype) || ldgx < channels))
        return GS_ERR_INVALID_ARG;
    if ((grad_weight && !array_ok(grad_weight, param_dtype)) ||
        (grad_bias && !array_ok(grad_bias, param_dtype)))
        return GS_ERR_INVALID_ARG;
    const bool params = grad_weight || grad_bias;
    if (params && (!words_ok(workspace) ||
                   workspace_bytes < gs_layer_norm_bwd_workspace_size(rows, channels)))
        return GS_ERR_WORKSPACE;
    if (!params && (!grad_x || rows == 0)) return GS_OK;
    launch_norm_bwd(NormArgs{x, ldx, weight, rows, channels, dtype, param_dtype}, grad_y, ldgy,
                    mean, rstd, rows > 0 ? grad_x : nullptr, ldgx, grad_weight, grad_bias,
                    static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
    return check_launch();
}

size_t gs_expert_sort_workspace_size(int64_t tokens, int topk, int experts) {
    if (!pairs_ok(tokens, topk, experts)) return 0;
    if (sort_units(tokens * topk) == 0) return 0;
    return sort_counts_bytes(tokens * topk, experts) +
           align_up((size_t)experts * sizeof(int32_t));
}

int gs_expert_sort(const int32_t* expert_ids, int64_t tokens, int topk, int experts,
                   int32_t* offsets, int32_t* order, int32_t* slots, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (!pairs_ok(tokens, topk, experts) || !words_ok(offsets)) return GS_ERR_INVALID_ARG;
    if (tokens > 0 && (!words_ok(expert_ids) || !words_ok(order) || !words_ok(slots)))
        return GS_ERR_INVALID_ARG;
    const size_t need = gs_expert_sort_workspace_size(tokens, topk, experts);
    if (need && (!words_ok(workspace) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
    int32_t* counts = static_cast<int32_t*>(workspace);
    int32_t* totals = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) +
                                                 sort_counts_bytes(tokens * topk, experts));
    launch_expert_sort(expert_ids, tokens * topk, experts, offsets, order, slots, counts, totals,
                       static_cast<cudaStream_t>(stream));
    return check_launch();
}

int gs_expert_dispatch(const void* x, int64_t ldx, const int32_t* slots, const int32_t* offsets,
                       int64_t tokens, int topk, int experts, int channels, int dtype, void* xs,
                       int32_t* d_status, void* stream) {
    if (!rows_ok(tokens, topk, experts, channels, dtype) || !words_ok(offsets))
        return GS_ERR_INVALID_ARG;
    if (tokens == 0) return GS_OK;
    if (!array_ok(x, dtype) || ldx < channels || !words_ok(slots) || !array_ok(xs, dtype))
        return GS_ERR_INVALID_ARG;
    launch_dispatch(RowArgs{tokens, topk, experts, channels, dtype, d_status}, x, ldx, slots,
                    offsets, xs, static_cast<cudaStream_t>(stream));
    return check_launch();
}

int gs_expert_combine(const void* ys, const int32_t* slots, const float* weights, int64_t tokens,
                      int topk, int channels, int dtype, void* y, int64_t ldy, int32_t* d_status,
                      void* stream) {
    if (!rows_ok(tokens, topk, 1, channels, dtype)) return GS_ERR_INVALID_ARG;
    if (tokens == 0) return GS_OK;
    if (!array_ok(ys, dtype) || !words_ok(slots) || (weights && !words_ok(weights)) ||
        !array_ok(y, dtype) || ldy < channels)
        return GS_ERR_INVALID_ARG;
    launch_combine(RowArgs{tokens, topk, 1, channels, dtype, d_status}, ys, slots, weights, y,
                   ldy, static_cast<cudaStream_t>(stream));
    return check_launch();
}

int gs_expert_combine_bwd(const void* grad_y, int64_t ldgy, const void* ys, const int32_t* slots,
                          const float* weights, const int32_t* offsets, int64_t tokens, int topk,
                          int experts, int channels, int dtype, void* grad_ys,
                          float* grad_weights, int32_t* d_status, void* stream) {
    if (!rows_ok(tokens, topk, experts, channels, dtype) || !words_ok(offsets))
        return GS_ERR_INVALID_ARG;
    if (tokens == 0) return GS_OK;
    if (!array_ok(grad_y, dtype) || ldgy < channels || !words_ok(slots) ||
        (weights && !words_ok(weights)) || !array_ok(grad_ys, dtype))
        return GS_ERR_INVALID_ARG;
    if (grad_weights && (!words_ok(grad_weights) || !array_ok(ys, dtype)))
        return GS_ERR_INVALID_ARG;
    launch_combine_bwd(RowArgs{tokens, topk, experts, channels, dtype, d_status}, grad_y, ldgy,
                       ys, slots, weights, offsets, grad_ys, grad_weights,
                       static_cast<cudaStream_t>(stream));
    return check_launch();
}

size_t gs_expert_linear_fwd_workspace_size(int64_t rows, int experts, int in_features,
                                           int out_features, int dtype, int aligned) {
    if (!linear_ok(&kSomeOffsets, rows, experts, in_features, out_features, dtype)) return 0;
    const LinearArgs a{nullptr, rows, experts, in_features, out_features, dtype, nullptr};
    const size_t with_weight = linear_fwd_workspace(a, some_array(aligned), some_array(true));
    if (aligned) return with_weight;
    // a misaligned weight may choose the kernel of few rows, which needs
    // nothing; with xs alone misaligned its rows are laid out
    return std::max(with_weight, linear_fwd_workspace(a, some_array(false), some_array(false)));
}

int gs_expert_linear_fwd(const void* xs, const int32_t* offsets, const void* weight,
                         const void* bias, int64_t rows, int experts, int in_features,
                         int out_features, int dtype, void* ys, void* workspace,
                         size_t workspace_bytes, int32_t* d_status, void* stream) {
    if (!linear_ok(offsets, rows, experts, in_features, out_features, dtype))
        return GS_ERR_INVALID_ARG;
    if (rows == 0) return GS_OK;
    if (!array_ok(xs, dtype) || !array_ok(weight, dtype) || (bias && !array_ok(bias, dtype)) ||
        !array_ok(ys, dtype))
        return GS_ERR_INVALID_ARG;
    const LinearArgs a{offsets, rows, experts, in_features, out_features, dtype, d_status};
    if (!workspace_ok(workspace, workspace_bytes, linear_fwd_workspace(a, xs, weight)))
        return GS_ERR_WORKSPACE;
    const int rc = launch_linear_fwd(a, xs, weight, bias, ys, workspace,
                                     static_cast<cudaStream_t>(stream));
    return rc == GS_OK ? check_launch() : rc;
}

size_t gs_expert_linear_bwd_workspace_size(int64_t rows, int experts, int in_features,
                                           int out_features, int dtype, int aligned) {
    if (!linear_ok(&kSomeOffsets, rows, experts, in_features, out_features, dtype)) return 0;
    const LinearArgs a{nullptr, rows, experts, in_features, out_features, dtype, nullptr};
    // all off the boundary needs the most: where a misaligned weight is read as
    // it lies, an aligned one is too
    const void* p = some_array(aligned);
    return linear_bwd_workspace(a, p, p, p);
}

int gs_expert_linear_bwd(const void* grad_ys, const void* xs, const int32_t* offsets,
                         const void* weight, int64_t rows, int experts, int in_features,
                         int out_features, int dtype, void* grad_xs, void* grad_weight,
                         void* grad_bias, void* workspace, size_t workspace_bytes,
                         int32_t* d_status, void* stream) {
    if (!linear_ok(offsets, rows, experts, in_features, out_features, dtype))
        return GS_ERR_INVALID_ARG;
    if (rows > 0 && !array_ok(grad_ys, dtype)) return GS_ERR_INVALID_ARG;
    if (rows > 0 && grad_xs && (!array_ok(grad_xs, dtype) || !array_ok(weight, dtype)))
        return GS_ERR_INVALID_ARG;
    if (grad_weight && (!array_ok(grad_weight, dtype) || (rows > 0 && !array_ok(xs, dtype))))
        return GS_ERR_INVALID_ARG;
    if (grad_bias && (!array_ok(grad_bias, dtype) || !grad_weight)) return GS_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LinearArgs a{offsets, rows, experts, in_features, out_features, dtype, d_status};
    if (!workspace_ok(workspace, workspace_bytes, linear_bwd_workspace(a, grad_ys, xs, weight)))
        return GS_ERR_WORKSPACE;
    if (rows == 0) {  // sums over nothing
        const size_t row = (size_t)experts * out_features * dtype_size(dtype);
        if ((grad_weight && cudaMemsetAsync(grad_weight, 0, row * in_features, s) != cudaSuccess) ||
            (grad_bias && cudaMemsetAsync(grad_bias, 0, row, s) != cudaSuccess))
            return GS_ERR_CUDA;
        return GS_OK;
    }
    if (!grad_xs && !grad_weight) return GS_OK;
    const int rc = launch_linear_bwd(a, grad_ys, xs, weight, grad_xs, grad_weight, grad_bias,
                                     workspace, s);
    return rc == GS_OK ? check_launch() : rc;
}

}  // extern "C"
