// head_internal.h -- what the host side of the training-head calls (head.cpp)
// passes to their kernels (norm.cu, loss.cu, gated.cu, clip.cu,
// adamw.cu).  Every launch function
// gets checked arguments: pointers aligned as include/zero.h asks, strides and
// dims multiples of 8 where it asks so.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace zk {

struct NormArgs {
    const void *x;
    int64_t x_stride;
    const void *residual;  // NULL: none
    int64_t residual_stride;
    const void *weight;
    float eps;
    int64_t rows;
    int dim;
    int lp;
    void *out;  // lp rows, or NULL when codes are written
    int64_t out_stride;
    void *sum;  // NULL: not written
    int64_t sum_stride;
    int fp8;         // codes: their format
    int8_t *codes;   // NULL unless quantized
    float *scales;
};
cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream);
cudaError_t launch_dequantize_rows(const int8_t *codes, const float *scales, int fp8, int64_t rows, int dim,
                                   int lp, void *out, int64_t out_stride, cudaStream_t stream);

struct NormBackwardArgs {
    const void *sum;
    int64_t sum_stride;
    const void *weight;
    const void *grad_out;
    int64_t grad_out_stride;
    const void *grad_sum;  // NULL: none
    int64_t grad_sum_stride;
    float eps;
    int64_t rows;
    int dim;
    int lp;
    void *grad_in;
    int64_t grad_in_stride;
    void *grad_weight;
    void *workspace;
};
int64_t norm_backward_bytes(int64_t rows, int dim);
cudaError_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream);

struct LossArgs {
    const void *hidden;
    int64_t hidden_stride;
    const void *weight;
    int64_t weight_stride;
    const int64_t *target;
    int64_t ignore;
    int64_t tokens, vocab;
    int dim;
    int lp;
    float *loss;  // forward: written
    float *lse;   // forward: written; backward: read
    const float *grad_loss;
    void *grad_hidden;
    int64_t grad_hidden_stride;
    void *grad_weight;
    int64_t grad_weight_stride;
    int32_t *status;
    void *workspace;
};
void set_loss_wait(int64_t cycles);
int64_t loss_wait();  // of every product's bounded waits
cudaError_t launch_take_status(int32_t *status, int32_t *bits, cudaStream_t stream);
int64_t loss_forward_bytes(int64_t tokens, int64_t vocab, int dim);
int64_t loss_backward_bytes(int64_t tokens, int64_t vocab, int dim);
cudaError_t launch_loss_forward(const LossArgs &a, cudaStream_t stream);
cudaError_t launch_loss_backward(const LossArgs &a, cudaStream_t stream);

struct GatedArgs {
    const void *x;
    int64_t x_stride;
    const void *gate;
    int64_t gate_stride;
    const void *up;
    int64_t up_stride;
    int act;  // ZERO_ACT_*
    int64_t tokens;
    int wide, dim;
    int lp;
    void *out;  // forward
    int64_t out_stride;
    const void *grad_out;  // backward, with all that follows
    int64_t grad_out_stride;
    void *grad_x;
    int64_t grad_x_stride;
    void *grad_gate;
    int64_t grad_gate_stride;
    void *grad_up;
    int64_t grad_up_stride;
    int32_t *status;
    void *workspace;
};
int64_t gated_forward_bytes(int64_t tokens, int64_t wide, int dim);
int64_t gated_backward_bytes(int64_t tokens, int64_t wide, int dim);
cudaError_t launch_gated_forward(const GatedArgs &a, cudaStream_t stream);
cudaError_t launch_gated_backward(const GatedArgs &a, cudaStream_t stream);

int64_t clip_bytes(int n, const int64_t *lens);
cudaError_t launch_clip(int n, const void *const *grads, const int64_t *lens, int dtype, void *const *out,
                        float loss_scale, float max_norm, float *norm, float *coef, int32_t *nonfinite,
                        void *workspace, cudaStream_t stream);

struct AdamwArgs {
    int n;
    float *const *params;
    const void *const *grads;
    int grad_dtype;
    void *const *copies;  // NULL: none
    int copy_type;
    const int64_t *lens;
    bool eight;  // the moments' format
    void *m, *v;
    float *m_scales, *v_scales;
    int64_t *record;
    double lr, beta1, beta2, eps, wd;
    float loss_scale;
    const float *coef;
    const int32_t *skip;
    uint32_t seed;
};
cudaError_t launch_adamw_step(const AdamwArgs &a, cudaStream_t stream);
cudaError_t launch_adamw_values(const int8_t *m, const uint8_t *v, const float *m_scales, const float *v_scales,
                                int64_t blocks, int dtype, void *m_out, void *v_out, cudaStream_t stream);

}  // namespace zk
