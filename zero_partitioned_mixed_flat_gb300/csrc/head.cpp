// head.cpp -- host side of the training-head calls of include/zero.h: argument
// checks, then the launches.  No state, no allocation.
#include "head_internal.h"
#include "zero.h"
#include "zero_internal.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - (1 << 16);

zero_status refuse(zero_status code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    zk::set_last_error(buf);
    return code;
}

zero_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return ZERO_OK;
    cudaGetLastError();
    return refuse(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// rows x cols lp elements at p, rows `stride` apart
zero_status matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t stride) {
    if (!p && rows > 0) return refuse(ZERO_EINVAL, "%s is NULL", name);
    if (!aligned(p, 16)) return refuse(ZERO_EALIGN, "%s is not 16-byte aligned", name);
    if (stride < cols) return refuse(ZERO_EINVAL, "%s: stride %lld is less than a row's %lld elements", name,
                                     (long long)stride, (long long)cols);
    if (stride % 8 != 0) return refuse(ZERO_EALIGN, "%s: stride %lld is not a multiple of 8", name, (long long)stride);
    if (rows > 1 && stride > (int64_t(1) << 40) / rows) return refuse(ZERO_EINVAL, "%s: rows * stride is too large", name);
    return ZERO_OK;
}

zero_status vector(const char *name, const void *p, int64_t n) {
    if (!p && n > 0) return refuse(ZERO_EINVAL, "%s is NULL", name);
    if (!aligned(p, 16)) return refuse(ZERO_EALIGN, "%s is not 16-byte aligned", name);
    return ZERO_OK;
}

zero_status shape(int64_t rows, int32_t dim, zero_lp lp) {
    if (rows < 0 || rows >= kMaxRows) return refuse(ZERO_EINVAL, "%lld rows outside [0, 2^31 - 2^16)", (long long)rows);
    if (dim < 8 || dim > ZERO_HEAD_MAX_DIM) return refuse(ZERO_EINVAL, "dim %d outside [8, %d]", dim, ZERO_HEAD_MAX_DIM);
    if (dim % 8 != 0) return refuse(ZERO_EALIGN, "dim %d is not a multiple of 8", dim);
    if (lp != ZERO_FP16 && lp != ZERO_BF16) return refuse(ZERO_EINVAL, "unknown lp type %d", int(lp));
    return ZERO_OK;
}

zero_status scratch(const void *p, int64_t have, int64_t need) {
    if (have < need) return refuse(ZERO_EINVAL, "workspace of %lld bytes, %lld needed", (long long)have, (long long)need);
    if (!p && need > 0) return refuse(ZERO_EINVAL, "workspace is NULL");
    if (!aligned(p, 16)) return refuse(ZERO_EALIGN, "workspace is not 16-byte aligned");
    return ZERO_OK;
}

#define TRY(call)                                   \
    do {                                            \
        const zero_status st_ = (call);             \
        if (st_ != ZERO_OK) return st_;             \
    } while (0)

// the arguments that both forms of the norm share
zero_status norm_arguments(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                           const void *weight, float eps, int64_t n_rows, int32_t dim, zero_lp lp, void *sum,
                           int64_t sum_stride) {
    TRY(shape(n_rows, dim, lp));
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return refuse(ZERO_EINVAL, "eps must be finite and >= 0");
    TRY(matrix("x", x, n_rows, dim, x_stride));
    if (residual) TRY(matrix("residual", residual, n_rows, dim, residual_stride));
    TRY(vector("weight", weight, dim));
    if (sum) TRY(matrix("sum", sum, n_rows, dim, sum_stride));
    return ZERO_OK;
}

zero_status check_format(int32_t format) {
    if (format != ZERO_QUANT_INT8 && format != ZERO_QUANT_FP8_E4M3)
        return refuse(ZERO_EINVAL, "format is not ZERO_QUANT_INT8 / ZERO_QUANT_FP8_E4M3");
    return ZERO_OK;
}

zero_status loss_shape(int64_t n_tokens, int64_t vocab, int32_t dim, zero_lp lp) {
    TRY(shape(n_tokens, dim, lp));
    if (vocab < 1 || vocab >= kMaxRows) return refuse(ZERO_EINVAL, "vocab %lld outside [1, 2^31 - 2^16)", (long long)vocab);
    return ZERO_OK;
}

zero_status loss_arguments(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride,
                           const int64_t *target, int64_t n_tokens, int64_t vocab, int32_t dim, zero_lp lp,
                           const int32_t *status) {
    TRY(loss_shape(n_tokens, vocab, dim, lp));
    TRY(matrix("hidden", hidden, n_tokens, dim, hidden_stride));
    TRY(matrix("weight", weight, vocab, dim, weight_stride));
    if (!target && n_tokens > 0) return refuse(ZERO_EINVAL, "target is NULL");
    if (!aligned(target, 8)) return refuse(ZERO_EALIGN, "target is not 8-byte aligned");
    if (!status) return refuse(ZERO_EINVAL, "status is NULL");
    if (!aligned(status, 4)) return refuse(ZERO_EALIGN, "status is not 4-byte aligned");
    return ZERO_OK;
}

zero_status clip_lengths(int32_t n_tensors, const int64_t *lens) {
    if (n_tensors < 0 || (n_tensors > 0 && !lens)) return refuse(ZERO_EINVAL, "n_tensors < 0 or lens is NULL");
    for (int32_t i = 0; i < n_tensors; ++i)
        if (lens[i] < 0 || lens[i] > (int64_t(1) << 40)) return refuse(ZERO_EINVAL, "lens[%d] outside [0, 2^40]", i);
    return ZERO_OK;
}

}  // namespace

extern "C" {

zero_status zero_norm_forward(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                              const void *weight, float eps, int64_t n_rows, int32_t dim, zero_lp lp, void *out,
                              int64_t out_stride, void *sum, int64_t sum_stride, void *stream) {
    TRY(norm_arguments(x, x_stride, residual, residual_stride, weight, eps, n_rows, dim, lp, sum, sum_stride));
    TRY(matrix("out", out, n_rows, dim, out_stride));
    if (n_rows == 0) return ZERO_OK;
    const zk::NormArgs a = {x,   x_stride, residual, residual_stride, weight, eps, n_rows,  dim,
                            lp,  out,      out_stride, sum,           sum_stride, 0, nullptr, nullptr};
    return launched(zk::launch_norm_forward(a, static_cast<cudaStream_t>(stream)), "norm kernel launch");
}

zero_status zero_norm_forward_quantized(const void *x, int64_t x_stride, const void *residual,
                                        int64_t residual_stride, const void *weight, float eps, int64_t n_rows,
                                        int32_t dim, zero_lp lp, int32_t format, int8_t *codes, float *scales,
                                        void *sum, int64_t sum_stride, void *stream) {
    TRY(norm_arguments(x, x_stride, residual, residual_stride, weight, eps, n_rows, dim, lp, sum, sum_stride));
    TRY(check_format(format));
    TRY(vector("codes", codes, n_rows));
    TRY(vector("scales", scales, n_rows));
    if (n_rows == 0) return ZERO_OK;
    const zk::NormArgs a = {x,  x_stride, residual, residual_stride, weight, eps, n_rows, dim,
                            lp, nullptr,  0,        sum,             sum_stride,
                            format == ZERO_QUANT_FP8_E4M3, codes, scales};
    return launched(zk::launch_norm_forward(a, static_cast<cudaStream_t>(stream)), "norm kernel launch");
}

zero_status zero_dequantize_rows(const int8_t *codes, const float *scales, int32_t format, int64_t n_rows,
                                 int32_t dim, zero_lp lp, void *out, int64_t out_stride, void *stream) {
    TRY(shape(n_rows, dim, lp));
    TRY(check_format(format));
    TRY(vector("codes", codes, n_rows));
    TRY(vector("scales", scales, n_rows));
    TRY(matrix("out", out, n_rows, dim, out_stride));
    if (n_rows == 0) return ZERO_OK;
    return launched(zk::launch_dequantize_rows(codes, scales, format == ZERO_QUANT_FP8_E4M3, n_rows, dim, lp, out,
                                               out_stride, static_cast<cudaStream_t>(stream)),
                    "dequantize kernel launch");
}

zero_status zero_norm_backward_workspace(int64_t n_rows, int32_t dim, int64_t *bytes) {
    TRY(shape(n_rows, dim, ZERO_BF16));
    if (!bytes) return refuse(ZERO_EINVAL, "bytes is NULL");
    *bytes = zk::norm_backward_bytes(n_rows, dim);
    return ZERO_OK;
}

zero_status zero_norm_backward(const void *sum, int64_t sum_stride, const void *weight, const void *grad_out,
                               int64_t grad_out_stride, const void *grad_sum, int64_t grad_sum_stride, float eps,
                               int64_t n_rows, int32_t dim, zero_lp lp, void *grad_in, int64_t grad_in_stride,
                               void *grad_weight, void *workspace, int64_t workspace_bytes, void *stream) {
    TRY(shape(n_rows, dim, lp));
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return refuse(ZERO_EINVAL, "eps must be finite and >= 0");
    TRY(matrix("sum", sum, n_rows, dim, sum_stride));
    TRY(vector("weight", weight, dim));
    TRY(matrix("grad_out", grad_out, n_rows, dim, grad_out_stride));
    if (grad_sum) TRY(matrix("grad_sum", grad_sum, n_rows, dim, grad_sum_stride));
    TRY(matrix("grad_in", grad_in, n_rows, dim, grad_in_stride));
    TRY(vector("grad_weight", grad_weight, dim));
    TRY(scratch(workspace, workspace_bytes, zk::norm_backward_bytes(n_rows, dim)));
    const zk::NormBackwardArgs a = {sum, sum_stride, weight, grad_out, grad_out_stride, grad_sum, grad_sum_stride, eps,
                                    n_rows, dim, lp, grad_in, grad_in_stride, grad_weight, workspace};
    return launched(zk::launch_norm_backward(a, static_cast<cudaStream_t>(stream)), "norm backward kernel launch");
}

zero_status zero_loss_set_wait_limit(int64_t cycles) {
    if (cycles < 0) return refuse(ZERO_EINVAL, "cycles < 0");
    zk::set_loss_wait(cycles);
    return ZERO_OK;
}

zero_status zero_loss_take_status(int32_t *status, int32_t *bits, void *stream) {
    if (!status || !bits) return refuse(ZERO_EINVAL, "status or bits is NULL");
    if (!aligned(status, 4) || !aligned(bits, 4)) return refuse(ZERO_EALIGN, "status or bits is not 4-byte aligned");
    return launched(zk::launch_take_status(status, bits, static_cast<cudaStream_t>(stream)), "status kernel launch");
}

zero_status zero_loss_workspace(int64_t n_tokens, int64_t vocab, int32_t dim, int64_t *forward_bytes,
                                int64_t *backward_bytes) {
    TRY(loss_shape(n_tokens, vocab, dim, ZERO_BF16));
    if (forward_bytes) *forward_bytes = zk::loss_forward_bytes(n_tokens, vocab, dim);
    if (backward_bytes) *backward_bytes = zk::loss_backward_bytes(n_tokens, vocab, dim);
    return ZERO_OK;
}

zero_status zero_loss_forward(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride,
                              const int64_t *target, int64_t ignore, int64_t n_tokens, int64_t vocab, int32_t dim,
                              zero_lp lp, float *loss, float *lse, int32_t *status, void *workspace,
                              int64_t workspace_bytes, void *stream) {
    TRY(loss_arguments(hidden, hidden_stride, weight, weight_stride, target, n_tokens, vocab, dim, lp, status));
    TRY(vector("loss", loss, n_tokens));
    TRY(vector("lse", lse, n_tokens));
    TRY(scratch(workspace, workspace_bytes, zk::loss_forward_bytes(n_tokens, vocab, dim)));
    if (n_tokens == 0) return ZERO_OK;
    const zk::LossArgs a = {hidden, hidden_stride, weight, weight_stride, target, ignore, n_tokens, vocab, dim, lp,
                            loss, lse, nullptr, nullptr, 0, nullptr, 0, status, workspace};
    return launched(zk::launch_loss_forward(a, static_cast<cudaStream_t>(stream)), "loss kernel launch");
}

zero_status zero_loss_backward(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride,
                               const int64_t *target, int64_t ignore, int64_t n_tokens, int64_t vocab, int32_t dim,
                               zero_lp lp, const float *lse, const float *grad_loss, void *grad_hidden,
                               int64_t grad_hidden_stride, void *grad_weight, int64_t grad_weight_stride,
                               int32_t *status, void *workspace, int64_t workspace_bytes, void *stream) {
    TRY(loss_arguments(hidden, hidden_stride, weight, weight_stride, target, n_tokens, vocab, dim, lp, status));
    TRY(vector("lse", lse, n_tokens));
    TRY(vector("grad_loss", grad_loss, n_tokens));
    TRY(matrix("grad_hidden", grad_hidden, n_tokens, dim, grad_hidden_stride));
    TRY(matrix("grad_weight", grad_weight, vocab, dim, grad_weight_stride));
    TRY(scratch(workspace, workspace_bytes, zk::loss_backward_bytes(n_tokens, vocab, dim)));
    const zk::LossArgs a = {hidden, hidden_stride, weight, weight_stride, target, ignore, n_tokens, vocab, dim, lp,
                            nullptr, const_cast<float *>(lse), grad_loss, grad_hidden, grad_hidden_stride,
                            grad_weight, grad_weight_stride, status, workspace};
    return launched(zk::launch_loss_backward(a, static_cast<cudaStream_t>(stream)), "loss backward kernel launch");
}

zero_status zero_clip_workspace(int32_t n_tensors, const int64_t *lens, int64_t *bytes) {
    TRY(clip_lengths(n_tensors, lens));
    if (!bytes) return refuse(ZERO_EINVAL, "bytes is NULL");
    *bytes = zk::clip_bytes(n_tensors, lens);
    return ZERO_OK;
}

zero_status zero_clip_gradients(int32_t n_tensors, const void *const *grads, const int64_t *lens, int32_t dtype,
                                void *const *out, float loss_scale, float max_norm, float *norm, float *coef,
                                int32_t *nonfinite, void *workspace, int64_t workspace_bytes, void *stream) {
    TRY(clip_lengths(n_tensors, lens));
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32) return refuse(ZERO_EINVAL, "unknown dtype %d", dtype);
    if (n_tensors > 0 && !grads) return refuse(ZERO_EINVAL, "grads is NULL");
    if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale)) return refuse(ZERO_EINVAL, "loss_scale must be finite and > 0");
    if (std::isnan(max_norm)) return refuse(ZERO_EINVAL, "max_norm is NaN");
    const uintptr_t size = dtype == ZERO_FP32 ? 4 : 2;
    for (int32_t i = 0; i < n_tensors; ++i) {
        if (lens[i] == 0) continue;
        if (!grads[i] || (out && !out[i])) return refuse(ZERO_EINVAL, "grads[%d] or out[%d] is NULL", i, i);
        if (!aligned(grads[i], size) || (out && !aligned(out[i], size)))
            return refuse(ZERO_EALIGN, "grads[%d] or out[%d] is not aligned to its elements", i, i);
    }
    if (!aligned(norm, 4) || !aligned(coef, 4) || !aligned(nonfinite, 4))
        return refuse(ZERO_EALIGN, "norm, coef or nonfinite is not 4-byte aligned");
    TRY(scratch(workspace, workspace_bytes, zk::clip_bytes(n_tensors, lens)));
    return launched(zk::launch_clip(n_tensors, grads, lens, dtype, out, loss_scale, max_norm, norm, coef, nonfinite,
                                    workspace, static_cast<cudaStream_t>(stream)),
                    "clip kernel launch");
}

}  // extern "C"
