// norm.cu -- residual addition + root-mean-square norm of rows, its 8-bit
// outputs, and its gradients (sm_103a).
#include "head_internal.h"
#include "launch.h"
#include "quant_codes.cuh"
#include "zero_internal.h"

namespace zk {
namespace {

constexpr int kNormRowThreads = 256;

template <bool BF16>
__device__ __forceinline__ float lp_load(const void *p, long long i) {
    if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}

template <bool BF16>
__device__ __forceinline__ void lp_store(void *p, long long i, float v) {
    if constexpr (BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

__device__ float block_sum(float v, float *shared) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < kNormRowThreads / 32; ++w) t += shared[w];
    __syncthreads();
    return t;
}

template <bool BF16>
__global__ void norm_row(const NormArgs a) {
    pdl_enter();
    __shared__ float shared[kNormRowThreads / 32];
    const long long row = blockIdx.x;
    const long long x0 = row * a.x_stride, r0 = row * a.residual_stride;
    auto at = [&](int i) {
        const float x = lp_load<BF16>(a.x, x0 + i);
        return a.residual ? x + lp_load<BF16>(a.residual, r0 + i) : x;
    };
    float sq = 0.0f;
    for (int i = threadIdx.x; i < a.dim; i += kNormRowThreads) {
        const float s = at(i);
        sq += s * s;
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, shared) / a.dim + a.eps);
    if (a.out) {
        for (int i = threadIdx.x; i < a.dim; i += kNormRowThreads) {
            const float s = at(i);
            lp_store<BF16>(a.out, row * a.out_stride + i, s * rstd * lp_load<BF16>(a.weight, i));
            if (a.sum) lp_store<BF16>(a.sum, row * a.sum_stride + i, s);
        }
        return;
    }
    // codes: a warp takes a block of 128, four elements a lane
    const int n_blocks = (a.dim + 127) / 128, lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < n_blocks; b += kNormRowThreads / 32) {
        float y[4], top = 0.0f;
        for (int k = 0; k < 4; ++k) {
            const int i = b * 128 + lane * 4 + k;
            y[k] = 0.0f;
            if (i < a.dim) {
                const float s = at(i);
                if (a.sum) lp_store<BF16>(a.sum, row * a.sum_stride + i, s);
                y[k] = s * rstd * lp_load<BF16>(a.weight, i);
            }
            top = fmaxf(top, fabsf(y[k]));
        }
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float scale;
        uint32_t word;
        if (a.fp8) {
            quant_codes_fp8<4>(y, top, scale, &word);
        } else {
            scale = __fdiv_rn(top, 127.0f);
            quant_codes<4>(y, scale, &word);
        }
        if (lane == 0) a.scales[row * n_blocks + b] = scale;
        if (b * 128 + lane * 4 < a.dim) reinterpret_cast<uint32_t *>(a.codes + row * a.dim)[b * 32 + lane] = word;
    }
}

template <bool BF16>
__global__ void dequantize_row(const int8_t *codes, const float *scales, int fp8, int dim, void *out,
                               long long out_stride) {
    pdl_enter();
    const long long row = blockIdx.x;
    const int n_blocks = (dim + 127) / 128;
    for (int i = threadIdx.x; i < dim; i += kNormRowThreads) {
        const uint32_t c = (uint8_t)codes[row * dim + i];
        const float v = fp8 ? from_e4m3x2(c).x : (float)(int8_t)c;
        lp_store<BF16>(out, row * out_stride + i, v * scales[row * n_blocks + i / 128]);
    }
}

template <bool BF16>
__global__ void norm_row_backward(const NormBackwardArgs a) {
    pdl_enter();
    __shared__ float shared[kNormRowThreads / 32];
    const long long row = blockIdx.x;
    auto s_at = [&](int i) { return lp_load<BF16>(a.sum, row * a.sum_stride + i); };
    auto g_at = [&](int i) { return lp_load<BF16>(a.grad_out, row * a.grad_out_stride + i); };
    float sq = 0.0f, dot = 0.0f;
    for (int i = threadIdx.x; i < a.dim; i += kNormRowThreads) {
        const float s = s_at(i);
        sq += s * s;
        dot += g_at(i) * lp_load<BF16>(a.weight, i) * s;
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, shared) / a.dim + a.eps);
    const float along = block_sum(dot, shared) / a.dim * rstd * rstd;
    for (int i = threadIdx.x; i < a.dim; i += kNormRowThreads) {
        const float s = s_at(i);
        float g = rstd * (g_at(i) * lp_load<BF16>(a.weight, i) - s * along);
        if (a.grad_sum) g += lp_load<BF16>(a.grad_sum, row * a.grad_sum_stride + i);
        static_cast<float *>(a.workspace)[row * a.dim + i] = g_at(i) * s * rstd;
        lp_store<BF16>(a.grad_in, row * a.grad_in_stride + i, g);
    }
}

template <bool BF16>
__global__ void norm_weight_sum(const NormBackwardArgs a) {
    pdl_enter();
    const int i = blockIdx.x * kNormRowThreads + threadIdx.x;
    if (i >= a.dim) return;
    float t = 0.0f;
    for (long long r = 0; r < a.rows; ++r) t += static_cast<const float *>(a.workspace)[r * a.dim + i];
    lp_store<BF16>(a.grad_weight, i, t);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream) {
    return launch_pdl(a.lp ? norm_row<true> : norm_row<false>, dim3((unsigned)a.rows), dim3(kNormRowThreads), 0,
                      stream, a);
}

cudaError_t launch_dequantize_rows(const int8_t *codes, const float *scales, int fp8, int64_t rows, int dim,
                                   int lp, void *out, int64_t out_stride, cudaStream_t stream) {
    return launch_pdl(lp ? dequantize_row<true> : dequantize_row<false>, dim3((unsigned)rows), dim3(kNormRowThreads),
                      0, stream, codes, scales, fp8, dim, out, (long long)out_stride);
}

int64_t norm_backward_bytes(int64_t rows, int dim) { return rows * dim * (int64_t)sizeof(float); }

cudaError_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream) {
    if (a.rows > 0) {
        cudaError_t e = launch_pdl(a.lp ? norm_row_backward<true> : norm_row_backward<false>, dim3((unsigned)a.rows),
                                   dim3(kNormRowThreads), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(a.lp ? norm_weight_sum<true> : norm_weight_sum<false>,
                      dim3((unsigned)((a.dim + kNormRowThreads - 1) / kNormRowThreads)), dim3(kNormRowThreads), 0,
                      stream, a);
}

}  // namespace zk
