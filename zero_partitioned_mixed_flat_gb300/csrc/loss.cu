// loss.cu -- softmax cross entropy of hidden states against a vocabulary
// matrix, without keeping the logits, and its gradients (sm_103a).
#include "head_internal.h"
#include "launch.h"
#include "zero.h"
#include "zero_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace zk {
namespace {

constexpr int kT = 64;    // tile: kT x kT outputs, kK products at a time
constexpr int kK = 16;
constexpr int kThreads = 256;  // 16 x 16 threads, 4 x 4 outputs each

template <bool BF16>
__device__ __forceinline__ float lp_get(const void *p, long long i) {
    if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}

template <bool BF16>
__device__ __forceinline__ void lp_put(void *p, long long i, float v) {
    if constexpr (BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// acc[4][4] of the tile at (m0, n0): sum over k of a(m, k) b(n, k)
template <typename A, typename B>
__device__ void tile_product(A a, B b, long long m0, long long n0, long long k1, float acc[4][4]) {
    __shared__ float as[kK][kT + 1], bs[kK][kT + 1];
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    for (long long k0 = 0; k0 < k1; k0 += kK) {
        for (int e = threadIdx.x; e < kT * kK; e += kThreads) {
            as[e % kK][e / kK] = k0 + e % kK < k1 ? a(m0 + e / kK, k0 + e % kK) : 0.0f;
            bs[e % kK][e / kK] = k0 + e % kK < k1 ? b(n0 + e / kK, k0 + e % kK) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

// the logits' tile of block (x: vocabulary, y: tokens)
template <bool BF16>
__device__ void logits_tile(const LossArgs &p, long long m0, long long n0, float acc[4][4]) {
    tile_product(
        [&](long long m, long long k) { return m < p.tokens ? lp_get<BF16>(p.hidden, m * p.hidden_stride + k) : 0.0f; },
        [&](long long n, long long k) { return n < p.vocab ? lp_get<BF16>(p.weight, n * p.weight_stride + k) : 0.0f; },
        m0, n0, p.dim, acc);
}

// forward workspace: partial (maximum, sum) [tile][token], then target logits
template <bool BF16>
__global__ void loss_tiles(const LossArgs p) {
    pdl_enter();
    const long long m0 = (long long)blockIdx.y * kT, n0 = (long long)blockIdx.x * kT;
    float acc[4][4];
    logits_tile<BF16>(p, m0, n0, acc);
    __shared__ float z[kT][kT + 1];
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) z[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    const long long t = m0 + threadIdx.x;
    if (threadIdx.x >= kT || t >= p.tokens) return;
    const int n = p.vocab - n0 < kT ? (int)(p.vocab - n0) : kT;
    float top = -INFINITY, sum = 0.0f;
    for (int j = 0; j < n; ++j) top = fmaxf(top, z[threadIdx.x][j]);
    for (int j = 0; j < n; ++j) sum += expf(z[threadIdx.x][j] - top);
    float2 *part = static_cast<float2 *>(p.workspace);
    part[blockIdx.x * p.tokens + t] = make_float2(top, sum);
    const long long at = p.target[t] - n0;
    if (at >= 0 && at < n) reinterpret_cast<float *>(part + (long long)gridDim.x * p.tokens)[t] = z[threadIdx.x][at];
}

__global__ void loss_join(const LossArgs p, int tiles) {
    pdl_enter();
    const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (t >= p.tokens) return;
    const float2 *part = static_cast<const float2 *>(p.workspace);
    float top = -INFINITY, sum = 0.0f;
    for (int i = 0; i < tiles; ++i) top = fmaxf(top, part[i * p.tokens + t].x);
    for (int i = 0; i < tiles; ++i) sum += part[i * p.tokens + t].y * expf(part[i * p.tokens + t].x - top);
    const float lse = top + logf(sum);
    p.lse[t] = lse;
    const long long y = p.target[t];
    if (y == p.ignore) {
        p.loss[t] = 0.0f;
    } else if (y < 0 || y >= p.vocab) {
        p.loss[t] = NAN;
        atomicOr(p.status, ZERO_LOSS_BAD_TARGET);
    } else {
        p.loss[t] = lse - reinterpret_cast<const float *>(part + (long long)tiles * p.tokens)[t];
    }
}

__device__ __forceinline__ bool counted(const LossArgs &p, long long t) {
    const long long y = p.target[t];
    return y != p.ignore && y >= 0 && y < p.vocab;
}

// backward workspace: one float (the largest finite |grad_loss|), then at byte
// 256 the float gradients of a piece of the vocabulary, then grad_hidden's sums
constexpr long long kPiece = 4096;

__global__ void loss_largest(const LossArgs p) {
    pdl_enter();
    __shared__ float shared[kThreads];
    float top = 0.0f;
    for (long long t = threadIdx.x; t < p.tokens; t += kThreads) {
        const float g = fabsf(p.grad_loss[t]);
        if (counted(p, t) && g <= 3.402823466e38f) top = fmaxf(top, g);
        if (p.target[t] != p.ignore && !counted(p, t)) atomicOr(p.status, ZERO_LOSS_BAD_TARGET);
    }
    shared[threadIdx.x] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads; ++i) top = fmaxf(top, shared[i]);
        *static_cast<float *>(p.workspace) = top;
    }
}

__device__ __forceinline__ float *slopes(const LossArgs &p) { return static_cast<float *>(p.workspace) + 64; }

template <bool BF16>
__global__ void loss_slopes(const LossArgs p, long long piece0) {
    pdl_enter();
    const long long m0 = (long long)blockIdx.y * kT, n0 = piece0 + (long long)blockIdx.x * kT;
    float acc[4][4];
    logits_tile<BF16>(p, m0, n0, acc);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i) {
        const long long t = m0 + ty * 4 + i;
        if (t >= p.tokens) continue;
        const bool counts = counted(p, t);
        for (int j = 0; j < 4; ++j) {
            const long long v = n0 + tx * 4 + j;
            float q = 0.0f;
            if (counts && v < p.vocab) q = (expf(acc[i][j] - p.lse[t]) - (v == p.target[t] ? 1.0f : 0.0f)) * p.grad_loss[t];
            slopes(p)[t * kPiece + v - piece0] = q;
        }
    }
}

template <bool BF16>
__global__ void loss_grad_hidden(const LossArgs p, long long piece0) {
    pdl_enter();
    const long long m0 = (long long)blockIdx.y * kT, n0 = (long long)blockIdx.x * kT;
    const long long n = p.vocab - piece0 < kPiece ? p.vocab - piece0 : kPiece;
    float acc[4][4];
    tile_product([&](long long m, long long k) { return m < p.tokens ? slopes(p)[m * kPiece + k] : 0.0f; },
                 [&](long long d, long long k) {
                     return d < p.dim ? lp_get<BF16>(p.weight, (piece0 + k) * p.weight_stride + d) : 0.0f;
                 },
                 m0, n0, n, acc);
    float *sums = slopes(p) + p.tokens * kPiece;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long t = m0 + ty * 4 + i, d = n0 + tx * 4 + j;
            if (t >= p.tokens || d >= p.dim) continue;
            const float v = acc[i][j] + (piece0 ? sums[t * p.dim + d] : 0.0f);
            sums[t * p.dim + d] = v;
            if (piece0 + n == p.vocab) lp_put<BF16>(p.grad_hidden, t * p.grad_hidden_stride + d, v);
        }
}

template <bool BF16>
__global__ void loss_grad_weight(const LossArgs p, long long piece0) {
    pdl_enter();
    const long long m0 = (long long)blockIdx.y * kT, n0 = (long long)blockIdx.x * kT;
    float acc[4][4];
    tile_product([&](long long m, long long k) { return m < kPiece ? slopes(p)[k * kPiece + m] : 0.0f; },
                 [&](long long d, long long k) {
                     return d < p.dim && counted(p, k) ? lp_get<BF16>(p.hidden, k * p.hidden_stride + d) : 0.0f;
                 },
                 m0, n0, p.tokens, acc);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long v = piece0 + m0 + ty * 4 + i, d = n0 + tx * 4 + j;
            if (v < p.vocab && d < p.dim) lp_put<BF16>(p.grad_weight, v * p.grad_weight_stride + d, acc[i][j]);
        }
}

unsigned tiles(int64_t n) { return (unsigned)((n + kT - 1) / kT); }

}  // namespace

int64_t loss_forward_bytes(int64_t tokens, int64_t vocab) { return (int64_t)tiles(vocab) * tokens * 8 + tokens * 4; }

cudaError_t launch_loss_forward(const LossArgs &a, cudaStream_t stream) {
    if (tiles(a.tokens) > 65535u) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(a.lp ? loss_tiles<true> : loss_tiles<false>, dim3(tiles(a.vocab), tiles(a.tokens)),
                               dim3(kThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(loss_join, dim3((unsigned)((a.tokens + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, a,
                      (int)tiles(a.vocab));
}

int64_t loss_backward_bytes(int64_t tokens, int64_t vocab, int dim) { return 256 + tokens * (kPiece + dim) * 4; }

cudaError_t launch_loss_backward(const LossArgs &a, cudaStream_t stream) {
    if (tiles(a.tokens) > 65535u) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(loss_largest, dim3(1), dim3(kThreads), 0, stream, a);
    for (long long piece0 = 0; piece0 < a.vocab; piece0 += kPiece) {
        const dim3 by_token(tiles(kPiece), tiles(a.tokens)), sums(tiles(a.dim), tiles(a.tokens));
        const dim3 rows(tiles(a.dim), tiles(std::min<long long>(kPiece, a.vocab - piece0)));
        if (e == cudaSuccess && a.tokens)
            e = launch_pdl(a.lp ? loss_slopes<true> : loss_slopes<false>, by_token, dim3(kThreads), 0, stream, a, piece0);
        if (e == cudaSuccess && a.tokens)
            e = launch_pdl(a.lp ? loss_grad_hidden<true> : loss_grad_hidden<false>, sums, dim3(kThreads), 0, stream, a,
                           piece0);
        if (e == cudaSuccess)
            e = launch_pdl(a.lp ? loss_grad_weight<true> : loss_grad_weight<false>, rows, dim3(kThreads), 0, stream, a,
                           piece0);
    }
    return e;
}

}  // namespace zk
