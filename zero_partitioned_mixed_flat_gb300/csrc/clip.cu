// clip.cu -- the global norm over a list of gradient tensors, and the clipped
// gradients, packed where the caller wants them (sm_103a).
//
// Two streaming passes.  The first cuts every tensor into chunks, one block
// each, and writes a double sum of squares per chunk; the last block to finish
// adds the chunk sums in a fixed order and decides the coefficient (the rule of
// the step's decision).  The second multiplies.
#include "head_internal.h"
#include "launch.h"
#include "zero.h"
#include "zero_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace zk {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 16384;  // elements of one block
constexpr int kClipTable = 512;    // tensors of one launch

// the head of the workspace; the chunk sums follow at byte 256
struct ClipRecord {
    float coef;
    int nonfinite;
    unsigned arrivals;
};

struct ClipParams {
    const void *in[kClipTable];
    void *out[kClipTable];
    long long len[kClipTable];
    int chunk0[kClipTable + 1];  // first block of each tensor in this launch
    int n;
    long long base;   // chunks of the launches before this one
    long long total;  // chunks of every launch
    ClipRecord *record;
    double *sums;
    float scale, max_norm;
    float *norm, *coef;
    int *nonfinite;
    int last;  // this launch decides
};

template <int TYPE>
__device__ __forceinline__ float element(const void *p, long long i) {
    if constexpr (TYPE == ZERO_FP16) return __half2float(static_cast<const __half *>(p)[i]);
    if constexpr (TYPE == ZERO_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

__device__ int tensor_of(const ClipParams &p, int block) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {  // the last tensor that starts at or before the block
        const int mid = (lo + hi + 1) / 2;
        if (p.chunk0[mid] <= block) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ double block_sum(double v, double *shared) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < kClipThreads / 32; ++w) t += shared[w];
    __syncthreads();
    return t;
}

template <int TYPE>
__global__ void __launch_bounds__(kClipThreads) clip_norm(const __grid_constant__ ClipParams p) {
    pdl_enter();
    __shared__ double shared[kClipThreads / 32];
    __shared__ bool decide;
    double sum = 0.0;
    bool bad = false;
    if ((int)blockIdx.x < p.chunk0[p.n]) {
        const int i = tensor_of(p, blockIdx.x);
        const long long e0 = (long long)(blockIdx.x - p.chunk0[i]) * kClipChunk;
        const long long e1 = e0 + kClipChunk < p.len[i] ? e0 + kClipChunk : p.len[i];
        for (long long e = e0 + threadIdx.x; e < e1; e += kClipThreads) {
            const float g = element<TYPE>(p.in[i], e);
            bad |= !isfinite(g);
            sum += (double)g * (double)g;
        }
    }
    sum = block_sum(sum, shared);
    const bool any = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if ((int)blockIdx.x < p.chunk0[p.n]) p.sums[p.base + blockIdx.x] = sum;
        if (any) atomicOr(&p.record->nonfinite, 1);
        __threadfence();
        decide = atomicAdd(&p.record->arrivals, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!decide) return;
    __threadfence();
    if (threadIdx.x == 0) p.record->arrivals = 0u;
    if (!p.last) return;
    double total = 0.0;
    for (long long k = threadIdx.x; k < p.total; k += kClipThreads) total += __ldcg(p.sums + k);
    total = block_sum(total, shared);
    if (threadIdx.x != 0) return;
    const double norm = sqrt(total) / (double)p.scale;
    const int nonfinite = atomicOr(&p.record->nonfinite, 0);
    float coef = 1.0f;
    if (!nonfinite && p.max_norm > 0.0f) {
        const double c = (double)p.max_norm / (norm + 1e-6);
        if (c < 1.0) coef = (float)c;
    }
    p.record->coef = coef;
    if (p.norm) *p.norm = (float)norm;
    if (p.coef) *p.coef = coef;
    if (p.nonfinite) *p.nonfinite = nonfinite;
}

template <int TYPE>
__global__ void __launch_bounds__(kClipThreads) clip_scale(const __grid_constant__ ClipParams p) {
    pdl_enter();
    const float coef = p.record->coef;
    const int i = tensor_of(p, blockIdx.x);
    const long long e0 = (long long)(blockIdx.x - p.chunk0[i]) * kClipChunk;
    const long long e1 = e0 + kClipChunk < p.len[i] ? e0 + kClipChunk : p.len[i];
    for (long long e = e0 + threadIdx.x; e < e1; e += kClipThreads) {
        const float g = element<TYPE>(p.in[i], e) * coef;
        if constexpr (TYPE == ZERO_FP16) static_cast<__half *>(p.out[i])[e] = __float2half_rn(g);
        if constexpr (TYPE == ZERO_BF16) static_cast<__nv_bfloat16 *>(p.out[i])[e] = __float2bfloat16_rn(g);
        if constexpr (TYPE == ZERO_FP32) static_cast<float *>(p.out[i])[e] = g;
    }
}

long long chunks_of(int64_t len) { return (len + kClipChunk - 1) / kClipChunk; }

template <int TYPE>
cudaError_t clip_impl(int n, const void *const *grads, const int64_t *lens, void *const *out, ClipParams &p,
                      cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(p.record, 0, sizeof(ClipRecord), stream);
    for (int pass = 0; pass < (out ? 2 : 1) && e == cudaSuccess; ++pass) {
        p.base = 0;
        int i = 0;
        do {
            long long blocks = 0;
            p.n = 0;
            for (; i < n && p.n < kClipTable; ++i) {
                if (lens[i] == 0) continue;
                if (p.n > 0 && blocks + chunks_of(lens[i]) > 0x3fffffffll) break;
                p.in[p.n] = grads[i];
                p.out[p.n] = out ? out[i] : nullptr;
                p.len[p.n] = lens[i];
                p.chunk0[p.n++] = (int)blocks;
                blocks += chunks_of(lens[i]);
            }
            p.chunk0[p.n] = (int)blocks;
            p.last = i == n;
            if (pass == 0)
                e = launch_pdl(clip_norm<TYPE>, dim3(blocks ? (unsigned)blocks : 1u), dim3(kClipThreads), 0, stream, p);
            else if (blocks)
                e = launch_pdl(clip_scale<TYPE>, dim3((unsigned)blocks), dim3(kClipThreads), 0, stream, p);
            p.base += blocks;
        } while (i < n && e == cudaSuccess);
    }
    return e;
}

}  // namespace

int64_t clip_bytes(int n, const int64_t *lens) {
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) chunks += chunks_of(lens[i]);
    return 256 + chunks * (int64_t)sizeof(double);
}

cudaError_t launch_clip(int n, const void *const *grads, const int64_t *lens, int dtype, void *const *out,
                        float loss_scale, float max_norm, float *norm, float *coef, int32_t *nonfinite,
                        void *workspace, cudaStream_t stream) {
    ClipParams p;
    p.record = static_cast<ClipRecord *>(workspace);
    p.sums = reinterpret_cast<double *>(static_cast<char *>(workspace) + 256);
    p.total = (clip_bytes(n, lens) - 256) / (int64_t)sizeof(double);
    p.scale = loss_scale;
    p.max_norm = max_norm;
    p.norm = norm;
    p.coef = coef;
    p.nonfinite = nonfinite;
    if (dtype == ZERO_FP16) return clip_impl<ZERO_FP16>(n, grads, lens, out, p, stream);
    if (dtype == ZERO_BF16) return clip_impl<ZERO_BF16>(n, grads, lens, out, p, stream);
    return clip_impl<ZERO_FP32>(n, grads, lens, out, p, stream);
}

}  // namespace zk
