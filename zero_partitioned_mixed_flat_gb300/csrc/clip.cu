// clip.cu -- the global norm over a list of gradient tensors, and the clipped
// gradients, packed where the caller wants them (sm_103a).
//
//   norm = sqrt(sum g^2) / S,  coef = min(1, c / (norm + 1e-6)),  out = g coef
//
// Bound by memory: the coefficient needs every element, so a list larger than
// L2 is read twice and written once (6 bytes an element in 16 bits).  Two
// passes.  The first cuts every tensor into chunks, one block each, and writes a
// double sum of squares per chunk.  The second adds the chunk sums in a fixed
// order, decides the coefficient (the rule of the step's decision) and
// multiplies, the last chunks first: the first pass has left those in L2.  Up to
// kClipEach chunks every block of the second pass decides for itself, which
// saves a launch; a longer list has one block decide in between.
#include "head_internal.h"
#include "launch.h"
#include "zero.h"
#include "zero_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace zk {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVecs = 8;      // 16-byte vectors a thread has in flight
constexpr int kClipChunkBytes = kClipThreads * kClipVecs * 16;  // of one block
constexpr int kClipTable = 640;   // tensors of one launch
constexpr int kClipEach = 1024;   // chunk sums a block of the second pass adds itself

struct ClipParams {
    const void *in[kClipTable];
    void *out[kClipTable];
    long long len[kClipTable];
    int chunk0[kClipTable + 1];  // first block of each tensor in this launch
    int n;
    long long base;   // chunks of the launches before this one
    long long total;  // chunks of every launch
    double *sums;     // one per chunk
    float *decided;   // the coefficient, where a launch of its own decides it; else NULL
    float scale, max_norm;
    float *norm, *coef;
    int *nonfinite;
};

template <int TYPE>
struct Element {
    static constexpr int kBytes = TYPE == ZERO_FP32 ? 4 : 2;
    static constexpr int kPerVec = 16 / kBytes;
    using Word = typename std::conditional<TYPE == ZERO_FP32, uint32_t, uint16_t>::type;

    static __device__ __forceinline__ float value(Word w) {
        if constexpr (TYPE == ZERO_FP16) return __half2float(__ushort_as_half(w));
        if constexpr (TYPE == ZERO_BF16) return __uint_as_float((uint32_t)w << 16);
        if constexpr (TYPE == ZERO_FP32) return __uint_as_float(w);
    }
    static __device__ __forceinline__ Word word(float v) {
        if constexpr (TYPE == ZERO_FP16) return __half_as_ushort(__float2half_rn(v));
        if constexpr (TYPE == ZERO_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
        if constexpr (TYPE == ZERO_FP32) return __float_as_uint(v);
    }
    // the vector's values, and back
    static __device__ __forceinline__ void widen(uint4 q, float v[kPerVec]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (kBytes == 4) {
                v[k] = __uint_as_float(w[k]);
            } else {
                v[2 * k] = value((uint16_t)(w[k] & 0xffffu));
                v[2 * k + 1] = value((uint16_t)(w[k] >> 16));
            }
        }
    }
    static __device__ __forceinline__ uint4 narrow(const float v[kPerVec]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (kBytes == 4)
                w[k] = __float_as_uint(v[k]);
            else
                w[k] = (uint32_t)word(v[2 * k]) | (uint32_t)word(v[2 * k + 1]) << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// the block's chunk: tensor i, elements [e0, e1)
struct Chunk {
    int i;
    long long e0, e1;
};

template <int TYPE>
__device__ __forceinline__ Chunk chunk_of(const ClipParams &p, int block) {
    constexpr int kElems = kClipChunkBytes / Element<TYPE>::kBytes;
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {  // the last tensor that starts at or before the block
        const int mid = (lo + hi + 1) / 2;
        if (p.chunk0[mid] <= block) lo = mid; else hi = mid - 1;
    }
    Chunk c;
    c.i = lo;
    c.e0 = (long long)(block - p.chunk0[lo]) * kElems;
    c.e1 = c.e0 + kElems < p.len[lo] ? c.e0 + kElems : p.len[lo];
    return c;
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

// A chunk is read in 16-byte vectors from its first aligned address; the few
// elements before and after go one by one.  Chunks start a whole number of
// vectors into their tensor, so every chunk of a tensor has the same head.
template <int TYPE>
struct Span {
    using E = Element<TYPE>;
    const typename E::Word *p;
    int head, vecs, tail;  // elements, vectors, elements

    __device__ __forceinline__ Span(const void *tensor, const Chunk &c) {
        p = static_cast<const typename E::Word *>(tensor) + c.e0;
        const int n = (int)(c.e1 - c.e0);
        const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / E::kBytes);
        head = off ? E::kPerVec - off : 0;
        if (head > n) head = n;
        vecs = (n - head) / E::kPerVec;
        tail = n - head - vecs * E::kPerVec;
    }
};

// Sum of squares of a chunk: floats over a thread's own few (four sums of 8 or
// 16 squares), then doubles.  Where a square may have left float's range -- a
// chunk's sum that is not finite although every element is, or so small that
// lost squares could count -- the chunk is summed again in double.  An element
// that is not finite leaves a sum that is not finite, and nothing else does.
template <int TYPE>
__global__ void __launch_bounds__(kClipThreads) clip_norm(const __grid_constant__ ClipParams p) {
    pdl_enter();
    using E = Element<TYPE>;
    __shared__ double shared[kClipThreads / 32];
    if ((int)blockIdx.x < p.chunk0[p.n]) {
        const Chunk c = chunk_of<TYPE>(p, blockIdx.x);
        const Span<TYPE> s(p.in[c.i], c);
        const uint4 *vec = reinterpret_cast<const uint4 *>(s.p + s.head);
        uint4 q[kClipVecs];
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            q[j] = v < s.vecs ? vec[v] : make_uint4(0u, 0u, 0u, 0u);
        }
        // the elements outside the vectors: head and tail have under a vector each
        float edge = 0.0f;
        if (threadIdx.x < s.head) edge = E::value(s.p[threadIdx.x]);
        if (threadIdx.x >= 32 && threadIdx.x - 32 < s.tail)
            edge = E::value(s.p[s.head + s.vecs * E::kPerVec + threadIdx.x - 32]);
        float part[4] = {__fmul_rn(edge, edge), 0.0f, 0.0f, 0.0f}, high = fabsf(edge);
        bool bad = !isfinite(edge);
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            float f[E::kPerVec];
            E::widen(q[j], f);
#pragma unroll
            for (int k = 0; k < E::kPerVec; ++k) {
                part[k & 3] = __fmaf_rn(f[k], f[k], part[k & 3]);
                high = fmaxf(high, fabsf(f[k]));
                bad |= !(fabsf(f[k]) <= 3.402823466e38f);
            }
        }
        double sum = block_sum((double)__fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3])), shared);
        const bool lossy = !(sum <= 1.7e38) || sum < 0x1p-100;
        if (lossy && !__syncthreads_or(bad) && __syncthreads_or(high > 0.0f)) {
            sum = 0.0;
            for (long long e = c.e0 + threadIdx.x; e < c.e1; e += kClipThreads) {
                const double g = E::value(static_cast<const typename E::Word *>(p.in[c.i])[e]);
                sum = __fma_rn(g, g, sum);
            }
            sum = block_sum(sum, shared);
        }
        if (threadIdx.x == 0) p.sums[p.base + blockIdx.x] = sum;
    }
}

// The coefficient from the chunk sums, by a whole block; `write`: also the results.
__device__ float decide(const ClipParams &p, bool write, double *shared) {
    double total = 0.0;
    for (long long k0 = threadIdx.x; k0 < p.total; k0 += 8 * kClipThreads) {
        double v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long k = k0 + j * kClipThreads;
            v[j] = k < p.total ? __ldcg(p.sums + k) : 0.0;
        }
        total += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    total = block_sum(total, shared);
    const double norm = sqrt(total) / (double)p.scale;
    const bool finite = total <= 1.7976931348623157e308;
    float coef = 1.0f;
    if (finite && p.max_norm > 0.0f) {
        const double c = (double)p.max_norm / (norm + 1e-6);
        if (c < 1.0) coef = (float)c;
    }
    if (write && threadIdx.x == 0) {
        if (p.norm) *p.norm = (float)norm;
        if (p.coef) *p.coef = coef;
        if (p.nonfinite) *p.nonfinite = !finite;
    }
    return coef;
}

__global__ void __launch_bounds__(kClipThreads) clip_decide(const __grid_constant__ ClipParams p) {
    pdl_enter();
    __shared__ double shared[kClipThreads / 32];
    const float coef = decide(p, true, shared);
    if (threadIdx.x == 0 && p.decided) *p.decided = coef;
}

// Where source and destination lie alike within 16 bytes, vectors go straight
// through; else (a flat buffer whose tensors have odd lengths) the products go
// through shared memory, so that both sides still move in aligned vectors.
template <int TYPE>
__global__ void __launch_bounds__(kClipThreads) clip_scale(const __grid_constant__ ClipParams p) {
    pdl_enter();
    using E = Element<TYPE>;
    using Word = typename E::Word;
    __shared__ __align__(16) unsigned char staged[kClipChunkBytes + 32];
    __shared__ double shared[kClipThreads / 32];
    const float coef = p.decided ? *p.decided : decide(p, blockIdx.x == 0 && p.base == 0, shared);
    const Chunk c = chunk_of<TYPE>(p, gridDim.x - 1 - blockIdx.x);
    if (coef == 1.0f && p.in[c.i] == p.out[c.i]) return;  // in place, and nothing to change
    const Span<TYPE> s(p.in[c.i], c), d(p.out[c.i], c);
    const uint4 *vec = reinterpret_cast<const uint4 *>(s.p + s.head);
    Word *out = const_cast<Word *>(d.p);
    uint4 q[kClipVecs];
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        const int v = threadIdx.x + j * kClipThreads;
        q[j] = v < s.vecs ? __ldcs(vec + v) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int at = threadIdx.x < 32 ? (int)threadIdx.x : s.head + s.vecs * E::kPerVec + (int)threadIdx.x - 32;
    const bool edge = threadIdx.x < 32 ? (int)threadIdx.x < s.head : (int)threadIdx.x - 32 < s.tail;
    Word lone = 0;
    if (edge) lone = E::word(__fmul_rn(E::value(s.p[at]), coef));
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        float f[E::kPerVec];
        E::widen(q[j], f);
#pragma unroll
        for (int k = 0; k < E::kPerVec; ++k) f[k] = __fmul_rn(f[k], coef);
        q[j] = E::narrow(f);
    }
    if (s.head == d.head) {
        uint4 *to = reinterpret_cast<uint4 *>(out + s.head);
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            if (v < s.vecs) __stcs(to + v, q[j]);
        }
        if (edge) out[at] = lone;
        return;
    }
    // element e of the chunk lies at byte (shift + e) * kBytes of `staged`, so
    // that the source's vectors are aligned there
    Word *stage = reinterpret_cast<Word *>(staged);
    const int shift = s.head ? E::kPerVec - s.head : 0;
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        const int v = threadIdx.x + j * kClipThreads;
        if (v < s.vecs) reinterpret_cast<uint4 *>(stage + shift + s.head)[v] = q[j];
    }
    if (edge) stage[shift + at] = lone;
    __syncthreads();
    uint4 *to = reinterpret_cast<uint4 *>(out + d.head);
    for (int v = threadIdx.x; v < d.vecs; v += kClipThreads) {
        const Word *from = stage + shift + d.head + v * E::kPerVec;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (E::kBytes == 4)
                w[k] = from[k];
            else
                w[k] = (uint32_t)from[2 * k] | (uint32_t)from[2 * k + 1] << 16;
        }
        __stcs(to + v, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (threadIdx.x < d.head) out[threadIdx.x] = stage[shift + threadIdx.x];
    if (threadIdx.x >= 32 && threadIdx.x - 32 < d.tail) {
        const int e = d.head + d.vecs * E::kPerVec + (int)threadIdx.x - 32;
        out[e] = stage[shift + e];
    }
}

template <int TYPE>
long long chunks_of(int64_t len) {
    constexpr int kElems = kClipChunkBytes / Element<TYPE>::kBytes;
    return (len + kElems - 1) / kElems;
}

template <int TYPE>
cudaError_t clip_impl(int n, const void *const *grads, const int64_t *lens, void *const *out, ClipParams &p,
                      cudaStream_t stream) {
    p.total = 0;
    for (int i = 0; i < n; ++i) p.total += chunks_of<TYPE>(lens[i]);
    float *own = p.decided;
    p.decided = p.total > kClipEach ? own : nullptr;
    cudaError_t e = cudaSuccess;
    for (int pass = 0; pass < (out ? 2 : 1) && e == cudaSuccess; ++pass) {
        p.base = 0;
        for (int i = 0; i < n && e == cudaSuccess; p.base += p.chunk0[p.n]) {
            long long blocks = 0;
            p.n = 0;
            for (; i < n && p.n < kClipTable; ++i) {
                if (lens[i] == 0) continue;
                if (p.n > 0 && blocks + chunks_of<TYPE>(lens[i]) > 0x3fffffffll) break;
                p.in[p.n] = grads[i];
                p.out[p.n] = out ? out[i] : nullptr;
                p.len[p.n] = lens[i];
                p.chunk0[p.n++] = (int)blocks;
                blocks += chunks_of<TYPE>(lens[i]);
            }
            p.chunk0[p.n] = (int)blocks;
            if (blocks)
                e = launch_pdl(pass ? clip_scale<TYPE> : clip_norm<TYPE>, dim3((unsigned)blocks), dim3(kClipThreads), 0,
                               stream, p);
        }
        if (pass == 0 && e == cudaSuccess && (p.decided || !out || p.total == 0))
            e = launch_pdl(clip_decide, dim3(1), dim3(kClipThreads), 0, stream, p);
    }
    return e;
}

}  // namespace

int64_t clip_bytes(int n, const int64_t *lens) {
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) chunks += chunks_of<ZERO_FP32>(lens[i]);  // the type with the most chunks
    return 256 + chunks * (int64_t)sizeof(double);
}

cudaError_t launch_clip(int n, const void *const *grads, const int64_t *lens, int dtype, void *const *out,
                        float loss_scale, float max_norm, float *norm, float *coef, int32_t *nonfinite,
                        void *workspace, cudaStream_t stream) {
    ClipParams p;
    p.n = 0;
    p.decided = static_cast<float *>(workspace);  // then, at byte 256, the chunk sums
    p.sums = reinterpret_cast<double *>(static_cast<char *>(workspace) + 256);
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
