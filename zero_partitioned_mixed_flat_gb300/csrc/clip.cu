// clip.cu -- the global norm over a list of gradient tensors, and the clipped
// gradients, packed where the caller wants them (sm_103a).
//
//   norm = sqrt(sum g^2) / S,  coef = min(1, c / (norm + 1e-6)),  out = g coef
//
// Bound by memory: the coefficient needs every element, so a list larger than
// L2 is read twice and written once (6 bytes an element in 16 bits).  Two
// passes over chunks of 32 KB.  The first writes a double sum of squares per
// block, each block taking many chunks; the place of the next chunk is looked up
// while the loads of this one are on their way.  The second has a block for each
// chunk and goes from the list's end, which the first has left in L2.  Between
// them one block adds the sums in a fixed order and decides the coefficient (the
// rule of the step's decision); up to kClipBlocks chunks every block of the second
// pass does that for itself instead, in the same order, which saves the launch.
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
constexpr int kClipChunkBytes = kClipThreads * kClipVecs * 16;
// Tensors of one launch: its table is a kernel parameter, 28 bytes a tensor, which
// the launch copies.  A short list takes the short table.
constexpr int kClipShort = 64, kClipTable = 640;
constexpr int kClipBlocks = 608;  // of one launch: four on each of 152 SMs

template <int TABLE>
struct ClipParams {
    const void *in[TABLE];
    void *out[TABLE];
    long long len[TABLE];
    int chunk0[TABLE + 1];  // first chunk of each tensor in this launch
    int n;
    int base;        // sums of the launches before this one
    int total;       // sums of every launch
    double *sums;
    float *decided;  // the coefficient, where a launch of its own decides it; else NULL
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

// The chunks of a block: every gridDim-th, so that all blocks together move
// through the list in order, forwards or from its end.  A chunk is elements
// [e0, e1) of tensor i.
template <int TYPE, int TABLE>
struct Chunks {
    static constexpr int kElems = kClipChunkBytes / Element<TYPE>::kBytes;
    int at, i;
    long long e0, e1;

    __device__ __forceinline__ explicit Chunks(const ClipParams<TABLE> &p) : at((int)blockIdx.x) {}
    // false after the last; else finds the chunk's place
    __device__ __forceinline__ bool here(const ClipParams<TABLE> &p, bool forwards) {
        const int all = p.chunk0[p.n];
        if (at >= all) return false;
        const int c = forwards ? at : all - 1 - at;
        int hi = p.n - 1;
        i = 0;
        while (i < hi) {  // the last tensor that starts at or before the chunk
            const int mid = (i + hi + 1) / 2;
            if (p.chunk0[mid] <= c) i = mid; else hi = mid - 1;
        }
        e0 = (long long)(c - p.chunk0[i]) * kElems;
        e1 = e0 + kElems < p.len[i] ? e0 + kElems : p.len[i];
        return true;
    }
};

// the sum over the block, in thread 0 (double additions are slow here: no other
// thread does any that it need not)
__device__ __forceinline__ double block_sum(double v, double *shared) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kClipThreads / 32; ++w) t += shared[w];
    return t;
}

// A run of elements as single ones up to the first 16-byte address, vectors, and
// single ones again.
template <int TYPE>
struct Span {
    using E = Element<TYPE>;
    const typename E::Word *p;
    int head, vecs, tail;  // elements, vectors, elements

    __device__ __forceinline__ Span(const void *tensor, long long e0, long long e1) {
        p = static_cast<const typename E::Word *>(tensor) + e0;
        const int n = (int)(e1 - e0);
        const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / E::kBytes);
        head = off ? E::kPerVec - off : 0;
        if (head > n) head = n;
        vecs = (n - head) / E::kPerVec;
        tail = n - head - vecs * E::kPerVec;
    }
    // the single element this thread takes, or -1
    __device__ __forceinline__ int single() const {
        const int t = (int)threadIdx.x;
        if (t < 32) return t < head ? t : -1;
        return t - 32 < tail ? head + vecs * E::kPerVec + t - 32 : -1;
    }
};

// Sum of squares: floats over the 32 or 64 elements a thread has of a chunk (in
// four sums), doubles from there on.  Where a square may have left float's range
// -- the floats' sum not finite, or so small that lost squares could count
// although an element is not zero -- the thread squares the same elements in
// double.  So the sum is not finite exactly where an element is not.
template <int TYPE, int TABLE>
__global__ void __launch_bounds__(kClipThreads) clip_norm(const __grid_constant__ ClipParams<TABLE> p) {
    pdl_enter();
    using E = Element<TYPE>;
    __shared__ double shared[kClipThreads / 32];
    double sum = 0.0;
    Chunks<TYPE, TABLE> c(p);
    for (bool more = c.here(p, true); more;) {
        const Span<TYPE> s(p.in[c.i], c.e0, c.e1);
        const uint4 *vec = reinterpret_cast<const uint4 *>(s.p + s.head);
        uint4 q[kClipVecs];
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            q[j] = v < s.vecs ? vec[v] : make_uint4(0u, 0u, 0u, 0u);
        }
        const int one = s.single();
        const float edge = one >= 0 ? E::value(s.p[one]) : 0.0f;
        c.at += gridDim.x;
        more = c.here(p, true);
        float part[4] = {__fmul_rn(edge, edge), 0.0f, 0.0f, 0.0f};
        uint32_t bits = 0u;
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            float f[E::kPerVec];
            E::widen(q[j], f);
            bits |= q[j].x | q[j].y | q[j].z | q[j].w;
#pragma unroll
            for (int k = 0; k < E::kPerVec; ++k) part[k & 3] = __fmaf_rn(f[k], f[k], part[k & 3]);
        }
        const float few = __fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3]));
        constexpr uint32_t kMagnitude = E::kBytes == 4 ? 0x7fffffffu : 0x7fff7fffu;
        if (few >= 0x1p-100f && few <= 1.7e38f) {
            sum += (double)few;
        } else if ((bits & kMagnitude) || edge != 0.0f) {
            sum = __fma_rn((double)edge, (double)edge, sum);
#pragma unroll 1
            for (int j = 0; j < kClipVecs; ++j) {
                const int v = threadIdx.x + j * kClipThreads;
                float f[E::kPerVec];
                E::widen(v < s.vecs ? vec[v] : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
                for (int k = 0; k < E::kPerVec; ++k) sum = __fma_rn((double)f[k], (double)f[k], sum);
            }
        }
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) p.sums[p.base + blockIdx.x] = sum;
}

// The coefficient from the blocks' sums, by a whole block; `write`: also the results.
template <int TABLE>
__device__ __forceinline__ float decide(const ClipParams<TABLE> &p, bool write) {
    __shared__ double shared[kClipThreads / 32];
    __shared__ float decision;
    double total = 0.0;
    for (int k0 = threadIdx.x; k0 < p.total; k0 += 4 * kClipThreads) {
        double v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = k0 + j * kClipThreads < p.total ? __ldcg(p.sums + k0 + j * kClipThreads) : 0.0;
        total += (v[0] + v[1]) + (v[2] + v[3]);
    }
    total = block_sum(total, shared);
    if (threadIdx.x == 0) {
        const double norm = sqrt(total) / (double)p.scale;
        const bool finite = total <= 1.7976931348623157e308;
        float coef = 1.0f;
        if (finite && p.max_norm > 0.0f) {
            const double c = (double)p.max_norm / (norm + 1e-6);
            if (c < 1.0) coef = (float)c;
        }
        decision = coef;
        if (write) {
            if (p.norm) *p.norm = (float)norm;
            if (p.coef) *p.coef = coef;
            if (p.nonfinite) *p.nonfinite = !finite;
        }
    }
    __syncthreads();
    return decision;
}

template <int TABLE>
__global__ void __launch_bounds__(kClipThreads) clip_decide(const __grid_constant__ ClipParams<TABLE> p) {
    pdl_enter();
    const float coef = decide(p, true);
    if (p.decided && threadIdx.x == 0) *p.decided = coef;
}

// the 16 bytes that start `off` bytes (a multiple of the element's) into lo, hi
__device__ __forceinline__ uint4 straddle(const uint4 &lo, const uint4 &hi, int off) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const bool one = off & 4, two = off & 8;
    uint32_t a[6], b[5], r[4];
#pragma unroll
    for (int k = 0; k < 6; ++k) a[k] = two ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) b[k] = one ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __funnelshift_r(b[k], b[k + 1], (off & 3) * 8);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The destination's aligned vectors decide what a thread takes.  Where the source
// lies otherwise within 16 bytes (a flat buffer whose tensors have odd lengths),
// a vector's elements straddle two of the source's aligned vectors, this lane's and
// the next lane's; the first and last vector of a chunk are then read element by
// element, so that nothing outside the tensor is read.
template <int TYPE, int TABLE>
__global__ void __launch_bounds__(kClipThreads) clip_scale(const __grid_constant__ ClipParams<TABLE> p) {
    pdl_enter();
    using E = Element<TYPE>;
    using Word = typename E::Word;
    Chunks<TYPE, TABLE> c(p);
    c.here(p, false);
    const float coef = p.decided ? *p.decided : decide(p, blockIdx.x == 0 && p.base == 0);
    if (coef == 1.0f && p.in[c.i] == p.out[c.i]) return;  // in place, and nothing to change
    const Span<TYPE> d(p.out[c.i], c.e0, c.e1);
    const Word *src = static_cast<const Word *>(p.in[c.i]) + c.e0;
    Word *out = const_cast<Word *>(d.p);
    const Word *from = src + d.head;  // of the first vector
    const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15u);
    uint4 q[kClipVecs];
    if (off == 0) {
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            if (v < d.vecs) q[j] = __ldcs(reinterpret_cast<const uint4 *>(from) + v);
        }
    } else {
        const uint4 *low = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(from) - off);
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            q[j] = v > 0 && v < d.vecs ? __ldg(low + v) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            const int v = threadIdx.x + j * kClipThreads;
            uint4 hi;  // the next lane's
            hi.x = __shfl_down_sync(0xffffffffu, q[j].x, 1);
            hi.y = __shfl_down_sync(0xffffffffu, q[j].y, 1);
            hi.z = __shfl_down_sync(0xffffffffu, q[j].z, 1);
            hi.w = __shfl_down_sync(0xffffffffu, q[j].w, 1);
            if ((threadIdx.x & 31) == 31 && v + 1 < d.vecs) hi = __ldg(low + v + 1);
            q[j] = straddle(q[j], hi, off);
        }
    }
    const int one = d.single();
    if (one >= 0) out[one] = E::word(__fmul_rn(E::value(src[one]), coef));
    uint4 *to = reinterpret_cast<uint4 *>(out + d.head);
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        const int v = threadIdx.x + j * kClipThreads;
        if (v >= d.vecs) break;
        float f[E::kPerVec];
        if (off && (v == 0 || v + 1 == d.vecs)) {
#pragma unroll
            for (int k = 0; k < E::kPerVec; ++k) f[k] = E::value(from[v * E::kPerVec + k]);
        } else {
            E::widen(q[j], f);
        }
#pragma unroll
        for (int k = 0; k < E::kPerVec; ++k) f[k] = __fmul_rn(f[k], coef);
        __stcs(to + v, E::narrow(f));
    }
}

template <int TYPE>
long long chunks_of(int64_t len) {
    constexpr int kElems = kClipChunkBytes / Element<TYPE>::kBytes;
    return (len + kElems - 1) / kElems;
}

template <int TYPE, int TABLE>
cudaError_t clip_impl(int n, const void *const *grads, const int64_t *lens, void *const *out, float loss_scale,
                      float max_norm, float *norm, float *coef, int32_t *nonfinite, void *workspace,
                      cudaStream_t stream) {
    ClipParams<TABLE> p;
    p.n = 0;
    p.base = 0;
    p.total = 0;
    float *decided = static_cast<float *>(workspace);  // then, at byte 16, the sums
    p.sums = static_cast<double *>(workspace) + 2;
    p.scale = loss_scale;
    p.max_norm = max_norm;
    p.norm = norm;
    p.coef = coef;
    p.nonfinite = nonfinite;
    long long all = 0;
    for (int i = 0; i < n; ++i) all += chunks_of<TYPE>(lens[i]);
    p.decided = all > kClipBlocks ? decided : nullptr;
    cudaError_t e = cudaSuccess;
    for (int pass = 0; pass < (out ? 2 : 1) && e == cudaSuccess; ++pass) {
        p.base = 0;
        for (int i = 0; i < n && e == cudaSuccess;) {
            long long chunks = 0;
            p.n = 0;
            for (; i < n && p.n < TABLE; ++i) {
                if (lens[i] == 0) continue;
                if (p.n > 0 && chunks + chunks_of<TYPE>(lens[i]) > 0x3fffffffll) break;
                p.in[p.n] = grads[i];
                p.out[p.n] = out ? out[i] : nullptr;
                p.len[p.n] = lens[i];
                p.chunk0[p.n++] = (int)chunks;
                chunks += chunks_of<TYPE>(lens[i]);
            }
            p.chunk0[p.n] = (int)chunks;
            if (chunks == 0) continue;
            const int sums = (int)(chunks < kClipBlocks ? chunks : kClipBlocks);
            e = launch_pdl(pass ? clip_scale<TYPE, TABLE> : clip_norm<TYPE, TABLE>, dim3((unsigned)(pass ? chunks : sums)),
                           dim3(kClipThreads), 0, stream, p);
            p.base += sums;
        }
        if (pass > 0) break;
        p.total = p.base;
        if (e == cudaSuccess && (p.decided || !out || p.total == 0))
            e = launch_pdl(clip_decide<TABLE>, dim3(1), dim3(kClipThreads), 0, stream, p);
    }
    return e;
}

}  // namespace

int64_t clip_bytes(int n, const int64_t *lens) {
    // launches: one for every kClipTable tensors, or for every 2^30 chunks
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) chunks += chunks_of<ZERO_FP32>(lens[i]);  // the type with the most chunks
    const int64_t launches = n / kClipTable + 1 + 2 * (chunks >> 29);
    return 16 + (chunks < launches * kClipBlocks ? chunks : launches * kClipBlocks) * (int64_t)sizeof(double);
}

cudaError_t launch_clip(int n, const void *const *grads, const int64_t *lens, int dtype, void *const *out,
                        float loss_scale, float max_norm, float *norm, float *coef, int32_t *nonfinite,
                        void *workspace, cudaStream_t stream) {
    const auto clip = [&](auto type) {
        constexpr int kType = decltype(type)::value;
        if (n <= kClipShort)
            return clip_impl<kType, kClipShort>(n, grads, lens, out, loss_scale, max_norm, norm, coef, nonfinite, workspace,
                                                stream);
        return clip_impl<kType, kClipTable>(n, grads, lens, out, loss_scale, max_norm, norm, coef, nonfinite, workspace,
                                            stream);
    };
    if (dtype == ZERO_FP16) return clip(std::integral_constant<int, ZERO_FP16>());
    if (dtype == ZERO_BF16) return clip(std::integral_constant<int, ZERO_BF16>());
    return clip(std::integral_constant<int, ZERO_FP32>());
}

}  // namespace zk
