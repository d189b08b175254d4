// adamw.cu -- one AdamW step over a list of tensors, the moments in 32 or in 8 bits (sm_103a).
//
// For every element, with g' = g * coef / S, t the step and c = 1 - beta^t:
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps),  copy = lp(p)
// Bound by memory: 24 bytes an element and the gradient and copy with 32-bit moments, 12
// with 8-bit ones.  Everything is read once and written once: a warp takes blocks of 128
// elements, each lane four of them, holds a whole block in registers and finds the new
// scales there, so 8-bit moments need no second pass.
//
// 8 bits.  Of a block of 128: m as E4M3 times the block's scale (the largest |m| / 448), the
// root of v as an unsigned number of three exponent and five mantissa bits times its own (the
// largest root / the largest code's value).  Holding the root halves the exponents that are
// needed: steps of 2^-5 to 2^-6 of the root over 2^12, v over 2^24.  A moment decays by
// less than a step, so rounding to nearest would leave most codes as they are for ever;
// they are rounded up or down at random instead, in proportion, which leaves the
// mean right: 16 random bits each from a hash of seed, step and element.  The largest
// element of a block needs no rounding and its scale is a float, so what all of a block have in
// common is kept exactly.  A root above zero never becomes zero: m / eps would follow.
#include "head_internal.h"
#include "launch.h"
#include "per_device.h"
#include "quant_codes.cuh"
#include "zero.h"
#include "zero_internal.h"

#include <algorithm>
#include <type_traits>

namespace zk {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = ZERO_QUANT_BLOCK;  // a warp's 32 lanes x 4
// Blocks of 128 that a warp has in flight: 16 or 8 elements a lane.
template <int BITS>
constexpr int kDepth = BITS == 8 ? 4 : 2;
template <int BITS>
constexpr int kChunkBlocks = kWarps * kDepth<BITS>;  // blocks of 128 of a chunk
// Tensors of one launch: the table is a kernel parameter, 44 bytes a tensor.
constexpr int kShort = 64, kTable = 640;

constexpr float kTopM = 448.0f, kTopR = 1.96875f / 256.0f;
constexpr float kLeastScale = 0x1p-126f;  // a scale below it is 0, and so are its codes

struct AdamwScalars {
    float lr, beta1, beta2, omb1, omb2, eps, decay, inv_scale;
    double b1, b2;
    const float *coef;
    const int *skip;
    uint32_t seed;
    long long *record;  // [0] steps taken, [1] blocks of this step's last launch that are done
    int last;           // this launch ends the step
};

struct Moments {
    void *m, *v;
    float *m_scales, *v_scales;
};

template <int TABLE>
struct AdamwParams {
    float *p[TABLE];
    const void *g[TABLE];
    void *copy[TABLE];
    long long len[TABLE];
    long long block0[TABLE];  // the state's first block of each tensor
    int chunk0[TABLE + 1];    // first chunk of each tensor in this launch
    int n;
    Moments s;
    AdamwScalars c;
};

// ------------------------------------------------------------------ random bits

// Multiplicative hashing (Knuth, The Art of Computer Programming 3, 6.4) between shifts:
// the multipliers are 2^32 over the golden ratio and 2^31 times the root of two, both odd.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9E3779B1u;
    x ^= x >> 15;
    x *= 0xB504F333u;
    return x ^ x >> 16;
}

// ------------------------------------------------------------------------ codes

// A code with MANTISSA bits below the leading one, normal from 2^LOW on, of y >= 0 (at
// most the largest code's value, but for a rounding): the float's bits from the last kept
// one on, after adding 16 random bits below it.  Below 2^LOW, where steps are
// equal, y + 2^LOW has the same steps.
template <int MANTISSA, int LOW>
__device__ __forceinline__ uint32_t random_code(float y, uint32_t random16) {
    constexpr int kDrop = 23 - MANTISSA;
    constexpr uint32_t kFirst = (uint32_t)(127 + LOW) << MANTISSA;  // 2^LOW's kept bits
    constexpr float kLow = LOW == -6 ? 0x1p-6f : 0x1p-14f;
    static_assert(LOW == -6 || LOW == -14, "");
    const bool below = y < kLow;
    const uint32_t bits = __float_as_uint(below ? y + kLow : y);
    const uint32_t kept = (bits + (random16 << (kDrop - 16)) + (1u << (kDrop - 17))) >> kDrop;
    return kept - (below ? kFirst : kFirst - (1u << MANTISSA));
}

// the scale of a block whose largest magnitude has these bits, and its reciprocal
__device__ __forceinline__ float scale_of(uint32_t top_bits, float per_top, float &inverse) {
    const float top = __uint_as_float(top_bits);
    float s = top * per_top;
    if (!(s >= kLeastScale)) s = 0.0f;
    if (top_bits >= 0x7f800000u) s = __int_as_float(0x7fffffff);  // an infinity or NaN: all of the block reads as NaN
    inverse = s >= kLeastScale ? __frcp_rn(s) : 0.0f;
    return s;
}

// four bytes -> the four roots' halves, as floats
__device__ __forceinline__ void root_values(uint32_t codes, float v[4]) {
    const uint32_t lo = __byte_perm(codes, 0u, 0x4140) << 5, hi = __byte_perm(codes, 0u, 0x4342) << 5;
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

__device__ __forceinline__ void m_values(uint32_t codes, float v[4]) {
    const float2 a = from_e4m3x2(codes & 0xffffu), b = from_e4m3x2(codes >> 16);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// --------------------------------------------------------------------- elements

template <int TYPE>
struct Grad {
    static constexpr int kBytes = TYPE == ZERO_FP32 ? 4 : 2;
    using Four = typename std::conditional<TYPE == ZERO_FP32, uint4, uint2>::type;

    // elements [i, len) of up to four, zeros behind them
    static __device__ __forceinline__ Four few(const void *p, long long i, long long len) {
        if constexpr (TYPE == ZERO_FP32) {
            const uint32_t *w = static_cast<const uint32_t *>(p) + i;
            return make_uint4(w[0], i + 1 < len ? w[1] : 0u, i + 2 < len ? w[2] : 0u, i + 3 < len ? w[3] : 0u);
        } else {
            const uint16_t *w = static_cast<const uint16_t *>(p) + i;
            const uint32_t lo = i + 1 < len ? w[1] : 0, mid = i + 2 < len ? w[2] : 0, hi = i + 3 < len ? w[3] : 0;
            return make_uint2(w[0] | lo << 16, mid | hi << 16);
        }
    }
    static __device__ __forceinline__ Four none() {
        if constexpr (TYPE == ZERO_FP32) return make_uint4(0u, 0u, 0u, 0u);
        else return make_uint2(0u, 0u);
    }
    static __device__ __forceinline__ void widen(Four q, float f[4]) {
        if constexpr (TYPE == ZERO_FP32) {
            f[0] = __uint_as_float(q.x);
            f[1] = __uint_as_float(q.y);
            f[2] = __uint_as_float(q.z);
            f[3] = __uint_as_float(q.w);
        } else {
            from_lp4<TYPE == ZERO_BF16>(q, f);
        }
    }
};

__device__ __forceinline__ uint4 stream_load(const uint4 *p) { return __ldcs(p); }
__device__ __forceinline__ uint2 stream_load(const uint2 *p) { return __ldcs(p); }

// One tensor of the table: what a chunk needs of it.
struct Piece {
    float *p;
    const void *g;
    void *copy;
    long long len, block0, first;  // first: the chunk's first block within the tensor
    bool vectors;                  // p, g and copy are aligned to four elements
};

// COPY: the copies' type, or -1
template <int GRAD, int COPY, int TABLE>
__device__ __forceinline__ Piece piece_of(const AdamwParams<TABLE> &t, int chunk, int chunk_blocks) {
    int i = 0, hi = t.n - 1;
    while (i < hi) {  // the last tensor that starts at or before the chunk
        const int mid = (i + hi + 1) / 2;
        if (t.chunk0[mid] <= chunk) i = mid; else hi = mid - 1;
    }
    Piece q;
    q.p = t.p[i];
    q.g = t.g[i];
    q.copy = COPY >= 0 ? t.copy[i] : nullptr;
    q.len = t.len[i];
    q.block0 = t.block0[i];
    q.first = (long long)(chunk - t.chunk0[i]) * chunk_blocks;
    q.vectors = ((reinterpret_cast<uintptr_t>(q.p) & 15u) | (reinterpret_cast<uintptr_t>(q.g) & (4 * Grad<GRAD>::kBytes - 1)) |
                 (reinterpret_cast<uintptr_t>(q.copy) & 7u)) == 0;
    return q;
}

// A thread's four elements of a block, as loaded.
template <int GRAD>
__device__ __forceinline__ void take(const Piece &q, long long e, float4 &p, typename Grad<GRAD>::Four &g) {
    if (q.vectors && e + 4 <= q.len) {
        p = __ldcs(reinterpret_cast<const float4 *>(q.p + e));
        g = stream_load(reinterpret_cast<const typename Grad<GRAD>::Four *>(static_cast<const char *>(q.g) + e * Grad<GRAD>::kBytes));
    } else if (e < q.len) {
        p = make_float4(q.p[e], e + 1 < q.len ? q.p[e + 1] : 0.0f, e + 2 < q.len ? q.p[e + 2] : 0.0f, e + 3 < q.len ? q.p[e + 3] : 0.0f);
        g = Grad<GRAD>::few(q.g, e, q.len);
    } else {
        p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        g = Grad<GRAD>::none();
    }
}

template <int COPY>
__device__ __forceinline__ void put(const Piece &q, long long e, const float p[4]) {
    if (q.vectors && e + 4 <= q.len) {
        __stcs(reinterpret_cast<float4 *>(q.p + e), make_float4(p[0], p[1], p[2], p[3]));
        if constexpr (COPY >= 0)
            __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(q.copy) + e),
                   make_uint2(to_lp2_packed<COPY == ZERO_BF16>(p[0], p[1]), to_lp2_packed<COPY == ZERO_BF16>(p[2], p[3])));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (e + k >= q.len) break;
            q.p[e + k] = p[k];
            if constexpr (COPY >= 0) static_cast<uint16_t *>(q.copy)[e + k] = (uint16_t)to_lp2_packed<COPY == ZERO_BF16>(p[k], 0.0f);
        }
    }
}

// What one step needs of its number and the device's decisions.
struct StepScalars {
    float factor, bc1, bc2;
    uint32_t key;
    int skip;
};

template <int BITS, int GRAD, int COPY, int TABLE>
__global__ void __launch_bounds__(kThreads)
adamw_step(const __grid_constant__ AdamwParams<TABLE> t) {
    pdl_enter();
    __shared__ StepScalars shared;
    const AdamwScalars &c = t.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long step = c.record[0] + 1;
    if (threadIdx.x == 0) {
        shared.bc1 = (float)(1.0 - pow(c.b1, (double)step));
        shared.factor = __fmul_rn(c.coef ? *c.coef : 1.0f, c.inv_scale);
        shared.skip = c.skip ? *c.skip : 0;
        shared.key = mix(mix(c.seed) + (uint32_t)step);
    }
    if (threadIdx.x == 32) shared.bc2 = (float)(1.0 - pow(c.b2, (double)step));
    const int chunks = t.chunk0[t.n];
    constexpr int N = kDepth<BITS>;
    bool first = true;
    StepScalars s;
    float lr1 = 0.0f, rs2 = 0.0f;
    for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const Piece q = piece_of<GRAD, COPY>(t, chunk, kChunkBlocks<BITS>);
        const long long b0 = q.first + warp * N;  // this warp's blocks within the tensor
        const long long blocks = (q.len + kBlock - 1) / kBlock;
        float4 p4[N];
        typename Grad<GRAD>::Four g4[N];
        float4 m4[BITS == 32 ? N : 1], v4[BITS == 32 ? N : 1];
        uint32_t mc[BITS == 8 ? N : 1], vc[BITS == 8 ? N : 1];
        float ms[BITS == 8 ? N : 1], vs[BITS == 8 ? N : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (b0 + i >= blocks) break;
            const long long at = (q.block0 + b0 + i) * (kBlock / 4) + lane;  // four elements of the state
            if constexpr (BITS == 32) {
                m4[i] = __ldcs(static_cast<const float4 *>(t.s.m) + at);
                v4[i] = __ldcs(static_cast<const float4 *>(t.s.v) + at);
            } else {
                mc[i] = __ldcs(static_cast<const uint32_t *>(t.s.m) + at);
                vc[i] = __ldcs(static_cast<const uint32_t *>(t.s.v) + at);
                ms[i] = t.s.m_scales[q.block0 + b0 + i];
                vs[i] = t.s.v_scales[q.block0 + b0 + i];
            }
            take<GRAD>(q, (b0 + i) * kBlock + lane * 4, p4[i], g4[i]);
        }
        if (first) {
            first = false;
            __syncthreads();
            s = shared;
            lr1 = __fdiv_rn(c.lr, s.bc1);
            rs2 = __frcp_rn(__fsqrt_rn(s.bc2));
            if (s.skip) break;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (b0 + i >= blocks) break;
            const long long e = (b0 + i) * kBlock + lane * 4;
            const long long at = (q.block0 + b0 + i) * (kBlock / 4) + lane;
            float p[4] = {p4[i].x, p4[i].y, p4[i].z, p4[i].w}, grad[4];
            Grad<GRAD>::widen(g4[i], grad);
            if constexpr (BITS == 32) {
                float m[4] = {m4[i].x, m4[i].y, m4[i].z, m4[i].w}, v[4] = {v4[i].x, v4[i].y, v4[i].z, v4[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // every operation rounded on its own, in zero_adam_step's order
                    const float g = __fmul_rn(grad[k], s.factor);
                    m[k] = __fadd_rn(__fmul_rn(c.beta1, m[k]), __fmul_rn(c.omb1, g));
                    v[k] = __fadd_rn(__fmul_rn(c.beta2, v[k]), __fmul_rn(c.omb2, __fmul_rn(g, g)));
                    const float denom = __fadd_rn(__fsqrt_rn(__fdiv_rn(v[k], s.bc2)), c.eps);
                    const float update = __fdiv_rn(__fmul_rn(c.lr, __fdiv_rn(m[k], s.bc1)), denom);
                    p[k] = __fsub_rn(__fmul_rn(p[k], c.decay), update);
                }
                __stcs(static_cast<float4 *>(t.s.m) + at, make_float4(m[0], m[1], m[2], m[3]));
                __stcs(static_cast<float4 *>(t.s.v) + at, make_float4(v[0], v[1], v[2], v[3]));
                put<COPY>(q, e, p);
            } else {
                float m[4], r[4];
                m_values(mc[i], m);
                root_values(vc[i], r);
                uint32_t top_m = 0u, top_r = 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float g = grad[k] * s.factor;
                    const float root = r[k] * vs[i];
                    m[k] = __fmaf_rn(c.beta1, m[k] * ms[i], c.omb1 * g);
                    const float v = __fmaf_rn(c.beta2 * root, root, c.omb2 * g * g);
                    r[k] = sqrt_approx(v);
                    if (e + k >= q.len) m[k] = r[k] = 0.0f;  // behind the tensor's end
                    p[k] = __fmaf_rn(p[k], c.decay, -__fdividef(lr1 * m[k], __fmaf_rn(r[k], rs2, c.eps)));
                    top_m = max(top_m, __float_as_uint(m[k]) & 0x7fffffffu);
                    top_r = max(top_r, __float_as_uint(r[k]) & 0x7fffffffu);
                }
                put<COPY>(q, e, p);
                top_m = __reduce_max_sync(0xffffffffu, top_m);
                top_r = __reduce_max_sync(0xffffffffu, top_r);
                float inv_m, inv_r;
                const float scale_m = scale_of(top_m, 1.0f / kTopM, inv_m), scale_r = scale_of(top_r, 1.0f / kTopR, inv_r);
                const unsigned long long place = (unsigned long long)at * 4;
                const uint32_t key = mix(s.key + (uint32_t)(place >> 32));
                uint32_t new_m = 0u, new_r = 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t random = mix(((uint32_t)place + k) ^ key);
                    uint32_t code = random_code<3, -6>(fabsf(m[k]) * inv_m, random & 0xffffu);
                    code = min(code, 126u) | (__float_as_uint(m[k]) >> 31 << 7);
                    new_m |= (inv_m > 0.0f ? code : 0u) << (8 * k);
                    uint32_t root = random_code<5, -14>(r[k] * inv_r, random >> 16);
                    root = min(max(root, r[k] > 0.0f ? 1u : 0u), 255u);
                    new_r |= (inv_r > 0.0f ? root : 0u) << (8 * k);
                }
                __stcs(static_cast<uint32_t *>(t.s.m) + at, new_m);
                __stcs(static_cast<uint32_t *>(t.s.v) + at, new_r);
                if (lane == 0) {
                    t.s.m_scales[q.block0 + b0 + i] = scale_m;
                    t.s.v_scales[q.block0 + b0 + i] = scale_r;
                }
            }
        }
    }
    // The step counts once everyone has read its number.
    if (!c.last) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned long long done = atomicAdd(reinterpret_cast<unsigned long long *>(c.record + 1), 1ull);
        if (done + 1 == gridDim.x) {
            c.record[1] = 0;
            if (!shared.skip) c.record[0] = step;
        }
    }
}

// The values of 8-bit moments: m and v of every element of the state, four a thread.
template <int TYPE>
__global__ void __launch_bounds__(kThreads)
adamw_values(const uint32_t *__restrict__ m, const uint32_t *__restrict__ v, const float *__restrict__ m_scales,
             const float *__restrict__ v_scales, long long fours, void *m_out, void *v_out) {
    pdl_enter();
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < fours; i += (long long)gridDim.x * kThreads) {
        const float ms = m_scales[i / (kBlock / 4)], vs = v_scales[i / (kBlock / 4)];
        float a[4], b[4];
        m_values(m[i], a);
        root_values(v[i], b);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] *= ms;
            b[k] *= vs;
            b[k] *= b[k];
        }
        if constexpr (TYPE == ZERO_FP32) {
            static_cast<float4 *>(m_out)[i] = make_float4(a[0], a[1], a[2], a[3]);
            static_cast<float4 *>(v_out)[i] = make_float4(b[0], b[1], b[2], b[3]);
        } else {
            constexpr bool kBf = TYPE == ZERO_BF16;
            static_cast<uint2 *>(m_out)[i] = make_uint2(to_lp2_packed<kBf>(a[0], a[1]), to_lp2_packed<kBf>(a[2], a[3]));
            static_cast<uint2 *>(v_out)[i] = make_uint2(to_lp2_packed<kBf>(b[0], b[1]), to_lp2_packed<kBf>(b[2], b[3]));
        }
    }
}

// ------------------------------------------------------------------------ host

// blocks that run at once on the current device, or an error below zero
template <int BITS, int GRAD, int COPY, int TABLE>
int blocks_at_once() {
    static PerDevice kept;
    return kept.get([] {
        int each = 0;
        const int asked = done_or_error(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, adamw_step<BITS, GRAD, COPY, TABLE>, kThreads, 0));
        if (asked < 0) return asked;
        return each > 0 ? each * sm_count() : -(int)cudaErrorInvalidConfiguration;
    });
}

template <int BITS, int GRAD, int COPY, int TABLE>
cudaError_t step_impl(const AdamwArgs &a, cudaStream_t stream) {
    const int most = blocks_at_once<BITS, GRAD, COPY, TABLE>();
    if (most < 0) return (cudaError_t)-most;
    AdamwParams<TABLE> t;
    t.s = {a.m, a.v, a.m_scales, a.v_scales};
    t.c.lr = (float)a.lr;
    t.c.beta1 = (float)a.beta1;
    t.c.beta2 = (float)a.beta2;
    t.c.omb1 = (float)(1.0 - a.beta1);
    t.c.omb2 = (float)(1.0 - a.beta2);
    t.c.eps = (float)a.eps;
    t.c.decay = (float)(1.0 - a.lr * a.wd);
    t.c.inv_scale = 1.0f / a.loss_scale;
    t.c.b1 = a.beta1;
    t.c.b2 = a.beta2;
    t.c.coef = a.coef;
    t.c.skip = a.skip;
    t.c.seed = a.seed;
    t.c.record = reinterpret_cast<long long *>(a.record);
    cudaError_t e = cudaSuccess;
    long long block = 0;
    int i = 0;
    do {
        long long chunks = 0;
        t.n = 0;
        for (; i < a.n && t.n < TABLE; ++i) {
            const long long blocks = (a.lens[i] + kBlock - 1) / kBlock, more = (blocks + kChunkBlocks<BITS> - 1) / kChunkBlocks<BITS>;
            if (blocks == 0) continue;
            if (t.n > 0 && chunks + more > 0x3fffffffll) break;
            t.p[t.n] = a.params[i];
            t.g[t.n] = a.grads[i];
            t.copy[t.n] = COPY >= 0 ? a.copies[i] : nullptr;
            t.len[t.n] = a.lens[i];
            t.block0[t.n] = block;
            t.chunk0[t.n++] = (int)chunks;
            chunks += more;
            block += blocks;
        }
        while (i < a.n && a.lens[i] == 0) ++i;
        t.chunk0[t.n] = (int)chunks;
        t.c.last = i == a.n;
        const unsigned grid = (unsigned)std::max<long long>(1, std::min<long long>(most, chunks));
        e = launch_pdl(adamw_step<BITS, GRAD, COPY, TABLE>, dim3(grid), dim3(kThreads), 0, stream, t);
    } while (i < a.n && e == cudaSuccess);
    return e;
}

template <int BITS, int GRAD, int COPY>
cudaError_t step_table(const AdamwArgs &a, cudaStream_t stream) {
    return a.n <= kShort ? step_impl<BITS, GRAD, COPY, kShort>(a, stream) : step_impl<BITS, GRAD, COPY, kTable>(a, stream);
}

template <int BITS, int GRAD>
cudaError_t step_copy(const AdamwArgs &a, cudaStream_t stream) {
    if (!a.copies) return step_table<BITS, GRAD, -1>(a, stream);
    return a.copy_type == ZERO_BF16 ? step_table<BITS, GRAD, ZERO_BF16>(a, stream) : step_table<BITS, GRAD, ZERO_FP16>(a, stream);
}

template <int BITS>
cudaError_t step_grad(const AdamwArgs &a, cudaStream_t stream) {
    if (a.grad_dtype == ZERO_FP32) return step_copy<BITS, ZERO_FP32>(a, stream);
    return a.grad_dtype == ZERO_BF16 ? step_copy<BITS, ZERO_BF16>(a, stream) : step_copy<BITS, ZERO_FP16>(a, stream);
}

}  // namespace

cudaError_t launch_adamw_step(const AdamwArgs &a, cudaStream_t stream) {
    return a.eight ? step_grad<8>(a, stream) : step_grad<32>(a, stream);
}

cudaError_t launch_adamw_values(const int8_t *m, const uint8_t *v, const float *m_scales, const float *v_scales, int64_t blocks,
                                int dtype, void *m_out, void *v_out, cudaStream_t stream) {
    const long long fours = blocks * (kBlock / 4);
    const unsigned grid = (unsigned)std::min<long long>((fours + kThreads - 1) / kThreads, 16ll * sm_count());
    const auto values = dtype == ZERO_FP32 ? adamw_values<ZERO_FP32> : dtype == ZERO_BF16 ? adamw_values<ZERO_BF16> : adamw_values<ZERO_FP16>;
    return launch_pdl(values, dim3(grid), dim3(kThreads), 0, stream, reinterpret_cast<const uint32_t *>(m),
                      reinterpret_cast<const uint32_t *>(v), m_scales, v_scales, fours, m_out, v_out);
}

}  // namespace zk
