// adamw.cu -- one AdamW step over a list of tensors, the moments in 32 or in 8 bits (sm_103a).
//
// For every element, with g' = g * coef / S, t the step and c = 1 - beta^t:
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps),  copy = lp(p)
// Bound by memory: 24 bytes an element and the gradient and copy with 32-bit moments, 12
// with 8-bit ones.  Everything is read once and written once: a warp takes blocks of 128
// elements, each lane four of them, holds a whole block in registers and finds the new
// scales there, so 8-bit moments need no second pass.  On GB300: 124M elements with bf16 gradients
// and copies 0.526 ms with 32-bit moments (99 % of the measured copy rate), 0.340 ms with 8-bit ones
// (85 %: issue slots 73 % busy beside the copies); a list of 12 small tensors 5.7 us.
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

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBlock = ZERO_QUANT_BLOCK;  // a warp's 32 lanes x 4
// Blocks of 128 that a warp has in flight, 16 or 12 elements a lane, in one block of 16 warps on an
// SM.  More warps with less in flight each are slower: 117M elements with 32-bit moments 525 us
// so, 541 and 617 us with two and three blocks of 256 that take 2 at a time, 982 us with
// eight that take 1; 124M with 8-bit moments and their values 479 us then (454 now), 499 with two
// blocks of 256, 528 with 3 at a time, 531 with 24 warps that take 2.
template <int BITS>
constexpr int kDepth = BITS == 8 ? 4 : 3;
template <int BITS>
constexpr int kChunkBlocks = kWarps * kDepth<BITS>;  // blocks of 128 of a chunk
// Whether a chunk's lines are asked for while the one before is at work: 8-bit moments, whose
// arithmetic takes about as long as their copies (124M elements 551 us without it and 512
// with it; with 32-bit moments 4 % slower with it).
template <int BITS>
constexpr bool kAhead = BITS == 8;
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

// Codes with MANTISSA bits below the leading one, normal from 2^LOW on, of y >= 0 (at
// most the largest code's value, but for a rounding), each rounded by 16 random bits.
// y 2^(-126 - LOW) has float's own subnormal numbers where the code has its: its bits
// from the last kept one on are the code, after adding the random bits below that.
template <int MANTISSA, int LOW>
__device__ __forceinline__ uint32_t random_code(float y, uint32_t random16, uint32_t most) {
    constexpr int kDrop = 23 - MANTISSA;
    static_assert(LOW == -6 || LOW == -14, "");
    const float z = y * (LOW == -6 ? 0x1p-120f : 0x1p-112f);
    return min((__float_as_uint(z) + (random16 << (kDrop - 16)) + (1u << (kDrop - 17))) >> kDrop, most);
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// two floats at once, each operation rounded to nearest
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// (add.rn.f32x2 of two products came out as if they were fused into it)
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)),
          "l"(reinterpret_cast<const uint64_t &>(c)));
    return r;
}

// The square root and the reciprocal of normal numbers, rounded to nearest: the hardware's
// approximation and one step with an exact remainder (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990); equal to the
// IEEE operations for every mantissa.  (Those intrinsics, with their branches for all other
// numbers, made 124M elements 512 us and not 479; two numbers an operation 456.)  The root of 0 is 0, that of infinity NaN;
// below 2^-96 the remainder loses bits, and below 2^-126 the result may be far too small.
__device__ __forceinline__ float2 roots_of(float2 x) {
    float2 y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(x.x, 0x1p-126f)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(x.y, 0x1p-126f)));
    const float2 s = mul2(x, y), minus = mul2(x, make_float2(-y.x, -y.y));
    return fma2(fma2(minus, s, x), mul2(y, both(0.5f)), s);
}
// The same of any numbers: what is below 2^-96 is scaled by 2^64 and its root by 2^-32, both exactly; x / 2^64 is below the
// root of everything finite, and infinity's own.
__device__ __forceinline__ float2 any_roots_of(float2 x) {
    const bool small_x = x.x < 0x1p-96f, small_y = x.y < 0x1p-96f;
    const float2 r = roots_of(mul2(x, make_float2(small_x ? 0x1p64f : 1.0f, small_y ? 0x1p64f : 1.0f)));
    const float2 root = mul2(r, make_float2(small_x ? 0x1p-32f : 1.0f, small_y ? 0x1p-32f : 1.0f)), least = mul2(x, both(0x1p-64f));
    return make_float2(fmaxf(root.x, least.x), fmaxf(root.y, least.y));
}
__device__ __forceinline__ float reciprocal_of(float x) {
    const float r = rcp_approx(x);
    return __fmaf_rn(__fmaf_rn(-x, r, 1.0f), r, r);
}

// the larger of a and |b|; NaN if either is
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// the bits of a block's largest root, of the lanes' four each
__device__ __forceinline__ uint32_t largest_root(const float (&r)[4]) {
    return __reduce_max_sync(0xffffffffu, __float_as_uint(larger(larger(larger(r[0], r[1]), r[2]), r[3])));
}

// the scale of a block whose largest magnitude has these bits, and its reciprocal
__device__ __forceinline__ float scale_of(uint32_t top_bits, float per_top, float &inverse) {
    float s = __uint_as_float(top_bits) * per_top;
    s = s >= kLeastScale ? s : 0.0f;
    if (top_bits >= 0x7f800000u) s = __int_as_float(0x7fffffff);  // an infinity or NaN: all of the block reads as NaN
    inverse = s >= kLeastScale ? reciprocal_of(s) : 0.0f;
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

// --------------------------------------------------------------------- elements

// Four consecutive gradients as loaded, widened only once they are needed.
template <int TYPE>
struct Grad {
    static constexpr int kBytes = TYPE == ZERO_FP32 ? 4 : 2;
    // 16 bits: two words, or three where the first element is the upper half of a word
    static constexpr int kWords = TYPE == ZERO_FP32 ? 4 : 3;
    uint32_t w[kWords];

    // all four there, aligned together or (16 bits) with another element behind them
    template <bool TOGETHER>
    __device__ __forceinline__ void load(const char *p) {
        if constexpr (TYPE == ZERO_FP32) {
            if constexpr (TOGETHER) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p));
                w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __ldcs(reinterpret_cast<const uint32_t *>(p) + k);
            }
        } else if constexpr (TOGETHER) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(p));
            w[0] = q.x; w[1] = q.y; w[2] = 0u;
        } else {
            const bool upper = reinterpret_cast<uintptr_t>(p) & 2u;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p - (upper ? 2 : 0));
            w[0] = __ldcs(q);
            w[1] = __ldcs(q + 1);
            w[2] = upper ? __ldcs(q + 2) : 0u;
        }
    }
    // `left` of them there, zeros behind
    __device__ __forceinline__ void few(const char *p, long long left) {
        const bool upper = kBytes == 2 && (reinterpret_cast<uintptr_t>(p) & 2u);
        if constexpr (TYPE == ZERO_FP32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = k < left ? reinterpret_cast<const uint32_t *>(p)[k] : 0u;
        } else {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = k < left ? reinterpret_cast<const uint16_t *>(p)[k] : 0u;
            w[0] = upper ? h[0] << 16 : h[0] | h[1] << 16;
            w[1] = upper ? h[1] | h[2] << 16 : h[2] | h[3] << 16;
            w[2] = upper ? h[3] : 0u;
        }
    }
    template <bool TOGETHER>
    __device__ __forceinline__ void widen(const char *p, float f[4]) const {
        if constexpr (TYPE == ZERO_FP32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(w[k]);
        } else {
            const uint32_t by = TOGETHER ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(p) & 2u) * 8u;
            from_lp4<TYPE == ZERO_BF16>(make_uint2(__funnelshift_r(w[0], w[1], by), __funnelshift_r(w[1], w[2], by)), f);
        }
    }
};

// One tensor of the table: what a chunk needs of it.
struct Piece {
    float *p;
    const void *g;
    void *copy;
    long long len, block0, first;  // first: the chunk's first block within the tensor
    bool vectors;                  // p and copy are aligned to four elements
    bool together;                 // and g
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
    q.vectors = ((reinterpret_cast<uintptr_t>(q.p) & 15u) | (reinterpret_cast<uintptr_t>(q.copy) & 7u)) == 0;
    q.together = (reinterpret_cast<uintptr_t>(q.g) & (4 * Grad<GRAD>::kBytes - 1)) == 0;
    return q;
}

// b^n by squaring: b^n is off by at most about n 2^-53 of itself, which 1 - b^n in float does
// not show.  (pow took 1.1 us more of a short list's 8.2.)
__device__ __forceinline__ double power(double b, long long n) {
    double r = 1.0;
    for (; n > 0; n >>= 1) {
        if (n & 1) r = __dmul_rn(r, b);
        b = __dmul_rn(b, b);
    }
    return r;
}

// What one step needs of its number and the device's decisions.
struct StepScalars {
    float factor, bc1, bc2;
    uint32_t key;
    int skip;
};

// A warp's N blocks of 128 of one tensor, a lane four elements of each: loaded all at
// once, then updated and stored one after the other.  FORM: kWhole, all of them exist and
// are whole, parameters and copies are aligned, and no 2^32 lies between their places;
// kTogether, the gradients are aligned too, else another element stands behind them; kAny,
// whatever there is.
enum Form { kAny, kWhole, kTogether };

template <int BITS, int GRAD, int COPY, int FORM>
struct Span {
    static constexpr int N = kDepth<BITS>;
    static constexpr bool FULL = FORM != kAny;
    float *p;          // this lane's first element, and the same place in the others
    const char *g;
    uint16_t *copy;
    long long e, len;  // elements of the tensor before it, and in all
    long long block;   // the first block's place in the state
    int blocks;        // that exist
    bool vectors;
    float4 p4[N];
    Grad<GRAD> g4[N];
    float4 m4[BITS == 32 ? N : 1], v4[BITS == 32 ? N : 1];
    uint32_t mc[BITS == 8 ? N : 1], vc[BITS == 8 ? N : 1];
    float ms[BITS == 8 ? N : 1], vs[BITS == 8 ? N : 1];

    __device__ __forceinline__ Span(const Piece &q, long long b0, int lane) {
        e = b0 * kBlock + lane * 4;
        p = q.p + e;
        g = static_cast<const char *>(q.g) + e * Grad<GRAD>::kBytes;
        copy = COPY >= 0 ? static_cast<uint16_t *>(q.copy) + e : nullptr;
        len = q.len;
        block = q.block0 + b0;
        const long long left = (q.len + kBlock - 1) / kBlock - b0;
        blocks = FULL || left > N ? N : (int)left;
        vectors = q.vectors;
    }

    __device__ __forceinline__ void load(const Moments &s, int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!FULL && i >= blocks) break;
            if constexpr (BITS == 32) {
                m4[i] = __ldcs(static_cast<const float4 *>(s.m) + block * 32 + lane + i * 32);
                v4[i] = __ldcs(static_cast<const float4 *>(s.v) + block * 32 + lane + i * 32);
            } else {
                mc[i] = __ldcs(static_cast<const uint32_t *>(s.m) + block * 32 + lane + i * 32);
                vc[i] = __ldcs(static_cast<const uint32_t *>(s.v) + block * 32 + lane + i * 32);
                ms[i] = s.m_scales[block + i];
                vs[i] = s.v_scales[block + i];
            }
            const long long at = e + i * kBlock;
            const float *from = p + i * kBlock;
            const char *grad = g + i * kBlock * Grad<GRAD>::kBytes;
            if (FULL || (vectors && at + 4 <= len))
                p4[i] = __ldcs(reinterpret_cast<const float4 *>(from));
            else
                p4[i] = make_float4(at < len ? from[0] : 0.0f, at + 1 < len ? from[1] : 0.0f, at + 2 < len ? from[2] : 0.0f,
                                    at + 3 < len ? from[3] : 0.0f);
            if (FULL || at + 5 <= len)
                g4[i].template load<FORM == kTogether>(grad);
            else
                g4[i].few(grad, len - at);
        }
    }

    __device__ __forceinline__ void put(int i, const float (&w)[4]) const {
        const long long at = e + i * kBlock;
        float *to = p + i * kBlock;
        if (FULL || (vectors && at + 4 <= len)) {
            __stcs(reinterpret_cast<float4 *>(to), make_float4(w[0], w[1], w[2], w[3]));
            if constexpr (COPY >= 0)
                __stcs(reinterpret_cast<uint2 *>(copy) + i * 32,
                       make_uint2(to_lp2_packed<COPY == ZERO_BF16>(w[0], w[1]), to_lp2_packed<COPY == ZERO_BF16>(w[2], w[3])));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (at + k >= len) break;
                to[k] = w[k];
                if constexpr (COPY >= 0) copy[i * kBlock + k] = (uint16_t)to_lp2_packed<COPY == ZERO_BF16>(w[k], 0.0f);
            }
        }
    }

    __device__ __forceinline__ void step(const Moments &st, const AdamwScalars &c, const StepScalars &s, float lr1, float rs2, int lane) {
        // Blocks whose largest root is NaN, or 0 < root < `least`, take their roots by any_roots_of.  roots_of
        // is wrong below 2^-48 only, and by less than 2^-63.  Where the block's largest is 2^-34 or more, such a root's code is
        // 1 whatever it is, and an eps of 2^-38 rs2 or more hides it in the update: with a smaller eps every
        // block's roots are taken so.  (124M elements 457 -> 456 us, nothing; any_roots_of everywhere 474, a test of every
        // element 472, the intrinsic in the rare branch 465.)
        const uint32_t least = c.eps >= rs2 * 0x1p-38f ? 0x2e800000u : 0x7f800000u;
        uint32_t key = BITS == 8 ? mix(s.key + (uint32_t)((unsigned long long)block * kBlock >> 32)) : 0u;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!FULL && i >= blocks) break;
            float w[4] = {p4[i].x, p4[i].y, p4[i].z, p4[i].w}, grad[4];
            g4[i].template widen<FORM == kTogether>(g, grad);
            if constexpr (BITS == 32) {
                float m[4] = {m4[i].x, m4[i].y, m4[i].z, m4[i].w}, v[4] = {v4[i].x, v4[i].y, v4[i].z, v4[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // every operation rounded on its own, in zero_adam_step's order
                    const float f = __fmul_rn(grad[k], s.factor);
                    m[k] = __fadd_rn(__fmul_rn(c.beta1, m[k]), __fmul_rn(c.omb1, f));
                    v[k] = __fadd_rn(__fmul_rn(c.beta2, v[k]), __fmul_rn(c.omb2, __fmul_rn(f, f)));
                    const float denom = __fadd_rn(__fsqrt_rn(__fdiv_rn(v[k], s.bc2)), c.eps);
                    const float update = __fdiv_rn(__fmul_rn(c.lr, __fdiv_rn(m[k], s.bc1)), denom);
                    w[k] = __fsub_rn(__fmul_rn(w[k], c.decay), update);
                }
                __stcs(static_cast<float4 *>(st.m) + block * 32 + lane + i * 32, make_float4(m[0], m[1], m[2], m[3]));
                __stcs(static_cast<float4 *>(st.v) + block * 32 + lane + i * 32, make_float4(v[0], v[1], v[2], v[3]));
                put(i, w);
            } else {
                // What lies behind a tensor's end has gradient and codes 0, and keeps them.
                float m[4], r[4], v[4];
                m_values(mc[i], m);
                root_values(vc[i], r);
                const float2 old_m = both(ms[i]), old_r = both(vs[i]);
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    // The new moments as with 32 bits, every operation rounded on its own: codes beside a
                    // border are anybody's guess otherwise.  The update need not be.
                    const float2 f = mul2(make_float2(grad[k], grad[k + 1]), both(s.factor));
                    const float2 root = mul2(make_float2(r[k], r[k + 1]), old_r);
                    const float2 m2 = add2(mul2(both(c.beta1), mul2(make_float2(m[k], m[k + 1]), old_m)), mul2(both(c.omb1), f));
                    const float2 v2 = add2(mul2(both(c.beta2), mul2(root, root)), mul2(both(c.omb2), mul2(f, f)));
                    const float2 r2 = roots_of(v2);
                    m[k] = m2.x;
                    m[k + 1] = m2.y;
                    v[k] = v2.x;
                    v[k + 1] = v2.y;
                    r[k] = r2.x;
                    r[k + 1] = r2.y;
                }
                const float top_m = larger(larger(larger(larger(0.0f, m[0]), m[1]), m[2]), m[3]);
                const uint32_t bits_m = __reduce_max_sync(0xffffffffu, __float_as_uint(top_m));
                uint32_t bits_r = largest_root(r);
                if (bits_r != 0u && bits_r - least >= 0x7f800000u - least) {
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 r2 = any_roots_of(make_float2(v[k], v[k + 1]));
                        r[k] = r2.x;
                        r[k + 1] = r2.y;
                    }
                    bits_r = largest_root(r);
                }
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float2 denominator = fma2(make_float2(r[k], r[k + 1]), both(rs2), both(c.eps));
                    const float2 part = mul2(mul2(both(-lr1), make_float2(m[k], m[k + 1])), make_float2(rcp_approx(denominator.x), rcp_approx(denominator.y)));
                    const float2 p2 = fma2(make_float2(w[k], w[k + 1]), both(c.decay), part);
                    w[k] = p2.x;
                    w[k + 1] = p2.y;
                }
                put(i, w);
                float inv_m, inv_r;
                const float scale_m = scale_of(bits_m, 1.0f / kTopM, inv_m), scale_r = scale_of(bits_r, 1.0f / kTopR, inv_r);
                const unsigned long long place = (unsigned long long)(block + i) * kBlock;
                if (!FULL && i > 0 && (uint32_t)place == 0u) key = mix(s.key + (uint32_t)(place >> 32));
                uint32_t cm[4], cr[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t random = mix(((uint32_t)place + lane * 4 + k) ^ key);
                    cm[k] = random_code<3, -6>(fabsf(m[k]) * inv_m, random & 0xffffu, 126u);
                    cr[k] = random_code<5, -14>(r[k] * inv_r, random >> 16, 255u);
                    cr[k] = max(cr[k], min(__float_as_uint(r[k]), 1u));  // r >= 0
                }
                uint32_t new_m = pack_bytes(cm[0], cm[1], cm[2], cm[3]), new_r = pack_bytes(cr[0], cr[1], cr[2], cr[3]);
                const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0073),
                                                   __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0073), 0x5410);
                new_m |= signs & 0x80808080u;
                if (!(scale_m > 0.0f)) new_m = 0u;
                if (!(scale_r > 0.0f)) new_r = 0u;
                __stcs(static_cast<uint32_t *>(st.m) + block * 32 + lane + i * 32, new_m);
                __stcs(static_cast<uint32_t *>(st.v) + block * 32 + lane + i * 32, new_r);
                if (lane == 0) {
                    st.m_scales[block + i] = scale_m;
                    st.v_scales[block + i] = scale_r;
                }
            }
        }
    }
};

// Asks L2 for the lines of a warp's N blocks: the next chunk's, while this one's are at work.
template <int BITS, int GRAD, int N>
__device__ __forceinline__ void ask_ahead(const Piece &q, long long b0, const Moments &s, int lane) {
    constexpr int kP = 4, kG = Grad<GRAD>::kBytes, kM = BITS / 8, kLines = kP + kG + 2 * kM;  // of 128 bytes, of a block
#pragma unroll
    for (int j = 0; j < (N * kLines + 31) / 32; ++j) {
        const int l = lane + 32 * j, i = l / kLines, line = l % kLines;
        if (i >= N || (b0 + i + 1) * kBlock > q.len) break;
        const char *at;
        if (line < kP) at = reinterpret_cast<const char *>(q.p + (b0 + i) * kBlock) + line * 128;
        else if (line < kP + kG) at = static_cast<const char *>(q.g) + (b0 + i) * kBlock * kG + (line - kP) * 128;
        else if (line < kP + kG + kM) at = static_cast<const char *>(s.m) + (q.block0 + b0 + i) * kBlock * kM + (line - kP - kG) * 128;
        else at = static_cast<const char *>(s.v) + (q.block0 + b0 + i) * kBlock * kM + (line - kP - kG - kM) * 128;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
}

template <int BITS, int GRAD, int COPY, int TABLE>
__global__ void __launch_bounds__(kThreads, 1)
adamw_step(const __grid_constant__ AdamwParams<TABLE> t) {
    pdl_enter();
    __shared__ StepScalars shared;
    const AdamwScalars &c = t.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long step = c.record[0] + 1;
    if (threadIdx.x == 0) {
        shared.bc1 = (float)(1.0 - power(c.b1, step));
        shared.factor = __fmul_rn(c.coef ? *c.coef : 1.0f, c.inv_scale);
        shared.skip = c.skip ? *c.skip : 0;
        shared.key = mix(mix(c.seed) + (uint32_t)step);
    }
    if (threadIdx.x == 32) shared.bc2 = (float)(1.0 - power(c.b2, step));
    const int chunks = t.chunk0[t.n];
    constexpr int N = kDepth<BITS>;
    bool first = true;
    StepScalars s;
    float lr1 = 0.0f, rs2 = 0.0f;
    Piece q;
    if ((int)blockIdx.x < chunks) q = piece_of<GRAD, COPY>(t, blockIdx.x, kChunkBlocks<BITS>);
    for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const long long b0 = q.first + warp * N;  // this warp's blocks within the tensor
        Piece next;
        const auto meanwhile = [&] {  // the loads being on their way
            if (chunk + (int)gridDim.x < chunks) {
                next = piece_of<GRAD, COPY>(t, chunk + gridDim.x, kChunkBlocks<BITS>);
                if (kAhead<BITS>) ask_ahead<BITS, GRAD, N>(next, next.first + warp * N, t.s, lane);
            }
            if (!first) return;
            first = false;
            __syncthreads();
            s = shared;
            lr1 = __fdiv_rn(c.lr, s.bc1);
            rs2 = __frcp_rn(__fsqrt_rn(s.bc2));
        };
        const unsigned long long place = (unsigned long long)(q.block0 + b0) * kBlock;
        const auto update = [&](auto form) {
            Span<BITS, GRAD, COPY, decltype(form)::value> a(q, b0, lane);
            a.load(t.s, lane);
            meanwhile();
            if (!s.skip) a.step(t.s, c, s, lr1, rs2, lane);
        };
        const bool full = q.vectors && (BITS == 32 || (uint32_t)place <= 0xffffffffu - (N - 1) * kBlock);
        if (full && q.together && (b0 + N) * kBlock <= q.len)
            update(std::integral_constant<int, kTogether>());
        else if (full && (b0 + N) * kBlock < q.len)
            update(std::integral_constant<int, kWhole>());
        else
            update(std::integral_constant<int, kAny>());
        if (s.skip) break;
        q = next;
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
