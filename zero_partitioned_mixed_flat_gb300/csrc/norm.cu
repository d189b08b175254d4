// norm.cu -- residual addition + root-mean-square norm of rows, its 8-bit
// outputs, and its gradients (sm_103a).
//
//   s = x + r,  rstd = (mean(s^2) + eps)^(-1/2),  y = s rstd w
//   gs' = rstd (w gy - s rstd mean(w gy s rstd)) + gs,  gw = sum over rows of gy s rstd
//
// Bound by memory: forward reads x and r and writes y and s once (8 bytes an
// element in 16 bits), backward reads s, gy, gs and writes gs' (8 bytes).  A row
// stays in the registers of the warps that own it between the sum of its squares
// and its outputs, so nothing is read twice; the weight's row comes from L1.
// On GB300, of the measured copy rate: forward 8191 x 4096 41 us (96 %), 16384 x
// 4096 79 us (100 %), with fp8 codes 71 us (98 %), int8 74 us; 16384 x 1600 fp8 32 us
// (84 %: a quarter of its lanes has no vector); backward 8191 x 4096 47 us (84 %).
#include "head_internal.h"
#include "launch.h"
#include "per_device.h"
#include "quant_codes.cuh"
#include "zero_internal.h"

namespace zk {
namespace {

constexpr int kSms = 152;
constexpr int kVpt = 4;           // vectors of 8 elements a thread holds of a row, at most
constexpr int kRowsPerBlock = 4;  // rows of a block when one warp owns a row
constexpr int kMaxWarps = 16;     // that own a row: 16384 elements at 4 vectors a thread

template <bool BF16>
__device__ __forceinline__ void widen(uint4 q, float v[8]) {
    from_lp4<BF16>(make_uint2(q.x, q.y), v);
    from_lp4<BF16>(make_uint2(q.z, q.w), v + 4);
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow(const float v[8]) {
    return make_uint4(to_lp2_packed<BF16>(v[0], v[1]), to_lp2_packed<BF16>(v[2], v[3]), to_lp2_packed<BF16>(v[4], v[5]),
                      to_lp2_packed<BF16>(v[6], v[7]));
}

// Hides from the compiler that q is what it was, so that it widens q again
// instead of keeping eight floats alive across a row's exchange.
__device__ __forceinline__ void forget(uint4 &q) { asm volatile("" : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)); }

// the sum over the warps that own a row, all of a block's unless there is one
template <typename T>
__device__ __forceinline__ T row_sum(T v, int warps, T *shared) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (warps == 1) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) shared[warp] = v;
    __syncthreads();
    v = lane < warps ? shared[lane] : T(0);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Whether a row's sum of squares has left float's range: not finite (from 1.8e19 /
// sqrt(dim) on, or not finite itself), or so small beside eps that lost squares could
// count.  The row then adds its squares up again in double.  Only bfloat16 gets there: the
// least square of fp16 numbers is 2^-48, and the largest sum 3e14.
template <bool BF16>
__device__ __forceinline__ bool leaves_float(float sq, float eps, int dim) {
    return BF16 && !(__fmaf_rn(eps, (float)dim, sq) >= 0x1p-100f && sq <= 1.7e38f);
}

// the larger one; NaN where either is (fmaxf gives the other)
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct NormShape {
    int vecs;   // vectors of 8 in a row
    int warps;  // that own a row: 1 (kRowsPerBlock rows a block) or all of a block
};

enum NormOutput { kOutLp = 0, kOutInt8 = 1, kOutFp8 = 2 };

// Thread t of a row holds its vectors t, t + threads, ...: every load and store
// of a warp is one run of 512 bytes, and 16 neighbouring lanes hold one block of
// 128 elements, so a block's largest magnitude takes four exchanges.
template <bool BF16, int VPT, int OUT>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) norm_rows(const NormArgs a, const NormShape sh) {
    pdl_enter();
    __shared__ float shared[kMaxWarps];
    __shared__ double shared_wide[kMaxWarps];
    const int threads = sh.warps * 32;
    const int t = sh.warps == 1 ? threadIdx.x & 31 : threadIdx.x;
    const long long row = sh.warps == 1 ? (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
    const uint4 *weight = static_cast<const uint4 *>(a.weight);
    if (row >= a.rows) return;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + row * a.x_stride);
    const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.residual) + row * a.residual_stride);
    uint4 qx[VPT], qr[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * threads;
        qx[j] = qr[j] = make_uint4(0u, 0u, 0u, 0u);
        if (v < sh.vecs) {
            qx[j] = __ldcs(x + v);
            if (a.residual) qr[j] = __ldcs(r + v);
        }
    }
    float s[VPT][8], sq = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float f[8];
        widen<BF16>(qx[j], s[j]);
        widen<BF16>(qr[j], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // without a residual s is x itself: x + 0 would turn -0 into 0
            if (a.residual) s[j][k] = __fadd_rn(s[j][k], f[k]);
            sq = __fmaf_rn(s[j][k], s[j][k], sq);
        }
    }
    sq = row_sum(sq, sh.warps, shared);
    float rstd = rsqrtf(__fadd_rn(__fdiv_rn(sq, (float)a.dim), a.eps));
    if (leaves_float<BF16>(sq, a.eps, a.dim)) {
        double wide = 0.0;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) wide = __fma_rn((double)s[j][k], (double)s[j][k], wide);
        wide = row_sum(wide, sh.warps, shared_wide);
        rstd = (float)rsqrt(wide / a.dim + (double)a.eps);
    }
    uint4 *sum = a.sum ? reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.sum) + row * a.sum_stride) : nullptr;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * threads;
        if constexpr (OUT == kOutLp) {
            if (v >= sh.vecs) continue;
        }
        if (sum && v < sh.vecs) sum[v] = narrow<BF16>(s[j]);
        float w[8], y[8];
        widen<BF16>(v < sh.vecs ? __ldg(weight + v) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(__fmul_rn(s[j][k], rstd), w[k]);
        if constexpr (OUT == kOutLp) {
            reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * a.out_stride)[v] = narrow<BF16>(y);
        } else {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max_or_nan(top, v < sh.vecs ? fabsf(y[k]) : 0.0f);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
            float scale;
            uint32_t codes[2];
            if (top != top) {  // codes have no NaN (int8), so the block's scale says it
                scale = top;
                codes[0] = codes[1] = 0u;
            } else if constexpr (OUT == kOutFp8) {
                quant_codes_fp8<8>(y, top, scale, codes);
            } else {
                scale = __fdiv_rn(top, 127.0f);
                quant_codes<8>(y, scale, codes);
            }
            if (v < sh.vecs) {
                reinterpret_cast<uint2 *>(a.codes + row * a.dim)[v] = make_uint2(codes[0], codes[1]);
                if ((v & 15) == 0) a.scales[row * ((a.dim + 127) / 128) + v / 16] = scale;
            }
        }
    }
}

// One warp a row, eight codes a lane and step.
template <bool BF16, bool FP8>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
dequantize_rows(const int8_t *__restrict__ codes, const float *__restrict__ scales, long long rows, int vecs, uint16_t *out,
                long long out_stride) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int blocks = (vecs + 15) / 16;
    for (long long row = (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5); row < rows;
         row += (long long)gridDim.x * kRowsPerBlock) {
        const uint2 *c = reinterpret_cast<const uint2 *>(codes) + row * vecs;
        const float *s = scales + row * blocks;
        uint4 *o = reinterpret_cast<uint4 *>(out + row * out_stride);
        for (int v0 = lane; v0 < vecs; v0 += 4 * 32) {
            uint2 q[4];
            float sc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = v0 + 32 * j;
                if (v < vecs) {
                    q[j] = __ldcs(c + v);
                    sc[j] = __ldg(s + v / 16);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = v0 + 32 * j;
                if (v >= vecs) break;
                const uint32_t w[2] = {q[j].x, q[j].y};
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    if constexpr (FP8) {
                        const float2 two = from_e4m3x2((w[k / 4] >> (8 * (k & 3))) & 0xffffu);
                        f[k] = __fmul_rn(two.x, sc[j]);
                        f[k + 1] = __fmul_rn(two.y, sc[j]);
                    } else {
                        const uint32_t biased = w[k / 4] ^ 0x80808080u;
                        f[k] = __fmul_rn(code_to_float(biased, k & 3), sc[j]);
                        f[k + 1] = __fmul_rn(code_to_float(biased, (k & 3) + 1), sc[j]);
                    }
                }
                o[v] = narrow<BF16>(f);
            }
        }
    }
}

// The sums v[0], v[1] over the warps that own a row, of several rows a block:
// `group` is the row's place in the block and its barrier.
template <typename T>
__device__ __forceinline__ void group_sum(T (&v)[2], int warps, int group, T (*shared)[2]) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
    if (warps == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        shared[warp][0] = v[0];
        shared[warp][1] = v[1];
    }
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        T t = lane < warps ? shared[group * warps + lane][n] : T(0);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        v[n] = t;
    }
}

// 16 bytes to shared memory without passing through registers
__device__ __forceinline__ void copy_async(uint4 *to, const uint4 *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Backward: the warps of a row also keep the columns they own of grad_weight, over
// all the rows they take.  A block of up to kMaxWarps warps fills an SM's registers
// with as many rows as it holds; at the end these add their columns up in shared
// memory, in order, and the block writes one row of partial sums.  The row's two
// sums (s^2, and w gy s) are exchanged together.  The registers hold no second row,
// so the next one is copied to shared memory meanwhile; every thread reads back
// only what it copied itself.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_rows_backward(const NormBackwardArgs a, const NormShape sh) {
    pdl_enter();
    extern __shared__ uint4 ahead[];  // [two rows][s, gy, gs][vector][thread]
    __shared__ float shared[2][kMaxWarps][2];
    __shared__ double shared_wide[2][kMaxWarps][2];
    const int threads = sh.warps * 32, groups = (int)blockDim.x / threads;
    const int group = threadIdx.x / threads, t = threadIdx.x - group * threads;
    uint4 w[VPT];
    float gw[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * threads;
        w[j] = v < sh.vecs ? __ldg(static_cast<const uint4 *>(a.weight) + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k) gw[j][k] = 0.0f;
    }
    const long long step = (long long)gridDim.x * groups;
    auto place = [&](int stage, int tensor, int j) -> uint4 * {
        return ahead + ((stage * 3 + tensor) * VPT + j) * blockDim.x + threadIdx.x;
    };
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
            const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.sum) + row * a.sum_stride);
            const uint4 *g = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.grad_out) + row * a.grad_out_stride);
            const uint4 *e = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.grad_sum) + row * a.grad_sum_stride);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = t + j * threads;
                if (v >= sh.vecs) break;
                copy_async(place(stage, 0, j), s + v);
                copy_async(place(stage, 1, j), g + v);
                if (a.grad_sum) copy_async(place(stage, 2, j), e + v);
            }
        }
        copies_commit();
    };
    int slot = 0;
    const long long first = (long long)blockIdx.x * groups + group;
    fetch(first, 0);
    for (long long row = first; row < a.rows; row += step, slot ^= 1) {
        fetch(row + step, slot ^ 1);
        copies_wait<1>();
        uint4 qs[VPT], qg[VPT], qe[VPT];
        auto take = [&] {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                qs[j] = qg[j] = qe[j] = make_uint4(0u, 0u, 0u, 0u);
                if (t + j * threads < sh.vecs) {
                    qs[j] = *place(slot, 0, j);
                    qg[j] = *place(slot, 1, j);
                    if (a.grad_sum) qe[j] = *place(slot, 2, j);
                }
            }
        };
        take();
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float fs[8], fg[8], fw[8];
            widen<BF16>(qs[j], fs);
            widen<BF16>(qg[j], fg);
            widen<BF16>(w[j], fw);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sums[0] = __fmaf_rn(fs[k], fs[k], sums[0]);
                sums[1] = __fmaf_rn(__fmul_rn(fg[k], fw[k]), fs[k], sums[1]);
            }
        }
        group_sum(sums, sh.warps, group, shared[slot]);
        float rstd = rsqrtf(__fadd_rn(__fdiv_rn(sums[0], (float)a.dim), a.eps));
        float along = __fmul_rn(__fdiv_rn(sums[1], (float)a.dim), rstd);  // mean(w gy s rstd)
        if (leaves_float<BF16>(sums[0], a.eps, a.dim) || (BF16 && !(fabsf(sums[1]) <= 1.7e38f))) {
            double wide[2] = {0.0, 0.0};
#pragma unroll 1
            for (int v = t, j = 0; v < sh.vecs; v += threads, ++j) {
                float fs[8], fg[8], fw[8];
                widen<BF16>(*place(slot, 0, j), fs);
                widen<BF16>(*place(slot, 1, j), fg);
                widen<BF16>(__ldg(static_cast<const uint4 *>(a.weight) + v), fw);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    wide[0] = __fma_rn((double)fs[k], (double)fs[k], wide[0]);
                    wide[1] = __fma_rn((double)fg[k] * (double)fw[k], (double)fs[k], wide[1]);
                }
            }
            group_sum(wide, sh.warps, group, shared_wide[slot]);
            const double exact = rsqrt(wide[0] / a.dim + (double)a.eps);
            rstd = (float)exact;
            along = (float)(wide[1] / a.dim * exact);
            take();  // again, so that no register holds the row meanwhile
        }
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.grad_in) + row * a.grad_in_stride);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = t + j * threads;
            forget(qs[j]);
            forget(qg[j]);
            forget(w[j]);
            float fs[8], fg[8], fw[8], fe[8];
            widen<BF16>(qs[j], fs);
            widen<BF16>(qg[j], fg);
            widen<BF16>(w[j], fw);
            widen<BF16>(qe[j], fe);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float unit = __fmul_rn(fs[k], rstd);
                gw[j][k] = __fmaf_rn(fg[k], unit, gw[j][k]);
                // without grad_sum fe is 0, which leaves the value as it is
                fe[k] = __fmaf_rn(rstd, __fmaf_rn(-unit, along, __fmul_rn(fg[k], fw[k])), fe[k]);
            }
            if (v < sh.vecs) out[v] = narrow<BF16>(fe);
        }
    }
    copies_wait<0>();
    float4 *const columns = reinterpret_cast<float4 *>(ahead);
    float4 *part = static_cast<float4 *>(a.workspace) + (long long)blockIdx.x * sh.vecs * 2;
    for (int g = 0; g < groups; ++g) {
        __syncthreads();
        if (group != g) continue;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = t + j * threads;
            if (v >= sh.vecs) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 sum = make_float4(gw[j][4 * h], gw[j][4 * h + 1], gw[j][4 * h + 2], gw[j][4 * h + 3]);
                if (g > 0) {
                    const float4 before = columns[h * sh.vecs + v];
                    sum = make_float4(before.x + sum.x, before.y + sum.y, before.z + sum.z, before.w + sum.w);
                }
                if (g + 1 < groups)
                    columns[h * sh.vecs + v] = sum;
                else
                    part[2 * v + h] = sum;
            }
        }
    }
}

constexpr int kColumns = 32, kWays = 32;

// grad_weight of 32 columns: 32 ways along the partial rows, joined in order
template <bool BF16>
__global__ void __launch_bounds__(kColumns *kWays)
norm_weight_sum(const float *__restrict__ parts, int n, int dim, uint16_t *grad_weight) {
    pdl_enter();
    __shared__ float shared[kWays][kColumns + 1];
    const int x = threadIdx.x % kColumns, y = threadIdx.x / kColumns, d = blockIdx.x * kColumns + x;
    float sum = 0.0f;
    if (d < dim) {
#pragma unroll
        for (int j = 0; j < (kSms + kWays - 1) / kWays; ++j)
            if (y + j * kWays < n) sum += __ldcg(parts + (long long)(y + j * kWays) * dim + d);
    }
    shared[y][x] = sum;
    __syncthreads();
    if (y != 0 || d >= dim) return;
    for (int i = 1; i < kWays; ++i) sum += shared[i][x];
    grad_weight[d] = (uint16_t)(to_lp2_packed<BF16>(sum, 0.0f) & 0xffffu);
}

// How many warps own a row, and how many vectors each thread holds.
//  - Rows for every SM: as many warps as hold the row at kVpt vectors a thread
//    (one warp up to 1024 elements, which needs no exchange through shared
//    memory).  Rows of 16384 x 1600: 33 us at 4 vectors, 35 us at 2, 37 us at 8.
//  - Fewer rows than SMs: one vector a thread, up to kMaxWarps warps, so that one
//    round of loads holds the row.
NormShape shape_of(int64_t rows, int dim, int *vpt) {
    NormShape s;
    s.vecs = dim / 8;
    const int each = rows < kSms ? 32 : 32 * kVpt;
    s.warps = (s.vecs + each - 1) / each;
    if (s.warps > kMaxWarps) s.warps = kMaxWarps;
    *vpt = (s.vecs + 32 * s.warps - 1) / (32 * s.warps);
    return s;
}

// blocks that take every row once
unsigned blocks_for(int64_t rows, const NormShape &s) {
    return (unsigned)(s.warps == 1 ? (rows + kRowsPerBlock - 1) / kRowsPerBlock : rows);
}

// Backward: the rows that a block takes at once, and the blocks.  An SM's registers
// hold kMaxWarps warps, and every block adds a partial row of grad_weight, so
// a block takes as many rows as that -- unless there are not enough rows for every
// SM.  (8191 x 4096: 47 us; 49 us without the copies ahead, and as much with four
// blocks an SM and four times the partial rows.)
int rows_of_block(int64_t rows, const NormShape &s) { return rows < kSms ? 1 : kMaxWarps / s.warps; }
int backward_blocks(int64_t rows, const NormShape &s) {
    const int64_t blocks = (rows + rows_of_block(rows, s) - 1) / rows_of_block(rows, s);
    return (int)(blocks < kSms ? blocks : kSms);
}

template <bool BF16, int OUT, int VPT = 1>
cudaError_t forward_impl(const NormArgs &a, const NormShape &s, int vpt, cudaStream_t stream) {
    if (vpt == VPT)  // a block for every row: 4 % faster than rows taken again and again
        return launch_pdl(norm_rows<BF16, VPT, OUT>, dim3(blocks_for(a.rows, s)),
                          dim3((unsigned)(s.warps == 1 ? 32 * kRowsPerBlock : 32 * s.warps)), 0, stream, a, s);
    if constexpr (VPT < kVpt) return forward_impl<BF16, OUT, VPT + 1>(a, s, vpt, stream);
    return cudaErrorInvalidValue;
}

template <bool BF16, int VPT = 1>
cudaError_t backward_impl(const NormBackwardArgs &a, const NormShape &s, int vpt, cudaStream_t stream) {
    if (vpt == VPT) {
        // two rows ahead of three tensors; the columns of grad_weight, 4 bytes each, need less
        constexpr int kAhead = 2 * 3 * VPT * (int)sizeof(uint4);
        static PerDevice allowed;
        const int set = allowed.get([] {
            return done_or_error(cudaFuncSetAttribute(norm_rows_backward<BF16, VPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      kAhead * 32 * kMaxWarps));
        });
        if (set < 0) return (cudaError_t)-set;
        const int threads = 32 * s.warps * rows_of_block(a.rows, s);
        return launch_pdl(norm_rows_backward<BF16, VPT>, dim3((unsigned)backward_blocks(a.rows, s)), dim3((unsigned)threads),
                          size_t(kAhead) * threads, stream, a, s);
    }
    if constexpr (VPT < kVpt) return backward_impl<BF16, VPT + 1>(a, s, vpt, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream) {
    int vpt;
    const NormShape s = shape_of(a.rows, a.dim, &vpt);
    if (a.out) return a.lp ? forward_impl<true, kOutLp>(a, s, vpt, stream) : forward_impl<false, kOutLp>(a, s, vpt, stream);
    if (a.fp8) return a.lp ? forward_impl<true, kOutFp8>(a, s, vpt, stream) : forward_impl<false, kOutFp8>(a, s, vpt, stream);
    return a.lp ? forward_impl<true, kOutInt8>(a, s, vpt, stream) : forward_impl<false, kOutInt8>(a, s, vpt, stream);
}

cudaError_t launch_dequantize_rows(const int8_t *codes, const float *scales, int fp8, int64_t rows, int dim,
                                   int lp, void *out, int64_t out_stride, cudaStream_t stream) {
    const int64_t blocks = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), block(32 * kRowsPerBlock);
    uint16_t *o = static_cast<uint16_t *>(out);
    const long long n = rows, stride = out_stride;
    if (fp8)
        return lp ? launch_pdl(dequantize_rows<true, true>, grid, block, 0, stream, codes, scales, n, dim / 8, o, stride)
                  : launch_pdl(dequantize_rows<false, true>, grid, block, 0, stream, codes, scales, n, dim / 8, o, stride);
    return lp ? launch_pdl(dequantize_rows<true, false>, grid, block, 0, stream, codes, scales, n, dim / 8, o, stride)
              : launch_pdl(dequantize_rows<false, false>, grid, block, 0, stream, codes, scales, n, dim / 8, o, stride);
}

int64_t norm_backward_bytes(int64_t rows, int dim) {
    int vpt;
    return (int64_t)backward_blocks(rows, shape_of(rows, dim, &vpt)) * dim * (int64_t)sizeof(float);
}

cudaError_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream) {
    int vpt;
    const NormShape s = shape_of(a.rows, a.dim, &vpt);
    if (a.rows > 0) {
        cudaError_t e = a.lp ? backward_impl<true>(a, s, vpt, stream) : backward_impl<false>(a, s, vpt, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(a.lp ? norm_weight_sum<true> : norm_weight_sum<false>,
                      dim3((unsigned)((a.dim + kColumns - 1) / kColumns)), dim3(kColumns * kWays), 0, stream,
                      static_cast<const float *>(a.workspace), backward_blocks(a.rows, s), a.dim,
                      static_cast<uint16_t *>(a.grad_weight));
}

}  // namespace zk
