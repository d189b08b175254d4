// quant.cu -- the quantized stage-3 gather (sm_103a).
//
// ZeRO++ ("ZeRO-1/2/3 分别优化了什么" note, ZeRO++: the all-gathered
// parameters are quantized to cut the traffic): each rank turns its lp shard
// into 1-byte codes with one float scale per 128-element block -- int8
// (symmetric, block max -> 127, nearest-even) or OCP FP8 E4M3 with a
// power-of-two scale -- and the gather expands code * scale back to lp while
// it concatenates the ranks' shards.  Per layer element the gather
// moves 1 B + 4/128 B in and 2 B out, against 2 B in and 2 B out for the lp
// gather.  Both kernels are plain streaming kernels; each thread keeps several
// independent loads in flight before it computes, and every warp load and
// store is one contiguous run.
#include "launch.h"
#include "per_device.h"
#include "quant_codes.cuh"
#include "zero_internal.h"

namespace zk {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 4;   // blocks per warp (quantize) / items per thread (gather)

// Eight lanes per 128-element block, 16 contiguous elements per lane (two
// 16-byte loads), four blocks per warp, one group of four blocks per warp and
// iteration (1 to 4 groups per iteration were swept on GB300: 1 is fastest):
// lane l holds elements 16(l mod 8) .. 16(l mod 8) + 15 of block
// 4*group + l/8.  The block maximum takes three xor shuffles; scale =
// amax / 127 (correctly rounded, scale_of_amax), code = nearest-even integer of
// x / scale (the correctly rounded float quotient, see quant_codes), clamped to
// +-127.  FP8: the E4M3 codes and power-of-two scale of quant_codes_fp8
// instead.  Each lane writes its 16 codes with one 16-byte store.  (Versus a
// half-warp per block with 8 elements per lane: the per-block work -- the
// shuffles and the scale -- is shared by twice the elements.)

template <bool BF16, bool FP8>
__global__ void __launch_bounds__(kQuantThreads, 3)  // 16 values per lane without spills
quantize_shard_blocks(const uint4 *__restrict__ x, uint4 *__restrict__ q, float *__restrict__ scales,
                      long long n_blocks) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int l8 = lane & 7;
    const long long n_groups = (n_blocks + 3) / 4;
    const long long warps = (long long)gridDim.x * (kQuantThreads / 32);
    const long long w0 = (long long)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
    // int8: a software pipeline, the next group's two loads in flight while
    // this group is quantized (the exactness test makes the compute long: 0.081
    // -> 0.071 ms at 7.5B); fp8, whose compute is short, loads then computes
    // (the pipeline measured 3 % slower there)
    auto load = [&](long long group, uint4 r[2]) {
        const long long b = 4 * group + (lane >> 3);
        if (group < n_groups && b < n_blocks) {
            r[0] = __ldg(x + b * 16 + 2 * l8);
            r[1] = __ldg(x + b * 16 + 2 * l8 + 1);
        } else {
            r[0] = r[1] = make_uint4(0u, 0u, 0u, 0u);
        }
    };
    uint4 cur[2], nxt[2];
    if constexpr (!FP8) load(w0, cur);
    for (long long group = w0; group < n_groups; group += warps) {  // uniform across the warp
        if constexpr (FP8) {
            load(group, cur);
        } else {
            load(group + warps, nxt);
        }
        const long long b = 4 * group + (lane >> 3);
        float v[16];
        from_lp4<BF16>(make_uint2(cur[0].x, cur[0].y), v);
        from_lp4<BF16>(make_uint2(cur[0].z, cur[0].w), v + 4);
        from_lp4<BF16>(make_uint2(cur[1].x, cur[1].y), v + 8);
        from_lp4<BF16>(make_uint2(cur[1].z, cur[1].w), v + 12);
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(v[k]));
#pragma unroll
        for (int off = 4; off > 0; off >>= 1)  // within each group of 8 lanes
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        float scale;
        uint32_t packed[4];
        if constexpr (FP8) {
            quant_codes_fp8<16>(v, amax, scale, packed);
        } else {
            scale = scale_of_amax(amax);
            quant_codes<16>(v, scale, packed);
        }
        if (b < n_blocks) {
            __stcs(q + b * 8 + l8, make_uint4(packed[0], packed[1], packed[2], packed[3]));
            if (l8 == 0) scales[b] = scale;
        }
        if constexpr (!FP8) {
            cur[0] = nxt[0];
            cur[1] = nxt[1];
        }
    }
}

template <int MAXN>
struct DequantGatherParams {
    const uint2 *codes[MAXN];   // rank j's codes at this unit's offset (8 per uint2)
    const float *scales[MAXN];  // rank j's scales at this unit's first block
    uint4 *out;                 // 8 lp per uint4
    long long vec_per_shard;    // shard_len / 8
};

// out[j * shard + k] = lp(code_j[k] * scale_j[k / 128]).  blockIdx.y is the
// rank j; along x a thread takes kQuantUnroll items of 8 codes (one 8-byte
// load each, all issued before any use) and writes each item's 8 lp values
// with one 16-byte store, so a warp's loads and stores are contiguous runs.
// FP8: the codes are E4M3, widened exactly by the conversion instruction.
template <int MAXN, bool BF16, bool FP8>
__global__ void __launch_bounds__(kQuantThreads)
gather_dequant(const __grid_constant__ DequantGatherParams<MAXN> p) {
    pdl_enter();
    const int j = blockIdx.y;
    const uint2 *codes = p.codes[j];
    const float *scales = p.scales[j];
    uint4 *out = p.out + (long long)j * p.vec_per_shard;
    const long long stride = (long long)gridDim.x * kQuantThreads;
    for (long long k0 = (long long)blockIdx.x * kQuantThreads + threadIdx.x; k0 < p.vec_per_shard;
         k0 += stride * kQuantUnroll) {
        uint2 c[kQuantUnroll];
        float sc[kQuantUnroll];
#pragma unroll
        for (int u = 0; u < kQuantUnroll; ++u) {
            const long long k = k0 + u * stride;
            if (k < p.vec_per_shard) {
                c[u] = __ldcs(codes + k);
                sc[u] = __ldg(scales + (k >> 4));  // 8 codes lie in one 128-block
            }
        }
#pragma unroll
        for (int u = 0; u < kQuantUnroll; ++u) {
            const long long k = k0 + u * stride;
            if (k >= p.vec_per_shard) break;
            uint32_t o[4];
            if constexpr (FP8) {
                const uint32_t w[2] = {c[u].x, c[u].y};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float2 f = from_e4m3x2(w[t >> 1] >> (16 * (t & 1)));
                    o[t] = to_lp2_packed<BF16>(__fmul_rn(f.x, sc[u]), __fmul_rn(f.y, sc[u]));
                }
            } else {
                const uint32_t w[2] = {c[u].x ^ 0x80808080u, c[u].y ^ 0x80808080u};
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float y[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) y[q] = __fmul_rn(code_to_float(w[t], q), sc[u]);
                    o[2 * t] = to_lp2_packed<BF16>(y[0], y[1]);
                    o[2 * t + 1] = to_lp2_packed<BF16>(y[2], y[3]);
                }
            }
            __stcs(out + k, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

template <typename K>
int blocks_per_sm(PerDevice &kept, K kernel) {
    const int b = kept.get([&] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kQuantThreads, 0) == cudaSuccess ? n : 0;
    });
    return b < 1 ? 1 : b;
}

template <int MAXN, bool BF16, bool FP8>
cudaError_t dequant_gather_impl(const int8_t *const *codes, const float *const *scales, int n,
                                int64_t offset, int64_t shard_len, void *out, cudaStream_t stream) {
    DequantGatherParams<MAXN> p;
    for (int j = 0; j < n; ++j) {
        p.codes[j] = reinterpret_cast<const uint2 *>(codes[j] + offset);
        p.scales[j] = scales[j] + offset / 128;
    }
    for (int j = n; j < MAXN; ++j) {
        p.codes[j] = nullptr;
        p.scales[j] = nullptr;
    }
    p.out = static_cast<uint4 *>(out);
    p.vec_per_shard = shard_len / 8;
    if (p.vec_per_shard == 0 || n == 0) return cudaSuccess;
    static PerDevice kept;
    const int occ = blocks_per_sm(kept, gather_dequant<MAXN, BF16, FP8>);
    // about two waves of CTAs over all ranks
    const long long per_rank_need = (p.vec_per_shard + kQuantThreads * kQuantUnroll - 1) /
                                    (kQuantThreads * kQuantUnroll);
    long long gx = (2LL * sm_count() * occ + n - 1) / n;
    if (gx > per_rank_need) gx = per_rank_need;
    if (gx < 1) gx = 1;
    return launch_pdl(gather_dequant<MAXN, BF16, FP8>, dim3((unsigned)gx, (unsigned)n), dim3(kQuantThreads), 0,
                      stream, p);
}

template <bool BF16, bool FP8>
cudaError_t quantize_impl(const void *shard, int64_t len, int8_t *codes, float *scales, cudaStream_t stream) {
    const long long blocks = len / 128;
    if (blocks == 0) return cudaSuccess;
    static PerDevice kept;
    const int occ = blocks_per_sm(kept, quantize_shard_blocks<BF16, FP8>);
    long long grid = (long long)sm_count() * occ;
    const long long per_cta = (kQuantThreads / 32) * 4;  // blocks per CTA per iteration
    const long long need = (blocks + per_cta - 1) / per_cta;
    if (grid > need) grid = need;
    return launch_pdl(quantize_shard_blocks<BF16, FP8>, dim3((unsigned)grid), dim3(kQuantThreads), 0, stream,
                      static_cast<const uint4 *>(shard), reinterpret_cast<uint4 *>(codes), scales, blocks);
}

}  // namespace

cudaError_t launch_quantize(const void *shard, int lp, int fp8, int64_t len, int8_t *codes, float *scales,
                            cudaStream_t stream) {
    if (fp8)
        return lp ? quantize_impl<true, true>(shard, len, codes, scales, stream)
                  : quantize_impl<false, true>(shard, len, codes, scales, stream);
    return lp ? quantize_impl<true, false>(shard, len, codes, scales, stream)
              : quantize_impl<false, false>(shard, len, codes, scales, stream);
}

template <int MAXN>
cudaError_t dequant_dispatch(const int8_t *const *codes, const float *const *scales, int n, int lp, int fp8,
                             int64_t offset, int64_t shard_len, void *out, cudaStream_t stream) {
    if (fp8)
        return lp ? dequant_gather_impl<MAXN, true, true>(codes, scales, n, offset, shard_len, out, stream)
                  : dequant_gather_impl<MAXN, false, true>(codes, scales, n, offset, shard_len, out, stream);
    return lp ? dequant_gather_impl<MAXN, true, false>(codes, scales, n, offset, shard_len, out, stream)
              : dequant_gather_impl<MAXN, false, false>(codes, scales, n, offset, shard_len, out, stream);
}

cudaError_t launch_dequant_gather(const int8_t *const *codes, const float *const *scales, int n, int lp,
                                  int fp8, int64_t offset, int64_t shard_len, void *out, cudaStream_t stream) {
    if (n <= 64) return dequant_dispatch<64>(codes, scales, n, lp, fp8, offset, shard_len, out, stream);
    return dequant_dispatch<1024>(codes, scales, n, lp, fp8, offset, shard_len, out, stream);
}

}  // namespace zk
