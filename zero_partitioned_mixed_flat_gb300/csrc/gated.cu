// gated.cu -- the gated projections of a feed-forward block and their gradients (sm_103a).
//
// With x [T, D], the matrices Wg and Wu [F, D], and p = act(g):
//   g = x Wg^T,  u = x Wu^T,  out = act(g) u
//   dg = go u act'(g),  du = go act(g)
//   gx = dg Wg + du Wu,  gWg = dg^T x,  gWu = du^T x
// Forward is one product whose tiles hold 128 columns of g and the same 128 of u: CTA 0 of
// a pair loads the rows of Wg and CTA 1 those of Wu, which is how a pair's B operand
// is split anyhow, so both sums of an element are in one row of tensor memory and neither g
// nor u is ever stored.  Backward keeps nothing of the forward pass but x: it computes g
// and u again (4 T D F operations beside the 8 of the gradients), writes dg and du in lp
// and takes the three products in one launch: gx's sum runs over dg's columns and then du's.
// dg and du are rounded because the tensor core takes both operands in one type of 16 bits (f16's kind):
// two parts of each would keep twice the bits for 16 and not 8 T D F operations, which is what bounds
// the larger sizes.  It leaves the gradients sqrt(2) times as far off as their own rounding (of bf16
// gradients 0.0023 of their norm, and 0.0017): what a chain of separate products in lp rounds, too.
//
// On GB300: forward 8184 x 1600 x 4264 (T x D x F) 0.142 ms (1570 TFLOP/s; 0.127 cold), one token
// 4096 x 10928 30 us (6.0 TB/s), 48 tokens 1600 x 4264 8.9 us; forward and gradients 4096 x 4096 x
// 10928 1.73 to 1.80 ms (16 T D F operations, 1630 to 1690 TFLOP/s), 2048 x 1600 x 4264 0.17 ms,
// 1023 x 768 x 2048 0.041 ms.  The largest are bound by power, few tokens by memory, what lies
// between by whole rounds of tiles and by what a launch takes to start and to end.
#include "head_internal.h"
#include "launch.h"
#include "per_device.h"
#include "tile_product.cuh"
#include "zero.h"
#include "zero_internal.h"

#include <algorithm>

namespace zk {
namespace {

constexpr int kGatedSmem = 1024 + kStages * kStageBytes;
constexpr int kTileCost = 4;  // blocks of K that starting and storing a tile cost, about

enum Mode { kForward = 0, kSlopes = 1, kGradients = 2 };
enum Kind { kGates = 0, kGatesEdge = 1, kGradX = 2, kGradGate = 3, kGradUp = 4 };

// Where the workspace's regions begin: slopes and partial sums leave in sectors of 32 bytes, each
// written by one store that asks for that alignment, and a warp's rows in lines.  A workspace
// is any 16-byte boundary, so the calls round it up to this and ask for that much more.
constexpr int64_t kBase = 128, kBaseSlack = kBase - 16;

// Blocks that look for the largest |grad_out|, two on each SM.
constexpr int kTopBlocks = 304, kTopThreads = 256;

struct GatedLayout {
    int64_t rows;   // tokens rounded up to whole tiles
    int64_t stride; // of the slopes' rows: whole sectors
    int splits;     // partial sums of grad_x
    int64_t slope_gate, slope_up, sums;  // byte offsets from the rounded-up workspace
    int64_t bytes;                       // that a workspace needs wherever it begins
};

// What a tile costs, in blocks of K of 256 columns; starting and storing it take about kTileCost.
// Fewer columns take (columns + 128) / 384 of a block, as measured (see plan_gates).
double tile_cost(double blocks, int64_t columns) { return blocks * (double)(std::min<int64_t>(columns, kTileN) + 128) / 384 + kTileCost; }

// In how many partial sums grad_x comes: it has few tiles and long sums.  As many as leave no
// part longer than a pair's share of all three gradients (at most 16, 8 blocks of K each); or
// fewer, so that every tile has a pair of its own, where the longest then ends before a
// pair that has one of each kind would.
int splits_of(int64_t tokens, int64_t wide, int dim) {
    const int64_t dim_tiles = up(dim, kTileN) / kTileN, row_tiles = up(std::max<int64_t>(tokens, 1), kTileM) / kTileM;
    const int64_t long_sum = 2 * (up(wide, kTileK) / kTileK), short_sum = up(tokens, kTileK) / kTileK;
    const int64_t n_x = row_tiles * dim_tiles, n_weight = 2 * (up(wide, kTileM) / kTileM) * dim_tiles;
    const int64_t share = (n_x * long_sum + n_weight * short_sum) / kPairs;
    int splits = 1;
    while (splits < 16 && long_sum / splits > share && long_sum / (splits + 1) >= 8) ++splits;
    const int64_t alone = (kPairs - n_weight) / n_x;
    if (alone >= 1 && alone < splits &&
        tile_cost((double)long_sum / alone, kTileN) < tile_cost((double)long_sum / splits, kTileN) + tile_cost((double)short_sum, kTileN))
        splits = (int)alone;  // 1023 x 768 x 2048: two parts and 72 tiles, and not four and 96
    return splits;
}

GatedLayout gated_layout(int64_t tokens, int64_t wide, int dim) {
    GatedLayout l;
    l.rows = up(std::max<int64_t>(tokens, 1), kTileM);
    l.splits = splits_of(tokens, wide, dim);
    int64_t at = up(kTopBlocks * 4, 1024);
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at = up(at + bytes, 1024);
        return here;
    };
    l.stride = up(wide, 16);
    l.slope_gate = take(tokens * l.stride * 2);
    l.slope_up = take(tokens * l.stride * 2);
    l.sums = take(l.splits > 1 ? l.splits * l.rows * dim * 4 : 0);
    l.bytes = at + kBaseSlack;
    return l;
}

// ----------------------------------------------------------------- activations

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two elements at a time, which halves the instructions: the thread that feeds the tensor core
// needs its turns too.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 rcp2(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 one_minus(float2 x) { return fma2(x, both(-1.0f), both(1.0f)); }

// 1 / (1 + exp(-x)); 0 and 1 far out
__device__ __forceinline__ float2 sigmoid(float2 x) { return rcp2(add2(exp2_2(mul2(x, both(-kLog2e))), both(1.0f))); }

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

// P = erfc(-g / sqrt(2)) / 2 from q = erfc(x) / 2 at x = |g| / sqrt(2): (1 + 2 x) exp(x^2) erfc(x)
// is a smooth function of t = (x - 2.5) / (x + 2.5) over all x >= 0 (Shepherd and Laframboise,
// "Chebyshev approximation of (1 + 2x) exp(x^2) erfc x in 0 <= x < infinity", Math. Comp. 36,
// 1981); the coefficients are a Chebyshev fit of degree 9 of half of it, 1.5e-7 off.  With the
// exponential rounded as it is here q is off by at most 0.4 (g^2 / 2 + 16) 2^-22 of itself.
// bell: exp(-g^2 / 2).  (erfcf took 120 cycles an element.)
__device__ __forceinline__ float2 normal_share(float2 g, float2 bell) {
    constexpr float kFit[10] = {2.022946865e-04f, 1.512481249e-04f,  -2.088966779e-03f, 5.443191039e-04f,  1.633777283e-02f,
                                -5.151086301e-02f, 7.882248610e-02f, -4.950888082e-02f, -6.117876619e-02f, 6.324190497e-01f};
    const float2 y = mul2(g, both(0.70710678118654752f));
    const float2 x = make_float2(fminf(fabsf(y.x), 16.0f), fminf(fabsf(y.y), 16.0f));
    const float2 above = add2(x, both(2.5f)), twice = fma2(x, both(2.0f), both(1.0f));
    const float2 r = rcp2(mul2(above, twice));  // at most 18.5 * 33
    const float2 t = mul2(mul2(add2(x, both(-2.5f)), twice), r);
    float2 h = both(kFit[0]);
#pragma unroll
    for (int i = 1; i < 10; ++i) h = fma2(h, t, both(kFit[i]));
    const float2 q = mul2(bell, mul2(h, mul2(above, r))), rest = one_minus(q);
    return make_float2(g.x < 0.0f ? q.x : rest.x, g.y < 0.0f ? q.y : rest.y);
}

// Each activation is g P(g), its derivative P + g P'.
//   silu       P = 1 / (1 + exp(-g))
//   gelu       P = erfc(-g / sqrt(2)) / 2
//   gelu_tanh  P = (1 + tanh(y)) / 2 = 1 / (1 + exp(-2 y)),  2 y = kTanhScale (g + kTanhCube g^3)
template <int ACT>
__device__ __forceinline__ float2 share_of(float2 g, float2 &derivative) {
    const float2 square = mul2(g, g);
    if constexpr (ACT == ZERO_ACT_GELU) {
        const float2 bell = exp2_2(mul2(square, both(-0.5f * kLog2e)));
        derivative = mul2(bell, both(0.3989422804014327f));
        return normal_share(g, bell);
    } else if constexpr (ACT == ZERO_ACT_SILU) {
        const float2 p = sigmoid(g);
        derivative = mul2(p, one_minus(p));
        return p;
    } else {
        const float2 p = sigmoid(mul2(fma2(mul2(g, both(kTanhCube)), square, g), both(kTanhScale)));
        derivative = mul2(mul2(p, one_minus(p)), fma2(square, both(3.0f * kTanhCube * kTanhScale), both(kTanhScale)));
        return p;
    }
}

// out of n columns, g and u in place
template <int ACT, int N>
__device__ __forceinline__ void outs_of(const float (&g)[N], float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 a = make_float2(g[i], g[i + 1]);
        float2 unused;
        const float2 out = mul2(mul2(a, share_of<ACT>(a, unused)), make_float2(u[i], u[i + 1]));
        u[i] = out.x;
        u[i + 1] = out.y;
    }
}

// dg and du of n columns, in g's and u's place
template <int ACT, int N>
__device__ __forceinline__ void slopes_of(const float (&go)[N], float (&g)[N], float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 a = make_float2(g[i], g[i + 1]), grad = make_float2(go[i], go[i + 1]);
        float2 derivative;
        const float2 p = share_of<ACT>(a, derivative);
        const float2 slope = fma2(a, derivative, p), du = mul2(grad, mul2(a, p));
        const float2 dg = mul2(mul2(grad, make_float2(u[i], u[i + 1])), slope);
        g[i] = dg.x;
        g[i + 1] = dg.y;
        u[i] = du.x;
        u[i + 1] = du.y;
    }
}

// Results go from registers to memory, 32 bytes of its row a lane: a whole sector, where the
// rows begin at one.  (Through shared memory and TMA a warp took 540 cycles for 32 rows of 64
// bytes, most of them waiting to fill, fence and start the store: as long as the sums of a
// tile with a K of 512, and the products read shared memory meanwhile.)
__device__ __forceinline__ void store_sector(void *to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void load_sector(const void *from, uint4 &a, uint4 &b) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(from));
}

__device__ __forceinline__ void ask_page(const void *at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

// A matrix of lp results.
struct Rows {
    uint16_t *at;
    long long stride;
    int cols;
};

// Writes a stretch of one row, 16 elements at a time, in whole sectors: where the row lies 16
// bytes off one, the last eight elements wait for the next eight, and only the stretch's two
// ends are half sectors.  (With halves everywhere 129 x 4088 x 10920's gradients took 198 us
// and not 163.)
struct RowWriter {
    uint16_t *at;     // of column 0
    int cols;
    bool odd, first;
    uint32_t carry[4];

    __device__ __forceinline__ RowWriter(const Rows &m, long long row, int col) {
        at = m.at + row * m.stride;
        cols = m.cols;
        odd = reinterpret_cast<uintptr_t>(at + col) & 16u;
        first = true;
    }
    static __device__ __forceinline__ void store_four(uint16_t *to, const uint32_t *w) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // columns col to col + 15, or as many of them as there are (a multiple of 8)
    __device__ __forceinline__ void put(int col, const uint32_t (&w)[8]) {
        uint32_t s[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = odd ? carry[i] : w[i];
            s[4 + i] = odd ? w[i] : w[4 + i];
            carry[i] = w[4 + i];
        }
        const int from = odd ? col - 8 : col;  // eight and eight elements from here
        const bool lo = !(odd && first) && from < cols, hi = from + 8 < cols;
        if (lo && hi) store_sector(at + from, s);
        else if (lo) store_four(at + from, s);
        else if (hi) store_four(at + from + 8, s + 4);
        first = false;
    }
    // after the last column before `end`
    __device__ __forceinline__ void finish(int end) const {
        if (odd && !first && end - 8 < cols) store_four(at + end - 8, carry);
    }
};

struct GatedParams {
    CUtensorMap x_k;             // x: boxes 64 of D x 128 tokens
    CUtensorMap gate_k, up_k, gate_k_edge, up_k_edge;  // matrices: 64 of D x half a tile's columns
    CUtensorMap x_mn;            // x: 64 of D x 64 tokens
    CUtensorMap gate_mn, up_mn;  // matrices: 64 of D x 64 of F
    CUtensorMap dg_k, du_k;      // slopes: 64 of F x 128 tokens
    CUtensorMap dg_mn, du_mn;    // slopes: 64 of F x 64 tokens
    long long tokens, rows;
    int wide, dim, splits;
    int step, whole, step_edge;  // columns of a tile of both projections, tiles of them, and columns of the others'
    int catch_up, start;         // see GatedWork
    int act;
    Rows out;                // forward
    Rows dg, du;             // slopes
    Rows gx, ggate, gup;     // gradients
    float *sums;             // of gx, where splits > 1: [split][rows][dim]
    const uint4 *grad_out;
    long long grad_stride;  // vectors
    const float *tops;      // NULL: the slopes are not scaled
    int *status;
    long long wait_cycles;
};

// The work of one launch, and which of it each pair does, in order: every pair-th tile,
// gradients first the tiles of grad_x, few and long; the pairs that get one fewer of
// them then take `catch_up` tiles of the matrices' gradients each; the rest of those goes round
// all pairs from `start` on.  Of every kind the tiles of many columns come first and those of
// fewer after them, as what is left over is best made of short ones.  plan_gates chooses
// the columns, plan_gradients catch_up and start.
template <int MODE>
struct GatedWork {
    Tiles whole, edge;           // both projections; grad_x
    Tiles weight, weight_edge;   // gradients of the matrices, gate's rows before up's
    int step, step_edge, edge_column;
    int pair, pairs, n_whole, n_weight, n_weights, weight_m;
    int fuller, catch_up, from, mine;

    __device__ __forceinline__ explicit GatedWork(const GatedParams &p) {
        const int row_tiles = (int)((p.tokens + kTileM - 1) / kTileM);
        pair = blockIdx.x >> 1;
        pairs = gridDim.x >> 1;
        step = p.step;
        step_edge = p.step_edge;
        if constexpr (MODE != kGradients) {
            const int blocks = (p.dim + kTileK - 1) / kTileK;
            edge_column = p.whole * p.step;
            const int left = 2 * p.wide - edge_column;
            whole.set(row_tiles, p.whole, edge_column, blocks, 1);
            edge.set(row_tiles, (left + p.step_edge - 1) / p.step_edge, left, blocks, 1);
            n_whole = whole.size();
        } else {
            const int columns = p.dim / kTileN, last = p.dim % kTileN, some = last ? 1 : 0;
            const int x_blocks = 2 * ((p.wide + kTileK - 1) / kTileK), weight_blocks = (int)((p.tokens + kTileK - 1) / kTileK);
            weight_m = (p.wide + kTileM - 1) / kTileM;
            edge_column = columns * kTileN;
            whole.set(row_tiles, columns, edge_column, x_blocks, p.splits);
            edge.set(row_tiles, some, last, x_blocks, p.splits);
            weight.set(2 * weight_m, columns, edge_column, weight_blocks, 1);
            weight_edge.set(2 * weight_m, some, last, weight_blocks, 1);
            n_whole = whole.size();
            n_weight = weight.size();
            n_weights = n_weight + weight_edge.size();
            const int n_x = n_whole + edge.size();
            fuller = n_x % pairs;
            catch_up = p.catch_up;
            from = pair >= p.start ? pair - p.start : pair - p.start + pairs;
            mine = n_x > pair ? (n_x - pair + pairs - 1) / pairs : 0;
        }
    }

    __device__ __forceinline__ bool at(int j, Tile &t) const {
        if constexpr (MODE != kGradients) {
            const int i = pair + j * pairs;
            if (i >= n_whole + edge.size()) return false;
            if (i < n_whole) {
                t = whole.at(i, kGates);
                t.n0 = t.n * step;
                t.width = step;
            } else {
                t = edge.at(i - n_whole, kGatesEdge);
                t.n0 = t.n * step_edge;
                const int left = (edge.columns - t.n0 + 31) / 32 * 32;
                t.width = left < step_edge ? left : step_edge;
                t.n0 += edge_column;
            }
            return true;
        }
        bool last;
        if (j < mine) {
            const int i = pair + j * pairs;
            last = i >= n_whole;
            t = last ? edge.at(i - n_whole, kGradX) : whole.at(i, kGradX);
        } else {
            j -= mine;
            const int others = pairs - fuller;
            int i;
            if (catch_up && pair >= fuller && j < catch_up) {
                i = pair - fuller + j * others;
            } else {
                if (catch_up && pair >= fuller) j -= catch_up;
                i = catch_up * others + from + j * pairs;
            }
            if (i >= n_weights) return false;
            last = i >= n_weight;
            t = last ? weight_edge.at(i - n_weight, kGradGate) : weight.at(i, kGradGate);
            if (t.m0 >= weight_m * kTileM) {
                t.m0 -= weight_m * kTileM;
                t.kind = kGradUp;
            }
        }
        if (last) t.n0 = edge_column;
        return true;
    }
};

template <bool BF16, int MODE>
__device__ __forceinline__ Feed feed_of(const Tile &t, uint32_t stage0) {
    return Feed(t.width, MODE == kGradients && t.kind != kGradX, MODE == kGradients, stage0, BF16);
}

// fp16 slopes are scaled by a power of two that puts the largest finite |grad_out| into
// [1/4, 1/2): u act'(g) and act(g) may be 2^17 before a slope overflows, and what is
// 2^-12 of the largest still has all its bits.  (bf16 has float's range.)  By a whole warp.
__device__ __forceinline__ float scale_of(const float *tops) {
    if (!tops) return 1.0f;
    float top = 0.0f;
    for (int i = threadIdx.x & 31; i < kTopBlocks; i += 32) top = fmaxf(top, tops[i]);
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // top is 0 or an fp16 number: 2^-24 at least
    return top > 0.0f ? __uint_as_float((252u - (__float_as_uint(top) >> 23)) << 23) : 1.0f;
}

template <bool BF16, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
gated_products(const __grid_constant__ GatedParams p) {
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t stage0 = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            bar_init(smem_addr(&sh.full[s]), 1);
            bar_init(smem_addr(&sh.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(smem_addr(&sh.acc_full[b]), 1);
            bar_init(smem_addr(&sh.acc_empty[b]), 2 * kResultWarps);
        }
        bar_init(smem_addr(&sh.drained), 1);
        sh.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(kTmemColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (threadIdx.x == 0) {  // the maps of the operands, while the kernel before this one ends
        if constexpr (MODE != kGradients) {
            ask_for(&p.x_k);
            ask_for(rank == 0 ? &p.gate_k : &p.up_k);
        } else {
            ask_for(&p.x_mn);
            ask_for(&p.dg_k);
            ask_for(&p.du_k);
            ask_for(&p.gate_mn);
            ask_for(&p.up_mn);
            ask_for(&p.dg_mn);
            ask_for(&p.du_mn);
        }
    }
    const GatedWork<MODE> work(p);
    // fp16 slopes follow gated_top, whose result only the results' warps read.  The others need
    // not wait for it: every block of it has waited for all that came before, x and the
    // matrices among it, or this kernel would not have started.
    if (MODE != kSlopes || BF16 || warp >= 2) pdl_enter();

    volatile int *dead = &sh.dead;
    const long long limit = p.wait_cycles;
    Tile t;

    if (warp == 0) {
        if (lane == 0) {  // ------------------------------------------ loads
            int stage = 0, placed = 0;
            uint32_t phase = 0;
            bool ok = true;
            Tile next;
            bool more = work.at(0, t);
            for (int j = 1; ok && more; ++j) {
                more = false;
                // this CTA's rows of A, and its half of the columns of B
                const int m0 = t.m0 + (int)rank * kHalf, n0 = t.n0 + (int)rank * (t.width / 2);
                const bool two = MODE != kGradients || t.width > kTileN / 2;  // boxes of 64 columns that hold its half
                const bool last = MODE != kGradients && t.kind == kGatesEdge;
                const uint32_t bytes = MODE != kGradients ? 2 * kOperandBytes + (last ? p.step_edge : p.step) * kTileK * 2
                                                          : 2 * (two ? kBlockBytes : kBlockBytes - kBoxBytes);
                const int half_k = MODE == kGradients ? (p.wide + kTileK - 1) / kTileK : 0;
                for (int k = t.k0; k < t.k1; k += kStageBlocks) {
                    ok = wait_for(&sh.empty[stage], phase ^ 1, dead, limit, p.status);
                    if (!ok) break;
                    const int blocks = t.k1 - k < kStageBlocks ? t.k1 - k : kStageBlocks;
                    const uint32_t bar = in_cta(smem_addr(&sh.full[stage]), 0);
                    sh.bytes[rank][stage] = blocks * bytes;
                    if (rank == 0) bar_expect(smem_addr(&sh.full[stage]), blocks * bytes);
                    for (int i = 0; i < blocks; ++i) {
                        const uint32_t a = stage0 + stage * kStageBytes + i * kBlockBytes, b = a + kOperandBytes;
                        if constexpr (MODE != kGradients) {
                            const int kk = (k + i) * kTileK;
                            tma_load(a, &p.x_k, kk, m0, bar);
                            tma_load(b, rank == 0 ? (last ? &p.gate_k_edge : &p.gate_k) : (last ? &p.up_k_edge : &p.up_k), kk, t.n0 / 2, bar);
                        } else if (t.kind == kGradX) {
                            const bool second = k + i >= half_k;
                            const int kk = (k + i - (second ? half_k : 0)) * kTileK;
                            const CUtensorMap *w = second ? &p.up_mn : &p.gate_mn;
                            tma_load(a, second ? &p.du_k : &p.dg_k, kk, m0, bar);
                            tma_load(b, w, n0, kk, bar);
                            if (two) tma_load(b + kBoxBytes, w, n0 + 64, kk, bar);
                        } else {
                            const int kk = (k + i) * kTileK;
                            const CUtensorMap *s = t.kind == kGradGate ? &p.dg_mn : &p.du_mn;
                            tma_load(a, s, m0, kk, bar);
                            tma_load(a + kBoxBytes, s, m0 + 64, kk, bar);
                            tma_load(b, &p.x_mn, n0, kk, bar);
                            if (two) tma_load(b + kBoxBytes, &p.x_mn, n0 + 64, kk, bar);
                        }
                    }
                    ++placed;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    // the divisions of the next tile's place, while loads are on their way
                    if (k == t.k0) more = work.at(j, next);
                }
                t = next;
            }
            store_in_cta(&sh.placed[rank], 0, placed);
            if (rank == 1)
                for (int s = 0; s < kStages; ++s) store_in_cta(&sh.bytes[1][s], 0, sh.bytes[1][s]);
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {  // ------------------------- products
            int stage = 0, buf = 0, consumed = 0;
            uint32_t phase = 0, acc_phase = 0;
            // as in loss.cu: this thread finds out what comes next while a stage is under way
            bool ok = true, ready = false, vacant = false;
            Tile after;
            bool more = work.at(0, t);
            Feed feed = feed_of<BF16, MODE>(t, stage0), feed_after;
            for (int j = 1; ok && more; ++j) {
                more = false;
                if (!vacant) ok = wait_for(&sh.acc_empty[buf], acc_phase ^ 1, dead, limit, p.status);
                if (!ok) break;
                const uint32_t acc = tmem + buf * kTileN;
                const uint32_t next_acc_phase = buf ? acc_phase ^ 1 : acc_phase;
                vacant = false;
                uint32_t add = 0;
                for (int k = t.k0; k < t.k1; k += kStageBlocks) {
                    if (!ready) ok = wait_for(&sh.full[stage], phase, dead, limit, p.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = feed.a + (uint32_t)stage * (kStageBytes >> 4), b = feed.b + (uint32_t)stage * (kStageBytes >> 4);
                    feed.block(acc, a, b, add);
                    if (k + 1 < t.k1) feed.block(acc, a + (kBlockBytes >> 4), b + (kBlockBytes >> 4), 1);
                    mma_commit(smem_addr(&sh.empty[stage]));
                    add = 1;
                    ++consumed;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    ready = bar_test(smem_addr(&sh.full[stage]), phase);
                    if (k + kStageBlocks >= t.k1) vacant = bar_test(smem_addr(&sh.acc_empty[buf ^ 1]), next_acc_phase ^ 1);
                    if (k == t.k0) {
                        more = work.at(j, after);
                        feed_after = feed_of<BF16, MODE>(after, stage0);
                    }
                }
                if (!ok) break;
                mma_commit(smem_addr(&sh.acc_full[buf]));
                buf ^= 1;
                acc_phase = next_acc_phase;
                t.k0 = after.k0;
                t.k1 = after.k1;
                feed = feed_after;
            }
            sh.consumed = consumed;
            // whoever gave up: no product reads shared memory or writes sums any more
            mma_commit_here(smem_addr(&sh.drained));
            if (!wait_out(&sh.drained, 0)) give_up(dead, p.status);
        }
    } else {  // ------------------------------------------------------ results
        const int quad = warp & 3;              // the quarter of the lanes this warp may read
        const int group = (warp - 2) >> 2;      // which half of the columns it takes
        const float scale = MODE == kForward ? 1.0f : scale_of(p.tops);
        const float factor = 1.0f / scale;      // powers of two
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int j = 0; work.at(j, t); ++j) {
            const int row0 = t.m0 + (int)rank * kHalf + quad * 32;  // this warp's first row of M
            const long long row = row0 + lane;
            // grad_out of the 64 elements of this lane's row, asked for while the sums are under way, whole
            // sectors where they lie so.  (16 at a time, the next 16 asked for between the results: the
            // backward pass of 2048 x 1600 x 4264 116.9 -> 116.2 us, of 5000 x 776 x 3000 135.5 -> 133.9,
            // of 1023 x 768 x 2048 31.9 -> 31.2, of 200 x 544 x 1200 19.6 -> 19.7.)
            uint4 grad[MODE == kSlopes ? 8 : 1];
            if constexpr (MODE == kSlopes) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const int f = t.n0 / 2 + group * 64 + 8 * i;
                    const uint4 *at = p.grad_out + row * p.grad_stride + f / 8;
                    const bool here = row < p.tokens && f < p.wide, both_here = here && f + 8 < p.wide;
                    grad[i] = grad[i + 1] = make_uint4(0u, 0u, 0u, 0u);
                    if (both_here && (reinterpret_cast<uintptr_t>(at) & 31u) == 0) {
                        load_sector(at, grad[i], grad[i + 1]);
                    } else {
                        if (here) grad[i] = __ldg(at);
                        if (both_here) grad[i + 1] = __ldg(at + 1);
                    }
                }
            }
            if (j == 0) {  // the first results' pages (1023 x 768 x 2048 forward 9.15 -> 8.96 us)
                if constexpr (MODE != kGradients) {
                    const int f = t.n0 / 2 + group * 64;
                    if (row < p.tokens && f < p.wide) {
                        ask_page((MODE == kForward ? p.out : p.dg).at + row * (MODE == kForward ? p.out : p.dg).stride + f);
                        if (MODE == kSlopes) ask_page(p.du.at + row * p.du.stride + f);
                    }
                } else {
                    const Rows &to = t.kind == kGradX ? p.gx : t.kind == kGradGate ? p.ggate : p.gup;
                    const int col = t.n0 + group * kResultColumns;
                    if (t.kind == kGradX && p.splits > 1) {
                        if (col < p.dim) ask_page(p.sums + (t.split * p.rows + row) * p.dim + col);
                    } else if (row < (t.kind == kGradX ? p.tokens : (long long)p.wide) && col < p.dim) {
                        ask_page(to.at + row * to.stride + col);
                    }
                }
            }
            const bool got = wait_for(&sh.acc_full[buf], acc_phase, dead, limit, p.status);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kTileN + ((uint32_t)(quad * 32) << 16);
            if constexpr (MODE != kGradients) {
                // 16 elements at a time
                const int f0 = t.n0 / 2 + group * 64;
                RowWriter first(MODE == kForward ? p.out : p.dg, row, f0), second(p.du, row, f0);
                const int end = group * 64 + 64 < t.width / 2 ? group * 64 + 64 : t.width / 2;
                if constexpr (MODE == kForward) {
                    int c = group * 64;
#pragma unroll 1
                    for (; c < end; c += 16) {
                        float g[16], u[16];
                        uint32_t w[8];
                        tmem_load16(acc + c, g);
                        tmem_load16(acc + t.width / 2 + c, u);
                        if (p.act == ZERO_ACT_SILU) outs_of<ZERO_ACT_SILU>(g, u);
                        else if (p.act == ZERO_ACT_GELU) outs_of<ZERO_ACT_GELU>(g, u);
                        else outs_of<ZERO_ACT_GELU_TANH>(g, u);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pack_lp<BF16>(u[2 * i], u[2 * i + 1]);
                        if (row < p.tokens) first.put(t.n0 / 2 + c, w);
                    }
                    if (row < p.tokens) first.finish(t.n0 / 2 + c);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int c = group * 64 + 16 * h;
                        if (c >= end) break;
                        float g[16], u[16], go[16];
                        uint32_t w[8];
                        tmem_load16(acc + c, g);
                        tmem_load16(acc + t.width / 2 + c, u);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float x[8];
                            widen8<BF16>(grad[2 * h + i], x);
#pragma unroll
                            for (int k = 0; k < 8; ++k) go[8 * i + k] = BF16 ? x[k] : x[k] * scale;
                        }
                        if (p.act == ZERO_ACT_SILU) slopes_of<ZERO_ACT_SILU>(go, g, u);
                        else if (p.act == ZERO_ACT_GELU) slopes_of<ZERO_ACT_GELU>(go, g, u);
                        else slopes_of<ZERO_ACT_GELU_TANH>(go, g, u);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pack_lp<BF16>(g[2 * i], g[2 * i + 1]);
                        if (row < p.tokens) first.put(t.n0 / 2 + c, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pack_lp<BF16>(u[2 * i], u[2 * i + 1]);
                        if (row < p.tokens) second.put(t.n0 / 2 + c, w);  // (the slopes' rows begin at sectors)
                    }
                }
            } else {
                const bool sums = t.kind == kGradX && p.splits > 1;
                const Rows to = t.kind == kGradX ? p.gx : t.kind == kGradGate ? p.ggate : p.gup;
                const bool mine = row < (t.kind == kGradX ? p.tokens : (long long)p.wide);
                float *const part = p.sums + (t.split * p.rows + row) * p.dim;
                RowWriter writer(to, row, t.n0 + group * kResultColumns);
                int c = group * kResultColumns;
#pragma unroll 1
                for (; c < group * kResultColumns + kResultColumns && c < t.width; c += 32) {
                    float z[32];
                    tmem_load32(acc + c, z);
                    const int col = t.n0 + c;
                    uint32_t w[8];
                    if (sums) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(z[8 * h + i] * factor);
                            if (mine && col + 8 * h < p.dim) store_sector(part + col + 8 * h, w);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = pack_lp<BF16>(z[16 * h + 2 * i] * factor, z[16 * h + 2 * i + 1] * factor);
                            if (mine) writer.put(col + 16 * h, w);
                        }
                    }
                }
                if (mine && !sums) writer.finish(t.n0 + c);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_cluster(in_cta(smem_addr(&sh.acc_empty[buf]), 0));
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1;
        }
    }
    __syncwarp();
    __syncthreads();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    // as in loss.cu: after a wait that gave up, copies may still be on their way to either
    // CTA's shared memory
    if (*dead) {
        if (rank == 0 && threadIdx.x == 0) {
            FullBars bars{sh.full};
            if (!drain_copies(sh.placed, sh.bytes, sh.consumed, bars)) atomicOr(p.status, ZERO_LOSS_TIMEOUT);
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns) : "memory");
}

// ------------------------------------------------------------------- few tokens

// Up to kNarrow tokens the matrices are what takes time, read once, and a tile of 256 tokens
// would hold few.  Here the matrices are the A operand: a CTA takes 128 rows of both, x is B,
// and a row of tensor memory holds one f's sums for every token, g's columns before u's.
// A cluster of CTAs shares a tile's K between them, so that as many CTAs as run at once
// load at the same time; each then adds up its share of the elements from all of them.
constexpr int kNarrow = 128;
constexpr int kNarrowThreads = 192;          // loads, products, and a warp for each quarter of the lanes
constexpr int kNarrowSmem = 220 * 1024, kNarrowHalf = 112 * 1024;  // one CTA on an SM, or two
constexpr int kNarrowWays = 8;               // CTAs of a cluster, at most
constexpr int kNarrowStages = 5;

struct NarrowPlan {
    int columns;  // tokens rounded up to what a product takes
    int stages, stage_bytes, ways, tmem, smem;
};

// Clusters of 1 to 8 CTAs that run at once with one CTA on an SM (cudaOccupancyMaxActiveClusters:
// what the SMs of a GPC leave room for); with two on each, twice as many.
constexpr int kClusters[kNarrowWays] = {152, 76, 46, 36, 28, 23, 15, 15};

int ways_of(int64_t tiles, int64_t blocks, int on_each) {
    int ways = (int)std::max<int64_t>(1, std::min<int64_t>(kNarrowWays, blocks / 2));
    while (ways > 1 && tiles > on_each * kClusters[ways - 1]) --ways;
    return ways;
}

// One CTA on an SM, with a long ring, if that leaves each tile two of them; else two.  As many ways
// as run at once: 34 tiles of 25 blocks (1600 x 4264, 24 tokens) 14.4, 10.9, 10.2, 9.9 us
// with 1 to 4 ways and one CTA on an SM, 15.4 and 21 with 5 and 8, which are two rounds; 86 tiles
// of 64 (4096 x 10928) 35.7 us whole and 32.2 three ways with two on an SM.
NarrowPlan narrow_plan(int64_t tokens, int64_t wide, int dim) {
    NarrowPlan n;
    n.columns = (int)up(tokens, 16);
    n.stage_bytes = 2 * kOperandBytes + n.columns * 128;
    n.tmem = 32;
    while (n.tmem < 2 * n.columns) n.tmem *= 2;
    const int64_t tiles = up(wide, kHalf) / kHalf, blocks = up(dim, kTileK) / kTileK;
    n.ways = ways_of(tiles, blocks, 1);
    // (the sums of more than 64 tokens take more than half an SM's shared memory)
    n.smem = n.ways > 1 || blocks < 4 || n.columns > 64 ? kNarrowSmem : kNarrowHalf;
    if (n.smem == kNarrowHalf) n.ways = ways_of(tiles, blocks, 2);
    n.stages = std::min(kNarrowStages, (n.smem - 1024) / n.stage_bytes);
    return n;
}

// Whether so few tokens are better off here than in tiles of 256, by what either takes beyond a
// launch, in us as measured: here the matrices at 6 TB/s and 0.045 for a token's sums, there 0.3
// for a block of K in each round of tiles, or the matrices at 4.2 TB/s.  (768 x 2048: 5.8 us here
// and 7.4 there with 8 tokens, 7.5 and 7.3 with 48; 4088 x 400: 8.6 and 20.3 with 32; 200 x 400:
// 4.6 and 4.8 with 8, 5.3 and 4.9 with 24.)
bool few(int64_t tokens, int64_t wide, int dim) {
    if (tokens > kNarrow) return false;
    const double bytes = 4.0 * (double)wide * dim, blocks = (double)(up(dim, kTileK) / kTileK);
    const double rounds = (double)(up(up(2 * wide, kTileN) / kTileN, kPairs) / kPairs);
    return 0.045 * (double)tokens + bytes / 6.0e6 < std::max(0.3 * blocks * rounds, bytes / 4.2e6);
}

struct NarrowParams {
    CUtensorMap gate_k, up_k;  // 64 of D x 128 of F
    CUtensorMap x_k;           // 64 of D x all tokens' columns
    int tokens, wide, k_blocks, act;
    int columns, stages, stage_bytes, ways, tmem;
    uint16_t *out;             // forward
    long long out_stride;
    const uint16_t *grad_out;  // slopes
    long long grad_stride;
    uint16_t *dg, *du;
    long long slope_stride;
    const float *tops;
    int *status;
    long long wait_cycles;
};

__device__ __forceinline__ void tma_load_here(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void commit_one(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float4 load_in_cta(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(in_cta(addr, rank)) : "memory");
    return v;
}

// A bounded wait of this CTA's: false once `limit` cycles have passed, or another wait of it has given up.
__device__ __forceinline__ bool narrow_wait(uint64_t *bar, uint32_t parity, volatile int *dead, long long limit, int *status) {
    const uint32_t b = smem_addr(bar);
    if (bar_try(b, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(b, parity)) {
        if (*dead || clock64() - t0 >= limit) {
            *dead = 1;
            atomicOr(status, ZERO_LOSS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// the results of four neighbouring elements from their sums
template <bool BF16, int MODE>
__device__ __forceinline__ void narrow_results(const NarrowParams &p, long long t, long long f, float scale, float (&g)[4], float (&u)[4]) {
    if constexpr (MODE == kForward) {
        if (p.act == ZERO_ACT_SILU) outs_of<ZERO_ACT_SILU>(g, u);
        else if (p.act == ZERO_ACT_GELU) outs_of<ZERO_ACT_GELU>(g, u);
        else outs_of<ZERO_ACT_GELU_TANH>(g, u);
        *reinterpret_cast<uint2 *>(p.out + t * p.out_stride + f) = make_uint2(pack_lp<BF16>(u[0], u[1]), pack_lp<BF16>(u[2], u[3]));
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(p.grad_out + t * p.grad_stride + f);
        float w[8];
        widen8<BF16>(make_uint4(q.x, q.y, 0u, 0u), w);
        const float go[4] = {w[0] * scale, w[1] * scale, w[2] * scale, w[3] * scale};
        if (p.act == ZERO_ACT_SILU) slopes_of<ZERO_ACT_SILU>(go, g, u);
        else if (p.act == ZERO_ACT_GELU) slopes_of<ZERO_ACT_GELU>(go, g, u);
        else slopes_of<ZERO_ACT_GELU_TANH>(go, g, u);
        *reinterpret_cast<uint2 *>(p.dg + t * p.slope_stride + f) = make_uint2(pack_lp<BF16>(g[0], g[1]), pack_lp<BF16>(g[2], g[3]));
        *reinterpret_cast<uint2 *>(p.du + t * p.slope_stride + f) = make_uint2(pack_lp<BF16>(u[0], u[1]), pack_lp<BF16>(u[2], u[3]));
    }
}

template <bool BF16, int MODE>
__global__ void __launch_bounds__(kNarrowThreads)
gated_narrow(const __grid_constant__ NarrowParams p) {
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t full[kNarrowStages], empty[kNarrowStages], done;
    __shared__ uint32_t tmem_at;
    __shared__ int dead_flag, placed_count, consumed_count;
    const uint32_t stage0 = (smem_addr(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            bar_init(smem_addr(&full[s]), 1);
            bar_init(smem_addr(&empty[s]), 1);
        }
        bar_init(smem_addr(&done), 1);
        dead_flag = placed_count = consumed_count = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)), "r"(p.tmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    if (threadIdx.x == 0) {
        ask_for(&p.gate_k);
        ask_for(&p.up_k);
        ask_for(&p.x_k);
    }
    pdl_enter();

    volatile int *dead = &dead_flag;
    const int tile = blockIdx.x / p.ways, f0 = tile * kHalf;
    const int k0 = p.k_blocks * (int)rank / p.ways, k1 = p.k_blocks * ((int)rank + 1) / p.ways;
    if (warp == 0) {
        if (lane == 0) {  // ------------------------------------------ loads
            int stage = 0, placed = 0;
            uint32_t phase = 0;
            for (int k = k0; k < k1; ++k) {
                if (!narrow_wait(&empty[stage], phase ^ 1, dead, p.wait_cycles, p.status)) break;
                const uint32_t bar = smem_addr(&full[stage]), a = stage0 + stage * p.stage_bytes;
                bar_expect(bar, p.stage_bytes);
                tma_load_here(a, &p.gate_k, k * kTileK, f0, bar);
                tma_load_here(a + kOperandBytes, &p.up_k, k * kTileK, f0, bar);
                tma_load_here(a + 2 * kOperandBytes, &p.x_k, k * kTileK, 0, bar);
                ++placed;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            placed_count = placed;
        }
    } else if (warp == 1) {
        if (lane == 0) {  // --------------------------------------- products
            uint32_t idesc = 1u << 4 | (BF16 ? 1u << 7 | 1u << 10 : 0u);  // float sums
            idesc |= (uint32_t)(p.columns >> 3) << 17 | (uint32_t)(kHalf >> 4) << 24;
            int stage = 0, consumed = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int k = k0; k < k1; ++k) {
                ok = narrow_wait(&full[stage], phase, dead, p.wait_cycles, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = stage0 + stage * p.stage_bytes;
                const uint64_t g = operand_desc(at, false), u = operand_desc(at + kOperandBytes, false), x = operand_desc(at + 2 * kOperandBytes, false);
#pragma unroll
                for (int i = 0; i < kTileK / 16; ++i) {
                    mma_one(tmem, g + 2 * i, x + 2 * i, idesc, k > k0 || i > 0);
                    mma_one(tmem + p.columns, u + 2 * i, x + 2 * i, idesc, k > k0 || i > 0);
                }
                commit_one(smem_addr(&empty[stage]));
                ++consumed;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            consumed_count = consumed;
            // also after a wait that gave up: no product reads shared memory any more
            commit_one(smem_addr(&done));
            if (!wait_out(&done, 0)) {
                *dead = 1;
                atomicOr(p.status, ZERO_LOSS_TIMEOUT);
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    __syncthreads();  // the products are done, and every copy that they waited for has landed
    tc_fence_after();
    if (*dead && threadIdx.x == 0) {  // copies on their way would land in what follows
        for (int n = consumed_count; n < placed_count; ++n)
            if (!wait_out(&full[n % p.stages], (uint32_t)(n / p.stages) & 1u)) atomicOr(p.status, ZERO_LOSS_TIMEOUT);
    }
    const float scale = MODE == kForward ? 1.0f : scale_of(p.tops);
    __syncthreads();  // thread 0 may have waited for copies
    // this CTA's sums to its shared memory: [g, then u][token][128 of f]
    if (warp >= 2) {
        const int quad = warp & 3;
        const uint32_t row = tmem + ((uint32_t)(quad * 32) << 16);
        for (int c = 0; c < 2 * p.columns; c += 16) {
            float z[16];
            tmem_load16(row + c, z);
            const int first = c < p.columns ? c : c - p.columns, left = p.tokens - first;
            const uint32_t to = stage0 + (((c < p.columns ? 0 : p.tokens) + first) * kHalf + quad * 32 + lane) * 4;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + i * kHalf * 4), "f"(z[i]) : "memory");
        }
    }
    __syncthreads();
    if (p.ways > 1) cluster_sync();
    const int fours = p.tokens * (kHalf / 4);
    const int i0 = fours * (int)rank / p.ways, i1 = fours * ((int)rank + 1) / p.ways;
    for (int i = i0 + (int)threadIdx.x; i < i1; i += kNarrowThreads) {
        const long long f = f0 + i % (kHalf / 4) * 4;
        if (f >= p.wide) continue;
        float4 part[2][kNarrowWays];
#pragma unroll
        for (int r = 0; r < kNarrowWays; ++r)
            if (r < p.ways) {
                part[0][r] = load_in_cta(stage0 + i * 16, r);
                part[1][r] = load_in_cta(stage0 + (fours + i) * 16, r);
            }
        float sum[2][4] = {};
#pragma unroll
        for (int r = 0; r < kNarrowWays; ++r)
            if (r < p.ways)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h][0] += part[h][r].x;
                    sum[h][1] += part[h][r].y;
                    sum[h][2] += part[h][r].z;
                    sum[h][3] += part[h][r].w;
                }
        narrow_results<BF16, MODE>(p, i / (kHalf / 4), f, scale, sum[0], sum[1]);
    }
    __syncthreads();
    if (p.ways > 1) cluster_sync();  // the others have read this CTA's
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem) : "memory");
}

// ---------------------------------------------------------- the smaller kernels

// The largest finite |grad_out| of a block's share of the rows, fp16.
__global__ void __launch_bounds__(kTopThreads)
gated_top(const uint4 *__restrict__ grad, long long stride, long long tokens, int vecs, float *tops) {
    pdl_enter();
    __shared__ uint32_t warp_top[kTopThreads / 32];
    uint32_t top = 0u;
    const auto look = [&](uint32_t w) {
        const uint32_t lo = w & 0x7fffu, hi = w >> 16 & 0x7fffu;
        top = max(top, max(lo < 0x7c00u ? lo : 0u, hi < 0x7c00u ? hi : 0u));
    };
    // a warp takes a row's stretch of 32 x 4 vectors at a time
    const long long parts = (vecs + 127) / 128, all = parts * tokens;
    const int lane = threadIdx.x & 31;
    for (long long i = (long long)blockIdx.x * (kTopThreads / 32) + threadIdx.x / 32; i < all; i += (long long)gridDim.x * (kTopThreads / 32)) {
        const long long t = i / parts;
        const int v0 = (int)(i - t * parts) * 128 + lane;
        uint4 q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = v0 + 32 * k < vecs ? grad[t * stride + v0 + 32 * k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            look(q[k].x);
            look(q[k].y);
            look(q[k].z);
            look(q[k].w);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) warp_top[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kTopThreads / 32; ++w) top = max(top, warp_top[w]);
        tops[blockIdx.x] = __half2float(__ushort_as_half((unsigned short)top));
    }
}

constexpr int kFinishThreads = 128;

// grad_x: the partial sums in order, rounded once.  A thread takes eight elements and asks for
// four parts at a time.
template <bool BF16>
__global__ void __launch_bounds__(kFinishThreads)
gated_finish(const float4 *__restrict__ sums, long long tokens, long long rows, int splits, int vecs, uint4 *out, long long stride) {
    pdl_enter();
    const long long all = tokens * vecs;
    for (long long i = (long long)blockIdx.x * kFinishThreads + threadIdx.x; i < all; i += (long long)gridDim.x * kFinishThreads) {
        const long long t = i / vecs, v = i - t * vecs;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        for (int s0 = 0; s0 < splits; s0 += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (s0 + k >= splits) break;
                const float4 *src = sums + (((s0 + k) * rows + t) * vecs + v) * 2;
                a[k] = src[0];
                b[k] = src[1];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (s0 + k >= splits) break;
                lo.x += a[k].x; lo.y += a[k].y; lo.z += a[k].z; lo.w += a[k].w;
                hi.x += b[k].x; hi.y += b[k].y; hi.z += b[k].z; hi.w += b[k].w;
            }
        }
        out[t * stride + v] = make_uint4(pack_lp<BF16>(lo.x, lo.y), pack_lp<BF16>(lo.z, lo.w), pack_lp<BF16>(hi.x, hi.y),
                                         pack_lp<BF16>(hi.z, hi.w));
    }
}

// ------------------------------------------------------------------------ host

// Pairs of CTAs that run at once on the current device, their shared memory having been
// allowed: or an error below zero.
template <bool BF16, int MODE>
int pairs_at_once() {
    static PerDevice kept;
    return kept.get([] {
        const int set = done_or_error(
            cudaFuncSetAttribute(gated_products<BF16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGatedSmem));
        if (set < 0) return set;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kProductThreads);
        cfg.dynamicSmemBytes = kGatedSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const int asked = done_or_error(cudaOccupancyMaxActiveClusters(&clusters, gated_products<BF16, MODE>, &cfg));
        if (asked < 0) return asked;
        return clusters > 0 ? clusters : -(int)cudaErrorInvalidConfiguration;
    });
}

// GatedWork's catch_up and start: of a few near what evens out the pairs' shares, those with
// which the last pair ends first.  (Without, and with the edge tiles among the others,
// 2048 x 1600 x 4264 took 246 blocks of K and not 210, 5000 x 776 x 3000 279 and not 213.)
void plan_gradients(GatedParams &p, int pairs) {
    constexpr int kMost = 256;
    p.catch_up = p.start = 0;
    if (pairs > kMost) return;
    const int64_t rows = up(p.tokens, kTileM) / kTileM, columns = p.dim / kTileN, last = p.dim % kTileN;
    const double blocks = 2.0 * (double)(up(p.wide, kTileK) / kTileK) / p.splits;
    const int64_t short_blocks = up(p.tokens, kTileK) / kTileK, weight_m = 2 * (up(p.wide, kTileM) / kTileM);
    const int64_t n_whole = rows * columns * p.splits, n_x = n_whole + (last ? rows * p.splits : 0);
    const int64_t n_weight = weight_m * columns, n_weights = n_weight + (last ? weight_m : 0);
    const double x = tile_cost(blocks, kTileN), x_last = tile_cost(blocks, last);
    const double w = tile_cost((double)short_blocks, kTileN), w_last = tile_cost((double)short_blocks, last);
    // tiles i, i + by, ... below n
    const auto count = [](int64_t n, int64_t i, int64_t by) { return n > i ? (n - i + by - 1) / by : 0; };
    const int64_t fuller = n_x % pairs, others = pairs - fuller;
    double first[kMost];
    for (int q = 0; q < pairs; ++q) {
        const int64_t whole = count(n_whole, q, pairs);
        first[q] = (double)whole * x + (double)(count(n_x, q, pairs) - whole) * x_last;
    }
    const int64_t even = fuller ? (int64_t)(x / w + 0.5) : 0;
    const int64_t starts[3] = {0, fuller, n_whole % pairs};
    double best = -1.0;
    for (int64_t c = std::max<int64_t>(0, even - 2); c <= even + 1; ++c) {
        if (c > 0 && (fuller == 0 || c * others > n_weights)) break;
        const int64_t taken = c * others, whole_left = std::max<int64_t>(0, n_weight - taken), left = n_weights - taken;
        for (const int64_t start : starts) {
            double end = 0.0;
            for (int q = 0; q < pairs; ++q) {
                double mine = first[q];
                if (q >= fuller && c > 0) {
                    const int64_t whole = std::min(c, count(n_weight, q - fuller, others));
                    mine += (double)whole * w + (double)(c - whole) * w_last;
                }
                const int64_t i = q >= start ? q - start : q - start + pairs, whole = count(whole_left, i, pairs);
                mine += (double)whole * w + (double)(count(left, i, pairs) - whole) * w_last;
                end = std::max(end, mine);
            }
            if (best < 0.0 || end < best) {
                best = end;
                p.catch_up = (int)c;
                p.start = (int)start;
            }
        }
    }
}

// Tiles of both projections: `whole` of `step` columns each, then the others of step_edge, so that
// the last pair ends first.  A block of K takes (columns + 128) / 384 of what it takes with 256, as
// measured: 19 rounds of 256 and 24 of 192 (4096 x 4096 x 10928) 400 and 432 us, 15 and 19 (8184 x 1600
// x 4264) 134.6 and 140.6, but one round of 128 columns and not of 256 (300 x 1000 x 2000) 9.3
// and 11.4, two of 192 and not of 256 (129 x 4088 x 10920) 53.3 and 58.5.  With narrower ones for what
// whole rounds leave: 129 x 4088 x 10920 52.4 -> 48.8, 2048 x 1600 x 4264 36.6 -> 35.2, 700 x 2000 x
// 5000 26.8 -> 24.8.
int64_t plan_gates(GatedParams &p, int64_t tokens, int pairs) {
    const int64_t rows = up(tokens, kTileM) / kTileM, columns = 2 * (int64_t)p.wide;
    const double blocks = (double)(up(p.dim, kTileK) / kTileK);
    double best = -1.0;
    int64_t tiles = 0;
    const auto look = [&](int64_t step, int64_t whole, int64_t step_edge) {
        const int64_t left = columns - whole * step, first = whole * rows, others = up(left, step_edge) / step_edge * rows;
        const double c = tile_cost(blocks, step), c_edge = tile_cost(blocks, std::min(step_edge, up(left, 32)));
        // pairs with one tile more of the first than the rest; the others' go on behind the last of them
        const int64_t more = first % pairs, more_edge = others % pairs;
        const double even = (double)(first / pairs) * c + (double)(others / pairs) * c_edge;
        double end = even + (more_edge > 0 ? c_edge : 0.0);
        if (more > 0) end = std::max(end, even + c + (more + more_edge > pairs ? c_edge : 0.0));
        if (best >= 0.0 && end >= best * 0.995) return;  // nearly the same: as few tiles as that takes
        best = end;
        tiles = first + others;
        p.step = (int)step;
        p.whole = (int)whole;
        p.step_edge = (int)step_edge;
    };
    for (int64_t step = kTileN; step >= kTileN / 2; step -= 64) {
        const int64_t all = columns / step, rounds = all * rows / pairs;
        look(step, all, std::max<int64_t>(64, up(columns - all * step, 32)));
        for (int64_t less = 0; less < 2 && rounds - less > 0; ++less) {
            const int64_t whole = (rounds - less) * pairs / rows;
            if (whole >= all) continue;
            for (int64_t edge = step - 32; edge >= 96; edge -= 32) look(step, whole, edge);
        }
    }
    return tiles;
}

template <bool BF16, int MODE>
cudaError_t launch_products(const GatedParams &p, int64_t tiles, cudaStream_t stream) {
    const int pairs = pairs_at_once<BF16, MODE>();
    if (pairs < 0) return (cudaError_t)-pairs;
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    const int64_t use = std::max<int64_t>(1, std::min<int64_t>(pairs, tiles));
    return launch_pdl(gated_products<BF16, MODE>, dim3((unsigned)(2 * use)), dim3(kProductThreads), kGatedSmem, stream, p);
}

template <bool BF16, int MODE>
cudaError_t launch_narrow(const GatedArgs &a, uint16_t *dg, uint16_t *du, const float *tops, cudaStream_t stream) {
    static PerDevice allowed;
    const int set = allowed.get([] {
        return done_or_error(cudaFuncSetAttribute(gated_narrow<BF16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kNarrowSmem));
    });
    if (set < 0) return (cudaError_t)-set;
    const NarrowPlan n = narrow_plan(a.tokens, a.wide, a.dim);
    NarrowParams p = {};
    if (!encoder() || !make_map(&p.gate_k, a.gate, a.wide, a.dim, a.gate_stride, a.lp, false, kHalf) ||
        !make_map(&p.up_k, a.up, a.wide, a.dim, a.up_stride, a.lp, false, kHalf) ||
        !make_map(&p.x_k, a.x, a.tokens, a.dim, a.x_stride, a.lp, false, n.columns))
        return cudaErrorNotSupported;
    p.tokens = (int)a.tokens;
    p.wide = a.wide;
    p.k_blocks = (int)(up(a.dim, kTileK) / kTileK);
    p.act = a.act;
    p.columns = n.columns;
    p.stages = n.stages;
    p.stage_bytes = n.stage_bytes;
    p.ways = n.ways;
    p.tmem = n.tmem;
    p.out = static_cast<uint16_t *>(a.out);
    p.out_stride = a.out_stride;
    p.grad_out = static_cast<const uint16_t *>(a.grad_out);
    p.grad_stride = a.grad_out_stride;
    p.dg = dg;
    p.du = du;
    p.slope_stride = up(a.wide, 16);
    p.tops = tops;
    p.status = a.status;
    p.wait_cycles = loss_wait();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(up(a.wide, kHalf) / kHalf * n.ways));
    cfg.blockDim = dim3(kNarrowThreads);
    cfg.dynamicSmemBytes = n.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)n.ways;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gated_narrow<BF16, MODE>, p);
}

template <bool BF16>
cudaError_t forward_impl(const GatedArgs &a, cudaStream_t stream) {
    if (few(a.tokens, a.wide, a.dim)) return launch_narrow<BF16, kForward>(a, nullptr, nullptr, nullptr, stream);
    const int pairs = pairs_at_once<BF16, kForward>();
    if (pairs < 0) return (cudaError_t)-pairs;
    GatedParams p = {};
    p.wide = a.wide;
    p.dim = a.dim;
    const int64_t tiles = plan_gates(p, a.tokens, pairs);
    if (!encoder() || !make_map(&p.x_k, a.x, a.tokens, a.dim, a.x_stride, a.lp, false, kHalf) ||
        !make_map(&p.gate_k, a.gate, a.wide, a.dim, a.gate_stride, a.lp, false, p.step / 2) ||
        !make_map(&p.up_k, a.up, a.wide, a.dim, a.up_stride, a.lp, false, p.step / 2) ||
        !make_map(&p.gate_k_edge, a.gate, a.wide, a.dim, a.gate_stride, a.lp, false, p.step_edge / 2) ||
        !make_map(&p.up_k_edge, a.up, a.wide, a.dim, a.up_stride, a.lp, false, p.step_edge / 2))
        return cudaErrorNotSupported;
    p.out = {static_cast<uint16_t *>(a.out), a.out_stride, a.wide};
    p.tokens = a.tokens;
    p.act = a.act;
    p.splits = 1;
    p.status = a.status;
    p.wait_cycles = loss_wait();
    return launch_products<BF16, kForward>(p, tiles, stream);
}

template <bool BF16>
cudaError_t backward_impl(const GatedArgs &a, cudaStream_t stream) {
    const GatedLayout l = gated_layout(a.tokens, a.wide, a.dim);
    char *ws = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(a.workspace) + (kBase - 1)) & ~uintptr_t(kBase - 1));
    float *tops = reinterpret_cast<float *>(ws), *sums = reinterpret_cast<float *>(ws + l.sums);
    void *dg = ws + l.slope_gate, *du = ws + l.slope_up;
    const int pairs = pairs_at_once<BF16, kSlopes>();
    if (pairs < 0) return (cudaError_t)-pairs;
    GatedParams p = {};
    p.wide = a.wide;
    p.dim = a.dim;
    const int64_t gate_tiles = plan_gates(p, a.tokens, pairs);
    const auto map = [&](CUtensorMap *m, const void *at, int64_t rows, int64_t cols, int64_t stride, int box) {
        return make_map(m, at, rows, cols, stride, a.lp, false, box);
    };
    if (!encoder() || !map(&p.x_k, a.x, a.tokens, a.dim, a.x_stride, kHalf) || !map(&p.gate_k, a.gate, a.wide, a.dim, a.gate_stride, p.step / 2) ||
        !map(&p.up_k, a.up, a.wide, a.dim, a.up_stride, p.step / 2) ||
        !map(&p.gate_k_edge, a.gate, a.wide, a.dim, a.gate_stride, p.step_edge / 2) ||
        !map(&p.up_k_edge, a.up, a.wide, a.dim, a.up_stride, p.step_edge / 2) || !map(&p.x_mn, a.x, a.tokens, a.dim, a.x_stride, kTileK) ||
        !map(&p.gate_mn, a.gate, a.wide, a.dim, a.gate_stride, kTileK) || !map(&p.up_mn, a.up, a.wide, a.dim, a.up_stride, kTileK) ||
        !map(&p.dg_k, dg, a.tokens, a.wide, l.stride, kHalf) || !map(&p.du_k, du, a.tokens, a.wide, l.stride, kHalf) ||
        !map(&p.dg_mn, dg, a.tokens, a.wide, l.stride, kTileK) || !map(&p.du_mn, du, a.tokens, a.wide, l.stride, kTileK))
        return cudaErrorNotSupported;
    p.tokens = a.tokens;
    p.rows = l.rows;
    p.splits = l.splits;
    p.act = a.act;
    p.dg = {static_cast<uint16_t *>(dg), l.stride, a.wide};
    p.du = {static_cast<uint16_t *>(du), l.stride, a.wide};
    p.gx = {static_cast<uint16_t *>(a.grad_x), a.grad_x_stride, a.dim};
    p.ggate = {static_cast<uint16_t *>(a.grad_gate), a.grad_gate_stride, a.dim};
    p.gup = {static_cast<uint16_t *>(a.grad_up), a.grad_up_stride, a.dim};
    p.sums = sums;
    p.grad_out = static_cast<const uint4 *>(a.grad_out);
    p.grad_stride = a.grad_out_stride / 8;
    p.tops = BF16 ? nullptr : tops;
    p.status = a.status;
    p.wait_cycles = loss_wait();
    const int64_t row_tiles = l.rows / kTileM, dim_tiles = up(a.dim, kTileN) / kTileN;
    cudaError_t e = cudaSuccess;
    // (nothing may come between gated_top and the slopes, whose loads do not wait for it: launch.h)
    if (!BF16)
        e = launch_pdl(gated_top, dim3(kTopBlocks), dim3(kTopThreads), 0, stream, p.grad_out, p.grad_stride, (long long)a.tokens, a.wide / 8, tops);
    if (e == cudaSuccess && few(a.tokens, a.wide, a.dim))
        e = launch_narrow<BF16, kSlopes>(a, static_cast<uint16_t *>(dg), static_cast<uint16_t *>(du), p.tops, stream);
    else if (e == cudaSuccess)
        e = launch_products<BF16, kSlopes>(p, gate_tiles, stream);
    if (e != cudaSuccess) return e;
    const int64_t tiles = row_tiles * dim_tiles * l.splits + 2 * (up(a.wide, kTileM) / kTileM) * dim_tiles;
    const int gradient_pairs = pairs_at_once<BF16, kGradients>();
    if (gradient_pairs < 0) return (cudaError_t)-gradient_pairs;
    plan_gradients(p, (int)std::min<int64_t>(gradient_pairs, tiles));
    e = launch_products<BF16, kGradients>(p, tiles, stream);
    if (e == cudaSuccess && l.splits > 1)
        e = launch_pdl(gated_finish<BF16>, dim3((unsigned)std::min<int64_t>(up(a.tokens * (a.dim / 8), kFinishThreads) / kFinishThreads, 16 * sm_count())), dim3(kFinishThreads), 0, stream,
                       reinterpret_cast<const float4 *>(sums), (long long)a.tokens, (long long)l.rows, l.splits, a.dim / 8,
                       static_cast<uint4 *>(a.grad_x), (long long)(a.grad_x_stride / 8));
    return e;
}

}  // namespace

int64_t gated_forward_bytes(int64_t, int64_t, int) { return 0; }

int64_t gated_backward_bytes(int64_t tokens, int64_t wide, int dim) { return gated_layout(tokens, wide, dim).bytes; }

cudaError_t launch_gated_forward(const GatedArgs &a, cudaStream_t stream) {
    return a.lp ? forward_impl<true>(a, stream) : forward_impl<false>(a, stream);
}

cudaError_t launch_gated_backward(const GatedArgs &a, cudaStream_t stream) {
    if (a.tokens == 0) {  // no token: zero gradients of the matrices
        const cudaError_t e = cudaMemset2DAsync(a.grad_gate, size_t(a.grad_gate_stride) * 2, 0, size_t(a.dim) * 2, size_t(a.wide), stream);
        if (e != cudaSuccess) return e;
        return cudaMemset2DAsync(a.grad_up, size_t(a.grad_up_stride) * 2, 0, size_t(a.dim) * 2, size_t(a.wide), stream);
    }
    return a.lp ? backward_impl<true>(a, stream) : backward_impl<false>(a, stream);
}

}  // namespace zk
