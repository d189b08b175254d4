// loss.cu -- softmax cross entropy of hidden states against a vocabulary
// matrix, without keeping the logits, and its gradients (sm_103a).
//
// With H the hidden states [T, D], W the matrix [V, D], y the targets:
//   z = H W^T,  lse[t] = log sum_v exp(z[t][v]),  loss[t] = lse[t] - z[t][y[t]]
//   q[t][v] = g[t] (exp(z[t][v] - lse[t]) - [v == y[t]]),  gH = q W,  gW = q^T H
// Forward is one product whose tiles are reduced to a maximum and a sum of
// exponentials per row as they leave the tensor cores.  Backward takes the
// vocabulary in pieces: a piece's logits again, q of the piece in lp, then the
// two products that use it.  So 2 T D V operations forward and 6 T D V
// backward, and no buffer holds more than a piece.
//
// All four products run in one kernel (loss_products): pairs of CTAs, each pair
// one 256 x 256 tile, tcgen05.mma on 256 x 256 x 16 with operands that TMA
// places in shared memory and sums that stay in tensor memory.  A pair halves
// what each SM reads of B; two pairs that share B by multicast were 1-3 % slower
// (clusters of four fill 144 of 152 SMs).
//
// On GB300, vocabulary 50257: forward 8184 x 1600 0.81 ms (1620 TFLOP/s; 0.72 ms
// from a cold start); forward and gradients 4096 x 4096 4.3 ms (8 T D V operations,
// 1570 TFLOP/s), 2048 x 1600 0.93 ms, 1023 x 768 0.24 ms.  Warm, the larger ones are
// bound by power (a library's bf16 product sustains 1690 TFLOP/s), the tensor pipe
// being 84-96 % active cold; the smallest by the latency of its loads.
#include "head_internal.h"
#include "launch.h"
#include "per_device.h"
#include "tile_product.cuh"
#include "zero.h"
#include "zero_internal.h"

#include <algorithm>
#include <atomic>

namespace zk {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// The tensor core's float sum drops the low bits of every step of 16, always
// towards zero: a logit of 15 over 4096 products came out 6e-5 too small, a
// relative 4e-6 where float addition has 4e-8.  The losses are float, so the
// statistics take the sum off after at most 512 products (kChunk blocks) and add it up
// in registers, rounded to nearest; q, with lp's bits or twice as many, does without.
// What is still lost depends on the data: nothing where a sum is exact (one nonzero
// product, small whole numbers), up to 32 steps' last places otherwise.  Where one logit
// of 18 to 30 is all of lse, 1024 products, vocabulary 40000: bf16 9e-7 low, fp16, whose
// longer products lose bits too as they are aligned, 2.6e-6.
constexpr int kChunk = 8;  // whole stages
// Half as many where no pair has a second tile, whose product the parts' results would
// hold up: half the error (163 x 328 x 373, the tensor core's logits alone: lse 1.0e-6
// relative, 6e-7 so) for 0 to 14 % of time (200 x 4096 x 5000 25.1 -> 28.6 us, 500 x 1600 x 8000 16.4 -> 17.6, smaller ones the
// same); with ten tiles a pair (1023 x 768 x 50257) it took 69 us and not 55.
constexpr int kShortChunk = 4;
constexpr int kTileCost = 4;  // blocks of K that starting and storing a tile cost, about

// The largest |grad_loss| becomes this in the lp operand q: fp16 keeps 15 more
// binades below it, bf16 has float's range.
__host__ __device__ constexpr float operand_top(bool bf16) { return bf16 ? 1.0f : 32768.0f; }

// ------------------------------------------------------------------ workspace

// Rounding q to lp is no matter where many tokens count, but the target's slope of
// one or a few tokens is most of a gradient, and its rounding then the gradient's
// error: up to 2.8 times what rounding the result once costs with one token, at most
// 1.7 with 7 and 1.4 from 17 on (hidden states 392 wide, eight draws each).  So up to
// this many counted tokens take a second place each, kRest further, whose row holds
// what the rounding of q in the first left over: twice lp's bits.  The places of both
// are one block of K and one tile of rows, which fewer tokens would fill as well.
constexpr int kRest = kTileK / 2;

struct LossRecord {
    int count;     // tokens that count
    int places;    // rows of the products: as many, or kTileK where each has two
    float factor;  // q in the products' operands times this is q
};

struct BackwardLayout {
    int64_t rows;      // tokens rounded up to whole tiles
    int64_t piece;     // columns of a piece of the vocabulary (whole tiles)
    int pieces;
    int splits;        // partial sums of grad_hidden
    int64_t index, place, lse2, ratio, target, at_target, hidden, slopes, sums, bytes;  // byte offsets
};

// A piece of q takes about this much at most.  (64, 96 and 128 MB, which L2 would
// hold in part: 1 to 5 % slower, as grad_hidden's sums are added to more often.)
constexpr int64_t kSlopeBytes = int64_t(256) << 20;
// ... unless there are so many tokens that it would have fewer columns than this:
// every piece reads and adds to all of grad_hidden's sums.  (100001 x 768 x 50257:
// 30.8 ms with pieces of 1280, 23.6 with 2048, 18.4 with 4096, 18.6 with 8192.)
constexpr int64_t kLeastPiece = 4096;

BackwardLayout backward_layout(int64_t tokens, int64_t vocab, int dim) {
    BackwardLayout l;
    l.rows = up(std::max<int64_t>(tokens, 1), kTileM);
    const int64_t most = std::max<int64_t>(kLeastPiece, kSlopeBytes / 2 / l.rows / kTileN * kTileN);
    l.pieces = (int)((vocab + most - 1) / most);
    l.piece = up((vocab + l.pieces - 1) / l.pieces, kTileN);
    l.pieces = (int)((vocab + l.piece - 1) / l.piece);
    // grad_hidden has few tiles and long sums: cut its sums until no part is longer
    // than a pair's share of both gradients (at most 16 ways, 8 blocks of K each)
    const int64_t dim_tiles = (dim + kTileN - 1) / kTileN, row_tiles = l.rows / kTileM;
    const int64_t long_sum = l.piece / kTileK, short_sum = (tokens + kTileK - 1) / kTileK;
    const int64_t share = (row_tiles * dim_tiles * long_sum + l.piece / kTileN * dim_tiles * short_sum) / kPairs;
    l.splits = 1;
    while (l.splits < 16 && long_sum / l.splits > share && long_sum / (l.splits + 1) >= 8) ++l.splits;
    int64_t at = 256;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at = up(at + bytes, 1024);
        return here;
    };
    l.index = take(l.rows * 4);
    l.place = take(l.rows * 4);
    l.lse2 = take(l.rows * 4);
    l.ratio = take(l.rows * 4);
    l.target = take(l.rows * 4);
    l.at_target = take(l.rows * 4);
    l.hidden = take(l.rows * dim * 2);
    l.slopes = take(l.rows * l.piece * 2);
    l.sums = take(l.splits * l.rows * dim * 4);
    l.bytes = at;
    return l;
}

// the joint (maximum, sum of exponentials relative to it) of two parts
__device__ __forceinline__ float2 join_parts(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    const float base = top == -INFINITY ? 0.0f : top;
    return make_float2(top, a.y * exp2_approx((a.x - base) * kLog2e) + b.y * exp2_approx((b.x - base) * kLog2e));
}

// ------------------------------------------------------------------- products

enum Product { kLogits = 0, kGradHidden = 1, kGradWeight = 2 };

struct ProductParams {
    CUtensorMap h_k, hc_k;    // hidden states (all, the counted ones): boxes 64 of D x 128 tokens
    CUtensorMap w_k;          // weight: 64 of D x 128 vocabulary
    CUtensorMap w_mn;         // weight: 64 of D x 64 vocabulary
    CUtensorMap h_mn, hc_mn;  // hidden states: 64 of D x 64 tokens
    CUtensorMap q_k;          // q: 64 vocabulary x 128 tokens
    CUtensorMap q_mn;         // q: 64 vocabulary x 64 tokens
    CUtensorMap q_out;        // q: 64 vocabulary x 32 tokens
    CUtensorMap gh_out;       // partial grad_hidden: 32 of D x 32 tokens, float
    CUtensorMap gw_out;       // grad_weight: 64 of D x 32 vocabulary
    int gradients;  // both gradients of the piece, else its logits (statistics or q)
    long long tokens, vocab;
    int dim;
    long long piece0, piece;  // the piece of the vocabulary (statistics: all of it)
    long long rows;           // tokens rounded up to whole tiles
    int splits;
    int first_piece;
    const LossRecord *record;  // NULL: every token counts
    // statistics
    const int64_t *target;
    float2 *parts;  // [tile of the vocabulary][token]
    float *picked;  // the target's logit
    int chunk;      // blocks of K that the tensor core adds up, whole stages
    // q, by place among the counted tokens
    const float *lse2, *ratio, *at_target;
    const int *place_target;
    int *status;
    long long wait_cycles;
};

// The statistics' sums: parts of at most p.chunk blocks of K, as even as can be (a
// short last part would have the tensor core wait for its accumulator).
__device__ __forceinline__ int chunks_of(int k_blocks, int chunk) { return (k_blocks + chunk - 1) / chunk; }

// The work of one launch, and which of it each pair does, in order.  Logits:
// every pair-th tile.  Gradients: first the tiles of grad_hidden, few and long,
// every pair-th; the pairs that get one fewer of them then take `catch_up` tiles
// of grad_weight each, about as long together as one of the others; the rest of
// grad_weight goes round all pairs.  Both products run in one launch because
// grad_hidden alone leaves the last round of pairs mostly idle.
struct Work {
    Tiles logits, hidden, weight;
    int gradients;
    int pair, pairs, n_hidden, n_weight;
    int fuller;  // pairs with one more tile of grad_hidden than the others, if not all have as many
    int catch_up;
    int mine;      // tiles of grad_hidden of this pair

    __device__ __forceinline__ Work(const ProductParams &p, long long count) {
        const long long end = p.piece0 + p.piece < p.vocab ? p.piece0 + p.piece : p.vocab;
        const int columns = (int)(end - p.piece0);
        const int row_tiles = (int)((count + kTileM - 1) / kTileM);
        const int dim_tiles = (p.dim + kTileN - 1) / kTileN, piece_tiles = (columns + kTileN - 1) / kTileN;
        logits.set(row_tiles, piece_tiles, columns, (p.dim + kTileK - 1) / kTileK, 1);
        hidden.set(row_tiles, dim_tiles, p.dim, (columns + kTileK - 1) / kTileK, p.splits);
        weight.set(piece_tiles, dim_tiles, p.dim, (int)((count + kTileK - 1) / kTileK), 1);
        gradients = p.gradients;
        pair = blockIdx.x >> 1;
        pairs = gridDim.x >> 1;
        n_hidden = hidden.size();
        n_weight = weight.size();
        fuller = n_hidden % pairs;
        const int long_tile = hidden.k_blocks / hidden.splits + kTileCost, short_tile = weight.k_blocks + kTileCost;
        catch_up = fuller ? (long_tile + short_tile / 2) / short_tile : 0;
        const int most = fuller ? n_weight / (pairs - fuller) : 0;
        if (catch_up > most) catch_up = most;
        mine = n_hidden > pair ? (n_hidden - pair + pairs - 1) / pairs : 0;
    }

    __device__ __forceinline__ bool at(int j, Tile &t) const {
        if (!gradients) {
            const int i = pair + j * pairs;
            if (i >= logits.size()) return false;
            t = logits.at(i, kLogits);
            return true;
        }
        if (j < mine) {
            t = hidden.at(pair + j * pairs, kGradHidden);
            return true;
        }
        j -= mine;
        const int others = pairs - fuller;
        int i;
        if (catch_up && pair >= fuller && j < catch_up) {
            i = pair - fuller + j * others;
        } else {
            if (catch_up && pair >= fuller) j -= catch_up;
            i = catch_up * others + pair + j * pairs;
        }
        if (i >= n_weight) return false;
        t = weight.at(i, kGradWeight);
        return true;
    }
};

template <bool BF16, bool STATS>
__device__ __forceinline__ Feed feed_of(const Tile &t, uint32_t stage0) {
    return Feed(t.width, !STATS && t.kind == kGradWeight, !STATS && t.kind != kLogits, stage0, BF16);
}

// what rounding x to the pair w left over: exact; nothing of what is not finite
template <bool BF16>
__device__ __forceinline__ float2 left_over(float2 x, uint32_t w) {
    float2 f;
    if constexpr (BF16)
        f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    const float2 r = make_float2(x.x - f.x, x.y - f.y);
    return make_float2(isfinite(r.x) ? r.x : 0.0f, isfinite(r.y) ? r.y : 0.0f);
}

template <bool BF16, bool STATS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
loss_products(const __grid_constant__ ProductParams p) {
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
    pdl_enter();

    volatile int *dead = &sh.dead;
    const long long limit = p.wait_cycles;
    const bool twice = p.record && p.record->places != p.record->count;  // each token has two places
    const bool all = p.record == nullptr || (p.record->count == p.tokens && !twice);
    const long long count = p.record ? p.record->places : p.tokens;
    const Work work(p, count);
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
                const bool two = t.width > kTileN / 2;  // boxes of 64 columns that hold its half
                const uint32_t bytes = 2 * (t.kind == kLogits || two ? kBlockBytes : kBlockBytes - kBoxBytes);
                for (int k = t.k0; k < t.k1; k += kStageBlocks) {
                    ok = wait_for(&sh.empty[stage], phase ^ 1, dead, limit, p.status);
                    if (!ok) break;
                    const int blocks = t.k1 - k < kStageBlocks ? t.k1 - k : kStageBlocks;
                    const uint32_t bar = in_cta(smem_addr(&sh.full[stage]), 0);
                    sh.bytes[rank][stage] = blocks * bytes;
                    if (rank == 0) bar_expect(smem_addr(&sh.full[stage]), blocks * bytes);
                    for (int i = 0; i < blocks; ++i) {
                        const uint32_t a = stage0 + stage * kStageBytes + i * kBlockBytes, b = a + kOperandBytes;
                        const int kk = (k + i) * kTileK;
                        if (t.kind == kLogits) {
                            tma_load(a, all ? &p.h_k : &p.hc_k, kk, m0, bar);
                            tma_load(b, &p.w_k, kk, (int)p.piece0 + n0, bar);
                        } else if (t.kind == kGradHidden) {
                            tma_load(a, &p.q_k, kk, m0, bar);
                            tma_load(b, &p.w_mn, n0, (int)p.piece0 + kk, bar);
                            if (two) tma_load(b + kBoxBytes, &p.w_mn, n0 + 64, (int)p.piece0 + kk, bar);
                        } else {
                            const CUtensorMap *h = all ? &p.h_mn : &p.hc_mn;
                            tma_load(a, &p.q_mn, m0, kk, bar);
                            tma_load(a + kBoxBytes, &p.q_mn, m0 + 64, kk, bar);
                            tma_load(b, h, n0, kk, bar);
                            if (two) tma_load(b + kBoxBytes, h, n0 + 64, kk, bar);
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
                if (t.k0 >= t.k1) more = work.at(j, next);
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
            // The tensor core takes little ahead of what it computes, so this thread finds out
            // what comes next while a stage is under way: whether the next stage is
            // there (ready), whether the next accumulator is free (vacant), and the next
            // tile with its descriptors (after, feed).
            bool ok = true, ready = false, vacant = false;
            const int stages = (work.logits.k_blocks + kStageBlocks - 1) / kStageBlocks;  // statistics: of every tile
            const int chunks = STATS ? chunks_of(work.logits.k_blocks, p.chunk) : 1;
            const int each = stages / chunks * kStageBlocks, longer = stages % chunks;
            Tile after;
            bool more = work.at(0, t);
            Feed feed = feed_of<BF16, STATS>(t, stage0), feed_after;
            for (int j = 1; ok && more; ++j) {
                more = false;
                int k = t.k0;
                for (int c = 0; c < chunks; ++c) {
                    int k1 = t.k1;
                    if (STATS && c + 1 < chunks) k1 = k + each + (c < longer ? kStageBlocks : 0);
                    if (!vacant) ok = wait_for(&sh.acc_empty[buf], acc_phase ^ 1, dead, limit, p.status);
                    if (!ok) break;
                    const uint32_t acc = tmem + buf * kTileN;
                    const uint32_t next_acc_phase = buf ? acc_phase ^ 1 : acc_phase;
                    vacant = false;
                    uint32_t add = 0;
                    for (; k < k1; k += kStageBlocks) {
                        if (!ready) ok = wait_for(&sh.full[stage], phase, dead, limit, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        uint64_t a = feed.a + (uint32_t)stage * (kStageBytes >> 4), b = feed.b + (uint32_t)stage * (kStageBytes >> 4);
                        feed.block(acc, a, b, add);
                        if (k + 1 < k1) feed.block(acc, a + (kBlockBytes >> 4), b + (kBlockBytes >> 4), 1);
                        mma_commit(smem_addr(&sh.empty[stage]));
                        add = 1;
                        ++consumed;
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                        ready = bar_test(smem_addr(&sh.full[stage]), phase);
                        if (k + kStageBlocks >= k1) vacant = bar_test(smem_addr(&sh.acc_empty[buf ^ 1]), next_acc_phase ^ 1);
                        if (k == t.k0) {
                            more = work.at(j, after);
                            feed_after = feed_of<BF16, STATS>(after, stage0);
                        }
                    }
                    if (!ok) break;
                    mma_commit(smem_addr(&sh.acc_full[buf]));
                    buf ^= 1;
                    acc_phase = next_acc_phase;
                }
                if (t.k0 >= t.k1) {
                    more = work.at(j, after);
                    feed_after = feed_of<BF16, STATS>(after, stage0);
                }
                t.k0 = after.k0;
                t.k1 = after.k1;
                feed = feed_after;
            }
            sh.consumed = consumed;
            // whoever gave up: no product reads shared memory or writes sums any more
            mma_commit_here(smem_addr(&sh.drained));
            if (!wait_out(&sh.drained, 0)) give_up(dead, p.status);
        }
    } else if constexpr (STATS) {  // ------------------------------- statistics
        const int quad = warp & 3;  // the quarter of the lanes this warp may read
        const int group = (warp - 2) >> 2;  // which of the tile's columns it takes
        using Joined = float2[kResultWarps / 4][kHalf];
        Joined *const joined = reinterpret_cast<Joined *>(smem + kStages * kStageBytes);
        int buf = 0;
        uint32_t acc_phase = 0;
        const int chunks = chunks_of(work.logits.k_blocks, p.chunk);
        for (int j = 0; work.at(j, t); ++j) {
            const int row = quad * 32 + lane;
            const long long token = (long long)t.m0 + (int)rank * kHalf + row;
            const bool mine = token < p.tokens;
            const long long v0 = (long long)t.n0 + group * kResultColumns;
            const long long left = p.vocab - v0;  // columns that exist
            const long long at = mine ? p.target[token] - v0 : -1;
            float z[kResultColumns];
#pragma unroll
            for (int i = 0; i < kResultColumns; ++i) z[i] = 0.0f;
            bool ok = true;
            for (int c = chunks; c > 0; --c) {
                const bool got = wait_for(&sh.acc_full[buf], acc_phase, dead, limit, p.status);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + buf * kTileN + group * kResultColumns + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int i = 0; i < kResultColumns; i += 16) {
                    float part[16];
                    tmem_load16(acc + i, part);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float2 two = add2(make_float2(z[i + k], z[i + k + 1]), make_float2(part[k], part[k + 1]));
                        z[i + k] = two.x;
                        z[i + k + 1] = two.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_cluster(in_cta(smem_addr(&sh.acc_empty[buf]), 0));
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
            float2 part = make_float2(-INFINITY, 0.0f);
            if (ok && left > 0) {
                if (left < kResultColumns) {
#pragma unroll
                    for (int i = 0; i < kResultColumns; ++i)
                        if (i >= left) z[i] = -INFINITY;
                }
                if (__any_sync(0xffffffffu, at >= 0 && at < kResultColumns)) {
                    float z_y = 0.0f;
#pragma unroll
                    for (int i = 0; i < kResultColumns; ++i) z_y = i == at ? z[i] : z_y;
                    if (at >= 0 && at < kResultColumns) p.picked[token] = z_y;
                }
                float tops[4] = {z[0], z[1], z[2], z[3]}, sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 4; i < kResultColumns; ++i) tops[i & 3] = fmaxf(tops[i & 3], z[i]);
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                // a row of -inf: any finite base leaves its sum at 0
                const float high = top == -INFINITY ? 0.0f : top;
                const float base = __fmul_rn(high, kLog2e);
#pragma unroll
                for (int i = 0; i < kResultColumns; i += 2) {
                    const float2 x = fma2(make_float2(z[i], z[i + 1]), make_float2(kLog2e, kLog2e), make_float2(-base, -base));
                    const float2 e = add2(make_float2(sums[i & 2], sums[(i & 2) + 1]), make_float2(exp2_approx(x.x), exp2_approx(x.y)));
                    sums[i & 2] = e.x;
                    sums[(i & 2) + 1] = e.y;
                }
                // the sum is relative to 2^base, and base to top log2(e) rounded once
                const float miss = __fmaf_rn(high, kLog2e, -base);
                const float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                part = make_float2(top, __fmaf_rn(sum, -miss * kLn2, sum));
            }
            // the warps of a row join their parts; if one gave up, all stop
            joined[j & 1][group][row] = part;
            if (any_of(1 + quad, 32 * (kResultWarps / 4), !ok)) break;
            if (group == 0 && mine) {
#pragma unroll
                for (int g = 1; g < kResultWarps / 4; ++g) part = join_parts(part, joined[j & 1][g][row]);
                p.parts[t.n * p.tokens + token] = part;
            }
        }
    } else {  // ------------------------------------------------------ results
        const int quad = warp & 3;
        const int first = ((warp - 2) >> 2) * kResultColumns;  // its columns
        const uint32_t buffer = stage0 + kStages * kStageBytes + (warp - 2) * kStoreBytes;
        const float factor = p.record->factor;
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int j = 0; work.at(j, t); ++j) {
            const int row0 = t.m0 + (int)rank * kHalf + quad * 32;  // this warp's first row of M
            const bool got = wait_for(&sh.acc_full[buf], acc_phase, dead, limit, p.status);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kTileN + ((uint32_t)(quad * 32) << 16);
            if (t.kind == kLogits) {
                const int place = row0 + lane;
                const bool rest = twice && row0 == kRest;  // this warp's rows are the second places
                const float lse2 = p.lse2[place], ratio = p.ratio[place], at_target = p.at_target[place];
                const bool live = p.place_target[place] >= 0;  // not a row that fills the last tile
                const int y = p.place_target[place] - (int)p.piece0 - t.n0;
                const long long left = p.vocab - p.piece0 - (long long)t.n0;
                // q of 32 columns, packed
                auto q_of = [&](int col, uint32_t *w) __attribute__((always_inline)) {
                    float z[32];
                    tmem_load32(acc + col, z);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 x = fma2(make_float2(z[j], z[j + 1]), make_float2(kLog2e, kLog2e), make_float2(-lse2, -lse2));
                        z[j] = exp2_approx(x.x);
                        z[j + 1] = exp2_approx(x.y);
                    }
                    const uint32_t hit = y >= col && y < col + 32 ? 1u << (y - col) : 0u;
                    if (__any_sync(0xffffffffu, hit != 0u)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] = hit >> j & 1u ? at_target : z[j];
                    }
                    const long long keep = live ? left - col : 0;  // columns that exist, in a row that counts
                    if (keep < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] = j < keep ? z[j] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = mul2(make_float2(z[2 * j], z[2 * j + 1]), make_float2(ratio, ratio));
                        w[j] = pack_lp<BF16>(x.x, x.y);
                        z[2 * j] = x.x;
                        z[2 * j + 1] = x.y;
                    }
                    if (!rest) return;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 r = left_over<BF16>(make_float2(z[2 * j], z[2 * j + 1]), w[j]);
                        w[j] = pack_lp<BF16>(r.x, r.y);
                    }
                };
                for (int c = first; c < first + kResultColumns; c += 64) {
                    uint32_t w[32];
                    q_of(c, w);
                    q_of(c + 32, w + 16);
                    put_rows(w, buffer, lane, &p.q_out, t.n0 + c, row0, false, false);
                }
            } else if (t.kind == kGradHidden) {
                const bool any = t.k1 > t.k0;  // else the accumulator was never written
                for (int c = first; c < first + kResultColumns; c += 32) {
                    float z[32];
                    tmem_load32(acc + c, z);
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) w[j] = any ? __float_as_uint(z[j] * factor) : 0u;
                    put_rows(w, buffer, lane, &p.gh_out, t.n0 + c, (int)(t.split * p.rows) + row0, !p.first_piece,
                             t.n0 + c >= p.dim);
                }
            } else {
                const bool any = t.k1 > t.k0;  // no token counts: the accumulator was never written
                auto scaled = [&](int col, uint32_t *w) __attribute__((always_inline)) {
                    float z[32];
                    tmem_load32(acc + col, z);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[j] = any ? pack_lp<BF16>(z[2 * j] * factor, z[2 * j + 1] * factor) : 0u;
                };
                for (int c = first; c < first + kResultColumns; c += 64) {
                    uint32_t w[32];
                    scaled(c, w);
                    scaled(c + 32, w + 16);
                    put_rows(w, buffer, lane, &p.gw_out, t.n0 + c, (int)p.piece0 + row0, false,
                             t.n0 + c >= p.dim || p.piece0 + row0 >= p.vocab);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_cluster(in_cta(smem_addr(&sh.acc_empty[buf]), 0));
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1;
        }
        if (lane == 0) store_wait_all();
    }
    __syncwarp();
    __syncthreads();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    // After a wait that gave up (the flag is the pair's, so both CTAs come here or neither),
    // copies may still be on their way to either CTA's shared memory.  The other warps'
    // stores have been waited for, and both loaders have stopped.
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

// ---------------------------------------------------------- the smaller kernels

// Tokens of a block, which has a warp for each; a lane for each way.  (32 tokens leave the
// targets' rows to few SMs: 163 x 328 x 373 10.8 us for both kernels, with 8 10.1.)
constexpr int kJoinTokens = 8, kJoinWays = 32;

// A logit by a warp, in float rounded to nearest, the same bits as loss_few's: each lane's
// vectors in order, then lanes 16, 8, ... apart.  also(v, x): vector v of h, on its way.
template <bool BF16, typename Also>
__device__ __forceinline__ float warp_logit(const uint4 *h, const uint4 *w, int vecs, int lane, Also also) {
    float z = 0.0f;
#pragma unroll 4
    for (int v = lane; v < vecs; v += 32) {
        const uint4 x = h[v], m = w[v];
        also(v, x);
        float a[8], b[8];
        widen8<BF16>(x, a);
        widen8<BF16>(m, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) z = __fmaf_rn(a[k], b[k], z);
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return z;
}

// Where the hidden states and the matrix are, their rows in vectors.
struct Operands {
    const uint4 *hidden, *weight;
    long long stride, weight_stride;
    int vecs;
};

// lse and loss: 32 ways along the vocabulary for each token, joined in order.
// The target's logit is a float sum rounded to nearest, in lse as in the slope (take_rows):
// of a target of probability p the loss and the slope are what is left of z - lse, 1 - p,
// and z off by 1e-5 in one of the two made gradients 1 % off at p = 0.999 and 3 to 17 % at
// 0.9999.  With the tensor core's logit d below it, lse is higher by log(1 + p (e^d - 1)),
// and the loss lower by d less that.  (hidden NULL: the logits are such sums already.)
template <bool BF16>
__global__ void __launch_bounds__(kJoinTokens *kJoinWays)
loss_join(const __grid_constant__ Operands in, const float2 *__restrict__ parts, const float *__restrict__ picked, int tiles,
          const int64_t *__restrict__ target, long long ignore, long long tokens, long long vocab, float *loss, float *lse, int *status) {
    __shared__ float2 way[kJoinWays][kJoinTokens + 1];
    const int x = threadIdx.x % kJoinTokens, w = threadIdx.x / kJoinTokens;
    const long long t = (long long)blockIdx.x * kJoinTokens + x;
    // the token that this warp ends with
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long mine = (long long)blockIdx.x * kJoinTokens + warp;
    const long long y = mine < tokens ? target[mine] : ignore;
    const bool counts = y >= 0 && y < vocab && y != ignore;
    // The target and both rows are read before the wait for the statistics, while their
    // kernel still runs: it only reads them too, and no block of this one starts before every
    // block of that one has waited for all that came before.  (After the wait, 256 x 4096 x
    // 32000 took 64 us for both kernels; so 57, as without these rows.)
    float z_float = 0.0f;
    if (counts && in.hidden)
        z_float = warp_logit<BF16>(in.hidden + mine * in.stride, in.weight + y * in.weight_stride, in.vecs, lane, [](int, uint4) {});
    pdl_enter();
    const float z_y = counts ? picked[mine] : 0.0f;
    const float low = counts && in.hidden ? z_float - z_y : 0.0f;  // what the picked logit is too low by
    float2 acc = make_float2(-INFINITY, 0.0f);
    if (t < tokens) {
        for (int i = w; i < tiles; i += 8 * kJoinWays) {
            float2 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = i + j * kJoinWays < tiles ? parts[(long long)(i + j * kJoinWays) * tokens + t] : make_float2(-INFINITY, 0.0f);
            float top = acc.x;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, v[j].x);
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = acc.y * exp2_approx((acc.x - base) * kLog2e);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[j].y * exp2_approx((v[j].x - base) * kLog2e);
            acc = make_float2(top, sum);
        }
    }
    way[w][x] = acc;
    __syncthreads();
    // then a warp for each token, a lane for each way
    acc = way[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        acc = join_parts(acc, make_float2(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o)));
    if (lane != 0 || mine >= tokens) return;
    const float log_sum = log2f(acc.y) * kLn2;
    float more = 0.0f;
    if (counts) {
        const float off = (acc.x - z_y) + log_sum;  // -log p
        // (logits of a million and beyond are off by more, and nothing is left of any difference)
        const bool small = fabsf(low) <= 1.0f && isfinite(off);
        if (small) more = log1pf(expf(-off) * expm1f(low));
        loss[mine] = small ? off + (more - low) : off;
    } else if (y == ignore) {
        loss[mine] = 0.0f;
    } else {
        loss[mine] = __int_as_float(0x7fffffff);
        atomicOr(status, ZERO_LOSS_BAD_TARGET);
    }
    lse[mine] = acc.x + (log_sum + more);
}

// Statistics of a few tokens, without the tensor cores: a tile of theirs has 256
// tokens, and what takes the time is the matrix, read once.  The hidden states
// lie in shared memory as floats; a warp takes four or eight rows of the matrix
// at a time, its lanes the same vectors of each, and the sums of all rows and tokens
// are exchanged together: with N sums each step hands half of them over, so N - 1
// exchanges and not 5 N, and leaves every lane one sum to keep statistics of.
// One token, 768 x 50257 in fp16, the matrix in L2: 10.5 us, 24 us in a tile; four
// tokens 16 and 24 us; eight would be no faster than in a tile.
constexpr int kFewTokens = 4;
constexpr int kFewThreads = 256;
constexpr int kFewBlocks = 304;              // two on each SM
constexpr int kFewSmem = 96 * 1024;          // floats of the hidden states, at most

template <bool BF16, int T>
__global__ void __launch_bounds__(kFewThreads, 2)
loss_few(const uint4 *__restrict__ hidden, long long hidden_stride, const uint4 *__restrict__ weight, long long weight_stride,
         const int64_t *__restrict__ target, int tokens, long long vocab, int vecs, float2 *parts, float *picked) {
    pdl_enter();
    constexpr int R = T == 1 ? 8 : 4, N = R * T;  // rows at a time, sums
    extern __shared__ float4 h[];  // [token][half of a vector][vector]
    __shared__ float2 warp_part[kFewThreads / 32][T];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < T * vecs; i += kFewThreads) {
        const int t = i / vecs, v = i - t * vecs;
        float f[8] = {};
        if (t < tokens) widen8<BF16>(hidden[t * hidden_stride + v], f);
        h[2 * t * vecs + v] = make_float4(f[0], f[1], f[2], f[3]);
        h[(2 * t + 1) * vecs + v] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __syncthreads();
    constexpr int kBits = N == 8 ? 3 : 4;
    const int mine = lane >> (5 - kBits);  // the sum this lane keeps: row mine / T, token mine % T
    const int token = mine % T;
    const long long y = token < tokens ? target[token] : -1;
    float2 stat = make_float2(-INFINITY, 0.0f);
    const long long groups = (vocab + R - 1) / R;
    for (long long g = (long long)blockIdx.x * (kFewThreads / 32) + warp; g < groups;
         g += (long long)gridDim.x * (kFewThreads / 32)) {
        float acc[N];
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.0f;
        const uint4 *row[R];
#pragma unroll
        for (int r = 0; r < R; ++r) row[r] = weight + (g * R + r < vocab ? g * R + r : vocab - 1) * weight_stride;
        for (int v = lane; v < vecs; v += 32) {
            uint4 q[R];
#pragma unroll
            for (int r = 0; r < R; ++r) q[r] = __ldg(row[r] + v);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float4 a = h[2 * t * vecs + v], b = h[(2 * t + 1) * vecs + v];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float w[8];
                    widen8<BF16>(q[r], w);
                    float &s = acc[r * T + t];
                    s = __fmaf_rn(w[0], a.x, s);
                    s = __fmaf_rn(w[1], a.y, s);
                    s = __fmaf_rn(w[2], a.z, s);
                    s = __fmaf_rn(w[3], a.w, s);
                    s = __fmaf_rn(w[4], b.x, s);
                    s = __fmaf_rn(w[5], b.y, s);
                    s = __fmaf_rn(w[6], b.z, s);
                    s = __fmaf_rn(w[7], b.w, s);
                }
            }
        }
        int off = 16;
#pragma unroll
        for (int half = N / 2; half >= 1; half /= 2, off >>= 1) {
            const bool upper = lane & off;
#pragma unroll
            for (int n = 0; n < half; ++n) {
                const float give = upper ? acc[n] : acc[n + half], keep = upper ? acc[n + half] : acc[n];
                acc[n] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
#pragma unroll
        for (; off >= 1; off >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
        const long long v = g * R + mine / T;
        if (v < vocab) {
            if (v == y) picked[token] = acc[0];
            stat = join_parts(stat, make_float2(acc[0], 1.0f));
        }
    }
    // lanes that keep the same sum hold the same statistics; rows join, then warps
    for (int off = 32 / R; off < 32; off <<= 1) {
        const float2 other = make_float2(__shfl_xor_sync(0xffffffffu, stat.x, off), __shfl_xor_sync(0xffffffffu, stat.y, off));
        stat = join_parts(stat, other);
    }
    if (lane < 32 / R && (lane & ((1 << (5 - kBits)) - 1)) == 0) warp_part[warp][token] = stat;
    __syncthreads();
    if (threadIdx.x < tokens) {
        stat = warp_part[0][threadIdx.x];
        for (int w = 1; w < kFewThreads / 32; ++w) stat = join_parts(stat, warp_part[w][threadIdx.x]);
        parts[(long long)blockIdx.x * tokens + threadIdx.x] = stat;
    }
}

constexpr int kCopyThreads = 128;

// Hidden states of the counted tokens by place, and zeros up to whole blocks of K: the
// products' maps of them have this many rows.
struct RowSource {
    const uint4 *hidden, *weight;
    long long stride, weight_stride;
    const int64_t *target;
    const float *lse;
    long long tokens;
    int vecs;
};

__host__ __device__ constexpr long long compact_rows(long long tokens) { return tokens < kTileK ? kTileK : tokens; }

// A warp takes a place: it copies the hidden state (out, not NULL) and computes the
// target's slope from the target's logit in float.  The tensor core's logit is low by
// up to 2^-23 of itself for every 16 products, and exp(z - lse) - 1 of a likely target
// has nothing left beside that: gradients of targets of probability 0.999 were 3 %
// off with 40 tokens, 4096 wide, and 12 % with five.  (1 % of the time of both passes:
// 1023 x 768 240 -> 243 us, 2048 x 1600 934 -> 942, 4096 x 4096 4.32 -> 4.36 ms.)
template <bool BF16>
__device__ __forceinline__ void take_rows(const RowSource &r, const int *index, long long count, long long places, uint4 *out,
                                          float *at_target) {
    const int lane = threadIdx.x & 31, warps = (int)blockDim.x / 32;
    const long long whole = (places + kTileK - 1) / kTileK * kTileK, limit = compact_rows(r.tokens);
    const long long end = !out ? count : whole < limit ? whole : limit;
    for (long long i = (long long)(threadIdx.x / 32) * gridDim.x + blockIdx.x; i < end; i += (long long)gridDim.x * warps) {
        const long long n = places != count && i >= kRest ? i - kRest : i;
        if (n >= count) {
            for (int v = lane; v < r.vecs; v += 32) out[i * r.vecs + v] = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        const long long t = index[n], y = r.target[t];
        const uint4 *h = r.hidden + t * r.stride, *w = r.weight + y * r.weight_stride;
        const float z = warp_logit<BF16>(h, w, r.vecs, lane, [&](int v, uint4 x) {
            if (out) out[i * r.vecs + v] = x;
        });
        if (lane == 0) at_target[i] = expm1f(z - r.lse[t]);
    }
}

// the same after loss_place
template <bool BF16>
__global__ void __launch_bounds__(kCopyThreads)
loss_rows(const __grid_constant__ RowSource r, const LossRecord *record, const int *__restrict__ index, uint4 *out, float *at_target) {
    pdl_enter();
    const long long count = record->count, places = record->places;
    take_rows<BF16>(r, index, count, places, count < r.tokens || places != count ? out : nullptr, at_target);
}

constexpr int kPlaceThreads = 1024;

constexpr int kKept = 4;                            // tokens a thread keeps in registers
constexpr int kFewPlaces = kKept * kPlaceThreads;  // tokens up to which blocks copy rows too

// The counted tokens in order (index: token of a place; place: place of a token
// or -1), what the slopes need of each, and the largest finite |grad_loss|.
// A thread takes consecutive tokens.  One block; or, up to kFewPlaces tokens, as many
// as then take the rows of the counted ones (out, not NULL; see loss_rows): each finds
// every place for itself, which saves a launch, and the first writes them down.
template <bool BF16>
__global__ void __launch_bounds__(kPlaceThreads)
loss_place(const __grid_constant__ RowSource r, long long ignore, long long rows, long long vocab, const float *__restrict__ grad_loss,
           LossRecord *record, int *index, int *place, float *lse2, float *ratio, int *place_target, int *status, uint4 *out,
           float *at_target) {
    constexpr float top_operand = operand_top(BF16);
    const int64_t *__restrict__ target = r.target;
    const float *__restrict__ lse = r.lse;
    const long long tokens = r.tokens;
    pdl_enter();
    __shared__ int sums[kPlaceThreads / 32];
    __shared__ float tops[kPlaceThreads / 32];
    __shared__ int listed[kFewPlaces];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long each = (tokens + kPlaceThreads - 1) / kPlaceThreads;
    const long long t0 = threadIdx.x * each < tokens ? threadIdx.x * each : tokens;
    const long long t1 = t0 + each < tokens ? t0 + each : tokens;
    const bool writes = blockIdx.x == 0;
    long long kept_y[kKept];
    float kept_g[kKept], kept_lse[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const bool is = t0 + k < t1;
        kept_y[k] = is ? target[t0 + k] : ignore;
        kept_g[k] = is ? grad_loss[t0 + k] : 0.0f;
        kept_lse[k] = is ? lse[t0 + k] : 0.0f;
    }
    int mine = 0;
    float top = 0.0f;
    bool bad = false;
    const auto counts = [&](long long y) { return y != ignore && y >= 0 && y < vocab; };
    const auto look = [&](long long y, float grad) {
        const float g = fabsf(grad);
        bad |= y != ignore && !counts(y);
        mine += counts(y);
        if (counts(y) && g <= 3.402823466e38f) top = fmaxf(top, g);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) look(kept_y[k], kept_g[k]);
    for (long long t = t0 + kKept; t < t1; ++t) look(target[t], grad_loss[t]);
    if (bad) atomicOr(status, ZERO_LOSS_BAD_TARGET);
    int before = mine;  // inclusive sum over the warp's lanes, then over the warps
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 31) sums[warp] = before;
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kPlaceThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
        top = fmaxf(top, tops[w]);
    }
    const int places = all > 0 && all <= kRest ? kTileK : all;
    int at = before - mine;
    const auto put = [&](long long t, long long y, float grad, float l) {
        if (writes) place[t] = counts(y) ? at : -1;
        if (!counts(y)) return;
        if (out) listed[at] = (int)t;
        if (writes) {
            index[at] = (int)t;
            for (int i = at; i < places; i += places == all ? places : kRest) {
                lse2[i] = l * kLog2e;
                ratio[i] = top > 0.0f ? grad / top * top_operand : grad;
                place_target[i] = (int)y;
            }
        }
        ++at;
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (t0 + k < t1) put(t0 + k, kept_y[k], kept_g[k], kept_lse[k]);
    for (long long t = t0 + kKept; t < t1; ++t) put(t, target[t], grad_loss[t], lse[t]);
    if (writes) {
        for (long long i = all + threadIdx.x; i < rows; i += kPlaceThreads) {  // rows that fill the last tile
            if (places != all && i >= kRest && i < kRest + all) continue;
            lse2[i] = ratio[i] = 0.0f;
            place_target[i] = -1;
        }
        if (threadIdx.x == 0) {
            record->count = all;
            record->places = places;
            record->factor = top / top_operand;
        }
    }
    if (!out) return;
    __syncthreads();
    take_rows<BF16>(r, listed, all, places, all < tokens || places != all ? out : nullptr, at_target);
}

// grad_hidden of a token: the partial sums of its place, or of both, in order, rounded once
template <bool BF16>
__global__ void __launch_bounds__(kCopyThreads)
loss_finish(const float4 *__restrict__ sums, const int *__restrict__ place, const LossRecord *record, long long tokens,
            long long rows, int splits, int vecs, uint4 *out, long long stride) {
    pdl_enter();
    const int each = record->places != record->count ? 2 : 1;
    for (long long t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int i = place[t];
        for (int v = threadIdx.x; v < vecs; v += kCopyThreads) {
            float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
            for (int n = 0; n < splits * each && i >= 0; ++n) {
                const int s = n < splits ? n : n - splits;
                const float4 *src = sums + ((s * rows + (n < splits ? i : i + kRest)) * vecs + v) * 2;
                const float4 a = src[0], b = src[1];
                lo.x += a.x; lo.y += a.y; lo.z += a.z; lo.w += a.w;
                hi.x += b.x; hi.y += b.y; hi.z += b.z; hi.w += b.w;
            }
            out[t * stride + v] = make_uint4(pack_lp<BF16>(lo.x, lo.y), pack_lp<BF16>(lo.z, lo.w), pack_lp<BF16>(hi.x, hi.y),
                                             pack_lp<BF16>(hi.z, hi.w));
        }
    }
}

// one exchange, so that no bit is lost that another stream's call sets meanwhile
__global__ void loss_take_status(int *status, int *bits) {
    pdl_enter();
    *bits = atomicExch(status, 0);
}

// ------------------------------------------------------------------------ host

// Pairs of CTAs that run at once on the current device, their shared memory having been
// allowed: or an error below zero.
template <bool BF16, bool STATS>
int pairs_at_once() {
    static PerDevice kept;
    return kept.get([] {
        const int set = done_or_error(
            cudaFuncSetAttribute(loss_products<BF16, STATS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
        if (set < 0) return set;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kProductThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const int asked = done_or_error(cudaOccupancyMaxActiveClusters(&clusters, loss_products<BF16, STATS>, &cfg));
        if (asked < 0) return asked;
        return clusters > 0 ? clusters : -(int)cudaErrorInvalidConfiguration;
    });
}

std::atomic<long long> g_wait_cycles{4000000000ll};  // about two seconds

template <bool BF16, bool STATS>
cudaError_t launch_products(const ProductParams &p, int64_t tiles, cudaStream_t stream) {
    const int pairs = pairs_at_once<BF16, STATS>();
    if (pairs < 0) return (cudaError_t)-pairs;
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    const int64_t use = std::max<int64_t>(1, std::min<int64_t>(pairs, tiles));
    return launch_pdl(loss_products<BF16, STATS>, dim3((unsigned)(2 * use)), dim3(kProductThreads), kSmemBytes, stream, p);
}

// whether the few tokens' hidden states fit into shared memory twice on an SM
bool few(int64_t tokens, int dim) {
    const int64_t t = tokens <= 2 ? tokens : 4;
    return tokens <= kFewTokens && t * dim * 4 <= kFewSmem;
}

template <bool BF16, int T>
cudaError_t launch_few(const LossArgs &a, float2 *parts, float *picked, cudaStream_t stream) {
    static PerDevice allowed;
    const int set = allowed.get(
        [] { return done_or_error(cudaFuncSetAttribute(loss_few<BF16, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem)); });
    if (set < 0) return (cudaError_t)-set;
    return launch_pdl(loss_few<BF16, T>, dim3(kFewBlocks), dim3(kFewThreads), size_t(T) * a.dim * 4, stream,
                      static_cast<const uint4 *>(a.hidden), (long long)(a.hidden_stride / 8),
                      static_cast<const uint4 *>(a.weight), (long long)(a.weight_stride / 8), a.target, (int)a.tokens,
                      (long long)a.vocab, a.dim / 8, parts, picked);
}

// parts of the vocabulary that the statistics come in
int64_t parts_of(int64_t tokens, int64_t vocab, int dim) {
    return few(tokens, dim) ? kFewBlocks : up(vocab, kTileN) / kTileN;
}

template <bool BF16>
cudaError_t forward_impl(const LossArgs &a, cudaStream_t stream) {
    const int64_t n = parts_of(a.tokens, a.vocab, a.dim);
    float2 *parts = static_cast<float2 *>(a.workspace);
    float *picked = reinterpret_cast<float *>(parts + n * a.tokens);
    cudaError_t e;
    if (few(a.tokens, a.dim)) {
        e = a.tokens == 1   ? launch_few<BF16, 1>(a, parts, picked, stream)
            : a.tokens == 2 ? launch_few<BF16, 2>(a, parts, picked, stream)
                            : launch_few<BF16, 4>(a, parts, picked, stream);
    } else {
        ProductParams p = {};
        if (!encoder() || !make_map(&p.h_k, a.hidden, a.tokens, a.dim, a.hidden_stride, a.lp, false, kHalf) ||
            !make_map(&p.w_k, a.weight, a.vocab, a.dim, a.weight_stride, a.lp, false, kHalf))
            return cudaErrorNotSupported;
        p.tokens = a.tokens;
        p.vocab = p.piece = a.vocab;
        p.dim = a.dim;
        p.splits = 1;
        p.target = a.target;
        p.parts = parts;
        p.picked = picked;
        p.status = a.status;
        p.wait_cycles = g_wait_cycles.load();
        const int64_t tiles = up(a.tokens, kTileM) / kTileM * (up(a.vocab, kTileN) / kTileN);
        p.chunk = tiles <= pairs_at_once<BF16, true>() ? kShortChunk : kChunk;
        e = launch_products<BF16, true>(p, tiles, stream);
    }
    if (e != cudaSuccess) return e;
    Operands in;
    in.hidden = few(a.tokens, a.dim) ? nullptr : static_cast<const uint4 *>(a.hidden);
    in.weight = static_cast<const uint4 *>(a.weight);
    in.stride = a.hidden_stride / 8;
    in.weight_stride = a.weight_stride / 8;
    in.vecs = a.dim / 8;
    return launch_pdl(loss_join<BF16>, dim3((unsigned)((a.tokens + kJoinTokens - 1) / kJoinTokens)),
                      dim3(kJoinTokens * kJoinWays), 0, stream, in, (const float2 *)parts, (const float *)picked, (int)n,
                      a.target, (long long)a.ignore, (long long)a.tokens, (long long)a.vocab, a.loss, a.lse, a.status);
}

template <bool BF16>
cudaError_t backward_impl(const LossArgs &a, cudaStream_t stream) {
    const BackwardLayout l = backward_layout(a.tokens, a.vocab, a.dim);
    char *ws = static_cast<char *>(a.workspace);
    LossRecord *record = reinterpret_cast<LossRecord *>(ws);
    int *index = reinterpret_cast<int *>(ws + l.index), *place = reinterpret_cast<int *>(ws + l.place);
    float *lse2 = reinterpret_cast<float *>(ws + l.lse2), *ratio = reinterpret_cast<float *>(ws + l.ratio);
    int *place_target = reinterpret_cast<int *>(ws + l.target);
    float *at_target = reinterpret_cast<float *>(ws + l.at_target);
    void *compact = ws + l.hidden, *slopes = ws + l.slopes;
    float *sums = reinterpret_cast<float *>(ws + l.sums);
    ProductParams p = {};
    if (!encoder() || !make_map(&p.h_k, a.hidden, a.tokens, a.dim, a.hidden_stride, a.lp, false, kHalf) ||
        !make_map(&p.hc_k, compact, compact_rows(a.tokens), a.dim, a.dim, a.lp, false, kHalf) ||
        !make_map(&p.w_k, a.weight, a.vocab, a.dim, a.weight_stride, a.lp, false, kHalf) ||
        !make_map(&p.w_mn, a.weight, a.vocab, a.dim, a.weight_stride, a.lp, false, kTileK) ||
        !make_map(&p.h_mn, a.hidden, a.tokens, a.dim, a.hidden_stride, a.lp, false, kTileK) ||
        !make_map(&p.hc_mn, compact, compact_rows(a.tokens), a.dim, a.dim, a.lp, false, kTileK) ||
        !make_map(&p.q_k, slopes, l.rows, l.piece, l.piece, a.lp, false, kHalf) ||
        !make_map(&p.q_mn, slopes, l.rows, l.piece, l.piece, a.lp, false, kTileK) ||
        !make_map(&p.q_out, slopes, l.rows, l.piece, l.piece, a.lp, false, 32) ||
        !make_map(&p.gh_out, sums, l.splits * l.rows, a.dim, a.dim, a.lp, true, 32) ||
        !make_map(&p.gw_out, a.grad_weight, a.vocab, a.dim, a.grad_weight_stride, a.lp, false, 32))
        return cudaErrorNotSupported;
    p.tokens = a.tokens;
    p.vocab = a.vocab;
    p.dim = a.dim;
    p.piece = l.piece;
    p.rows = l.rows;
    p.splits = l.splits;
    p.record = record;
    p.lse2 = lse2;
    p.ratio = ratio;
    p.at_target = at_target;
    p.place_target = place_target;
    p.status = a.status;
    p.wait_cycles = g_wait_cycles.load();
    const bool joint = a.tokens <= kFewPlaces;
    const int copies = (int)std::min<int64_t>(a.tokens, 8 * sm_count());
    RowSource r;
    r.hidden = static_cast<const uint4 *>(a.hidden);
    r.weight = static_cast<const uint4 *>(a.weight);
    r.stride = a.hidden_stride / 8;
    r.weight_stride = a.weight_stride / 8;
    r.target = a.target;
    r.lse = a.lse;
    r.tokens = a.tokens;
    r.vecs = a.dim / 8;
    // a warp for each place, of a block of K at least
    const int64_t blocks = joint ? std::min<int64_t>(std::max<int64_t>(a.tokens, kTileK), sm_count()) : 1;
    cudaError_t e = launch_pdl(loss_place<BF16>, dim3((unsigned)blocks), dim3(kPlaceThreads), 0, stream, r, (long long)a.ignore,
                               (long long)l.rows, (long long)a.vocab, (const float *)a.grad_loss, record, index, place, lse2, ratio,
                               place_target, a.status, joint ? static_cast<uint4 *>(compact) : nullptr, at_target);
    if (e == cudaSuccess && !joint)
        e = launch_pdl(loss_rows<BF16>, dim3((unsigned)copies), dim3(kCopyThreads), 0, stream, r, (const LossRecord *)record,
                       (const int *)index, static_cast<uint4 *>(compact), at_target);
    const int64_t row_tiles = l.rows / kTileM, dim_tiles = up(a.dim, kTileN) / kTileN, piece_tiles = l.piece / kTileN;
    for (int i = 0; i < l.pieces && e == cudaSuccess; ++i) {
        p.piece0 = i * l.piece;
        p.first_piece = i == 0;
        p.gradients = 0;
        e = launch_products<BF16, false>(p, row_tiles * piece_tiles, stream);
        p.gradients = 1;
        if (e == cudaSuccess) e = launch_products<BF16, false>(p, row_tiles * dim_tiles * l.splits + piece_tiles * dim_tiles, stream);
    }
    if (e == cudaSuccess)
        e = launch_pdl(loss_finish<BF16>, dim3((unsigned)copies), dim3(kCopyThreads), 0, stream, reinterpret_cast<const float4 *>(sums),
                       (const int *)place, (const LossRecord *)record, (long long)a.tokens, (long long)l.rows, l.splits, a.dim / 8,
                       static_cast<uint4 *>(a.grad_hidden), (long long)(a.grad_hidden_stride / 8));
    return e;
}

}  // namespace

void set_loss_wait(int64_t cycles) { g_wait_cycles.store(cycles); }

int64_t loss_wait() { return g_wait_cycles.load(); }

cudaError_t launch_take_status(int32_t *status, int32_t *bits, cudaStream_t stream) {
    return launch_pdl(loss_take_status, dim3(1), dim3(1), 0, stream, status, bits);
}

int64_t loss_forward_bytes(int64_t tokens, int64_t vocab, int dim) {
    return parts_of(tokens, vocab, dim) * tokens * 8 + up(tokens * 4, 16);
}

cudaError_t launch_loss_forward(const LossArgs &a, cudaStream_t stream) {
    return a.lp ? forward_impl<true>(a, stream) : forward_impl<false>(a, stream);
}

int64_t loss_backward_bytes(int64_t tokens, int64_t vocab, int dim) { return backward_layout(tokens, vocab, dim).bytes; }

cudaError_t launch_loss_backward(const LossArgs &a, cudaStream_t stream) {
    if (a.tokens == 0)  // no token: a zero grad_weight
        return cudaMemset2DAsync(a.grad_weight, size_t(a.grad_weight_stride) * 2, 0, size_t(a.dim) * 2, size_t(a.vocab), stream);
    return a.lp ? backward_impl<true>(a, stream) : backward_impl<false>(a, stream);
}

}  // namespace zk
