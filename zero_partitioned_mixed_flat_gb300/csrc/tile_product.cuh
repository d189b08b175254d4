// tile_product.cuh -- what the kernels of matrix products have in common (loss.cu,
// gated.cu): pairs of CTAs, each pair one 256 x 256 tile, tcgen05.mma on 256 x 256 x 16
// with operands that TMA places in shared memory and sums that stay in tensor memory; the
// tiles' order; bounded waits; and the maps of the operands (host).
#pragma once

#include "loss_drain.h"
#include "zero.h"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace zk {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int kTileM = 256, kTileN = 256;  // outputs of a pair of CTAs
constexpr int kHalf = 128;                 // rows of A, and of B, that each CTA loads
constexpr int kTileK = 64;                 // 128 bytes: one swizzle row
constexpr int kOperandBytes = kHalf * kTileK * 2;
constexpr int kBlockBytes = 2 * kOperandBytes;  // both operands of a block of K
// A stage of shared memory holds two blocks of K, so that the thread that feeds
// the tensor core waits and commits half as often.  (Six stages of one: 8184 x 1600
// forward 3 % slower, 4096 x 4096 with gradients 2.5 %.)
constexpr int kStageBlocks = 2, kStages = 3;
constexpr int kStageBytes = kStageBlocks * kBlockBytes;
constexpr int kBoxBytes = 64 * kTileK * 2;  // a 64 x 64 box of an operand whose rows run along K
constexpr int kStoreBytes = 32 * 128;       // 32 rows of 128 bytes: one warp's store
// Warps that take a tile's results: two on each quarter of its rows, each half of
// the columns.  (Sixteen for the statistics: 8184 x 1600 forward 2 % slower: they take
// issue slots from the thread that feeds the tensor core.)
constexpr int kResultWarps = 8, kResultColumns = kTileN / 2;
constexpr int kProductThreads = 64 + 32 * kResultWarps;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kResultWarps * kStoreBytes;
constexpr int kTmemColumns = 512;  // two accumulators of 256 columns

constexpr int kPairs = 76;  // of SMs

int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// ------------------------------------------------------------- PTX primitives

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// the same without waiting for a moment where it is not yet
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// the address of this CTA's `addr` in CTA `rank` of the pair
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// a store to either CTA's shared memory
__device__ __forceinline__ void store_in_cta(const volatile void *p, uint32_t rank, uint32_t value) {
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(smem_addr(const_cast<const void *>(p)), rank)), "r"(value)
                 : "memory");
}

// bytes counted on `bar` as if a copy had landed
__device__ __forceinline__ void bar_count(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// a box of `map` at (x, y) to this CTA's shared memory; the bytes count on `bar`,
// which may be the other CTA's
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// a map, into the cache that copies read it from
__device__ __forceinline__ void ask_for(const CUtensorMap *map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }

__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void tma_add(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle.  Rows of 128 bytes, eight
// to a 1024-byte group (the stride offset).  K-major: a row holds 64 values of
// K.  MN-major: a row holds 64 values of M or N at one K, and the next 64 of M
// or N lie a whole box further (the leading offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
    uint64_t d = (addr & 0x3ffffu) >> 4;
    d |= (uint64_t)(mn ? kBoxBytes >> 4 : 1) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// arrive on `bar` of both CTAs once every product issued so far is done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// the same on a barrier of this CTA only
__device__ __forceinline__ void mma_commit_here(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive columns of this lane's accumulator row
__device__ __forceinline__ void tmem_load32(uint32_t addr, float v[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, float v[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// two floats at once, each rounded to nearest
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return r;
}
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

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_lp(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// ------------------------------------------------------------------- tiles

// A tile's product.
struct Tile {
    int kind;
    int m0, n0;   // its first row and column
    int width;    // columns of the product: fewer in a last tile that few columns need
    int k0, k1;   // blocks of K
    int split;    // which of the partial sums of grad_hidden
    int n;        // its number along the columns
};

// Division by a number that stays: the product with 2^32 / d rounded up gives the
// quotient or one more.  (A plain division took the thread that feeds the tensor
// core long enough to leave it idle at every tile.)
struct Divisor {
    uint32_t d, inverse;

    __device__ __forceinline__ void set(uint32_t by) {
        d = by ? by : 1u;
        inverse = 0xffffffffu / d + 1u;
    }
    __device__ __forceinline__ uint32_t into(uint32_t x) const {
        const uint32_t q = d == 1u ? x : __umulhi(x, inverse);
        return q * d > x ? q - 1u : q;
    }
};

// A grid of tiles.
struct Tiles {
    int m, n, columns, k_blocks, splits;
    Divisor per_split, per_group, last_group;
    static constexpr int kGroup = 8;

    __device__ __forceinline__ void set(int m_, int n_, int columns_, int k_blocks_, int splits_) {
        m = m_;
        n = n_;
        columns = columns_;
        k_blocks = k_blocks_;
        splits = splits_;
        per_split.set(m * n);
        per_group.set(kGroup * n);
        last_group.set(m % kGroup);
    }
    __device__ __forceinline__ int size() const { return m * n * splits; }

    // Consecutive tiles take 8 tiles of M for one of N before the next of N, so the
    // pairs that run together read few different rows of either operand from L2.
    __device__ __forceinline__ Tile at(uint32_t i, int kind) const {
        Tile t;
        t.kind = kind;
        t.split = splits == 1 ? 0 : (int)per_split.into(i);
        const uint32_t r = i - t.split * per_split.d;
        const uint32_t g = per_group.into(r), q = r - g * per_group.d;
        const bool whole = (int)(g + 1) * kGroup <= m;
        t.n = (int)(whole ? q / kGroup : last_group.into(q));
        t.n0 = t.n * kTileN;
        t.m0 = (int)(g * kGroup + (q - t.n * (whole ? kGroup : last_group.d))) * kTileM;
        const int left = (columns - t.n0 + 31) / 32 * 32;
        t.width = left < kTileN ? left : kTileN;
        t.k0 = splits == 1 ? 0 : k_blocks * t.split / splits;
        t.k1 = splits == 1 ? k_blocks : k_blocks * (t.split + 1) / splits;
        return t;
    }
};

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int dead;  // a wait of the pair gave up
    // what the first CTA has to know to wait for the pair's copies: see loss_drain.h
    int placed[2], consumed;
    uint32_t bytes[2][kStages];
};

// The longest that a pair which gives up waits for each of its copies and products in
// flight, in cycles: they end by themselves, in microseconds.
constexpr long long kDrainCycles = 4000000000ll;

// the pair stops, and the status says so
__device__ __noinline__ void give_up(volatile int *dead, int *status) {
    store_in_cta(dead, 0, 1u);
    store_in_cta(dead, 1, 1u);
    atomicOr(status, ZERO_LOSS_TIMEOUT);
}

// A bounded wait: false once `limit` cycles have passed, or another wait of the
// pair has given up.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *dead, long long limit, int *status) {
    const uint32_t b = smem_addr(bar);
    if (bar_try(b, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(b, parity)) {
        if (*dead || clock64() - t0 >= limit) {
            give_up(dead, status);
            return false;
        }
    }
    return true;
}

// the same, for what ends by itself
__device__ __forceinline__ bool wait_out(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!bar_try(smem_addr(bar), parity))
        if (clock64() - t0 >= kDrainCycles) return false;
    return true;
}

// drain_copies' barriers
struct FullBars {
    uint64_t *full;

    __device__ __forceinline__ void expect(int slot, uint32_t bytes) { bar_expect(smem_addr(full + slot), bytes); }
    __device__ __forceinline__ void count(int slot, uint32_t bytes) { bar_count(smem_addr(full + slot), bytes); }
    __device__ __forceinline__ bool wait(int slot, uint32_t parity) { return wait_out(full + slot, parity); }
};

// 32 rows of 128 bytes, one a lane, to a box of `map`: swizzled into the warp's
// buffer once its last store has read it, then one store.  (A second buffer a
// warp would cost operands 32 KB: 1 % slower at 4096 x 4096.)
__device__ __forceinline__ void put_rows(const uint32_t (&w)[32], uint32_t buffer, int lane, const CUtensorMap *map, int x,
                                         int y, bool add, bool skip) {
    if (lane == 0) store_wait_read();
    __syncwarp();
    const uint32_t row = buffer + lane * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((c ^ (lane & 7)) << 4)), "r"(w[4 * c]),
                     "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                     : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        if (!skip) {
            if (add)
                tma_add(map, x, y, buffer);
            else
                tma_store(map, x, y, buffer);
        }
        store_commit();
    }
}

// What the tensor core is told of a tile's blocks: the instruction, the operands'
// descriptors in the first stage, and how far 16 of K further is (32 bytes along
// a row, or 16 rows).  a_mn, b_mn: the operand's rows run along M or N, not along K.
struct Feed {
    uint32_t idesc, a_step, b_step;
    uint64_t a, b;

    __device__ __forceinline__ Feed() {}
    __device__ __forceinline__ Feed(int width, bool a_mn, bool b_mn, uint32_t stage0, bool bf16) {
        idesc = 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u);  // float sums
        idesc |= (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16;
        idesc |= (uint32_t)(width >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
        a_step = (a_mn ? 16 * 128 : 32) >> 4;
        b_step = (b_mn ? 16 * 128 : 32) >> 4;
        a = operand_desc(stage0, a_mn);
        b = operand_desc(stage0 + kOperandBytes, b_mn);
    }
    __device__ __forceinline__ void block(uint32_t acc, uint64_t at_a, uint64_t at_b, uint32_t add) const {
        mma_pair(acc, at_a, at_b, idesc, add);
#pragma unroll
        for (int i = 1; i < kTileK / 16; ++i) mma_pair(acc, at_a + i * a_step, at_b + i * b_step, idesc, 1);
    }
};

// an OR over `threads` threads that meet at barrier `id`
__device__ __forceinline__ bool any_of(int id, int threads, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)mine), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

template <bool BF16>
__device__ __forceinline__ void widen8(uint4 q, float f[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            f[2 * k] = t.x;
            f[2 * k + 1] = t.y;
        }
    }
}

// ------------------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// rows x cols elements (lp, or float) at p, read or written in boxes of 128
// bytes x box_rows with the 128-byte swizzle; what lies outside reads as zero.
bool make_map(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t stride, int lp, bool f32, int box_rows) {
    const int size = f32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(stride * size)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    const CUtensorMapDataType type = f32  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : lp ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const auto encode = [&] {
        return encoder()(m, type, 2, const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // The driver wants a context, which a thread has from its first call of the runtime that needs
    // one: this may be the thread's first.
    int device = 0;
    return cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess && encode();
}

}  // namespace
}  // namespace zk
