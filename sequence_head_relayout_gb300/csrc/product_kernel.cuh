// Device side of the experts' products (include/vf_relayout.h, "Expert
// products"): products of 16-bit rows grouped by expert, on the fifth-generation
// tensor cores.
//
// rows     out[r, n] = sum_m packed[r, m] * weights[e(r), n, m]
// weights  grad_weights[e, n, m] = sum over e's rows r of grad[r, n] * packed[r, m]
//
// Both are D[i, j] = sum_k A[i, k] * B[j, k] for each expert.  A holds output
// features: the weights [n][m], or the gradient's columns.  B holds the expert's
// rows [r][m], or the packed rows' columns.  With the features on the
// instruction's M side (128 rows of a CTA) and the rows on its N side (16 to 256
// of them, chosen tile by tile) an expert with few rows wastes no tensor work
// beyond a multiple of 16 rows, and one that has none reads no weights.
//
// A CTA is a pipeline of warps over its tiles: two warps copy (one for each operand)
// into a ring of stages (64 k of A and of B, 128-byte swizzle), one thread issues the
// products into one of two accumulators in tensor memory, and eight warps round the
// other one and store it.  Two CTAs of a pair share a tile of 256 features: each holds
// its features' half of A and half of B.  The segments are read from the plan on the
// device; every role walks the tiles for itself.
//
// Bound by the tensor cores where experts have some 300 rows and more, else by HBM, from
// which the weights are read once.  Measured on GB300 (bf16, device time after a pause;
// under the power cap long products take a fifth longer, as cuBLAS's do):
//   rows     T = 55,414, K = 2, E = 16, 3,584 to 4,096   1,630 us   1.92 PFLOP/s
//   rows     T = 4,096, K = 8, E = 64, 4,096 to 2,048      339 us   1.56 PFLOP/s
//   rows     T = 64, K = 4, E = 64, 2,048 to 3,584         135 us   7.0 TB/s
//   rows     T = 1, K = 8, E = 128, 4,096 to 2,048          24 us   5.6 TB/s
//   weights  T = 4,096, K = 8, E = 32, 4,096 x 2,048       321 us   1.71 PFLOP/s
//                                    in float32            391 us   1.41 PFLOP/s
//
// No wait is without an end: a role that waits for kWaitNs of the kernel's own time
// (wait.h) gives up, sets the CTA's flag, and what is still to be stored is stored as NaN.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "shift.cuh"
#include "wait.h"

namespace vfp {

constexpr int kBlockK = 64;                    // k of a stage: 128 bytes of 16-bit elements
constexpr int kTileM = 128;                    // features of a CTA's tile
constexpr int kStageA = kTileM * kBlockK * 2;  // bytes
constexpr int kMaxStages = 12;
constexpr int kBoxes = 4;                      // heights of the copies of B, multiples of one
constexpr int kEpilogueWarps = 8;              // two for each quarter of the tile's features
// Staging of an epilogue warp: 32 rows of 64 bytes, or of up to 144.
constexpr int kStagingRows = 2048, kStagingWeights = 4608;
constexpr int kPartBytes = 2 * 32 * kTileM * 4; // SPLIT: 32 columns of each turn's, in float32
constexpr int kThreads = 32 * (4 + kEpilogueWarps);
constexpr uint64_t kDrainNs = 100000000ull;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct ProductArgs {
    // rows form: b_maps[i] has boxes of (i + 1) box rows
    CUtensorMap a_map, b_maps[kBoxes];
    const int32_t *counts, *offsets;
    void *out;                    // rows: [rows][feat]; weights: [E][feat][cols]
    int32_t E, rows;
    int32_t feat, cols, red;      // features; weights: columns; rows: length of the sums
    int32_t feat_tiles, col_tiles;
    int32_t part;                 // most rows (rows form: features) of one accumulation
    int32_t step_experts, step_tiles;    // weights: the grid's tiles, in experts and the rest
    int32_t tile_n;               // most rows (columns) of a tile
    int32_t split;                // CTAs that share the sums of a tile
    int32_t box;                  // rows form: a copy of B has one to kBoxes times as many rows
    int32_t stages, stage_bytes;
    int32_t acc_stride, tmem_cols;
    int32_t a_slabs, b_slabs;     // operands with i contiguous: 64 i to a slab, a CTA's share
                                  // by one copy of so many; 0: a copy for each
    int32_t bf16, gaps, vec;
};

// ---- synchronisation -----------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return uint32_t(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void barrier_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Whether it has, without a wait: a try may hold its thread for some 4 us (every
// product took as much longer when the last block of its last tile was issued behind a
// try for a block that would not come).
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Waits for the phase of the given parity to end; false when it gave up, or another
// role did.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity,
                                             volatile int *failed) {
    for (int i = 0; i < 64; ++i)
        if (barrier_try(bar, parity)) return true;
    const bool done = wait_until([&] { return barrier_try(bar, parity); },
                                 [&] { return *failed != 0; }, [] { return now_ns(); });
    if (!done) *failed = 1;
    return done;
}

// The same by a whole warp, `ready`: the result of an earlier test.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *failed,
                                          bool ready = false) {
    if (!ready) ready = barrier_wait(bar, parity, failed);
    return __all_sync(kAll, int(ready));
}

// True in one lane of the warp, the same one every time.
__device__ __forceinline__ bool elected() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// A value that all lanes hold, known to be uniform by the compiler: copies and
// products take their arguments from uniform registers, and a thread that had to move
// them there one by one issued a block of products in some 400 cycles of the 512 that
// they run (product of 16,384 rows, 3,584 to 4,096 features: 55% of the tensor pipe).
template <class T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(kAll, v, 0); }

__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The address of CTA `to` of the cluster that is `addr` here.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t to) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(to));
    return r;
}

// Arrival at the barrier of CTA `to`.
__device__ __forceinline__ void barrier_arrive_at(uint32_t bar, uint32_t to) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                 ::"r"(cluster_addr(bar, to)) : "memory");
}

__device__ __forceinline__ float cluster_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                 ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- copies --------------------------------------------------------------------

// The barrier of a pair's copies is that of its first CTA.
template <int CTAS>
__device__ __forceinline__ uint32_t first_barrier(uint32_t bar) {
    return CTAS == 1 ? bar : cluster_addr(bar, 0);
}

template <int CTAS>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                        int x, int y) {
    if constexpr (CTAS == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
}

template <int CTAS>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                        int x, int y, int z) {
    if constexpr (CTAS == 1)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}

template <int CTAS>
__device__ __forceinline__ void copy_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                        int x, int y, int z, int w) {
    if constexpr (CTAS == 1)
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
                     ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// ---- tensor cores --------------------------------------------------------------

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (CTAS == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     ::"r"(addr), "r"(cols) : "memory");
}

// Descriptor of an operand in shared memory, 128-byte swizzle.  k contiguous: rows of
// 128 bytes, groups of 8 rows 1,024 bytes apart.  i contiguous: 64 i to a row of 128
// bytes, one row for each k, groups of 8 k 1,024 bytes apart and the next 64 i
// 64 rows on.  The low word holds the address, in units of 16 bytes.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t operand(uint32_t addr) {
    return (uint32_t((kBlockK * 128) >> 4) << 16) | ((addr & 0x3FFFF) >> 4);
}

template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                    bool accumulate) {
    if constexpr (CTAS == 1)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                     ::"r"(d), "r"(a), "r"(b), "r"(instr), "r"(uint32_t(accumulate)),
                       "n"(kDescHigh) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}"
                     ::"r"(d), "r"(a), "r"(b), "r"(instr), "r"(uint32_t(accumulate)),
                       "n"(kDescHigh) : "memory");
}

// The barrier (of both CTAs of a pair) is arrived at when the products issued so
// far are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"(uint16_t(3)) : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of the warp's 32 lanes: lane l's float of column c in v[c].
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(addr) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 16 columns likewise.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// From one step of 16 k to the next, in units of 16 bytes.
template <bool MN> constexpr uint32_t kStep16 = MN ? 16 * 128 / 16 : 2;

// ---- tiles ---------------------------------------------------------------------

// ceil(n / d), for n up to 2^31 - 1
__device__ __forceinline__ int parts(int n, int d) { return n / d + (n % d != 0); }

struct Tile {
    int e, f0;         // expert, first feature
    int row0, valid;   // first row and rows of the tile; weights: of this part of the sum
    int c0;            // weights: first column
    int k0;            // rows form in parts: first feature of this part of the sum
    int n;             // rows or columns of the product, a multiple of 16 CTAS
    int kblocks;
    int gap;           // rows to be written as zeros behind the tile
    bool more;         // a later part of the sum
};

// The CTA's (pair's) tiles, by all lanes of a warp together.  Rows form: the
// experts' tiles in order, an expert's row tiles fastest (they share a tile of
// weights), each expert's rows cut into equal tiles.  A lane holds four experts, a
// warp 128 at a time.
template <int CTAS, bool WEIGHTS, bool PARTS, bool SPLIT>
struct Tiles {
    static constexpr int kStep = 16 * CTAS;
    const ProductArgs &a;
    int lane;
    // rows form
    int64_t t, step;              // this tile, and what is added for the next
    int base = -128;              // first expert of the warp's 128
    int64_t before = 0;           // tiles before it
    int64_t total = 0;            // tiles of the 128
    int64_t first = 0;            // tiles of the 128 before the lane's four experts
    int count[4], begin[4];
    // weights form: the tile as a number within its expert
    int e, in, each;
    int next_offset, next_count;  // of the next tile's expert, loaded a tile ahead
    int slice = 0;                // SPLIT: this CTA's of a.split shares of the sums
    int row0, rest;               // what is left of the expert's rows (sums in parts), or
                                  // of the features
    bool inside = false;

    __device__ __forceinline__ explicit Tiles(const ProductArgs &args)
        : a(args), lane(int(threadIdx.x & 31)) {
        const uint32_t group = SPLIT ? uint32_t(a.split) : CTAS;
        t = blockIdx.x / group;
        step = gridDim.x / group;
        if constexpr (SPLIT) slice = int(cluster_rank());
        if constexpr (WEIGHTS) {
            each = a.feat_tiles * a.col_tiles;
            e = int(t) / each;
            in = int(t) - e * each;
            ahead();
        }
    }

    __device__ __forceinline__ void ahead() {
        const int expert = min(e, a.E - 1);
        next_offset = a.offsets[expert];
        next_count = a.counts[expert];
    }

    // Rows of an expert that exist, whatever the plan says.
    __device__ __forceinline__ void segment(int offset, int n, int &begin_, int &count_) const {
        begin_ = min(max(offset, 0), a.rows);
        count_ = min(max(n, 0), a.rows - begin_);
    }

    __device__ __forceinline__ int64_t tiles_of(int n) const {
        return int64_t(parts(n, a.tile_n)) * a.feat_tiles;
    }

    __device__ __forceinline__ bool next(Tile &o) {
        const bool there = WEIGHTS ? next_weights(o) : next_rows(o);
        o.e = uniform(o.e);
        o.f0 = uniform(o.f0);
        o.c0 = uniform(o.c0);
        o.k0 = uniform(o.k0);
        o.row0 = uniform(o.row0);
        o.valid = uniform(o.valid);
        o.n = uniform(o.n);
        o.kblocks = uniform(o.kblocks);
        return __all_sync(kAll, int(there));
    }

    __device__ __forceinline__ bool next_weights(Tile &o) {
        if (inside) {                                      // the same tile's next part
            o.more = true;
        } else {
            if (e >= a.E) return false;
            o.e = e;
            o.f0 = in % a.feat_tiles * (kTileM * CTAS);
            o.c0 = in / a.feat_tiles * a.tile_n;
            // (each CTA's share of B starts at a whole slab)
            const int multiple = a.b_slabs ? 64 * CTAS : kStep;
            o.n = (min(a.tile_n, a.cols - o.c0) + multiple - 1) / multiple * multiple;
            o.gap = 0;
            o.more = false;
            segment(next_offset, next_count, row0, rest);
            if constexpr (SPLIT) {
                // this CTA's share of the blocks
                const int64_t n = parts(rest, kBlockK);
                const int from = int(n * slice / a.split) * kBlockK;
                const int to = int(min(n * (slice + 1) / a.split * kBlockK, int64_t(rest)));
                row0 += from;
                rest = to - from;
            }
            e += a.step_experts;
            in += a.step_tiles;
            if (in >= each) {
                in -= each;
                ++e;
            }
            ahead();
        }
        o.row0 = row0;
        o.valid = min(rest, a.part);
        o.kblocks = parts(o.valid, kBlockK);
        row0 += o.valid;
        rest -= o.valid;
        inside = rest > 0;
        return true;
    }

    // The next part of a tile's sums; parts are whole blocks.
    __device__ __forceinline__ void next_part(Tile &o, bool first) {
        o.more = !first;
        o.k0 = first ? 0 : o.k0 + a.part;
        rest = first ? a.red : rest - a.part;
        o.kblocks = parts(min(rest, a.part), kBlockK);
        inside = rest > a.part;
    }

    __device__ __forceinline__ bool next_rows(Tile &o) {
        if constexpr (PARTS)
            if (inside) {
                next_part(o, false);
                return true;
            }
        while (t >= before + total) {
            base += 128;
            if (base >= a.E) return false;
            before += total;
            int64_t sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = base + 4 * lane + i;
                count[i] = begin[i] = 0;
                if (e < a.E) segment(a.offsets[e], a.counts[e], begin[i], count[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += tiles_of(count[i]);
            first = sum;
#pragma unroll
            for (int o2 = 1; o2 < 32; o2 <<= 1) {
                const int64_t other = __shfl_up_sync(kAll, first, o2);
                if (lane >= o2) first += other;
            }
            total = __shfl_sync(kAll, first, 31);
            first -= sum;
        }
        // the last lane whose experts start at or before the tile holds it
        const int64_t at = t - before;
        const int owner = 31 - __clz(__ballot_sync(kAll, first <= at));
        int64_t rest = at - first;
        int i = 0, c = count[0], b = begin[0];
#pragma unroll
        for (int j = 1; j < 4; ++j)
            if (i == j - 1 && rest >= tiles_of(c)) {
                rest -= tiles_of(c);
                i = j;
                c = count[j];
                b = begin[j];
            }
        c = __shfl_sync(kAll, c, owner);
        b = __shfl_sync(kAll, b, owner);
        rest = __shfl_sync(kAll, rest, owner);
        o.e = base + 4 * owner + __shfl_sync(kAll, i, owner);
        const int row_tiles = parts(c, a.tile_n);
        const int part = parts(parts(c, row_tiles), kStep) * kStep;
        const int f = rest >> 32 ? int(rest / row_tiles) : int(uint32_t(rest) / uint32_t(row_tiles));
        const int r = int(rest - int64_t(f) * row_tiles);
        o.f0 = f * (kTileM * CTAS);
        o.row0 = b + r * part;
        o.valid = min(part, c - r * part);
        o.n = (o.valid + kStep - 1) / kStep * kStep;
        o.c0 = 0;
        if constexpr (PARTS) next_part(o, true);
        else o.kblocks = parts(a.red, kBlockK);
        o.gap = 0;
        if (a.gaps && r == row_tiles - 1)
            // (cut to the buffer before the difference, which could wrap else)
            o.gap = max(0, min(max(a.offsets[o.e + 1], 0), a.rows) - (b + c));
        t += step;
        return true;
    }
};

// ---- epilogue ------------------------------------------------------------------

__device__ __forceinline__ uint32_t round2(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Rows form: v[c] is row c of 32 from `row` on (`valid` of them exist), feature f +
// lane.  Through shared memory, so that a row's 32 features leave as 64 bytes.
__device__ __forceinline__ void store_rows(const ProductArgs &a, const uint32_t (&v)[32],
                                           int64_t row, int valid, int f, int lane,
                                           uint8_t *staging) {
    uint16_t *out = static_cast<uint16_t *>(a.out);
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j] = round2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), a.bf16);
    if (!a.vec) {
        if (f + lane >= a.feat) return;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < valid)
                out[(row + j) * a.feat + f + lane] = uint16_t(w[j / 2] >> (j % 2 * 16));
        return;
    }
    uint16_t *s = reinterpret_cast<uint16_t *>(staging);
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j * 32 + lane] = uint16_t(w[j / 2] >> (j % 2 * 16));
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int j = q * 8 + lane / 4, c = f + lane % 4 * 8;
        if (j < valid && c < a.feat)
            *reinterpret_cast<uint4 *>(out + (row + j) * a.feat + c) =
                *reinterpret_cast<const uint4 *>(s + j * 32 + lane % 4 * 8);
    }
    __syncwarp();
}

// Zeros for rows row .. row + n - 1, 32 features from f on.
__device__ __forceinline__ void zero_rows(const ProductArgs &a, int64_t row, int n, int f,
                                          int lane) {
    uint16_t *out = static_cast<uint16_t *>(a.out);
    if (!a.vec) {
        if (f + lane < a.feat)
            for (int j = 0; j < n; ++j) out[(row + j) * a.feat + f + lane] = 0;
        return;
    }
    const int c = f + lane % 4 * 8;
    if (c < a.feat)
        for (int j = lane / 4; j < n; j += 8)
            *reinterpret_cast<uint4 *>(out + (row + j) * a.feat + c) = make_uint4(0, 0, 0, 0);
}

// Weights form, float32: v[c] is column c0 + c of feature f + lane of expert e.  Through
// rows of 144 bytes in shared memory (both sides without bank conflicts), so that 32
// columns leave as 128 bytes.
__device__ __forceinline__ void store_weights32(const ProductArgs &a, const uint32_t (&v)[32],
                                                int e, int f, int c0, int lane,
                                                uint8_t *staging) {
    float *out = static_cast<float *>(a.out) + (int64_t(e) * a.feat + f) * a.cols + c0;
    const int rows = min(32, a.feat - f), cols = min(32, a.cols - c0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4 *>(staging + lane * 144 + j * 16) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    if (a.vec) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r = q * 4 + lane / 8, c = lane % 8 * 4;
            if (r < rows && c < cols)
                *reinterpret_cast<uint4 *>(out + int64_t(r) * a.cols + c) =
                    *reinterpret_cast<const uint4 *>(staging + r * 144 + c * 4);
        }
    } else if (lane < cols) {
#pragma unroll 8
        for (int r = 0; r < rows; ++r)
            out[int64_t(r) * a.cols + lane] =
                *reinterpret_cast<const float *>(staging + r * 144 + lane * 4);
    }
    __syncwarp();
}

// The same for 16-bit results, 64 columns to 128 bytes, in two steps: half `h` of the
// columns to shared memory, and both to the result.
__device__ __forceinline__ void stage_weights16(const ProductArgs &a, const uint32_t (&v)[32],
                                                int h, int lane, uint8_t *staging) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = round2(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]),
                          a.bf16);
        *reinterpret_cast<uint4 *>(staging + lane * 144 + h * 64 + j * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void store_weights16(const ProductArgs &a, int e, int f, int c0,
                                                int lane, uint8_t *staging) {
    uint16_t *out = static_cast<uint16_t *>(a.out) + (int64_t(e) * a.feat + f) * a.cols + c0;
    const int rows = min(32, a.feat - f), cols = min(64, a.cols - c0);
    __syncwarp();
    if (a.vec) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r = q * 4 + lane / 8, c = lane % 8 * 8;
            if (r < rows && c < cols)
                *reinterpret_cast<uint4 *>(out + int64_t(r) * a.cols + c) =
                    *reinterpret_cast<const uint4 *>(staging + r * 144 + c * 2);
        }
    } else if (cols == 64) {
        // each row in the 16-byte pieces that lie in it, and eight elements at its ends
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r = q * 4 + lane / 8, i = lane % 8;
            uint16_t *const row = out + int64_t(r) * a.cols;
            const int head = int(-(reinterpret_cast<uint64_t>(row) >> 1) & 7);
            if (r >= rows) continue;
            const uint4 lo = *reinterpret_cast<const uint4 *>(staging + r * 144 + i * 16);
            if (head == 0) {
                *reinterpret_cast<uint4 *>(row + i * 8) = lo;
                continue;
            }
            if (i < 7) {
                const uint4 hi = *reinterpret_cast<const uint4 *>(staging + r * 144 + i * 16 + 16);
                *reinterpret_cast<uint4 *>(row + head + i * 8) = vf::shifted(lo, hi, head * 2);
            }
            const int c = i < head ? i : 56 + i;
            row[c] = *reinterpret_cast<const uint16_t *>(staging + r * 144 + c * 2);
        }
    } else {
        const uint16_t *const s = reinterpret_cast<const uint16_t *>(staging) + lane;
        out += lane;
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            if (lane < cols) out[int64_t(r) * a.cols] = s[r * 72];
            if (lane + 32 < cols) out[int64_t(r) * a.cols + 32] = s[r * 72 + 32];
        }
    }
    __syncwarp();
}

// ---- the kernel ----------------------------------------------------------------

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    uint64_t part_full[2], part_empty[2];   // SPLIT, for each turn of the epilogue
    uint32_t tmem;
    int failed;
};

// The sum of a tile's 32 columns over the CTAs that share it.  A warp holds 32 features
// of them; the four warps of its turn leave theirs in `part`, CTA `owner` adds all
// CTAs' in their order, and its four warps get the result in v (true).  No part is
// written again before it has been read.
struct Join {
    uint32_t chunk = 0, owned = 0;                   // of this turn so far

    __device__ __forceinline__ bool operator()(const ProductArgs &a, Control &ctl, float *part,
                                               int turn, int quarter, int lane, int slice,
                                               int owner, volatile int *failed, bool &ok,
                                               uint32_t (&v)[32]) {
        const uint32_t full = smem_addr(&ctl.part_full[turn]);
        const uint32_t empty = smem_addr(&ctl.part_empty[turn]);
        if (chunk > 0 && ok) {
            ok = warp_wait(empty, (chunk - 1) & 1, failed);
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
        }
        ++chunk;
        float *const mine = part + turn * 32 * kTileM + quarter * 32 + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) mine[j * kTileM] = __uint_as_float(v[j]);
        __syncwarp();
        if (lane == 0) barrier_arrive_at(full, uint32_t(owner));
        if (slice != owner) return false;
        if (ok) ok = warp_wait(full, owned & 1, failed);
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        ++owned;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0;
        for (int q = 0; q < a.split; ++q) {
            const uint32_t from = cluster_addr(smem_addr(mine), uint32_t(q));
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = __float_as_uint(__uint_as_float(v[j]) +
                                       cluster_load(from + j * kTileM * 4));
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (!ok) v[j] = 0x7FC00000u;
        __syncwarp();
        if (lane < a.split) barrier_arrive_at(empty, uint32_t(lane));
        return true;
    }
};

// Shared memory: stages, staging, parts, Control; 1,024 more for the alignment.
__host__ __device__ constexpr int64_t shared_bytes(bool weights, bool split, int stages,
                                                   int stage_bytes) {
    return int64_t(stages) * stage_bytes +
           kEpilogueWarps * (weights ? kStagingWeights : kStagingRows) + (split ? kPartBytes : 0) +
           int64_t(sizeof(Control)) + 1024;
}

// CTAS     CTAs that share a tile (2: a pair, 256 features, each CTA holds half of B)
// WEIGHTS  the weights' gradient, else the rows' product
// A_MN     the first operand is stored with i contiguous
// PARTS    sums are taken in parts of a.part terms, which are added in registers
// SPLIT    the a.split CTAs of a cluster share the sums of a tile (weights)
// OUT32    the result is float32 (weights, in parts)
template <int CTAS, bool WEIGHTS, bool A_MN, bool PARTS = false, bool SPLIT = false,
          bool OUT32 = false>
__global__ void __launch_bounds__(kThreads, 1)
expert_product(const __grid_constant__ ProductArgs a) {
    static_assert(!SPLIT || (CTAS == 1 && WEIGHTS), "single CTAs share the weights' sums");
    static_assert(!OUT32 || (PARTS && WEIGHTS), "the weights' sums in float32 are in parts");
    constexpr bool B_MN = WEIGHTS;
    constexpr int kStagingBytes = WEIGHTS ? kStagingWeights : kStagingRows;
    extern __shared__ uint8_t raw[];
    uint8_t *const smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    uint8_t *const staging = smem + a.stages * a.stage_bytes;
    uint8_t *const part = staging + kEpilogueWarps * kStagingBytes;
    Control &ctl = *reinterpret_cast<Control *>(part + (SPLIT ? kPartBytes : 0));
    volatile int *const failed = &ctl.failed;
    const int warp = uniform(int(threadIdx.x >> 5)), lane = int(threadIdx.x & 31);
    const uint32_t rank = CTAS == 1 ? 0 : cluster_rank();

    // Every role walks the same tiles.  The first one is found while tensor memory is
    // being allocated.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) tmem_alloc<CTAS>(smem_addr(&ctl.tmem), uint32_t(a.tmem_cols));
    if (warp == 3 && lane == 0) {
        for (int s = 0; s < a.stages; ++s) {
            barrier_init(smem_addr(&ctl.full[s]), 1);
            barrier_init(smem_addr(&ctl.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            barrier_init(smem_addr(&ctl.acc_full[i]), 1);
            barrier_init(smem_addr(&ctl.acc_empty[i]), kEpilogueWarps * CTAS);
            if constexpr (SPLIT) {
                barrier_init(smem_addr(&ctl.part_full[i]), kEpilogueWarps / 2 * a.split);
                barrier_init(smem_addr(&ctl.part_empty[i]), kEpilogueWarps / 2);
            }
        }
        ctl.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Tiles<CTAS, WEIGHTS, PARTS, SPLIT> tiles(a);
    Tile o = {};
    bool more = tiles.next(o);
    fence_before();
    __syncthreads();
    if constexpr (CTAS > 1 || SPLIT) cluster_sync();
    fence_after();
    const uint32_t tmem = uniform(ctl.tmem);

    int s = 0;                                       // stage and its phase
    uint32_t phase = 0;
    const auto advance = [&] {
        if (++s == a.stages) {
            s = 0;
            phase ^= 1;
        }
    };

    const uint32_t ring = smem_addr(smem), full = smem_addr(&ctl.full[0]),
                   empty = smem_addr(&ctl.empty[0]);
    if (warp == 0 || warp == 3) {
        // copies: one warp for this CTA's A, one for its share of B
        const uint32_t bars = first_barrier<CTAS>(full);
        const bool one = elected();
        bool ok = true;
        for (; ok && more; more = tiles.next(o)) {
            const int half = o.n / CTAS;
            const int slabs = (half + 63) / 64;
            // rows form: one copy, as high as the tile needs
            const int boxes = WEIGHTS ? slabs : (half + a.box - 1) / a.box;
            const CUtensorMap *const b_map = &a.b_maps[WEIGHTS ? 0 : boxes - 1];
            const int copied = WEIGHTS ? (a.b_slabs ? a.b_slabs : slabs) * 64 : boxes * a.box;
            const uint32_t bytes = uint32_t(CTAS * (kStageA + copied * 128));
            const int fa = o.f0 + int(rank) * kTileM, cb = o.c0 + int(rank) * half;
            for (int kb = 0; kb < o.kblocks; ++kb) {
                ok = warp_wait(empty + s * 8, phase ^ 1, failed);
                if (!ok) break;
                const uint32_t bar = bars + s * 8;
                const uint32_t da = ring + s * a.stage_bytes, db = da + kStageA;
                const int k = kb * kBlockK + (PARTS && !WEIGHTS ? o.k0 : 0);
                // Weights form: the last block's rows lie at its end, behind zeros: the
                // maps' second coordinate runs over the same rows as the third, so that
                // what lies before it is outside the tensor.
                const int y = min(0, o.valid - k - kBlockK), z = o.row0 + k;
                if (!one) {
                } else if (warp == 0) {
                    if (rank == 0) barrier_expect(full + s * 8, bytes);
                    if constexpr (!A_MN) {
                        copy_3d<CTAS>(da, &a.a_map, bar, k, fa, o.e);
                    } else if (a.a_slabs) {
                        if constexpr (WEIGHTS)
                            copy_4d<CTAS>(da, &a.a_map, bar, 0, y, z, fa / 64);
                        else
                            copy_4d<CTAS>(da, &a.a_map, bar, 0, k, fa / 64, o.e);
                    } else {
                        for (int j = 0; j < 2; ++j)
                            if constexpr (WEIGHTS)
                                copy_3d<CTAS>(da + j * 8192, &a.a_map, bar, fa + j * 64, y, z);
                            else
                                copy_3d<CTAS>(da + j * 8192, &a.a_map, bar, fa + j * 64, k, o.e);
                    }
                } else if constexpr (!WEIGHTS) {
                    copy_2d<CTAS>(db, b_map, bar, k, o.row0 + int(rank) * half);
                } else if (a.b_slabs) {
                    copy_4d<CTAS>(db, b_map, bar, 0, y, z, cb / 64);
                } else {
                    for (int j = 0; j < boxes; ++j)
                        copy_3d<CTAS>(db + j * 8192, b_map, bar, cb + j * 64, y, z);
                }
                __syncwarp();
                advance();
            }
        }
        // The products of the last blocks still arrive at the stages' barriers, of a pair
        // at those of both CTAs: neither leaves before they have.
        for (int i = 0; ok && i < a.stages; ++i, advance())
            ok = warp_wait(empty + s * 8, phase ^ 1, failed);
    } else if (warp == 1 && rank == 0) {
        // products; one thread issues them
        const uint32_t instr = (1u << 4) | (a.bf16 ? (1u << 7) | (1u << 10) : 0u) |
                               (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
                               (uint32_t(kTileM * CTAS / 16) << 24);
        const uint32_t first = operand(ring), stage16 = uint32_t(a.stage_bytes) >> 4;
        const bool one = elected();
        uint32_t it = 0;
        bool ok = true;
        for (; ok && more; more = tiles.next(o)) {
            if (o.kblocks == 0) continue;
            const uint32_t acc = it & 1, acc_phase = it >> 1 & 1;
            bool ready = barrier_test(full + s * 8, phase);
            ok = warp_wait(smem_addr(&ctl.acc_empty[acc]), acc_phase ^ 1, failed);
            fence_after();
            const uint32_t d = tmem + acc * uint32_t(a.acc_stride);
            const uint32_t in = instr | (uint32_t(o.n / 8) << 17);
            for (int kb = 0; ok && kb < o.kblocks; ++kb) {
                ok = warp_wait(full + s * 8, phase, failed, ready);
                if (!ok) break;
                fence_after();
                const uint32_t at = first + uint32_t(s) * stage16, bar = empty + s * 8;
                advance();
                ready = barrier_test(full + s * 8, phase);       // the next block's
                if (one) {
#pragma unroll
                    for (int q = 0; q < kBlockK / 16; ++q)
                        mma<CTAS>(d, at + q * kStep16<A_MN>,
                                  at + (kStageA >> 4) + q * kStep16<B_MN>, in, kb > 0 || q > 0);
                    mma_commit<CTAS>(bar);
                }
                __syncwarp();
            }
            if (ok && one) mma_commit<CTAS>(smem_addr(&ctl.acc_full[acc]));
            ++it;
        }
    } else if (OUT32 && warp >= 4) {
        const int quarter = warp % 4, turn = (warp - 4) / 4;
        uint8_t *const mine = staging + (warp - 4) * kStagingBytes;
        uint32_t it = 0;
        bool ok = true;
        float sum[4][32];                            // half of the columns, by 32
        Join join;
        for (; more; more = tiles.next(o)) {
            const uint32_t acc = it & 1, acc_phase = it >> 1 & 1;
            const int n = min(o.n, a.cols - o.c0);
            if (!o.more) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
            }
            if (o.kblocks > 0) {
                ok = ok && warp_wait(smem_addr(&ctl.acc_full[acc]), acc_phase, failed);
                fence_after();
                ++it;
                const uint32_t d =
                    tmem + acc * uint32_t(a.acc_stride) + (uint32_t(quarter * 32) << 16);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = 32 * turn + 64 * (i / 2) + 16 * (i % 2);
                    uint32_t v[16];
                    if (!ok || c >= n) continue;
                    tmem_load(d + uint32_t(c), v);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum[i / 2][16 * (i % 2) + j] += __uint_as_float(v[j]);
                }
                fence_before();
                __syncwarp();
                if (ok && lane == 0) {
                    if constexpr (CTAS == 1) barrier_arrive(smem_addr(&ctl.acc_empty[acc]));
                    else barrier_arrive_at(smem_addr(&ctl.acc_empty[acc]), 0);
                }
            }
            const int f = o.f0 + int(rank) * kTileM + quarter * 32;
            if (tiles.inside || (!SPLIT && f >= a.feat)) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 32 * turn + 64 * i;
                if (c >= n) continue;
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = ok ? __float_as_uint(sum[i][j]) : 0x7FC00000u;
                if constexpr (SPLIT)
                    if (!join(a, ctl, reinterpret_cast<float *>(part), turn, quarter, lane,
                              tiles.slice, i % a.split, failed, ok, v))
                        continue;
                if (f >= a.feat) continue;
                store_weights32(a, v, o.e, f, o.c0 + c, lane, mine);
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp % 4, turn = (warp - 4) / 4;
        uint8_t *const mine = staging + (warp - 4) * kStagingBytes;
        uint32_t it = 0, d = 0;
        bool ok = true;
        Join join;
        // the next accumulator, and its return
        const auto take = [&] {
            const uint32_t acc = it & 1, acc_phase = it >> 1 & 1;
            // (a sum may have some 2^19 parts: none is waited for once a role gave up)
            ok = !*failed && barrier_wait(smem_addr(&ctl.acc_full[acc]), acc_phase, failed);
            ok = __all_sync(kAll, int(ok));
            fence_after();
            d = tmem + acc * uint32_t(a.acc_stride) + (uint32_t(quarter * 32) << 16);
            ++it;
        };
        const auto give = [&] {
            const uint32_t acc = smem_addr(&ctl.acc_empty[(it - 1) & 1]);
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CTAS == 1) barrier_arrive(acc);
                else barrier_arrive_at(acc, 0);
            }
        };
        for (; more; more = tiles.next(o)) {
            ok = true;
            const int f = o.f0 + int(rank) * kTileM + quarter * 32;
            const int n = WEIGHTS ? min(o.n, a.cols - o.c0) : o.valid;
            // 32 columns at a time; of the weights 64, which leave together
            constexpr int kHalves = WEIGHTS ? 2 : 1, kCols = 32 * kHalves;
            bool store = false;                      // all lanes alike
            const auto leave = [&](int c0, int h, uint32_t(&v)[32]) {
                if (h == 0) store = f < a.feat;
                if constexpr (SPLIT)
                    if (!join(a, ctl, reinterpret_cast<float *>(part), turn, quarter, lane,
                              tiles.slice, c0 / 128 % a.split, failed, ok, v))
                        store = false;
                if constexpr (WEIGHTS) {
                    if (store) stage_weights16(a, v, h, lane, mine);
                    if (store && h == 1) store_weights16(a, o.e, f, o.c0 + c0, lane, mine);
                } else {
                    if (store) store_rows(a, v, int64_t(o.row0) + c0, n - c0, f, lane, mine);
                }
            };
            if (PARTS && tiles.inside) {
                // a sum of several parts: half of the columns in registers
                float sum[4][32] = {};
                bool all = true;
                while (true) {
                    take();
                    all = all && ok;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = kCols * (2 * (i / 2 / kHalves) + turn) +
                                      32 * (i / 2 % kHalves) + 16 * (i % 2);
                        uint32_t v[16];
                        if (!ok || c >= n) continue;
                        tmem_load(d + uint32_t(c), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[i / 2][16 * (i % 2) + j] += __uint_as_float(v[j]);
                    }
                    if (ok) give();
                    if (!tiles.inside) break;
                    tiles.next(o);
                }
                ok = all;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c0 = kCols * (2 * (i / kHalves) + turn);
                    if (c0 >= n) continue;
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = ok ? __float_as_uint(sum[i][j]) : 0x7FC00000u;
                    leave(c0, i % kHalves, v);
                }
            } else {
                if (o.kblocks > 0) take();
                for (int c0 = kCols * turn; c0 < n; c0 += 2 * kCols) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        const int c = c0 + 32 * h;
                        uint32_t v[32];
                        if (o.kblocks > 0 && ok && c < n) {
                            tmem_load(d + uint32_t(c), v);
                        } else {
                            // an empty sum, or one that was given up: NaN
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = ok ? 0u : 0x7FC00000u;
                        }
                        leave(c0, h, v);
                    }
                }
                if (o.kblocks > 0 && ok) give();
            }
            if (!WEIGHTS && o.gap > 0 && f < a.feat && turn == 0)
                zero_rows(a, int64_t(o.row0) + o.valid, o.gap, f, lane);
        }
    }

    __syncthreads();
    if (*failed) {
        // copies and products that were on their way when a role gave up land first
        const uint64_t start = now_ns();
        while (now_ns() - start < kDrainNs) {}
    }
    fence_before();
    __syncthreads();
    if constexpr (CTAS > 1 || SPLIT) cluster_sync();
    fence_after();
    if (warp == 2) tmem_free<CTAS>(tmem, uint32_t(a.tmem_cols));
}

// ---- operands at any address -----------------------------------------------------

// Lines of `len` 16-bit elements, at any address and any element stride, to lines that
// start at multiples of 16 bytes, as tensor maps need them: [outer][lines][pitch].
// Only what the product reads: the outer items whose count is above 0, or the lines
// below *limit.  Bound by HBM: each line is read and written once.
struct PadArgs {
    const uint16_t *src, *end;    // the operand, and behind its last element
    int64_t s_outer, s_line, s_el;
    uint16_t *dst;
    int64_t outer, lines, len, pitch;
    int64_t step_outer, step_lines;      // the grid's warps, in outer items and the rest
    const int32_t *counts;        // [outer], or null
    const int32_t *limit;         // null: all lines
};

// The 16 bytes at `at`, a multiple of 16; zeros outside the operand.
__device__ __forceinline__ uint4 piece(const PadArgs &a, uint64_t at) {
    const uint64_t lo = reinterpret_cast<uint64_t>(a.src), hi = reinterpret_cast<uint64_t>(a.end);
    if (at >= lo && at + 16 <= hi) return *reinterpret_cast<const uint4 *>(at);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint64_t q = at + 2 * j;
        if (q >= lo && q < hi)
            w[j / 2] |= uint32_t(*reinterpret_cast<const uint16_t *>(q)) << (j % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256)
pad_lines(const __grid_constant__ PadArgs a) {
    constexpr int U = 4;                                   // pieces of a lane in flight
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = int(threadIdx.x & 31);
    const int64_t limit = a.limit ? min(int64_t(max(*a.limit, 0)), a.lines) : a.lines;
    const int64_t chunks = (a.len + 7) / 8;
    const int64_t first = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
    int64_t e = first / a.lines, l = first - e * a.lines;
    for (; e < a.outer; e += a.step_outer, l += a.step_lines) {
        if (l >= a.lines) {
            l -= a.lines;
            if (++e >= a.outer) break;
        }
        if (l >= limit || (a.counts && a.counts[e] <= 0)) continue;
        const uint16_t *const p = a.src + e * a.s_outer + l * a.s_line;
        uint4 *const to = reinterpret_cast<uint4 *>(a.dst + (e * a.lines + l) * a.pitch);
        const int shift = int(reinterpret_cast<uint64_t>(p) & 15);
        const uint64_t at = reinterpret_cast<uint64_t>(p) - shift;
        for (int64_t c0 = 0; c0 < chunks; c0 += 32 * U) {
            uint4 v[U];
            if (a.s_el == 1) {
                uint4 hi[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + u * 32 + lane;
                    v[u] = hi[u] = make_uint4(0, 0, 0, 0);
                    if (c >= chunks) continue;
                    v[u] = piece(a, at + 16 * c);
                    if (shift) hi[u] = piece(a, at + 16 * c + 16);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = vf::shifted(v[u], hi[u], shift);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + u * 32 + lane;
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c * 8 + j < a.len)
                            w[j / 2] |= uint32_t(p[(c * 8 + j) * a.s_el]) << (j % 2 * 16);
                    v[u] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 + lane < chunks) to[c0 + u * 32 + lane] = v[u];
        }
    }
}

}  // namespace vfp
