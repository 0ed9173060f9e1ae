// A matrix product on the tensor cores (tcgen05, 16-bit values into fp32) with an
// operation's own way to finish its tiles: D[m, n] = sum over k of A[m, k] B[n, k].
//
// One persistent kernel.  Teams of one CTA (tiles of 128 rows) or of a pair (tiles
// of 256 rows: each CTA holds 128 of A's rows and of the accumulator's, and loads
// half of B) take tiles with a stride.  In each CTA one thread loads (TMA, boxes of
// 64 x 64 into a ring of stages), one thread multiplies, and eight warps empty one
// accumulator while the next tile fills the other.  No operand is transposed in
// memory: one whose k does not run along its rows is read as it lies and multiplied
// MN-major.
//
// An operation Op has
//   Job                      what its kernel is given, derived from Product
//   kAMn, kBMn, kFp16        how its operands lie and their type (bf16 otherwise)
//   kCounted, plan(job)      true: the tiles depend on what kernels before have counted,
//                            and plan() says how many there are
//   Ahead, ahead(job, plan, tile, row, share, cols, lane)
//                            what finish() needs of memory, asked for before the tile's
//                            products are there
//   kHeld                    false:
//     finish(job, plan, tile, acc, row, share, cols, ahead, out)   (not `out.real`: nothing
//                            leaves the registers and `out`'s shared memory)
//                            the warp's 32 rows (from `row` of the matrix) and its share of
//                            the columns of a tile, out of tensor memory
//                            true:
//     finish(job, plan, tile, v, row, part, half, ahead, out)
//                            the same with the thread's half row of the tile (part 0 or 1,
//                            at most 128 columns) in registers: tensor memory is free again at once.
//                            k goes in segments of a few steps, each into a sum of its
//                            own, added up in registers: the tensor cores cut their sums
//                            off instead of rounding them, which makes 64 steps of 16
//                            terms low by 1e-6 of their sum, and 256 by 4e-6.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "tiles.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

struct Product {
  int m_tiles, n_tiles;  // of one matrix
  int count;             // matrices
  int k_blocks;          // steps of kDepth
  int splits;            // parts of k, each a tile of its own
  int k_parts;           // CTAs of a cluster that sum parts of k of one tile (single CTAs)
  int width;             // rows of B that a CTA loads; a tile has CTAs x width columns
  int stages;
  int a_rows, b_rows;  // rows from one matrix to the next in A's and B's maps
  int symmetric;       // tiles left of the diagonal's are not made
  int b_boxes;         // MN-major: B's 2-D boxes of 64 columns in a step, or 0 for one 3-D
  int32_t* status;     // or null
};

struct ProductMaps {
  CUtensorMap a, b, out;
};

struct Plan {
  int m_tiles, k_blocks;
  int tiles;
  int rows;  // of a matrix, for the operation's own use
};

struct ProductTile {
  int z, split, m, n;
  int k_lo, k_hi;
};

// At most 512 terms, low by 5e-7 of their sum, and two segments from 5 steps on: with
// segments of 256 terms throughout, logits of 2048 rows take 16 % longer, of 128 terms 33 %.
// 128 rows or fewer are bound by B's bytes: there 128 terms, low by 1e-7, cost little
// (losses of 64 x 4096 x 32000 61.6 us with both, of 128 x 1024 x 65536 38.2, with
// gradients of 7 x 2360 x 3056 48 and 50).  From 129 rows on they cost something: 129 x 1024
// x 65536 41 us with 512 terms and 47 with 128, 512 x 1024 x 65536 52 and 66, 129 x 4096 x
// 32000 71 and 74, 512 x 4096 x 32000 99 and 109.
__host__ __device__ __forceinline__ int segment_steps(int k_blocks, int rows) {
  const bool few = rows <= 128;
  const int most = few ? 2 : 8;
  const int least = few || k_blocks <= 4 ? 1 : 2;
  const int parts = (k_blocks + most - 1) / most > least ? (k_blocks + most - 1) / most : least;
  return k_blocks > parts ? (k_blocks + parts - 1) / parts : 1;
}

// Half a row in registers needs more of them than 168: then the loader and the
// multiplier have a warpgroup of their own (two of its warps idle), which gives its
// registers up (2 x 128 x 224 + 128 x 56 = 384 x 168, what the block is launched with).
// Where the compiler had given a thread fewer, the warps that take more would wait for
// ever: such a build launches nothing (resident_teams).
template <typename Op>
constexpr int kProductThreads = Op::kHeld ? 384 : kThreads;
constexpr int kMoreRegisters = 224, kFewerRegisters = 56;
constexpr int kSplitRegisters = 256 * kMoreRegisters + 128 * kFewerRegisters;

// Accumulators that a tile fills one after another.
template <bool kHeld>
__device__ __forceinline__ int segments(const ProductTile& t, int steps) {
  return kHeld ? max(1, (t.k_hi - t.k_lo + steps - 1) / steps) : 1;
}

// A tile's half row: its segments' sums, added up in registers.  wait() until a segment's is
// there, load32(column, u) 32 of its columns, taken() when it has been read.  A wait that
// gives up leaves nothing of the tile known, and the segments before it are no result: the
// first value becomes NaN, and with it all that is made of the half row.  (All 128 of them:
// losses of 2048 x 65536 at depths of up to 256 took 91 us instead of 87.)
#pragma nv_exec_check_disable
template <typename Wait, typename Load, typename Taken>
__host__ __device__ __forceinline__ bool sum_segments(float (&v)[128], int parts, int half, bool ok,
                                                      Wait&& wait, Load&& load32, Taken&& taken) {
#pragma unroll
  for (int k = 0; k < 128; ++k) v[k] = 0.f;
  for (int g = 0; g < parts && ok; ++g) {
    ok = wait();
    if (!ok) break;
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c >= half) break;
      float u[32];
      load32(c, u);
#pragma unroll
      for (int k = 0; k < 32; ++k) v[c + k] += u[k];
    }
    taken();
  }
  if (!ok) v[0] = NAN;
  return ok;
}

constexpr int kMostStages = 12;
constexpr int kABytes = 2 * kBox;  // of a stage: A's 128 rows

// A symmetric product has tiles at least as high as wide: this many columns of tiles
// to a row of them.
__device__ __forceinline__ int symmetric_ratio(const Product& j) { return 128 / j.width; }

__device__ __forceinline__ int tiles_of_matrix(const Product& j, int m_tiles) {
  if (!j.symmetric) return m_tiles * j.n_tiles;
  const int q = symmetric_ratio(j);
  int n = 0;
  for (int m = 0; m < m_tiles; ++m) n += max(0, j.n_tiles - m * q);
  return n;
}

// All tiles that there can be.
__device__ __forceinline__ Plan whole_plan(const Product& j) {
  return {j.m_tiles, j.k_blocks, tiles_of_matrix(j, j.m_tiles) * j.count * j.splits, 0};
}

// Tiles in groups of 16 tile rows, down each group's columns: a wave of teams shares
// few rows of A and few of B, which then come from L2.
// (Some hundred cycles of divisions: each role asks for its next tile while it works on
// the present one.)
__device__ __forceinline__ ProductTile product_tile(const Product& j, const Plan& p, int i) {
  ProductTile t = {};
  if (i >= p.tiles) return t;
  if (j.splits > 1) {
    const int per_part = p.tiles / j.splits;
    t.split = i / per_part;
    i -= t.split * per_part;
    t.k_lo = (int)((int64_t)p.k_blocks * t.split / j.splits);
    t.k_hi = (int)((int64_t)p.k_blocks * (t.split + 1) / j.splits);
  } else {
    t.k_hi = p.k_blocks;
  }
  if (j.count > 1) {
    const int per = p.tiles / (j.splits * j.count);
    t.z = i / per;
    i -= t.z * per;
  }
  if (j.symmetric) {
    const int q = symmetric_ratio(j);
    while (i >= j.n_tiles - t.m * q) i -= j.n_tiles - t.m * q, ++t.m;
    t.n = t.m * q + i;
  } else {
    const int group = 16 * j.n_tiles, g = i / group, first = g * 16;
    const int high = min(16, p.m_tiles - first);
    i -= g * group;
    t.n = i / high;
    t.m = first + i - t.n * high;
  }
  return t;
}

// Where the CTAs of a cluster share a tile, 32 columns after another are each CTA's in
// turn: how many a CTA has at most, and a column's place among its owner's.
__host__ __device__ __forceinline__ int share_columns(int cols, int parts) {
  return (cols / 32 + parts - 1) / parts * 32;
}
__device__ __forceinline__ int share_column(int c, int parts) { return c / 32 / parts * 32 + c % 32; }

// For operations that need nothing.
struct None {};

// A tile's accumulator: in the CTA's tensor memory, or, when the CTAs of a cluster each
// summed a part of k, their sums of this CTA's share in its shared memory, in the CTAs'
// order ([part][column of the share][row]; `sums` is this thread's row).  Where nothing was
// multiplied (an empty sum, or a wait that gave up) every value is `fill`.
struct Accumulator {
  uint32_t at;
  bool there;
  float fill;
  const float* sums;
  int parts, columns;  // columns of a share
  template <int kN>
  __device__ __forceinline__ void get(int c, float* v) const {
    if (sums) {
      const float* from = sums + share_column(c, parts) * 128;
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = from[i * 128];
#pragma unroll 1
      for (int p = 1; p < parts; ++p) {
        from += columns * 128;
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += from[i * 128];
      }
    } else if (there) {
      if (kN == 32) tmem_load32(at + c, v);
      else tmem_load16(at + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = fill;
    }
  }
  __device__ __forceinline__ void load(int c, float* v) const { get<kCols>(c, v); }
  __device__ __forceinline__ void load32(int c, float* v) const { get<32>(c, v); }
};

// The columns of a tile that a warp finishes: 32 from `first`, and again after each
// `step`.
struct Share {
  int first, step;
};

// A warp's way to memory: 4 KB of shared memory, as two boxes of 32 rows of 64 bytes (or
// one of 128), which a tile's 32 rows and 32 columns go through.  Threads that store
// their own rows write 32 rows at a time, 16 bytes each: for 128 columns of 8 warps 1100
// cycles, all of it the load-store unit's; the same through here takes a third.
constexpr int kOutBytes = 4096;

struct Out {
  uint32_t at;
  uint32_t* words;  // the same, for rows that go one by one
  const CUtensorMap* map;
  int lane;
  bool real;  // false: nothing is sent

  // The boxes sent before have been read.
  __device__ __forceinline__ void room() const {
    if (elect_one()) stores_read();
    __syncwarp();
  }
  // The lane's row of a box: 32 16-bit columns, two in a word, in the 64-byte swizzle.
  __device__ __forceinline__ uint32_t place(int box, int chunk) const {
    return at + box * 2048 + lane * 64 + ((chunk ^ ((lane >> 1) & 3)) << 4);
  }
  __device__ __forceinline__ void put(int box, const uint32_t* w) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) shared_store16(place(box, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
  // The same values across the diagonal: the lane's column of a box.
  __device__ __forceinline__ void put_across(int box, const uint32_t* w) const {
    const uint32_t base = at + box * 2048 + (lane & 7) * 2;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      shared_store2(base + c * 64 + (((lane >> 3) ^ ((c >> 1) & 3)) << 4),
                    (uint16_t)(c & 1 ? w[c / 2] >> 16 : w[c / 2]));
  }
  // 32 fp32 columns of the lane's row, in the 128-byte swizzle.
  __device__ __forceinline__ void put_wide(const float* v) const {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      shared_store16(at + lane * 128 + ((c ^ (lane & 7)) << 4), __float_as_uint(v[4 * c]),
                     __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                     __float_as_uint(v[4 * c + 3]));
  }
  // 32 16-bit columns of the lane's row: the first or second half (0 or 1) of a box of 64, in
  // the 128-byte swizzle.
  __device__ __forceinline__ void put_half(int half, const uint32_t* w) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      shared_store16(at + lane * 128 + (((half * 4 + c) ^ (lane & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                     w[4 * c + 3]);
  }
  __device__ __forceinline__ void ready() const {
    store_fence();
    __syncwarp();
  }
  __device__ __forceinline__ void send(int box, int x, int y, int z) const {
    ready();
    if (real && elect_one()) {
      tma_store_3d(map, x, y, z, at + box * 2048);
      store_commit();
    }
  }
};

// The epilogue's warps meet.
__device__ __forceinline__ void epilogue_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpilogueWarps) : "memory");
}

template <int kCtas>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if (kCtas == 2) tma_load_pair(dst, map, x, y, bar);
  else tma_load(dst, map, x, y, bar);
}

// What a tile's loads have in common: the first coordinates of A and B.
struct LoadAt {
  int m0, n0, a0, b0;
};

template <int kCtas>
__device__ __forceinline__ LoadAt load_at(const Product& j, const ProductTile& t, int rank) {
  return {(t.m * kCtas + rank) * 128, (t.n * kCtas + rank) * j.width, t.z * j.a_rows, t.z * j.b_rows};
}

// One load for each operand of a k-step: the loading thread is what bounds the rate of
// steps (with four boxes of 64 x 64 a step took 700 cycles, its products 512 at most).
template <typename Op, int kCtas>
__device__ __forceinline__ void load_product_step(const Product& j, const ProductMaps& maps,
                                                  const LoadAt& at, int k, uint32_t smem,
                                                  uint32_t bar) {
  const int k0 = k * kDepth;
  if (Op::kAMn) tma_load_3d<kCtas>(smem, &maps.a, 0, at.a0 + k0, at.m0 / 64, bar);
  else load_box<kCtas>(smem, &maps.a, k0, at.a0 + at.m0, bar);
  if (!Op::kBMn) {
    load_box<kCtas>(smem + kABytes, &maps.b, k0, at.b0 + at.n0, bar);
  } else if (j.b_boxes == 0) {
    tma_load_3d<kCtas>(smem + kABytes, &maps.b, 0, at.b0 + k0, at.n0 / 64, bar);
  } else {
    for (int b = 0; b < j.b_boxes; ++b)
      load_box<kCtas>(smem + kABytes + b * kBox, &maps.b, at.n0 + 64 * b, at.b0 + k0, bar);
  }
}

template <typename Op, int kCtas>
__global__ void __launch_bounds__(kProductThreads<Op>, 1)
    product_kernel(const __grid_constant__ typename Op::Job j,
                   const __grid_constant__ ProductMaps maps) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[kMostStages], empty[kMostStages], done[2], taken[2];
  __shared__ uint32_t tmem_slot;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int k_parts = kCtas == 1 && !Op::kHeld ? j.k_parts : 1;
  const int k_part = k_parts > 1 ? (int)cluster_rank() : 0;
  const int teams = gridDim.x / (kCtas * k_parts), team = blockIdx.x / (kCtas * k_parts);
  const int cols = kCtas * j.width, stage_bytes = kABytes + j.width * 128;
  const uint32_t columns = 2 * cols;  // of tensor memory: two accumulators

  if (warp == kLoader) tmem_alloc<kCtas>(smem_u32(&tmem_slot), columns);
  if (warp == kMultiplier && lane == 0) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
    prefetch_map(&maps.out);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < j.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&done[b]), 1);
      mbar_init(smem_u32(&taken[b]), kCtas * kEpilogueWarps);
    }
    mbar_init_fence();
  }
  tmem_fence_before();
  __syncthreads();
  if (kCtas == 2 || k_parts > 1) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  let_next_kernel_start();
  // what can be worked out before the wait is (2000 to 6000 cycles, of code that is not in
  // the instruction cache yet)
  Plan p = whole_plan(j);
  ProductTile t = product_tile(j, p, team);
  wait_for_kernels_before();
  if constexpr (Op::kCounted) {
    const Plan counted = Op::template plan<kCtas>(j);
    if (counted.m_tiles != p.m_tiles || counted.k_blocks != p.k_blocks) {
      p = counted;
      t = product_tile(j, p, team);
    }
    p.rows = counted.rows;
  }
  const int segment = segment_steps(p.k_blocks, p.rows);
  if (k_parts > 1) {  // (one tile for each cluster)
    const int n = t.k_hi;
    t.k_lo = n * k_part / k_parts;
    t.k_hi = n * (k_part + 1) / k_parts;
  }
  // of the epilogue's warps
  const int quarter = warp & 3, part = warp >> 2;
  const Share share = {(k_part + part * k_parts) * 32, 64 * k_parts};
  // the cluster's sums of this CTA's share of the tile
  const int of_cta = share_columns(cols, k_parts);
  const int sums_at = j.stages * stage_bytes + kEpilogueWarps * kOutBytes;
  const float* sums = reinterpret_cast<const float*>(raw + (smem - smem_u32(raw)) + sums_at) + quarter * 32 + lane;
  const uint32_t out_at = j.stages * stage_bytes + warp * kOutBytes;
  Out out = {smem + out_at, reinterpret_cast<uint32_t*>(raw + (smem - smem_u32(raw)) + out_at),
             &maps.out, lane, true};

  if (warp < kEpilogueWarps) {
    if constexpr (Op::kHeld) more_registers<kMoreRegisters>();
    const uint64_t limit = wait_for_tile(p.k_blocks);
    const uint32_t at_rows = (uint32_t)(quarter * 32) << 16;  // of tensor memory
    uint32_t n = 0;
    // The first pass is a rehearsal: a box of the first tile, of zeros, that goes nowhere,
    // while that tile is loaded and multiplied.  It brings the epilogue's code into the
    // instruction cache, which small products wait for (five Newton-Schulz steps of 16
    // matrices of 704 x 256 take 118 us without it and 114 with, of 12 of 512 x 512 139 and
    // 132).  An accumulator held in registers has none: its code is long, and the
    // rehearsal ended after the products.
    for (int i = Op::kHeld ? team : team - teams; i < p.tiles && team < p.tiles; i += teams) {
      const bool real = Op::kHeld || i >= team;
      if (i > team) t = product_tile(j, p, i);
      const int row = (t.m * kCtas + (int)rank) * 128 + quarter * 32;
      out.real = real;
      typename Op::Ahead ahead = {};
      if (real) ahead = Op::ahead(j, p, t, row, share, cols, lane);
      if constexpr (Op::kHeld) {
        auto wait = [&]() {
          const bool there = __all_sync(~0u, mbar_wait(smem_u32(&done[n & 1]), (n >> 1) & 1, limit));
          tmem_fence_after();
          return there;
        };
        auto read = [&]() {
          tmem_fence_before();
          __syncwarp();
          const uint32_t bar = smem_u32(&taken[n & 1]);
          if (lane == 0) mbar_arrive_taken(kCtas == 2 ? map_to_cta(bar, 0) : bar);
          ++n;
        };
        float v[128];
        ok = sum_segments(
            v, segments<true>(t, segment), cols / 2, ok, wait,
            [&](int c, float* u) { tmem_load32(tmem + (n & 1) * cols + at_rows + part * (cols / 2) + c, u); },
            read);
        Op::finish(j, p, t, v, row, part, cols / 2, ahead, out);
      } else {
        const uint32_t b = n & 1;
        if (real) {
          ok = ok && __all_sync(~0u, mbar_wait(smem_u32(&done[b]), (n >> 1) & 1, limit));
          tmem_fence_after();
        }
        const uint32_t at = tmem + b * cols + at_rows;
        Accumulator acc = {at, real && ok && t.k_lo < t.k_hi, ok ? 0.f : NAN, nullptr, 1, cols};
        if (k_parts > 1) {
          // To their owners, written there: when the owners read them instead, each of
          // the parts cost a way there and back (five Newton-Schulz steps of 1024 x 1024
          // 153 us instead of 144, of 512 x 512 131 instead of 114).
#pragma unroll 1
          for (int c = part * 32; c < cols; c += real ? 64 : cols) {
            float u[32];
            acc.load32(c, u);
            const uint32_t to = map_to_cta(
                smem + sums_at + ((k_part * of_cta + share_column(c, k_parts)) * 128 + quarter * 32 + lane) * 4,
                real ? c / 32 % k_parts : k_part);
#pragma unroll
            for (int k = 0; k < 32; ++k) store_cluster(to + k * 512, u[k]);
          }
          if (real) cluster_sync();
          else epilogue_sync();  // (what it wrote is overwritten by other warps)
          acc.sums = sums;
          acc.parts = k_parts;
          acc.columns = of_cta;
        }
        Op::finish(j, p, t, acc, row, real ? share : Share{share.first, 1 << 20}, cols, ahead, out);
        if (!real) continue;
        ++n;
        if (!ok) continue;
        tmem_fence_before();
        __syncwarp();
        const uint32_t bar = smem_u32(&taken[b]);
        if (lane == 0) mbar_arrive_taken(kCtas == 2 ? map_to_cta(bar, 0) : bar);
      }
    }
    if (elect_one()) stores_read();  // (what they write is there at the kernel's end)
  } else {
    if constexpr (Op::kHeld) fewer_registers<kFewerRegisters>();
    if (warp == kLoader) {
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t counted0 = kCtas == 2 ? map_to_cta(full0, 0) : full0;
      int s = 0;
      uint32_t turn = 0;
      bool ready = true;  // the next stage is free: asked for a step ahead
      for (int i = team; ok && i < p.tiles; i += teams) {
        const LoadAt at = load_at<kCtas>(j, t, (int)rank);
        const int k_lo = t.k_lo, k_hi = t.k_hi;
        if (k_lo == k_hi) t = product_tile(j, p, i + teams);
        for (int k = k_lo; k < k_hi; ++k) {
          if (!__all_sync(~0u, ready)) ok = mbar_wait_warp(empty0 + 8 * s, (turn & 1) ^ 1);
          if (!ok) break;
          if (elect_one()) {
            if (rank == 0) mbar_expect(full0 + 8 * s, kCtas * stage_bytes);
            load_product_step<Op, kCtas>(j, maps, at, k, smem + s * stage_bytes, counted0 + 8 * s);
          }
          if (++s == j.stages) s = 0, ++turn;
          ready = mbar_test(empty0 + 8 * s, (turn & 1) ^ 1);
          if (k == k_lo) t = product_tile(j, p, i + teams);
        }
      }
    } else if (warp == kMultiplier && rank == 0) {
      const uint32_t desc = mma_descriptor(kCtas * 128, cols, Op::kAMn, Op::kBMn, Op::kFp16);
      const uint64_t da0 = tile_descriptor(smem, Op::kAMn ? kBox : 16);
      const uint64_t db0 = tile_descriptor(smem + kABytes, Op::kBMn ? kBox : 16);
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t done0 = smem_u32(done), taken0 = smem_u32(taken);
      int s = 0;
      uint32_t turn = 0, n = 0;
      bool ready = false;  // the next stage is full: asked for a step ahead
      for (int i = team; ok && i < p.tiles; i += teams) {
        const int parts = segments<Op::kHeld>(t, segment), k_lo = t.k_lo, k_hi = t.k_hi;
        if (k_lo == k_hi) t = product_tile(j, p, i + teams);
        for (int g = 0; ok && g < parts; ++g, ++n) {
          const uint32_t b = n & 1, d = tmem + b * cols;
          const int lo = Op::kHeld ? k_lo + g * segment : k_lo;
          const int hi = Op::kHeld ? min(lo + segment, k_hi) : k_hi;
          ok = mbar_wait_warp(taken0 + 8 * b, ((n >> 1) & 1) ^ 1);
          if (!ok) break;
          tmem_fence_after();
          for (int k = lo; k < hi; ++k) {
            if (!__all_sync(~0u, ready)) ok = mbar_wait_warp(full0 + 8 * s, turn & 1);
            if (!ok) break;
            const uint64_t da = da0 + s * (stage_bytes >> 4), db = db0 + s * (stage_bytes >> 4);
            const uint32_t used = empty0 + 8 * s;
            if (++s == j.stages) s = 0, ++turn;
            ready = mbar_test(full0 + 8 * s, turn & 1);
            if (elect_one()) {
#pragma unroll
              for (int q = 0; q < kDepth / 16; ++q)
                mma_16bit<kCtas>(d, da + q * (Op::kAMn ? 2048 >> 4 : 32 >> 4),
                                 db + q * (Op::kBMn ? 2048 >> 4 : 32 >> 4), desc, k > lo || q > 0);
              mma_commit<kCtas>(used);
            }
            if (k == k_lo) t = product_tile(j, p, i + teams);
          }
          if (ok && elect_one()) mma_commit<kCtas>(done0 + 8 * b);
        }
      }
    }
  }
  // (a cluster that shares a tile's k has one: the epilogue's warps have met the others)
  __syncwarp();
  if (k_parts > 1 && warp >= kEpilogueWarps) cluster_sync();
  if (!ok) give_up(j.status);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (kCtas == 2) cluster_sync();
  if (warp == kLoader) tmem_free<kCtas>(tmem, columns);
}

// ------------------------------------------------------------ shapes of the tiles
// How a product is cut: teams of `ctas`, tiles of ctas x width columns, `splits` parts of
// k as tiles of their own, or `k_parts` summed in a cluster.
struct Cut {
  int ctas, width, splits, k_parts;
};

constexpr int kFixedSmem = 1024 + kEpilogueWarps * kOutBytes;

// Shared memory for the sums of a tile's parts (single CTAs).
inline int sums_bytes(int width, int k_parts) {
  return k_parts > 1 ? k_parts * share_columns(width, k_parts) * 512 : 0;
}

inline int64_t tiles_in(int64_t m, int64_t n, int ctas, int width, bool symmetric) {
  const int64_t m_tiles = over(m, 128 * ctas), n_tiles = over(n, ctas * width);
  if (!symmetric) return m_tiles * n_tiles;
  const int64_t q = 128 / width;
  int64_t t = 0;
  for (int64_t i = 0; i < m_tiles; ++i) t += n_tiles > i * q ? n_tiles - i * q : 0;
  return t;
}

// What a cut costs, in cycles, as measured on GB300 over rows of 200 and 2048, depths of
// 64 to 2048 and 65536 columns: a pair's k-step takes 200 and 3.44 for each row of B in
// a CTA (420 for 64, 640 for 128, whose products alone are 512), a single CTA's 430, or
// 246 and 1.83 for each column past 100; a tile's epilogue 2500 and `finish` for each
// column, hidden behind the next tile's products where there is one; a launch 6000 to
// fill its pipelines and drain.  A part of k more costs `part` for all its fp32 sums (0:
// k is not cut).  Both sides, 2048 x 65536 at depth 1024: pairs of 128 154 us, of 64 210,
// single CTAs of 256 171, of 64 424.
// Where few tiles leave SMs idle, 2 or 4 CTAs of a cluster may share a tile's k
// (`clusters`); adding their sums up costs 2500, and their shared memory leaves a tile of 256
// columns too few stages.  Five Newton-Schulz steps of 2731 x 1001: 177 us with clusters, 193
// without, of 1024 x 4096 178 and 216.
inline Cut best_cut(int64_t m, int64_t n, int64_t k_blocks, int64_t count, bool symmetric,
                    int finish, double part, bool clusters = false) {
  Cut best = {};
  double least = 0;
  const int64_t sms = sm_count();
  for (int ctas = 1; ctas <= 2; ++ctas)
    for (int width = 64; width <= (ctas == 1 && !symmetric ? 256 : 128); width *= 2) {
      const int64_t one = tiles_in(m, n, ctas, width, symmetric) * count;
      for (int splits = 1; splits == 1 || (part > 0 && splits <= 64 && splits * 2 <= k_blocks);
           ++splits) {
        const int cols = ctas * width;
        const int64_t tiles = one * splits;
        const int64_t teams = sms / ctas;
        const double waves = (double)over(tiles, teams);
        const double single = 246 + 1.83 * cols;
        const double step = ctas == 2 ? 200 + 3.44 * width : single < 430 ? 430 : single;
        const double products = (double)over(k_blocks, splits) * step;
        const double end = 2500 + (double)finish * cols;
        const double c = waves * (products > end ? products : end) + end + 6000 +
                         (splits > 1 ? 3000 : 0) + part * splits;
        if (best.ctas == 0 || c < least) least = c, best = {ctas, width, splits, 1};
        if (tiles > 4 * teams) break;  // more parts would only cost more sums
      }
      for (int k_parts = 2; clusters && ctas == 1 && width <= 128 && k_parts <= 4 && one * k_parts <= sms &&
                            k_parts * 2 <= k_blocks;
           k_parts *= 2) {
        const double single = 246 + 1.83 * width, step = single < 430 ? 430 : single;
        const double c = (double)over(k_blocks, k_parts) * step + 2500 + (double)finish * width + 8500;
        if (c < least) least = c, best = {ctas, width, 1, k_parts};
      }
    }
  return best;
}

// Teams that can be resident (per device and kernel, found once); 0 on an error.
template <typename Op, int kCtas>
int resident_teams() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(product_kernel<Op, kCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemLimit) != cudaSuccess)
    return 0;
  if (Op::kHeld) {
    cudaFuncAttributes f = {};
    if (cudaFuncGetAttributes(&f, product_kernel<Op, kCtas>) != cudaSuccess ||
        f.numRegs * kProductThreads<Op> < kSplitRegisters)
      return 0;
  }
  n = sm_count();
  if (kCtas == 2) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count() / 2 * 2);
    cfg.blockDim = dim3(kProductThreads<Op>);
    cfg.dynamicSmemBytes = kSmemLimit;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, product_kernel<Op, kCtas>, &cfg) != cudaSuccess || n < 1)
      return 0;
  }
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <typename Op, int kCtas>
zr_status product_launch_of(const typename Op::Job& j, const ProductMaps& maps, int64_t tiles,
                            cudaStream_t stream) {
  const int teams = resident_teams<Op, kCtas>();
  if (teams == 0) return ZR_ERR_CUDA;
  const int stage = kABytes + j.width * 128;
  // (a cluster that shares a tile's k has no second one)
  const unsigned grid =
      (unsigned)(j.k_parts > 1 ? tiles * j.k_parts : kCtas * (tiles < teams ? tiles : teams));
  return launched(launch_kernel(product_kernel<Op, kCtas>, grid, kProductThreads<Op>,
                                (size_t)j.stages * stage + kFixedSmem + sums_bytes(j.width, j.k_parts),
                                kCtas * j.k_parts, stream, j, maps));
}

// Fills in the cut of an [m, n] product over k_blocks.
inline void apply_cut(Product& j, Cut cut, int64_t m, int64_t n, int64_t k_blocks) {
  j.m_tiles = (int)over(m, 128 * cut.ctas);
  j.n_tiles = (int)over(n, cut.ctas * cut.width);
  j.k_blocks = (int)k_blocks;
  j.splits = cut.splits;
  j.k_parts = cut.k_parts;
  j.width = cut.width;
  const int stages =
      (kSmemLimit - kFixedSmem - sums_bytes(cut.width, cut.k_parts)) / (kABytes + cut.width * 128);
  j.stages = stages < kMostStages ? stages : kMostStages;
  j.b_boxes = 0;
}

template <typename Op>
zr_status product_launch(const typename Op::Job& j, const ProductMaps& maps, int ctas, int64_t m,
                         int64_t n, cudaStream_t stream) {
  const int64_t tiles = tiles_in(m, n, ctas, j.width, j.symmetric) * j.count * j.splits;
  if (tiles > INT32_MAX / 2) return ZR_ERR_UNSUPPORTED;  // (the callers refuse them earlier)
  return ctas == 2 ? product_launch_of<Op, 2>(j, maps, tiles, stream)
                   : product_launch_of<Op, 1>(j, maps, tiles, stream);
}

}  // namespace
}  // namespace zr
