// Gated feed-forward block: h = a(x Wg^T) (x Wu^T), and its gradients (zr.h
// has the formulas).
//
// Every product runs on the tensor cores (tcgen05, bf16 into fp32), in one of
// two kernels (pairs of CTAs for large products, single CTAs for small ones)
// with four uses:
//   forward      [g | u] = x [Wg ; Wu]^T, and h in the epilogue;
//   projections  the same, and dg, du from dh in the epilogue (to the
//                workspace);
//   input        dx = [dg | du] [Wg ; Wu], one product over k = 2 f;
//   weights      [dWg ; dWu] = [dg | du]^T x, over k = rows.
// No operand is transposed in memory: an operand whose k does not run along
// its rows is read as it lies and multiplied MN-major.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "tcgen05.cuh"
#include "zr.h"
#include "zr_device.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

using bf16 = __nv_bfloat16;

// a(g), and with it a'(g) where it is asked for.
template <bool kSlope>
__device__ __forceinline__ float silu(float g, float* slope) {
  const float s = __fdividef(1.f, 1.f + __expf(-g)), a = g * s;
  if (kSlope) *slope = s * (1.f + g * (1.f - s));
  return a;
}

// The normal distribution's tail, erfc(x) / 2 at x = |g| / sqrt 2, from the power
// that the slope needs as well: erfc(x) exp(x^2) is t times a polynomial of degree 7
// in t = 1 / (1 + 0.43 x), fitted to the function for x up to 9.4 with the least
// relative error (8.4e-8), so that the tail keeps its digits where it is small
// (evaluated in fp32, without the power's own error, it is off by 6e-7 of itself
// down to g = -4 and by 4e-6 down to -12.9).
template <bool kSlope>
__device__ __forceinline__ float gelu(float g, float* slope) {
  const float t = __fdividef(1.f, fmaf(0.43f * 0.70710678118654752f, fabsf(g), 1.f));
  const float e = __expf(-0.5f * g * g);
  float poly = fmaf(0.07370788f, t, -0.3103732f);
  poly = fmaf(poly, t, 0.3837054f);
  poly = fmaf(poly, t, -0.085725509f);
  poly = fmaf(poly, t, 0.24684432f);
  poly = fmaf(poly, t, 0.20495114f);
  poly = fmaf(poly, t, 0.24437544f);
  poly = fmaf(poly, t, 0.24251461f);
  const float tail = 0.5f * poly * t * e;
  const float cdf = g < 0.f ? tail : 1.f - tail;
  if (kSlope) *slope = fmaf(g * e, 0.39894228040143268f, cdf);
  return g * cdf;
}

// (1 + tanh x) / 2 = 1 / (1 + exp(-2x)), and its complement from the same power:
// neither is a difference, so small results keep their digits.
template <bool kSlope>
__device__ __forceinline__ float gelu_tanh(float g, float* slope) {
  const float c = 0.79788456080286536f, g2 = g * g;
  const float e = __expf(-2.f * c * g * fmaf(0.044715f, g2, 1.f));
  const float half = __fdividef(1.f, 1.f + e);
  if (kSlope) {
    const float flat = half == 0.f ? 0.f : half * (e * half);  // (1 - tanh^2) / 4
    *slope = half + (flat == 0.f ? 0.f : 2.f * c * g * flat * fmaf(0.134145f, g2, 1.f));
  }
  return g * half;
}

constexpr int kCols = 16;  // columns that an epilogue thread takes at a time

// g -> a(g), slope -> a'(g).  The choice is made once for 16 values: code that
// jumps for each of them costs more in instruction fetches than the values do
// (5 us of a 37 us call).
template <bool kSlope>
__device__ __forceinline__ void activate(float* g, float* slope, int act) {
  if (act == ZR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) g[i] = silu<kSlope>(g[i], slope + i);
  } else if (act == ZR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) g[i] = gelu<kSlope>(g[i], slope + i);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i) g[i] = gelu_tanh<kSlope>(g[i], slope + i);
  }
}

// ------------------------------------------------------------ what a product is given
enum class Use { kForward, kProjections, kInput, kWeights };

template <Use kUse>
constexpr bool kTwoOutputs = kUse == Use::kForward || kUse == Use::kProjections;

constexpr int kDepth = 64;         // k of one step
constexpr int kBox = 64 * 64 * 2;  // bytes of a 64 x 64 box

struct Maps {
  CUtensorMap x, w_gate, w_up, grads;
};

struct Job {
  FfArgs a;
  bf16* grads;  // [rows, 2 padded]: dg, then du from column `padded`
  int64_t ld_grads;
  int padded;  // f, up to a multiple of 64; the columns between are 0
  int m_tiles, n_tiles, k_blocks;
  int width;   // columns of a tile (of one projection); of a CTA's half in a pair
  int splits;  // parts of k, summed by the CTAs of a cluster
  int stages;
  int tail;     // where the epilogue's staging areas start
  int a_rows;  // rows of A's boxes: 64, or fewer where fewer exist
  int a_bytes;  // of a stage's A
  bool beside;  // weights: the kernel ahead is the input gradient's
  int32_t* status;
  int32_t* waited;  // backward: set when the input gradient's kernel has waited
};

struct Tile {
  int m, n;
};

// Tiles in groups of 16 tile rows, down each group's columns: a wave of CTAs
// shares few rows of A and few of B, which then come from L2.
__device__ __forceinline__ Tile tile_at(const Job& j, int i) {
  const int per = 16 * j.n_tiles, g = i / per, first = g * 16;
  const int high = min(16, j.m_tiles - first), r = i - g * per;
  return {first + r % high, r / high};
}

// ------------------------------------------------------------ rows of 16 values
// An epilogue thread holds 16 columns of one row.  Rows on 16-byte boundaries
// go as vectors; others through the warp's staging area, so that a warp reads
// or writes two rows at a time and not 32 rows two bytes each.
constexpr int kStageWords = kCols / 2 + 1;  // a row and one word: no bank twice
constexpr int kStaging = 32 * kStageWords * 4;
constexpr int kRowsAtOnce = 32 / kCols, kPasses = 32 / kRowsAtOnce;

__device__ __forceinline__ bool on16(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0;
}

// Stores the warp's 32 rows (the first `rows` exist) of `left` columns at p.
__device__ __forceinline__ void store_rows(bf16* p, int64_t ld, bool fast, const float* v, int rows,
                                           int left, uint32_t* stage, int lane) {
  uint32_t w[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (fast && left % 8 == 0) {
    if (lane < rows) {
      uint4* q = reinterpret_cast<uint4*>(p + lane * ld);
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      if (left > 8) q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) stage[lane * kStageWords + i] = w[i];
  __syncwarp();
  // all of the staging area's words first, then all stores
  const uint16_t* s = reinterpret_cast<const uint16_t*>(stage);
  uint16_t* q = reinterpret_cast<uint16_t*>(p);
  const int col = lane % kCols, r0 = lane / kCols;
  uint16_t x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) x[i] = s[(r0 + i * kRowsAtOnce) * 2 * kStageWords + col];
  if (col < left) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (r0 + i * kRowsAtOnce < rows) q[(r0 + i * kRowsAtOnce) * ld + col] = x[i];
  }
  __syncwarp();
}

__device__ __forceinline__ void load_rows(const bf16* p, int64_t ld, bool fast, float* v, int rows,
                                          int left, uint32_t* stage, int lane) {
  uint32_t w[kCols / 2];
  if (fast && left == kCols) {
    uint4 x = {}, y = {};
    if (lane < rows) {
      const uint4* q = reinterpret_cast<const uint4*>(p + lane * ld);
      x = q[0];
      y = q[1];
    }
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  } else {
    // all loads first: their latency is most of what this takes
    uint16_t* s = reinterpret_cast<uint16_t*>(stage);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    const int col = lane % kCols, r0 = lane / kCols;
    uint16_t x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      x[i] = 0;
      if (col < left && r0 + i * kRowsAtOnce < rows) x[i] = q[(r0 + i * kRowsAtOnce) * ld + col];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPasses; ++i) s[(r0 + i * kRowsAtOnce) * 2 * kStageWords + col] = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) w[i] = stage[lane * kStageWords + i];
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// ------------------------------------------------------------ epilogues
// Where an accumulator's columns come from: the CTA's tensor memory, or, when
// the CTAs of a cluster each summed a part of k, all their shared memories, in
// the CTAs' order ([column][row], fp32; `shared` is this thread's row).
struct InTmem {
  uint32_t at;
  __device__ __forceinline__ void load(int c, float* v) const { tmem_load16(at + c, v); }
};

// A wait gave up: what the tile would have held is not known, and says so.
struct InNothing {
  __device__ __forceinline__ void load(int, float* v) const {
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = NAN;
  }
};

struct InCluster {
  uint32_t shared;
  int parts;
  __device__ __forceinline__ void load(int c, float* v) const {
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = 0.f;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) {
      const uint32_t at = map_to_cta(shared, p) + c * 512;
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] += load_cluster(at + i * 512);
    }
  }
};

// The warp's 32 rows from row m on, columns c .. c + 15 of a tile of `width`
// columns that starts at column n0; u's columns are `u_off` after g's.
template <Use kUse, typename Source>
__device__ __forceinline__ void finish_projections(const Job& j, int64_t m, int64_t n0, int c,
                                                   int width, const Source& acc, int u_off,
                                                   uint32_t* stage, int lane) {
  const FfArgs& a = j.a;
  const int rows = (int)max((int64_t)0, min((int64_t)32, a.rows - m));
  const int64_t n = n0 + c;
  const int there = (int)min((int64_t)min(kCols, width - c), a.f - n);  // columns of f
  if (rows == 0) return;
  float g[kCols], u[kCols];
  if (kUse == Use::kForward) {
    if (there <= 0) return;
    acc.load(c, g);
    acc.load(u_off + c, u);
    activate<false>(g, nullptr, a.act);
#pragma unroll
    for (int i = 0; i < kCols; ++i) g[i] *= u[i];
    store_rows(static_cast<bf16*>(a.h) + m * a.ld_h + n, a.ld_h, on16(a.h, a.ld_h), g, rows, there,
               stage, lane);
  } else {
    const int cols = (int)min((int64_t)min(kCols, width - c), j.padded - n);  // with the zeros
    if (cols <= 0) return;
    float dh[kCols], slope[kCols];
    if (there > 0)
      load_rows(static_cast<const bf16*>(a.dh) + m * a.ld_dh + n, a.ld_dh, on16(a.dh, a.ld_dh), dh,
                rows, there, stage, lane);
    acc.load(c, g);
    activate<true>(g, slope, a.act);
    acc.load(u_off + c, u);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      slope[i] = i < there ? dh[i] * u[i] * slope[i] : 0.f;  // dg
      u[i] = i < there ? dh[i] * g[i] : 0.f;                 // du
    }
    bf16* out = j.grads + m * j.ld_grads + n;
    store_rows(out, j.ld_grads, true, slope, rows, cols, stage, lane);
    store_rows(out + j.padded, j.ld_grads, true, u, rows, cols, stage, lane);
  }
}

struct Output {
  bf16* p;
  int64_t ld, rows;
};

// Where a gradient tile goes; the weights' tile rows are the gate's, then the up's.
template <Use kUse>
__device__ __forceinline__ Output output_of(const Job& j, int& m_tile) {
  const FfArgs& a = j.a;
  if (kUse == Use::kInput) return {static_cast<bf16*>(a.dx), a.ld_dx, a.rows};
  const int half = j.m_tiles / 2;
  const bool gate = m_tile < half;
  if (!gate) m_tile -= half;
  return {static_cast<bf16*>(gate ? a.dw_gate : a.dw_up), a.ld_dw, a.f};
}

template <Use kUse>
__device__ __forceinline__ void finish_gradient(const Job& j, const Output& out, int64_t m,
                                                int64_t n, float* v, uint32_t* stage, int lane) {
  const int rows = (int)max((int64_t)0, min((int64_t)32, out.rows - m));
  const int left = (int)min((int64_t)kCols, j.a.d - n);
  if (rows == 0 || left <= 0) return;
  bf16* p = out.p + m * out.ld + n;
  const bool fast = on16(out.p, out.ld);
  if (kUse == Use::kWeights && j.a.accumulate) {
    float old[kCols];
    load_rows(p, out.ld, fast, old, rows, left, stage, lane);
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] += old[i];
  }
  store_rows(p, out.ld, fast, v, rows, left, stage, lane);
}

constexpr int kEpilogueWarps = 8;  // two for each quarter of the accumulator's rows
constexpr int kLoader = kEpilogueWarps, kMultiplier = kEpilogueWarps + 1;
constexpr int kThreads = 32 * (kEpilogueWarps + 2);

// A tile's products: a k-step of them takes some 0.3 us, and is given 2.
__device__ __forceinline__ uint64_t wait_for_tile(const Job& j) {
  return kWaitNs + (uint64_t)j.k_blocks * 2000;
}

// A wait gave up: reports it, and lets the copies in flight land before the
// shared memory is given back.
__device__ __noinline__ void give_up(int32_t* status) {
  if (status) *status = ZR_ERR_TIMEOUT;
  const uint64_t t0 = global_time_ns();
  while (global_time_ns() - t0 < 5000000ull) __nanosleep(1000);
}

// The weights' gradients need nothing of the input's gradient: where they follow
// it, their CTAs start on the SMs that it leaves free.  It lets them start only
// after its own wait, when the projections' results are there, and notes that wait
// in the workspace; a CTA that reads the note (an acquire) sees those results, and
// all that came before them, without a wait.  One that does not read it there yet
// waits as any other kernel does.  Each waits before it ends, so that what follows
// this kernel follows both.  Backward, 777 x 1001 x 2731: 61.1 -> 59.4 us; 300 x 2048
// x 5504: 84.9 -> 78.7; 4096 x 4096 x 11008: 1413 -> 1407 (on one card).
template <Use kUse>
__device__ __forceinline__ void start_after(const Job& j) {
  if (kUse == Use::kWeights && j.beside) {
    if (!published(j.waited)) wait_for_kernels_before();
    return;
  }
  wait_for_kernels_before();
  if (kUse == Use::kInput) {
    if (blockIdx.x == 0 && threadIdx.x == 32 * kLoader) publish(j.waited);
    let_next_kernel_start();
  }
}

template <Use kUse>
__device__ __forceinline__ void end_after(const Job& j) {
  if (kUse == Use::kWeights && j.beside) wait_for_kernels_before();
}

// The call's first product clears the status word, and the note of the input
// gradient's wait (whose kernel waits for this one's end before it sets it).
template <Use kUse>
__device__ __forceinline__ void first_kernel(const Job& j) {
  if (blockIdx.x != 0 || threadIdx.x != 0) return;
  if (j.status) *j.status = ZR_OK;
  if (kUse == Use::kProjections) *j.waited = 0;
}

// ------------------------------------------------------------ large products
// A pair of CTAs makes one tile of 256 rows and up to 256 columns: each CTA
// holds 128 of the rows (of A and of the accumulator) and loads half of B.  One
// k-step is 32 KB of shared memory in each CTA, loaded as boxes of 64 x 64.
// The columns (2 `width`) are chosen so that the waves of pairs come out full.
//
// Split: one loader and one multiplier thread, eight epilogue warps that empty
// one accumulator while the next tile fills the other (two of 256 columns are
// all of tensor memory), six stages.
// Bound: the matrix instructions and the loads are close to one another.
// 4096 x 4096 x 11008 forward takes 420 us (1760 TFLOP/s) from rest; its
// products alone 377, its loads alone 410 (32 KB a step for 8.4 MFLOP, about 50
// bytes a cycle and SM out of L2).  Run back to back the power limit sets in:
// 446 to 460 us by the GPU (1600 to 1660 TFLOP/s, 93 to 96 % of the library's
// sustained rate).  The tensor pipe
// is active 69 % of the time at 2048 rows, where the last of ten waves is all
// but empty.
constexpr int kTile = 256, kHalf = 128;
constexpr int kPairStage = 4 * kBox;  // A half, then B half
constexpr int kPairStages = 6;
constexpr int kColumns = 512;  // tensor memory: two accumulators of 256
constexpr int kPairSmem = kPairStages * kPairStage + 1024 + kEpilogueWarps * kStaging;

// The loader's boxes of one k-step: A's 128 rows of this CTA, then B's.
template <Use kUse>
__device__ __forceinline__ void load_pair_step(const Job& j, const Maps& maps, Tile t, int k,
                                               uint32_t rank, uint32_t smem, uint32_t bar) {
  const int k0 = k * kDepth;
  const int m0 = t.m * kTile + (int)rank * kHalf;
  if (kTwoOutputs<kUse>) {
    const CUtensorMap* w = rank == 0 ? &maps.w_gate : &maps.w_up;
    const int n0 = t.n * j.width;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.x, k0, m0 + 64 * b, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, w, k0, n0 + 64 * b, bar);
  } else if (kUse == Use::kInput) {
    const bool second = k0 >= j.padded;
    const CUtensorMap* w = second ? &maps.w_up : &maps.w_gate;
    const int n0 = (2 * t.n + (int)rank) * j.width, f0 = second ? k0 - j.padded : k0;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.grads, k0, m0 + 64 * b, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, w, n0 + 64 * b, f0, bar);
  } else {
    const int half = j.m_tiles / 2;
    const int f0 = t.m < half ? m0 : m0 - half * kTile + j.padded;
    const int n0 = (2 * t.n + (int)rank) * j.width;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.grads, f0 + 64 * b, k0, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, &maps.x, n0 + 64 * b, k0, bar);
  }
}

// A tile's columns, 16 at a time, for the warp's rows (from `row` of the tile).
template <Use kUse, typename Source>
__device__ __forceinline__ void finish_pair_tile(const Job& j, Tile t, const Source& acc, int row,
                                                 int part, uint32_t* stage, int lane) {
  if (kTwoOutputs<kUse>) {
#pragma unroll 1
    for (int c = part * kCols; c < j.width; c += 2 * kCols) {
      finish_projections<kUse>(j, (int64_t)t.m * kTile + row, (int64_t)t.n * j.width, c, j.width,
                               acc, j.width, stage, lane);
      __syncwarp();
    }
  } else {
    const Output out = output_of<kUse>(j, t.m);
#pragma unroll 1
    for (int c = part * kCols; c < 2 * j.width; c += 2 * kCols) {
      float v[kCols];
      acc.load(c, v);
      finish_gradient<kUse>(j, out, (int64_t)t.m * kTile + row, (int64_t)t.n * 2 * j.width + c, v,
                            stage, lane);
      __syncwarp();
    }
  }
}

template <Use kUse>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ff_pair_kernel(const __grid_constant__ Job j, const __grid_constant__ Maps maps) {
  constexpr bool kAMn = kUse == Use::kWeights;
  constexpr bool kBMn = !kTwoOutputs<kUse>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], done[2], taken[2];
  __shared__ uint32_t tmem_slot;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int tiles = j.m_tiles * j.n_tiles;

  if (warp == kLoader) tmem_alloc<2>(smem_u32(&tmem_slot), kColumns);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&done[b]), 1);
      mbar_init(smem_u32(&taken[b]), 2 * kEpilogueWarps);  // of both CTAs
    }
    mbar_init_fence();
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  if (kUse != Use::kInput) let_next_kernel_start();
  start_after<kUse>(j);
  if (kTwoOutputs<kUse>) first_kernel<kUse>(j);

  if (warp == kLoader) {
    if (lane == 0) {
      uint32_t step = 0;
      for (int i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_at(j, i);
        for (int k = 0; k < j.k_blocks; ++k, ++step) {
          const uint32_t s = step % kPairStages, turn = step / kPairStages;
          ok = mbar_wait(smem_u32(&empty[s]), (turn & 1) ^ 1);
          if (!ok) break;
          if (rank == 0) mbar_expect(smem_u32(&full[s]), 2 * kPairStage);
          load_pair_step<kUse>(j, maps, t, k, rank, smem + s * kPairStage,
                               map_to_cta(smem_u32(&full[s]), 0));
        }
      }
    }
  } else if (warp == kMultiplier) {
    if (rank == 0 && lane == 0) {
      const uint32_t desc = mma_descriptor(kTile, 2 * j.width, kAMn, kBMn);
      uint32_t step = 0, n = 0;
      for (int i = pair; ok && i < tiles; i += pairs, ++n) {
        const uint32_t b = n & 1;
        ok = mbar_wait(smem_u32(&taken[b]), ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        tmem_fence_after();
        for (int k = 0; k < j.k_blocks; ++k, ++step) {
          const uint32_t s = step % kPairStages;
          ok = mbar_wait(smem_u32(&full[s]), (step / kPairStages) & 1);
          if (!ok) break;
          tmem_fence_after();
          const uint32_t base = smem + s * kPairStage;
          const uint64_t da = tile_descriptor(base, kAMn ? kBox : 16);
          const uint64_t db = tile_descriptor(base + 2 * kBox, kBMn ? kBox : 16);
#pragma unroll
          for (int q = 0; q < kDepth / 16; ++q)
            mma_bf16<2>(tmem + b * kTile, da + q * (kAMn ? 2048 >> 4 : 32 >> 4),
                        db + q * (kBMn ? 2048 >> 4 : 32 >> 4), desc, k > 0 || q > 0);
          mma_commit<2>(smem_u32(&empty[s]));
        }
        if (ok) mma_commit<2>(smem_u32(&done[b]));
      }
    }
  } else {
    uint32_t* stage = reinterpret_cast<uint32_t*>(
        raw + (smem - smem_u32(raw)) + kPairStages * kPairStage + warp * kStaging);
    const int quarter = warp & 3, part = warp >> 2;
    const int row = (int)rank * kHalf + quarter * 32;
    uint32_t n = 0;
    for (int i = pair; i < tiles; i += pairs, ++n) {
      const uint32_t b = n & 1;
      const Tile t = tile_at(j, i);
      ok = ok && __all_sync(~0u, mbar_wait(smem_u32(&done[b]), (n >> 1) & 1, wait_for_tile(j)));
      if (!ok) {
        finish_pair_tile<kUse>(j, t, InNothing{}, row, part, stage, lane);
        continue;
      }
      tmem_fence_after();
      finish_pair_tile<kUse>(j, t, InTmem{tmem + b * kTile + ((uint32_t)(quarter * 32) << 16)}, row,
                             part, stage, lane);
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&taken[b]), 0));
    }
  }
  if (!ok) give_up(j.status);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kLoader) tmem_free<2>(tmem, kColumns);
  end_after<kUse>(j);
}

// ------------------------------------------------------------ small products
// One CTA makes one tile of 128 rows and `width` columns (of each projection),
// a width that spreads the work over all SMs.  A long k can be cut into parts,
// summed by the CTAs of a cluster: each leaves its accumulator in its shared
// memory, and finishes a share of the columns from all of theirs.
//
// Bound: for few rows the weights' bytes.  One row of 4096 x 11008 takes 32.3
// us (180 MB, 5.6 TB/s): 6.9 TB/s while it streams (from a fit over d), the rest
// is the launch, the first loads' latency and the epilogue.  138 CTAs of 80
// features make one wave; nine stages of 21 KB hold 26 MB in flight.  For more
// rows L2's bandwidth, about 65 bytes a cycle and SM: 16 KB of A and 128 bytes
// a column each step.  777 x 1001 x 2731: projections 21 us, of which the
// products are 8 and the epilogue's activations and odd rows 6.
constexpr int kMaxStages = 12;

// Columns of the accumulator, and of tensor memory that its loads may touch.
template <Use kUse>
__device__ __forceinline__ int columns_of(const Job& j) {
  return kTwoOutputs<kUse> ? 2 * j.width : j.width;
}

template <Use kUse>
__device__ __forceinline__ void load_step(const Job& j, const Maps& maps, Tile t, int k,
                                          int a_boxes, uint32_t smem, uint32_t bar) {
  const int k0 = k * kDepth, m0 = t.m * 128, n0 = t.n * j.width;
  const uint32_t b_at = smem + j.a_bytes;
  if (kTwoOutputs<kUse>) {
    for (int b = 0; b < a_boxes; ++b) tma_load(smem + b * kBox, &maps.x, k0, m0 + 64 * b, bar);
    tma_load(b_at, &maps.w_gate, k0, n0, bar);
    tma_load(b_at + j.width * 128, &maps.w_up, k0, n0, bar);
  } else if (kUse == Use::kInput) {
    const bool second = k0 >= j.padded;
    const CUtensorMap* w = second ? &maps.w_up : &maps.w_gate;
    const int f0 = second ? k0 - j.padded : k0;
    for (int b = 0; b < a_boxes; ++b) tma_load(smem + b * kBox, &maps.grads, k0, m0 + 64 * b, bar);
    for (int b = 0; b < j.width / 64; ++b) tma_load(b_at + b * kBox, w, n0 + 64 * b, f0, bar);
  } else {
    const int half = j.m_tiles / 2;
    const int f0 = t.m < half ? m0 : m0 - half * 128 + j.padded;
    for (int b = 0; b < 2; ++b) tma_load(smem + b * kBox, &maps.grads, f0 + 64 * b, k0, bar);
    for (int b = 0; b < j.width / 64; ++b) tma_load(b_at + b * kBox, &maps.x, n0 + 64 * b, k0, bar);
  }
}

// Columns c0, c0 + step, ... of a tile, 16 at a time, for the warp's rows.
template <Use kUse, typename Source>
__device__ __forceinline__ void finish_tile(const Job& j, Tile t, const Source& acc, int row,
                                            int c0, int step, uint32_t* stage, int lane) {
  const int64_t m0 = (int64_t)t.m * 128 + row;
  if (kTwoOutputs<kUse>) {
    if (m0 >= j.a.rows) return;
#pragma unroll 1
    for (int c = c0; c < j.width; c += step) {
      finish_projections<kUse>(j, m0, (int64_t)t.n * j.width, c, j.width, acc, j.width, stage,
                               lane);
      __syncwarp();
    }
  } else {
    const Output out = output_of<kUse>(j, t.m);
#pragma unroll 1
    for (int c = c0; c < j.width; c += step) {
      float v[kCols];
      acc.load(c, v);
      finish_gradient<kUse>(j, out, (int64_t)t.m * 128 + row, (int64_t)t.n * j.width + c, v, stage,
                            lane);
      __syncwarp();
    }
  }
}

template <Use kUse>
__global__ void __launch_bounds__(kThreads, 2)
    ff_tile_kernel(const __grid_constant__ Job j, const __grid_constant__ Maps maps) {
  constexpr bool kAMn = kUse == Use::kWeights;
  constexpr bool kBMn = !kTwoOutputs<kUse>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_slot;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int index = blockIdx.x / j.splits, split = blockIdx.x - index * j.splits;
  Tile t = tile_at(j, index);
  const int k_lo = (int)((int64_t)j.k_blocks * split / j.splits),
            k_hi = (int)((int64_t)j.k_blocks * (split + 1) / j.splits);
  const int columns = columns_of<kUse>(j), stage_bytes = j.a_bytes + columns * 128;
  // loads read 16 columns at a time, from the second projection's too
  const uint32_t reach = kTwoOutputs<kUse> ? j.width + (j.width + 15) / 16 * 16 : columns;
  float* sums = reinterpret_cast<float*>(raw + (smem - smem_u32(raw)));
  unsigned char* tail = raw + (smem - smem_u32(raw)) + j.tail;
  const uint32_t tmem_columns = reach <= 32 ? 32 : reach <= 64 ? 64 : reach <= 128 ? 128 : 256;

  // rows past the end are not loaded: what their lanes hold is never read
  const int a_boxes = kAMn || t.m * 128 + 64 < j.a.rows ? 2 : 1;
  const uint32_t step_bytes = a_boxes * (kAMn ? 64 : j.a_rows) * 128 + columns * 128;
  const int early = min(j.stages, k_hi - k_lo);  // steps that need not wait for a free stage

  if (kUse != Use::kInput) let_next_kernel_start();
  if (warp == kMultiplier) tmem_alloc<1>(smem_u32(&tmem_slot), tmem_columns);
  if (warp == kLoader && lane == 0) {
    for (int s = 0; s < j.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    mbar_init_fence();
    start_after<kUse>(j);
    for (int s = 0; s < early; ++s) {  // while the others set up
      mbar_expect(smem_u32(&full[s]), step_bytes);
      load_step<kUse>(j, maps, t, k_lo + s, a_boxes, smem + s * stage_bytes, smem_u32(&full[s]));
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  start_after<kUse>(j);
  if (kTwoOutputs<kUse>) first_kernel<kUse>(j);

  if (warp == kLoader) {
    if (lane == 0) {
      int s = early % j.stages;
      uint32_t turn = early / j.stages;
      for (int k = k_lo + early; k < k_hi; ++k) {
        ok = mbar_wait(smem_u32(&empty[s]), (turn & 1) ^ 1);
        if (!ok) break;
        mbar_expect(smem_u32(&full[s]), step_bytes);
        load_step<kUse>(j, maps, t, k, a_boxes, smem + s * stage_bytes, smem_u32(&full[s]));
        if (++s == j.stages) s = 0, ++turn;
      }
    }
  } else if (warp == kMultiplier) {
    if (lane == 0) {
      const uint32_t desc = mma_descriptor(128, columns, kAMn, kBMn);
      int s = 0;
      uint32_t turn = 0;
      for (int k = k_lo; k < k_hi; ++k) {
        ok = mbar_wait(smem_u32(&full[s]), turn & 1);
        if (!ok) break;
        tmem_fence_after();
        const uint32_t base = smem + s * stage_bytes;
        const uint64_t da = tile_descriptor(base, kAMn ? kBox : 16);
        const uint64_t db = tile_descriptor(base + j.a_bytes, kBMn ? kBox : 16);
#pragma unroll
        for (int q = 0; q < kDepth / 16; ++q)
          mma_bf16<1>(tmem, da + q * (kAMn ? 2048 >> 4 : 32 >> 4),
                      db + q * (kBMn ? 2048 >> 4 : 32 >> 4), desc, k > k_lo || q > 0);
        mma_commit<1>(smem_u32(&empty[s]));
        if (++s == j.stages) s = 0, ++turn;
      }
      if (ok) mma_commit<1>(smem_u32(&done));
    }
  } else {
    uint32_t* stage = reinterpret_cast<uint32_t*>(tail + warp * kStaging);
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32;
    ok = __all_sync(~0u, mbar_wait(smem_u32(&done), 0, wait_for_tile(j)));
    tmem_fence_after();
    const InTmem mine = {tmem + ((uint32_t)row << 16)};
    if (j.splits == 1) {
      if (ok) finish_tile<kUse>(j, t, mine, row, part * kCols, 2 * kCols, stage, lane);
      else finish_tile<kUse>(j, t, InNothing{}, row, part * kCols, 2 * kCols, stage, lane);
    } else {
      // the loader's stages are free: the accumulator goes there
#pragma unroll 1
      for (int c = part * kCols; c < columns; c += 2 * kCols) {
        float v[kCols];
        mine.load(c, v);
#pragma unroll
        for (int i = 0; i < kCols; ++i) sums[(c + i) * 128 + row + lane] = ok ? v[i] : NAN;
      }
    }
  }
  if (j.splits > 1) {
    __syncwarp();
    cluster_sync();
    if (warp < kEpilogueWarps) {
      const int row = (warp & 3) * 32, part = warp >> 2;
      const InCluster all = {smem_u32(sums + row + lane), j.splits};
      finish_tile<kUse>(j, t, all, row, (split + part * j.splits) * kCols, 2 * j.splits * kCols,
                        reinterpret_cast<uint32_t*>(tail + warp * kStaging), lane);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are read
  }
  if (!ok) give_up(j.status);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kMultiplier) tmem_free<1>(tmem, tmem_columns);
  end_after<kUse>(j);
}

// ------------------------------------------------------------ layout
// Matrices whose rows do not start on 16 bytes, laid out again with rows that
// do (TMA reads no others).  A thread makes eight columns; 777 + 2 x 2731 rows of
// 1001 take 6.8 us, bound by the latency of 2-byte loads.
struct Copy {
  const bf16* in;
  bf16* out;
  int64_t ld_in, rows;
};
struct Copies {
  Copy c[3];
  int n;
  int64_t cols, ld_out;
};

__global__ void __launch_bounds__(256) ff_layout_kernel(const Copies a) {
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t per_row = a.ld_out / 8;
  int64_t i = blockIdx.x * 256ll + threadIdx.x;
  Copy c = a.c[0];
  if (i >= c.rows * per_row) {
    i -= c.rows * per_row;
    c = a.c[1];
    if (i >= c.rows * per_row) {
      i -= c.rows * per_row;
      c = a.c[2];
      if (i >= c.rows * per_row) return;
    }
  }
  const int64_t r = i / per_row, col = (i - r * per_row) * 8;
  const uint16_t* p = reinterpret_cast<const uint16_t*>(c.in) + r * c.ld_in + col;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = col + 2 * k < a.cols ? p[2 * k] : 0;
    const uint32_t hi = col + 2 * k + 1 < a.cols ? p[2 * k + 1] : 0;
    w[k] = lo | hi << 16;
  }
  *reinterpret_cast<uint4*>(c.out + r * a.ld_out + col) = make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void ff_clear_status_kernel(int32_t* status) { *status = ZR_OK; }

zr_status launched(cudaError_t e) { return e == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

int64_t up_to(int64_t n, int64_t step) { return (n + step - 1) / step * step; }
int64_t over(int64_t n, int64_t d) { return (n + d - 1) / d; }

// ------------------------------------------------------------ shapes of the tiles
// How a product of m x n (n columns of each projection) over k_blocks steps is
// cut: in pairs' tiles of 256 x 2 width, or in tiles of 128 x width with
// `splits` parts of k.
struct Cut {
  bool pairs;
  int width, splits;
};

// What a cut costs, in cycles, as measured on GB300:
//   a pair's k-step takes 330 and 1.65 for each column of a half (narrow tiles
//   save little), a tile's what its loads need at 65 bytes a cycle and SM, 256
//   + 2 for each column;
//   an output column of the epilogue takes 60 (projections) or 35 to 45, hidden
//   behind the next tile's products where there is one;
//   a launch takes 5000 (10000 for pairs) to fill its pipelines and drain.
// Two tiles share an SM where each has two stages in half its shared memory;
// they overlap one's epilogue with the other's products.
// Over 40 shapes from 1 to 4096 rows (widths 64 to 11008) the forward call with the
// rule's choice was within 5 % of the best of all cuts for 29, and within 16 % for
// all; dx 34 and 12 %, the weight gradients 37 and 13 % (calls with their
// projections).  Both sides forward at 777 x 1000 x 2736: pairs 19.3 us, tiles of 64
// 17.0; at 4096 x 4096 x 11008: pairs 420, tiles of 128 482; pairs of 112 instead of
// 128 columns 458.
// The best pairs' tiles for m_tiles rows of tiles and n columns.
Cut best_pairs(int64_t m_tiles, int64_t n, int64_t k_blocks, bool two, int64_t* cost) {
  Cut best = {};
  for (int w = kHalf; w >= 96; w -= 8) {
    const int columns = two ? w : 2 * w;
    const int64_t waves = over(m_tiles * over(n, columns), sm_count() / 2);
    const int64_t products = k_blocks * (330 + w * 5 / 3), finish = (two ? 60 : 45) * columns;
    const int64_t c =
        waves * (products > finish ? products : finish) + finish + 10000;
    if (best.width == 0 || c < *cost) *cost = c, best = {true, w, 1};
  }
  return best;
}

constexpr int kSmemLimit = 227 * 1024 - 1024;  // a CTA's, less what is static

// What a tile's CTA needs besides its stages: alignment, and the staging areas
// or what a short A leaves of the 128 rows that its last stage is read as.
int fixed_smem(int a_bytes) {
  const int staging = kEpilogueWarps * kStaging, overhang = 2 * kBox - a_bytes;
  return 1024 + (staging > overhang ? staging : overhang);
}

int usable_sms(int s);

// The best tiles for m_tiles rows of tiles and n columns (of each projection),
// or `best` if they do not beat its cost.
Cut best_tiles(int64_t m_tiles, int64_t n, int64_t k_blocks, int first, int last, int step,
               bool two, Cut best, int64_t cost) {
  for (int w = first; w <= last; w += step)
    for (int s = 1; s == 1 || (s <= 8 && s * 4 <= k_blocks); s *= 2) {
      const int columns = two ? 2 * w : w;
      if (s > 1 && columns > 128) break;
      const double sms = usable_sms(s);
      const int shared =
          (kSmemLimit / 2 - 1024 - fixed_smem(2 * kBox)) / (2 * kBox + columns * 128) >= 2 ? 2 : 1;
      const double load = (double)(m_tiles * over(n, w) * s) / sms;
      const double rounds = ceil(load / shared);
      const double waves = shared == 1 || load <= 1 ? ceil(load) : load <= 2 ? 1 + load / 2 : load + 0.5;
      const double products = (double)(over(k_blocks, s) * (256 + 2 * columns));
      const double finish = (two ? 60.0 : 35.0) * w;
      const double c = waves * products + (shared == 1 ? waves : rounds) * finish +
                       rounds * 5000 + (load > 1 ? 1000 : 0) + (s > 1 ? 2500 : 0);
      if (c < (double)cost) cost = (int64_t)c, best = {false, w, s};
    }
  return best;
}

Cut cut_projections(int64_t rows, int64_t n, int64_t k_blocks) {
  int64_t cost = 0;
  const Cut pairs = best_pairs(over(rows, kTile), n, k_blocks, true, &cost);
  return best_tiles(over(rows, 128), n, k_blocks, 8, 128, 8, true, pairs, cost);
}

Cut cut_input(int64_t rows, int64_t d, int64_t k_blocks) {
  int64_t cost = 0;
  const Cut pairs = best_pairs(over(rows, kTile), d, k_blocks, false, &cost);
  return best_tiles(over(rows, 128), d, k_blocks, 64, 192, 64, false, pairs, cost);
}

Cut cut_weights(int64_t f, int64_t d, int64_t k_blocks) {
  int64_t cost = 0;
  const Cut pairs = best_pairs(2 * over(f, kTile), d, k_blocks, false, &cost);
  return best_tiles(2 * over(f, 128), d, k_blocks, 64, 192, 64, false, pairs, cost);
}

// Workspace: status (256 bytes), the matrices laid out again, and [dg | du].
struct Layout {
  size_t x, w_gate, w_up, grads, total;
  int64_t ld_x, ld_w;  // as the product reads them
};

// Rows of [dg | du] a power of two apart would meet in few of L2's slices.
int64_t ld_of_grads(int64_t f) {
  const int64_t n = 2 * up_to(f, 64);
  return n % 2048 ? n : n + 64;
}

Layout layout(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w, int backward) {
  Layout l = {};
  size_t at = 256;  // the status word
  auto take = [&at](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  l.ld_x = ld_x;
  l.ld_w = ld_w;
  if (ld_x % 8) l.x = take((size_t)rows * (l.ld_x = up_to(d, 8)) * 2);
  if (ld_w % 8) {
    l.ld_w = up_to(d, 8);
    l.w_gate = take((size_t)f * l.ld_w * 2);
    l.w_up = take((size_t)f * l.ld_w * 2);
  }
  if (backward) l.grads = take((size_t)rows * ld_of_grads(f) * 2);
  // a forward call that needs nothing else needs no status word either
  l.total = at > 256 || backward ? at : 0;
  return l;
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

Encode encoder() {
  static std::atomic<Encode> cached{nullptr};
  Encode e = cached.load(std::memory_order_acquire);
  if (!e) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    e = reinterpret_cast<Encode>(p);
    cached.store(e, std::memory_order_release);
  }
  return e;
}

// A [rows, cols] matrix read in boxes of 64 columns and box_rows rows; what lies
// outside reads as 0.
zr_status make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld,
                   int box_rows) {
  const Encode encode = encoder();
  if (!encode) return ZR_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? ZR_OK
             : ZR_ERR_UNSUPPORTED;
}

// Pairs of CTAs that can be resident (per device, found once).
template <Use kUse>
int resident_pairs() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(ff_pair_kernel<kUse>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kPairSmem) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sm_count() / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  if (cudaOccupancyMaxActiveClusters(&n, ff_pair_kernel<kUse>, &cfg) != cudaSuccess || n < 1)
    return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Lets the tile kernel use all of an SM's shared memory (per device, once).
template <Use kUse>
bool tile_kernel_ready() {
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (ready[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(ff_tile_kernel<kUse>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemLimit) != cudaSuccess)
    return false;
  ready[dev].store(true, std::memory_order_relaxed);
  return true;
}

// SMs that clusters of s CTAs, one on an SM, can fill (per device, found once):
// a cluster stays inside one of the GPU's processing clusters, so some are left
// over.
int usable_sms(int s) {
  static std::atomic<int> cached[64][4];
  int dev = 0, log = 0;
  while ((1 << log) < s) ++log;
  if (s == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm_count();
  int n = cached[dev][log].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)s;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() / s * s));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemLimit;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!tile_kernel_ready<Use::kInput>() ||
      cudaOccupancyMaxActiveClusters(&n, ff_tile_kernel<Use::kInput>, &cfg) != cudaSuccess || n < 1)
    return sm_count() / 2;
  n *= s;
  cached[dev][log].store(n, std::memory_order_relaxed);
  return n;
}

// m is cut into tile rows (once for each of the weights' halves).
template <Use kUse>
zr_status product(Job j, const Maps& maps, Cut cut, int64_t m, int64_t n, int64_t k_blocks,
                  cudaStream_t stream) {
  const int halves = kUse == Use::kWeights ? 2 : 1;
  const int64_t m_tiles = halves * over(m, cut.pairs ? kTile : 128);
  const int64_t n_tiles =
      over(n, cut.pairs && !kTwoOutputs<kUse> ? 2 * cut.width : cut.width);
  if (m_tiles * n_tiles * cut.splits > INT32_MAX - (1 << 20)) return ZR_ERR_UNSUPPORTED;
  j.m_tiles = (int)m_tiles;
  j.n_tiles = (int)n_tiles;
  j.k_blocks = (int)k_blocks;
  j.splits = cut.splits;
  j.width = cut.width;
  const int tiles = j.m_tiles * j.n_tiles;
  if (cut.pairs) {
    const int pairs = resident_pairs<kUse>();
    if (pairs == 0) return ZR_ERR_CUDA;
    return launched(launch_kernel(ff_pair_kernel<kUse>, 2 * (tiles < pairs ? tiles : pairs),
                                  kThreads, kPairSmem, 1, stream, j, maps));
  }
  if (!tile_kernel_ready<kUse>()) return ZR_ERR_CUDA;
  // One CTA an SM takes all the shared memory, two take half each.
  // The matrix instruction reads 128 rows of A; those that are not there are
  // whatever the shared memory holds (fixed_smem).
  j.a_bytes = kUse == Use::kWeights || j.a.rows > 64 ? 2 * kBox : j.a_rows * 128;
  const int stage = j.a_bytes + (kTwoOutputs<kUse> ? 2 : 1) * cut.width * 128;
  const int half = kSmemLimit / 2 - 1024;
  const int fixed = fixed_smem(j.a_bytes);
  const bool shared = tiles * cut.splits > usable_sms(cut.splits) && (half - fixed) / stage >= 2;
  // Over 200 KB in flight an SM's loads are no faster: one row of 4096 x 11008
  // takes 3 % longer with ten stages of 21 KB than with nine, 1 % with seven.
  const int room = (shared ? half : kSmemLimit) - fixed;
  j.stages = (room < 200 * 1024 ? room : 200 * 1024) / stage;
  if (j.stages > kMaxStages) j.stages = kMaxStages;
  j.tail = j.stages * stage;
  const int sums = cut.splits > 1 ? (kTwoOutputs<kUse> ? 2 : 1) * cut.width * 512 : 0;
  if (j.tail < sums) j.tail = sums;
  return launched(launch_kernel(ff_tile_kernel<kUse>, tiles * cut.splits, kThreads,
                                (size_t)j.tail + fixed, cut.splits, stream, j, maps));
}

// Lays out what needs it, and makes the job and the maps; `w_rows` are the
// rows of the weights' boxes.
zr_status begin(const FfArgs& a, const Layout& l, void* ws, int w_rows, int a_rows, Job* j,
                Maps* maps, cudaStream_t stream) {
  char* w = static_cast<char*>(ws);
  *j = Job{};
  j->a = a;
  j->padded = (int)up_to(a.f, 64);
  j->ld_grads = ld_of_grads(a.f);
  j->grads = reinterpret_cast<bf16*>(w + l.grads);
  j->status = reinterpret_cast<int32_t*>(w);
  j->waited = j->status + 1;
  j->a_rows = a_rows;
  const void* x = l.x ? w + l.x : a.x;
  const void* wg = l.w_gate ? w + l.w_gate : a.w_gate;
  const void* wu = l.w_up ? w + l.w_up : a.w_up;
  zr_status st = make_map(&maps->x, x, a.rows, a.d, l.ld_x, a_rows);
  if (st == ZR_OK) st = make_map(&maps->w_gate, wg, a.f, a.d, l.ld_w, w_rows);
  if (st == ZR_OK) st = make_map(&maps->w_up, wu, a.f, a.d, l.ld_w, w_rows);
  if (st == ZR_OK && l.grads)
    st = make_map(&maps->grads, j->grads, a.rows, 2 * (int64_t)j->padded, j->ld_grads, 64);
  if (st != ZR_OK) return st;
  Copies c = {};
  c.cols = a.d;
  c.ld_out = up_to(a.d, 8);
  auto add = [&](const void* in, int64_t ld_in, size_t at, int64_t rows) {
    c.c[c.n++] = {static_cast<const bf16*>(in), reinterpret_cast<bf16*>(w + at), ld_in, rows};
  };
  if (l.x) add(a.x, a.ld_x, l.x, a.rows);
  if (l.w_gate) {
    add(a.w_gate, a.ld_w, l.w_gate, a.f);
    add(a.w_up, a.ld_w, l.w_up, a.f);
  }
  if (c.n == 0) return ZR_OK;
  int64_t all = 0;
  for (int i = 0; i < c.n; ++i) all += c.c[i].rows * (c.ld_out / 8);
  if (over(all, 256) > INT32_MAX) return ZR_ERR_UNSUPPORTED;
  return launched(
      launch_kernel(ff_layout_kernel, (unsigned)over(all, 256), 256, 0, 1, stream, c));
}

}  // namespace

size_t gated_ff_workspace_bytes(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w,
                                int backward) {
  return layout(rows, d, f, ld_x, ld_w, backward).total;
}

zr_status gated_ff_launch(const FfArgs& a, void* ws, cudaStream_t stream) {
  Job j;
  Maps maps = {};
  const int64_t k_blocks = over(a.d, kDepth);
  const Cut cut = cut_projections(a.rows, a.f, k_blocks);
  const zr_status st = begin(a, layout(a.rows, a.d, a.f, a.ld_x, a.ld_w, 0), ws,
                             cut.pairs ? 64 : cut.width,
                             cut.pairs ? 64 : (int)up_to(a.rows < 64 ? a.rows : 64, 8), &j, &maps,
                             stream);
  if (st != ZR_OK) return st;
  return product<Use::kForward>(j, maps, cut, a.rows, a.f, k_blocks, stream);
}

zr_status gated_ff_backward_launch(const FfArgs& a, void* ws, cudaStream_t stream) {
  if (a.rows == 0) {
    ff_clear_status_kernel<<<1, 1, 0, stream>>>(static_cast<int32_t*>(ws));
    if (launched(cudaGetLastError()) != ZR_OK) return ZR_ERR_CUDA;
    if (a.dw_gate && !a.accumulate)
      for (void* p : {a.dw_gate, a.dw_up})
        if (cudaMemset2DAsync(p, (size_t)a.ld_dw * 2, 0, (size_t)a.d * 2, (size_t)a.f, stream) !=
            cudaSuccess)
          return ZR_ERR_CUDA;
    return ZR_OK;
  }
  Job j;
  Maps maps = {};
  const Layout l = layout(a.rows, a.d, a.f, a.ld_x, a.ld_w, 1);
  const int64_t d_blocks = over(a.d, kDepth);
  const Cut cut = cut_projections(a.rows, up_to(a.f, 64), d_blocks);
  zr_status st = begin(a, l, ws, cut.pairs ? 64 : cut.width, 64, &j, &maps, stream);
  if (st == ZR_OK)
    st = product<Use::kProjections>(j, maps, cut, a.rows, j.padded, d_blocks, stream);
  if (st == ZR_OK && a.dx) {
    // the weights again, in square boxes
    if (!cut.pairs) {
      const char* w = static_cast<const char*>(ws);
      st = make_map(&maps.w_gate, l.w_gate ? w + l.w_gate : a.w_gate, a.f, a.d, l.ld_w, 64);
      if (st == ZR_OK)
        st = make_map(&maps.w_up, l.w_up ? w + l.w_up : a.w_up, a.f, a.d, l.ld_w, 64);
    }
    if (st == ZR_OK)
      st = product<Use::kInput>(j, maps, cut_input(a.rows, a.d, 2 * (int64_t)j.padded / kDepth),
                                a.rows, a.d, 2 * (int64_t)j.padded / kDepth, stream);
  }
  j.beside = a.dx != nullptr;
  if (st == ZR_OK && a.dw_gate)
    st = product<Use::kWeights>(j, maps, cut_weights(a.f, a.d, over(a.rows, kDepth)), a.f, a.d,
                                over(a.rows, kDepth), stream);
  return st;
}

}  // namespace zr
