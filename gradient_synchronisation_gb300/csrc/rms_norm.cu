// Root-mean-square norm with the residual's addition, and its gradients (zr.h has
// the formulas).
//
// A row is held in registers, 16 values a thread (8 in the backward pass), so that
// memory is read once: 32 to 1024 threads a row by its length, and rows longer than
// 16384 in a kernel that reads them again.  Rows on 16-byte boundaries go as vectors of
// 16 bytes, others value by value with neighbouring threads at neighbouring values.
//
// Memory bounds both directions.  16384 x 4096 in bf16 with a residual, 537 MB each way:
// forward 78 us (6.9 TB/s; some of what it writes is still in L2 at its end, a copy of 2 GB
// reaches 6.7), backward 93 us, of which the rows take 89 (5.8 to 6.0 TB/s) and the sums of
// the weight's gradient 4.

#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "tcgen05.cuh"
#include "tiles.cuh"
#include "zr.h"
#include "zr_device.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

constexpr int kMostHeld = 16384;  // values of a row

template <typename T>
constexpr int kPerVector = 16 / (int)sizeof(T);

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 narrow<bf16>(float x) { return __float2bfloat16_rn(x); }

// The values of a row that a thread holds: kVec at a time, the threads' vectors
// beside one another.  v past the row's end is 0.
template <typename T, int kVec, int kThreads, int kHeld>
__device__ __forceinline__ void load_held(const T* row, int d, int t, float (&v)[kHeld]) {
#pragma unroll
  for (int i = 0; i < kHeld / kVec; ++i) {
    const int at = (i * kThreads + t) * kVec;
    if (kVec == 1) {
      v[i] = at < d ? widen(row[at]) : 0.f;
    } else {
      uint4 w = {};
      if (at < d) w = *reinterpret_cast<const uint4*>(row + at);
      const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[i * kVec + k] = widen(x[k]);
    }
  }
}

template <typename T, int kVec, int kThreads, int kHeld>
__device__ __forceinline__ void store_held(T* row, int d, int t, const float (&v)[kHeld]) {
#pragma unroll
  for (int i = 0; i < kHeld / kVec; ++i) {
    const int at = (i * kThreads + t) * kVec;
    if (at >= d) continue;
    if (kVec == 1) {
      row[at] = narrow<T>(v[i]);
    } else {
      uint4 w;
      T* x = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = narrow<T>(v[i * kVec + k]);
      *reinterpret_cast<uint4*>(row + at) = w;
    }
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// The sum over the kThreads threads of a row; every one of them has it.  `turn`
// counts the calls: the words of two calls in a row are apart, so that one barrier is
// enough.
template <int kThreads>
__device__ __forceinline__ float row_sum(float x, float (*words)[32], int turn) {
  x = warp_sum(x);
  if (kThreads == 32) return x;
  float* w = words[turn & 1];
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < kThreads / 32 ? w[lane] : 0.f);
}

// The mean of the squares and eps; rstd is 1 / sqrt of it.  Where it leaves fp32's range it
// is taken of 2^-80 of the values: the largest square is then 2^96, 2^31 of them still no
// infinity, and the values that make up such a sum (2^48 in the mean at least) no zeros.
// What comes out, 2^80 of the row's rstd, is applied before the 2^-80: the rstd itself may
// be subnormal.
__device__ __forceinline__ float mean_of(float sum, int64_t d, float eps) {
  return sum / (float)d + eps;
}
constexpr float kDown = 0x1p-80f;
__device__ __forceinline__ float mean_of_small(float sum, int64_t d, float eps) {
  return mean_of(sum, d, eps * kDown * kDown);
}

template <int kThreads>
constexpr int kBlock = kThreads < 128 ? 128 : kThreads;

template <typename T, int kVec, int kThreads>
__global__ void __launch_bounds__(kBlock<kThreads>) norm_kernel(const NormArgs a) {
  constexpr int kHeld = 16;
  constexpr int kRows = kBlock<kThreads> / kThreads;
  __shared__ float words[2][32];
  const int t = threadIdx.x % kThreads;
  const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kThreads;
  const int d = (int)a.d;
  let_next_kernel_start();
  wait_for_kernels_before();
  if (kThreads == 32 && r >= a.rows) return;  // (a wider row's CTA has a row of its own)
  float s[kHeld], v[kHeld];
  load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.x) + r * a.ld_x, d, t, s);
  if (a.residual) {
    load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.residual) + r * a.ld_res, d, t, v);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) s[i] = widen(narrow<T>(s[i] + v[i]));
    store_held<T, kVec, kThreads, kHeld>(static_cast<T*>(a.sum) + r * a.ld_sum, d, t, s);
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) q = fmaf(s[i], s[i], q);
  q = row_sum<kThreads>(q, words, 0);
  const float mean = mean_of(q, d, a.eps);
  float rstd = 1.f / sqrtf(mean), scale = rstd;
  if (mean > FLT_MAX) {
    q = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) q = fmaf(s[i] * kDown, s[i] * kDown, q);
    const float up = 1.f / sqrtf(mean_of_small(row_sum<kThreads>(q, words, 1), d, a.eps));
#pragma unroll
    for (int i = 0; i < kHeld; ++i) s[i] *= up;
    scale = kDown;
    rstd = up * kDown;
  }
  if (a.rstd && t == 0) a.rstd[r] = rstd;
  load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.weight), d, t, v);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) v[i] = s[i] * scale * v[i];
  store_held<T, kVec, kThreads, kHeld>(static_cast<T*>(a.y) + r * a.ld_y, d, t, v);
}

// A row of any length, read twice (the second time out of L2 where it fits), value by
// value: 2000 x 20000 in fp32 85 us, 3.8 TB/s.  A thread's sums are one chain up to d =
// 2^18, and chains of 256 values with a Long over them past that: one chain of 16384 fp32
// terms of a size, d = 2^24, is off by 1e-4.  (Two loops where one would do cost shorter
// rows 4 %, 2000 x 20000 89 us instead of 85.)
constexpr int64_t kChain = 256 * 1024;  // values of a row to a chain of each thread

// A sum of fp32 terms and what its roundings left out (Knuth's sum of two; fp64 is slow
// enough here that two sums of it take 6 of the 85 us of 2000 x 20000).
struct Long {
  float sum = 0.f, rest = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = sum + x, z = t - sum;
    rest += (sum - (t - z)) + (x - z);
    sum = t;
  }
  // (what an infinite sum left out is not a number)
  __device__ __forceinline__ float total() const { return isfinite(sum) ? sum + rest : sum; }
};

template <typename T, bool kChains>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  __shared__ float words[2][32];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + r * a.ld_res : nullptr;
  T* sum = a.residual ? static_cast<T*>(a.sum) + r * a.ld_sum : nullptr;
  float q = 0.f, small = 0.f;
  auto add = [&](int64_t i) {
    float s = widen(x[i]);
    if (res) {
      const T w = narrow<T>(s + widen(res[i]));
      sum[i] = w;
      s = widen(w);
    }
    q = fmaf(s, s, q);
    small = fmaf(s * kDown, s * kDown, small);
  };
  if (!kChains) {
    for (int64_t i = threadIdx.x; i < a.d; i += 1024) add(i);
  } else {
    Long all, all_small;
    for (int64_t lo = 0; lo < a.d; lo += kChain) {
      const int64_t hi = lo + kChain < a.d ? lo + kChain : a.d;
      q = small = 0.f;
#pragma unroll 16
      for (int64_t i = lo + threadIdx.x; i < hi; i += 1024) add(i);
      all.add(q);
      all_small.add(small);
    }
    q = all.total();
    small = all_small.total();
  }
  q = row_sum<1024>(q, words, 0);
  small = row_sum<1024>(small, words, 1);
  const float mean = mean_of(q, a.d, a.eps);
  const bool huge = mean > FLT_MAX;
  const float up = 1.f / sqrtf(huge ? mean_of_small(small, a.d, a.eps) : mean);
  const float scale = huge ? kDown : 1.f;
  if (a.rstd && threadIdx.x == 0) a.rstd[r] = up * scale;
  const T* s = res ? sum : x;  // what this thread itself has written, or an input
  const T* weight = static_cast<const T*>(a.weight);
  T* y = static_cast<T*>(a.y) + r * a.ld_y;
  for (int64_t i = threadIdx.x; i < a.d; i += 1024)
    y[i] = narrow<T>(widen(s[i]) * up * scale * widen(weight[i]));
}

// ------------------------------------------------------------ backward
// Rows are dealt to the CTAs with a stride; each thread keeps the sums of the
// weight's gradient for its columns in registers over all its rows, and a CTA leaves
// one row of sums, which the second kernel adds up in the CTAs' order.
constexpr int kBackThreads = 1024;  // of an SM, in as many CTAs as that makes

template <int kThreads>
constexpr int kBackBlock = kThreads < 256 ? 256 : kThreads;

// A thread's values of a row as they come from memory.
template <typename T, int kVec, int kHeld>
struct Raw {
  uint4 w[kHeld / kVec];
};
template <typename T, int kHeld>
struct Raw<T, 1, kHeld> {
  T w[kHeld];
};

template <typename T, int kVec, int kThreads, int kHeld>
__device__ __forceinline__ void load_raw(const T* row, int d, int t, Raw<T, kVec, kHeld>& raw) {
#pragma unroll
  for (int i = 0; i < kHeld / kVec; ++i) {
    const int at = (i * kThreads + t) * kVec;
    if constexpr (kVec == 1) {
      raw.w[i] = at < d ? row[at] : narrow<T>(0.f);
    } else {
      raw.w[i] = make_uint4(0, 0, 0, 0);
      if (at < d) raw.w[i] = *reinterpret_cast<const uint4*>(row + at);
    }
  }
}

template <typename T, int kVec, int kHeld>
__device__ __forceinline__ float value_of(const Raw<T, kVec, kHeld>& raw, int i) {
  if constexpr (kVec == 1) return widen(raw.w[i]);
  else return widen(reinterpret_cast<const T*>(&raw.w[i / kVec])[i % kVec]);
}

// A 16-bit row's successor is on its way while the row is worked on (an fp32 row's
// would take 24 registers more, and has twice the bytes in flight as it is).
template <typename T, int kVec, int kThreads, int kHeld>
__global__ void __launch_bounds__(kBackBlock<kThreads>, kBackThreads / kBackBlock<kThreads>)
    norm_backward_kernel(const NormBackArgs a, float* parts) {
  constexpr int kRows = kBackBlock<kThreads> / kThreads;
  constexpr bool kAhead = sizeof(T) == 2 && kVec > 1 && kHeld == 8;
  __shared__ float words[kRows][2][32];
  __shared__ float shared_sums[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? kThreads * kHeld : 1];
  const int t = threadIdx.x % kThreads, group = threadIdx.x / kThreads;
  const int d = (int)a.d;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  wait_for_kernels_before();
  float dw[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) dw[i] = 0.f;
  const T *s = static_cast<const T*>(a.s), *dy = static_cast<const T*>(a.dy);
  const T* ds = static_cast<const T*>(a.ds);
  Raw<T, kVec, kHeld> rs = {}, ry = {}, rd = {};
  float rstd = 0.f;
  auto load = [&](int64_t r) {
    rstd = a.rstd[r];
    load_raw<T, kVec, kThreads, kHeld>(s + r * a.ld_s, d, t, rs);
    load_raw<T, kVec, kThreads, kHeld>(dy + r * a.ld_dy, d, t, ry);
  };
  auto load_ds = [&](int64_t r) {
    if (ds) load_raw<T, kVec, kThreads, kHeld>(ds + r * a.ld_ds, d, t, rd);
  };
  int turn = 0;
  int64_t first = (int64_t)blockIdx.x * kRows;
  if (kAhead && first + group < a.rows) load(first + group), load_ds(first + group);
  for (; first < a.rows; first += stride, ++turn) {
    const int64_t r = first + group;
    const bool there = r < a.rows;
    if (!kAhead && there) load(r), load_ds(r);
    const Raw<T, kVec, kHeld> cs = rs, cy = ry;
    const float scale = there ? rstd : 0.f;
    if (kAhead && r + stride < a.rows) load(r + stride);
    float w[kHeld];  // out of L1: kept over the rows it would cost 16 registers more
    load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.weight), d, t, w);
    float c = 0.f;
    if (there) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const float hat = value_of<T, kVec, kHeld>(cs, i) * scale, g = value_of<T, kVec, kHeld>(cy, i);
        dw[i] = fmaf(g, hat, dw[i]);
        c = fmaf(g * w[i], hat, c);
      }
    }
    if (!a.dx) continue;
    c = warp_sum(c);
    if (kThreads > 32) {
      float* p = words[group][turn & 1];
      if ((threadIdx.x & 31) == 0) p[t >> 5] = c;
      __syncthreads();
      const int lane = threadIdx.x & 31;
      c = warp_sum(lane < kThreads / 32 ? p[lane] : 0.f);
    }
    if (!there) continue;
    c /= (float)d;
    load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.weight), d, t, w);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const float hat = value_of<T, kVec, kHeld>(cs, i) * scale;
      const float v = fmaf(-hat, c, value_of<T, kVec, kHeld>(cy, i) * w[i]);
      w[i] = ds ? fmaf(scale, v, value_of<T, kVec, kHeld>(rd, i)) : scale * v;
    }
    if (kAhead && r + stride < a.rows) load_ds(r + stride);
    store_held<T, kVec, kThreads, kHeld>(static_cast<T*>(a.dx) + r * a.ld_dx, d, t, w);
  }
  let_next_kernel_start();  // (not before: see below)
  if (!parts) return;
  if (kRows > 1) {  // the groups' sums, in their order
    if (group > 0)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) shared_sums[group - 1][i * kThreads + t] = dw[i];
    __syncthreads();
    if (group > 0) return;
#pragma unroll 1
    for (int g = 0; g < kRows - 1; ++g)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) dw[i] += shared_sums[g][i * kThreads + t];
  }
  float* out = parts + (int64_t)blockIdx.x * d;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int at = (i / kVec * kThreads + t) * kVec + i % kVec;
    if (at < d) out[at] = dw[i];
  }
}

// The same for rows on 16-byte boundaries, of which two or more stages fit: whole rows
// come by bulk copies into a ring in shared memory, a few ahead of the one that is worked
// on, so that enough bytes are on their way whatever the threads wait for (16384 x 4096
// in bf16 89 us; out of registers, with the next row's loads ahead, 115).  A row's stage is
// free when every thread has passed the next row's barrier.
constexpr int kRingThreads = 256;
constexpr int kRingCtas = 3;  // of an SM
constexpr int kRingBytes = 72 * 1024;
constexpr int kRingMost = 8;  // stages

template <typename T>
__global__ void __launch_bounds__(kRingThreads, kRingCtas)
    norm_backward_ring_kernel(const NormBackArgs a, float* parts, int stages) {
  constexpr int kVec = kPerVector<T>, kHeld = 16, kThreads = kRingThreads;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) uint64_t full[kRingMost];
  __shared__ float words[2][32];
  const int t = threadIdx.x, d = (int)a.d;
  const uint32_t row_bytes = (uint32_t)(a.d * sizeof(T)), tensors = a.ds ? 3 : 2;
  const uint32_t stage_bytes = tensors * row_bytes;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full[s]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  wait_for_kernels_before();
  const T *s = static_cast<const T*>(a.s), *dy = static_cast<const T*>(a.dy);
  const T* ds = static_cast<const T*>(a.ds);
  auto ask = [&](int64_t r, int stage) {
    const uint32_t at = smem_u32(ring) + stage * stage_bytes, bar = smem_u32(&full[stage]);
    mbar_expect(bar, stage_bytes);
    bulk_load(at, s + r * a.ld_s, row_bytes, bar);
    bulk_load(at + row_bytes, dy + r * a.ld_dy, row_bytes, bar);
    if (ds) bulk_load(at + 2 * row_bytes, ds + r * a.ld_ds, row_bytes, bar);
  };
  const int64_t stride = gridDim.x;
  if (t == 0)
    for (int i = 0; i < stages && blockIdx.x + i * stride < a.rows; ++i) ask(blockIdx.x + i * stride, i);
  float dw[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) dw[i] = 0.f;
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t r = blockIdx.x; r < a.rows; r += stride, ++turn) {
    const float rstd = a.rstd[r];
    ok = ok && mbar_wait(smem_u32(&full[stage]), phase);
    const T* row = reinterpret_cast<const T*>(ring + stage * stage_bytes);
    float w[kHeld], hat[kHeld], g[kHeld];
    load_held<T, kVec, kThreads, kHeld>(row, d, t, hat);
    load_held<T, kVec, kThreads, kHeld>(row + d, d, t, g);
    load_held<T, kVec, kThreads, kHeld>(static_cast<const T*>(a.weight), d, t, w);
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      hat[i] = ok ? hat[i] * rstd : NAN;  // a wait that gave up: what it would have held is not known
      dw[i] = fmaf(g[i], hat[i], dw[i]);
      g[i] *= w[i];
      c = fmaf(g[i], hat[i], c);
    }
    c = row_sum<kThreads>(c, words, turn) / (float)d;
    // every thread has the row before behind it: its stage takes the row `stages` after it
    if (t == 0 && ok && turn > 0) {
      const int before = stage == 0 ? stages - 1 : stage - 1;
      const int64_t next = r + (stages - 1) * stride;
      if (next < a.rows) ask(next, before);
    }
    if (a.dx) {
      if (ds) load_held<T, kVec, kThreads, kHeld>(row + 2 * d, d, t, w);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const float v = fmaf(-hat[i], c, g[i]);
        w[i] = ds ? fmaf(rstd, v, w[i]) : rstd * v;
      }
      store_held<T, kVec, kThreads, kHeld>(static_cast<T*>(a.dx) + r * a.ld_dx, d, t, w);
    }
    if (++stage == stages) stage = 0, phase ^= 1;
  }
  // Not before: the next kernel's CTAs would take places that this one's, which fill
  // each SM, still wait for (16384 x 4096: 131 us a call instead of 93).
  let_next_kernel_start();
  if (!ok) {  // copies in flight land before the shared memory is given back
    const uint64_t t0 = global_time_ns();
    while (global_time_ns() - t0 < 5000000ull) __nanosleep(1000);
  }
  if (!parts) return;
  float* out = parts + (int64_t)blockIdx.x * d;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int at = (i / kVec * kThreads + t) * kVec + i % kVec;
    if (at < d) out[at] = dw[i];
  }
}

// Rows of any length: the sums stay in the CTA's row of the workspace.
template <typename T, bool kChains>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormBackArgs a,
                                                                  float* parts) {
  __shared__ float words[2][32];
  let_next_kernel_start();
  wait_for_kernels_before();
  const T* w = static_cast<const T*>(a.weight);
  float* out = parts ? parts + (int64_t)blockIdx.x * a.d : nullptr;
  int turn = 0;
  bool first = true;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, ++turn, first = false) {
    const T* s = static_cast<const T*>(a.s) + r * a.ld_s;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    const float rstd = a.rstd[r];
    float c = 0.f;
    auto add = [&](int64_t i) { c = fmaf(widen(dy[i]) * widen(w[i]), widen(s[i]) * rstd, c); };
    if (!kChains) {
      for (int64_t i = threadIdx.x; i < a.d; i += 1024) add(i);
    } else {
      Long all;
      for (int64_t lo = 0; lo < a.d; lo += kChain) {
        const int64_t hi = lo + kChain < a.d ? lo + kChain : a.d;
        c = 0.f;
        for (int64_t i = lo + threadIdx.x; i < hi; i += 1024) add(i);
        all.add(c);
      }
      c = all.total();
    }
    c = row_sum<1024>(c, words, turn) / (float)a.d;
    const T* ds = a.ds ? static_cast<const T*>(a.ds) + r * a.ld_ds : nullptr;
    T* dx = a.dx ? static_cast<T*>(a.dx) + r * a.ld_dx : nullptr;
    for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
      const float hat = widen(s[i]) * rstd, g = widen(dy[i]);
      if (out) out[i] = first ? g * hat : fmaf(g, hat, out[i]);
      const float v = rstd * fmaf(-hat, c, g * widen(w[i]));
      if (dx) dx[i] = narrow<T>(ds ? v + widen(ds[i]) : v);
    }
  }
}

// The weight's gradient from the CTAs' sums: 32 columns a CTA, its warps each a part of
// the sums.
constexpr int kWeightWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kWeightWarps)
    norm_weight_kernel(const NormBackArgs a, const float* parts, int n) {
  __shared__ float sums[kWeightWarps][32];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = blockIdx.x * 32ll + lane;
  float x = 0.f;
  if (col < a.d) {
    const int hi = n * (warp + 1) / kWeightWarps;
#pragma unroll 8
    for (int i = n * warp / kWeightWarps; i < hi; ++i) x += parts[i * a.d + col];
  }
  sums[warp][lane] = x;
  __syncthreads();
  if (warp || col >= a.d) return;
#pragma unroll
  for (int i = 1; i < kWeightWarps; ++i) x += sums[i][lane];
  T* dw = static_cast<T*>(a.dweight);
  if (a.accumulate) x += widen(dw[col]);
  dw[col] = narrow<T>(x);
}

// ------------------------------------------------------------ launches
bool on_vectors(const void* p, int64_t ld, int64_t rows, size_t elem) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || ld * elem % 16 == 0));
}

template <typename T, int kVec, int kThreads>
zr_status norm_with(const NormArgs& a, cudaStream_t stream) {
  constexpr int kRows = kBlock<kThreads> / kThreads;
  return launched(launch_kernel(norm_kernel<T, kVec, kThreads>, (unsigned)over(a.rows, kRows),
                                kBlock<kThreads>, 0, 1, stream, a));
}

template <typename T, int kVec>
zr_status norm_by_length(const NormArgs& a, cudaStream_t stream) {
  if (a.d <= 512) return norm_with<T, kVec, 32>(a, stream);
  if (a.d <= 2048) return norm_with<T, kVec, 128>(a, stream);
  if (a.d <= 4096) return norm_with<T, kVec, 256>(a, stream);
  if (a.d <= 8192) return norm_with<T, kVec, 512>(a, stream);
  return norm_with<T, kVec, 1024>(a, stream);
}

template <typename T>
zr_status norm_by_type(const NormArgs& a, cudaStream_t stream) {
  if (a.d > kMostHeld)
    return launched(launch_kernel(a.d > kChain ? norm_long_kernel<T, true> : norm_long_kernel<T, false>,
                                  (unsigned)a.rows, 1024, 0, 1, stream, a));
  const bool vectors = a.d % kPerVector<T> == 0 && on_vectors(a.x, a.ld_x, a.rows, sizeof(T)) &&
                       on_vectors(a.residual, a.ld_res, a.rows, sizeof(T)) &&
                       on_vectors(a.sum, a.ld_sum, a.rows, sizeof(T)) &&
                       on_vectors(a.y, a.ld_y, a.rows, sizeof(T)) &&
                       on_vectors(a.weight, 0, 1, sizeof(T));
  return vectors ? norm_by_length<T, kPerVector<T>>(a, stream) : norm_by_length<T, 1>(a, stream);
}

// Rows of up to 1024 values go several to a CTA in the other kernel, rows past 4096 have no
// 256 threads to hold them.
bool may_ring(int64_t d) { return d > 1024 && d <= 16 * kRingThreads; }

// Stages of the ring kernel, 0 where it is not taken.
int ring_stages(int64_t d, size_t elem, bool ds) {
  if (!may_ring(d)) return 0;
  const int n = (int)(kRingBytes / ((ds ? 3 : 2) * d * (int64_t)elem));
  return n < 2 ? 0 : n < kRingMost ? n : kRingMost;
}

template <typename T>
zr_status ring_with(const NormBackArgs& a, float* parts, int n, int stages, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ZR_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(norm_backward_ring_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRingBytes) != cudaSuccess)
      return ZR_ERR_CUDA;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  const size_t smem = (size_t)stages * (a.ds ? 3 : 2) * a.d * sizeof(T);
  return launched(launch_kernel(norm_backward_ring_kernel<T>, (unsigned)n, kRingThreads, smem, 1,
                                stream, a, parts, stages));
}

// CTAs of the backward pass: as many as an SM holds at once, on each of 152, of the kernel
// that makes it.  (With the ring's 456 for the others too, 304 of 512 threads at once and
// the rest behind them: 16384 x 4096 in fp32 with ds 189 us instead of 169, 16384 x 3001 in
// bf16 136 instead of 115; of 256 threads, 608 at once, 16384 x 1501 in fp32 85 instead of 76.)
int back_parts(int64_t rows, int64_t d, bool ring) {
  const int64_t at_once = d <= 256 ? 8 : d <= 1024 ? 2 : 1;  // rows of a CTA
  const int64_t block = d <= 2048 ? 256 : d <= 4096 ? 512 : 1024;
  const int64_t n = over(rows, at_once), most = 152 * (ring ? kRingCtas : kBackThreads / block);
  return (int)(n < most ? n : most);
}

template <typename T, int kVec, int kThreads, int kHeld = 8>
zr_status back_with(const NormBackArgs& a, float* parts, int n, cudaStream_t stream) {
  return launched(launch_kernel(norm_backward_kernel<T, kVec, kThreads, kHeld>, (unsigned)n,
                                kBackBlock<kThreads>, 0, 1, stream, a, parts));
}

template <typename T, int kVec>
zr_status back_by_length(const NormBackArgs& a, float* parts, int n, cudaStream_t stream) {
  if (a.d <= 256) return back_with<T, kVec, 32>(a, parts, n, stream);
  if (a.d <= 1024) return back_with<T, kVec, 128>(a, parts, n, stream);
  if (a.d <= 2048) return back_with<T, kVec, 256>(a, parts, n, stream);
  if (a.d <= 4096) return back_with<T, kVec, 512>(a, parts, n, stream);
  if (a.d <= 8192) return back_with<T, kVec, 1024>(a, parts, n, stream);
  return back_with<T, kVec, 1024, 16>(a, parts, n, stream);
}

template <typename T>
zr_status back_by_type(const NormBackArgs& a, void* ws, cudaStream_t stream) {
  float* parts = a.dweight ? static_cast<float*>(ws) : nullptr;
  const bool vectors =
      a.d % kPerVector<T> == 0 && on_vectors(a.s, a.ld_s, a.rows, sizeof(T)) &&
      on_vectors(a.dy, a.ld_dy, a.rows, sizeof(T)) && on_vectors(a.ds, a.ld_ds, a.rows, sizeof(T)) &&
      on_vectors(a.dx, a.ld_dx, a.rows, sizeof(T)) && on_vectors(a.weight, 0, 1, sizeof(T));
  const int stages = vectors ? ring_stages(a.d, sizeof(T), a.ds) : 0;
  const int n = back_parts(a.rows, a.d, stages > 0);
  zr_status st = ZR_OK;
  if (a.rows > 0) {
    if (a.d > kMostHeld) {
      st = launched(launch_kernel(
          a.d > kChain ? norm_backward_long_kernel<T, true> : norm_backward_long_kernel<T, false>,
          (unsigned)n, 1024, 0, 1, stream, a, parts));
    } else {
      st = stages    ? ring_with<T>(a, parts, n, stages, stream)
           : vectors ? back_by_length<T, kPerVector<T>>(a, parts, n, stream)
                     : back_by_length<T, 1>(a, parts, n, stream);
    }
  }
  if (st != ZR_OK || !a.dweight) return st;
  return launched(launch_kernel(norm_weight_kernel<T>, (unsigned)over(a.d, 32), 32 * kWeightWarps, 0, 1, stream,
                                a, (const float*)parts, n));
}

}  // namespace

zr_status norm_launch(const NormArgs& a, zr_dtype dt, cudaStream_t stream) {
  return dt == ZR_F32 ? norm_by_type<float>(a, stream) : norm_by_type<bf16>(a, stream);
}

size_t norm_backward_workspace_bytes(int64_t rows, int64_t d) {
  const int other = back_parts(rows, d, false);
  const int ring = may_ring(d) ? back_parts(rows, d, true) : other;
  const size_t n = (size_t)(ring > other ? ring : other) * (size_t)d * sizeof(float);
  return n ? n : 16;
}

zr_status norm_backward_launch(const NormBackArgs& a, zr_dtype dt, void* ws, cudaStream_t stream) {
  return dt == ZR_F32 ? back_by_type<float>(a, ws, stream) : back_by_type<bf16>(a, ws, stream);
}

}  // namespace zr
