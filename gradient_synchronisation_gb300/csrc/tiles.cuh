// What the kernels with matrix products share: the tiles' boxes, rows of 16
// values on their way to and from memory, the maps that TMA reads by, and matrices
// laid out again for it.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tcgen05.cuh"
#include "zr.h"
#include "zr_device.cuh"

namespace zr {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kCols = 16;  // columns that an epilogue thread takes at a time

constexpr int kDepth = 64;         // k of one step
constexpr int kBox = 64 * 64 * 2;  // bytes of a 64 x 64 box

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

// Stores the warp's 32 rows (the first `rows` exist) of `left` columns at p; w holds
// the thread's 16 values, two in a word.
__device__ __forceinline__ void store_words(uint16_t* p, int64_t ld, bool fast,
                                            const uint32_t* w, int rows, int left,
                                            uint32_t* stage, int lane) {
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
  uint16_t* q = p;
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

__device__ __forceinline__ void store_rows(bf16* p, int64_t ld, bool fast, const float* v, int rows,
                                           int left, uint32_t* stage, int lane) {
  uint32_t w[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  store_words(reinterpret_cast<uint16_t*>(p), ld, fast, w, rows, left, stage, lane);
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

// ------------------------------------------------------------ the warps of a CTA
constexpr int kEpilogueWarps = 8;  // two for each quarter of the accumulator's rows
constexpr int kLoader = kEpilogueWarps, kMultiplier = kEpilogueWarps + 1;
constexpr int kThreads = 32 * (kEpilogueWarps + 2);

// A tile's products: a k-step of them takes some 0.3 us, and is given 2.
__device__ __forceinline__ uint64_t wait_for_tile(int k_blocks) {
  return kWaitNs + (uint64_t)k_blocks * 2000;
}

// A wait gave up: reports it, and lets the copies in flight land before the
// shared memory is given back.
__device__ __noinline__ void give_up(int32_t* status) {
  if (status) *status = ZR_ERR_TIMEOUT;
  const uint64_t t0 = global_time_ns();
  while (global_time_ns() - t0 < 5000000ull) __nanosleep(1000);
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

__global__ void __launch_bounds__(256) layout_kernel(const Copies a) {
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

// ------------------------------------------------------------ the host's side
inline zr_status launched(cudaError_t e) { return e == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

inline int64_t up_to(int64_t n, int64_t step) { return (n + step - 1) / step * step; }
inline int64_t over(int64_t n, int64_t d) { return (n + d - 1) / d; }

constexpr int kSmemLimit = 227 * 1024 - 1024;  // a CTA's, less what is static

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

inline Encode encoder() {
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

// A [rows, cols] matrix of 16-bit values read in boxes of 64 columns and box_rows
// rows; what lies outside reads as 0.
inline zr_status make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld,
                          int box_rows,
                          CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  const Encode encode = encoder();
  if (!encode) return ZR_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(p), dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? ZR_OK
             : ZR_ERR_UNSUPPORTED;
}

// The same matrix in boxes of `chunks` times 64 columns and 64 rows, one chunk behind
// another in shared memory.  Its rows are read up to a multiple of 64 columns, so the
// matrix's memory has to go that far.
inline zr_status make_chunk_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols,
                                int64_t ld, int chunks,
                                CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  const Encode encode = encoder();
  if (!encode) return ZR_ERR_CUDA;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)over(cols, 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
  const cuuint32_t box[3] = {64, 64, (cuuint32_t)chunks}, step[3] = {1, 1, 1};
  return encode(map, type, 3, const_cast<void*>(p), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? ZR_OK
             : ZR_ERR_UNSUPPORTED;
}

// `count` matrices of [rows, cols], `step` elements apart, as boxes of 32 rows and
// `box_cols` columns are stored to them: in rows of 64 or 128 bytes.
inline zr_status make_store_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols,
                                int64_t ld, int64_t count, int64_t step, CUtensorMapDataType type,
                                int box_cols = 32) {
  const Encode encode = encoder();
  if (!encode) return ZR_ERR_CUDA;
  const int64_t elem = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * elem),
                                 (cuuint64_t)((count > 1 ? step : ld) * elem)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, 32, 1}, one[3] = {1, 1, 1};
  return encode(map, type, 3, const_cast<void*>(p), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                box_cols * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? ZR_OK
             : ZR_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace zr
