// Orthogonalised matrices by Newton-Schulz steps (zr.h has the formulas):
//   X0 = G / (|G| + eps),   A = X X^T,   B = a I + b A + c A A,   X <- B X
// on the shorter side (A = X^T X and X <- X B where there are more rows than columns),
// for all matrices of a batch in each launch.
//
// Three products a step on the tensor cores.  A and B are symmetric: only their tiles
// on and right of the diagonal's are made, and written a second time across it.  No
// operand is transposed in memory.  Large matrices are bound by the tensor cores
// (4096 x 4096: 48, 51 and 83 us for the three, the tensor pipe active 66, 63 and 72 % of
// them), small ones by a kernel's latency: 5.5 to 7.5 us for each of 704 x 256, of which
// 1.2 pass between the kernel before and the wait's end, 1.3 until the first products, 2
// to 3 with them, and 1.5 to 2 in the epilogue.
//
// X, A and B are kept in fp16 times 2^11, with fp32 sums.  fp16 has three bits more
// than bf16 at the same rate: a rounding of X in an early step grows like the singular
// values around it, up to a^5 = 485 times, so that bf16 would leave an error of a
// percent and more where fp16 leaves 1e-3.  Its range is enough because X's entries are at
// most its largest singular value (1.2 with the usual coefficients, 1 at the start), A's
// its square and the polynomial's its largest value: times 2^11 they have a factor of 22
// to the largest fp16, and keep all their bits down to 2^-25.  What grows past that (X past
// 5.65 on entry to a step, whose A is 31.98) becomes infinite, not wrong.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "product.cuh"
#include "zr.h"

namespace zr {
namespace {

constexpr float kScale = 2048.f;

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------ norm
// A sum of squares that does not leave fp32's range, for values whose squares do: large
// and small values are summed apart, scaled by powers of two (Blue, "A portable Fortran
// program to find the Euclidean norm of a vector", 1978).
struct Squares {
  float large = 0.f, middle = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float u = fabsf(x);
    if (u > 0x1p46f) {
      const float y = x * 0x1p-80f;
      large = fmaf(y, y, large);
    } else if (u < 0x1p-46f) {
      const float y = x * 0x1p80f;
      small = fmaf(y, y, small);
    } else {  // NaN too
      middle = fmaf(x, x, middle);
    }
  }
  __device__ __forceinline__ double sum() const {
    return (double)middle + (double)large * 0x1p160 + (double)small * 0x1p-160;
  }
};

// The sum over the CTA's 256 threads, in thread 0 (the others get nothing: fp64 is slow
// enough here that 256 threads of it would take longer than the kernel's memory).
__device__ __forceinline__ double cta_sum(double x, double* words) {
  words[threadIdx.x] = x;
  __syncthreads();
  if (threadIdx.x >= 32) return 0;
  x = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) x += words[threadIdx.x + 32 * w];
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

struct Input {
  const void* g;
  int64_t ld, step, rows, cols;
  int vectors;   // rows on 16 bytes, of whole vectors
  int parts;     // CTAs for a matrix
  int lanes;     // threads for a row
  double* sums;  // [count, parts]
  int32_t* status;
  float eps;
  __half *x0, *x1;  // [count, rows_padded, ld_x]
  int64_t ld_x, rows_padded;
};

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float as_float<bf16>(bf16 x) { return __bfloat162float(x); }

// A thread's values of a row's columns from `lo` (a multiple of 16) up to `hi`, a vector at
// a time.
template <typename T, typename Use>
__device__ __forceinline__ void for_row(const Input& in, const T* row, int64_t lo, int64_t hi, int lane,
                                        const Use& use) {
  constexpr int kPer = 16 / (int)sizeof(T);
  if (in.vectors) {
#pragma unroll 4
    for (int64_t i = lo / kPer + lane; i < hi / kPer; i += in.lanes) {
      const uint4 v = reinterpret_cast<const uint4*>(row)[i];
      const T* x = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int k = 0; k < kPer; ++k) use(as_float(x[k]));
    }
  } else {
#pragma unroll 8
    for (int64_t i = lo + lane; i < hi; i += in.lanes) use(as_float(row[i]));
  }
}

// Columns of a row that fp32 sums go over: 1024 in each of 256 threads.  (One chain over a
// row of 2^26, 2^18 terms in a thread, was off by up to 4e-3 where all are of a size.)
constexpr int64_t kChain = 256 * 1024;

// Rows are dealt to a matrix's CTAs, and in a CTA to its groups of threads.  One read of
// G, memory-bound; a thread whose values of a row are all small, or one of them large,
// reads them again.
template <typename T, bool kChains>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const Input in) {
  __shared__ double words[256];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t z = blockIdx.x / in.parts;
  const int part = (int)(blockIdx.x - z * in.parts);
  const int lane = threadIdx.x % in.lanes, group = threadIdx.x / in.lanes, groups = 256 / in.lanes;
  const T* g = static_cast<const T*>(in.g) + z * in.step;
  double sum = 0;
  for (int64_t r = (int64_t)part * groups + group; r < in.rows; r += (int64_t)in.parts * groups) {
    auto add = [&](int64_t lo, int64_t hi) {
      float most = 0.f, plain = 0.f;
      for_row<T>(in, g + r * in.ld, lo, hi, lane, [&](float x) {
        most = fmaxf(most, fabsf(x));
        plain = fmaf(x, x, plain);
      });
      double part = plain;
      if (most > 0x1p46f || (most < 0x1p-40f && most > 0.f)) {
        Squares s;
        for_row<T>(in, g + r * in.ld, lo, hi, lane, [&](float x) { s.add(x); });
        part = s.sum();
      }
      sum += part;  // in fp64: no fp32 sum is long
    };
    if (!kChains) add(0, in.cols);
    else
      for (int64_t lo = 0; lo < in.cols; lo += kChain) add(lo, lo + kChain < in.cols ? lo + kChain : in.cols);
  }
  sum = cta_sum(sum, words);
  if (threadIdx.x == 0) in.sums[blockIdx.x] = sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *in.status = ZR_OK;
}

// X0 in fp16, rows to 16-byte boundaries, the rows up to a whole step of k zeros (in
// both of X's buffers).
template <typename T>
__global__ void __launch_bounds__(256) ortho_start_kernel(const Input in) {
  constexpr int kPer = 16 / (int)sizeof(T);
  __shared__ double words[256];
  __shared__ float powers[2];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t z = blockIdx.x / in.parts;
  const int part = (int)(blockIdx.x - z * in.parts);
  const int lane = threadIdx.x % in.lanes, group = threadIdx.x / in.lanes, groups = 256 / in.lanes;
  double sum = 0;
  for (int i = threadIdx.x; i < in.parts; i += 256) sum += in.sums[z * in.parts + i];
  sum = cta_sum(sum, words);
  if (threadIdx.x == 0) {
    // 2^11 / norm as a power of two, in two halves, times a factor from 1 to 2: its
    // parts stay in fp32's range whatever the norm's size
    const double norm = sqrt(sum) + (double)in.eps;
    int e = 0;
    const double inv = norm > 0 ? kScale / norm : 0.0;
    const float factor = (float)(2 * frexp(inv, &e));
    powers[0] = ldexpf(1.f, (e - 1) / 2);
    powers[1] = ldexpf(1.f, e - 1 - (e - 1) / 2) * factor;
  }
  __syncthreads();
  const float p0 = powers[0], p1 = powers[1];
  const T* g = static_cast<const T*>(in.g) + z * in.step;
  for (int64_t r = (int64_t)part * groups + group; r < in.rows_padded;
       r += (int64_t)in.parts * groups) {
    __half* out = in.x0 + (z * in.rows_padded + r) * in.ld_x;
    __half* other = in.x1 + (z * in.rows_padded + r) * in.ld_x;
    const T* row = g + r * in.ld;
    if (r >= in.rows) {
      for (int64_t i = lane; i < in.ld_x; i += in.lanes) out[i] = other[i] = __half(0.f);
    } else if (in.vectors) {
#pragma unroll 4
      for (int64_t i = lane; i < in.cols / kPer; i += in.lanes) {
        const uint4 v = reinterpret_cast<const uint4*>(row)[i];
        const T* x = reinterpret_cast<const T*>(&v);
        uint32_t w[kPer / 2];
#pragma unroll
        for (int k = 0; k < kPer; k += 2)
          w[k / 2] = pack_half2(as_float(x[k]) * p0 * p1, as_float(x[k + 1]) * p0 * p1);
        if (kPer == 8) reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[kPer / 2 - 1]);
        else reinterpret_cast<uint2*>(out)[i] = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll 8
      for (int64_t i = lane; i < in.cols; i += in.lanes)
        out[i] = __float2half_rn(as_float(row[i]) * p0 * p1);
    }
  }
}

// ------------------------------------------------------------ steps
struct OrthoJob : Product {
  const __half* in;  // square: A, [count, step elements] with ld
  int64_t ld, step;
  int rows, cols;
  float a, b, c;
  bf16* last;  // the last step's X, to the caller
  int64_t ld_last, step_last;
  float factor;  // that takes the scales of A or B and X off
  float scale;   // of the last X (apart from factor: together they may be subnormal)
  int boxes;  // X goes as boxes
};

// Sends a symmetric tile's 32 rows and 32 columns, and across the diagonal those of
// tiles right of the diagonal's.
__device__ __forceinline__ void send_symmetric(const OrthoJob& j, const ProductTile& t,
                                               const float* v, int row, int n, const Out& o) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_half2(v[2 * i], v[2 * i + 1]);
  const bool across = t.n / symmetric_ratio(j) > t.m;
  o.put(0, w);
  if (across) o.put_across(1, w);
  o.ready();
  if (o.real && elect_one()) {
    tma_store_3d(o.map, n, row, t.z, o.at);
    if (across) tma_store_3d(o.map, row, n, t.z, o.at + 2048);
    store_commit();
  }
}

template <bool kTall>
struct Gram {
  using Job = OrthoJob;
  static constexpr bool kAMn = kTall, kBMn = kTall, kFp16 = true, kCounted = false, kHeld = false;
  using Ahead = None;
  static __device__ __forceinline__ None ahead(const Job&, const Plan&, const ProductTile&, int, Share, int, int) {
    return {};
  }
  static __device__ __forceinline__ void finish(const Job& j, const Plan&, const ProductTile& t,
                                                const Accumulator& acc, int row, Share share, int cols, None,
                                                const Out& o) {
    if (row >= j.rows) return;
#pragma unroll 1
    for (int k = share.first; k < cols; k += share.step) {
      if (t.n * cols + k >= j.cols) break;
      float v[32];
      acc.load32(k, v);
      o.room();
      if (j.splits > 1) {  // a part of a long sum
        o.put_wide(v);
        o.send(0, t.n * cols + k, row, t.split * j.count + t.z);
        continue;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= 1.f / kScale;
      send_symmetric(j, t, v, row, t.n * cols + k, o);
    }
  }
};

// A from the parts of a long sum, in their order; `high` rows of tiles by `high` columns
// left of the diagonal's are not made, and come from across it.
struct GramSum {
  const float* parts;  // [splits, count, m, ld_parts]
  __half* a;           // [count, m, ld]
  int64_t count, m, ld_parts, ld;
  int splits, high;
};

__global__ void __launch_bounds__(256) ortho_gram_kernel(const GramSum s) {
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t all = s.count * s.m * s.m, part = s.count * s.m * s.ld_parts;
  for (int64_t n = blockIdx.x * 256ll + threadIdx.x; n < all; n += gridDim.x * 256ll) {
    const int64_t row = n / s.m, c = n - row * s.m, z = row / s.m, r = row - z * s.m;
    const bool made = c / s.high >= r / s.high;
    const float* p = s.parts + (z * s.m + (made ? r : c)) * s.ld_parts + (made ? c : r);
    float x = 0.f;
    for (int i = 0; i < s.splits; ++i) x += p[i * part];
    s.a[row * s.ld + c] = __float2half_rn(x * (1.f / kScale));
  }
}

// A's own tile comes in rows of 64 bytes, four lanes to a row, and each lane gets its row
// through the box that it is sent from afterwards.
struct Square {
  using Job = OrthoJob;
  static constexpr bool kAMn = false, kBMn = false, kFp16 = true, kCounted = false, kHeld = false;
  struct Ahead {
    uint4 next[4];  // rows lane / 4, and 8 further each: a box's
  };
  // (ld is a multiple of 64, and holds 32 columns from n on)
  static __device__ __forceinline__ void ask(const Job& j, const ProductTile& t, int row, int k, int cols,
                                             int lane, Ahead& a) {
    const int n = t.n * cols + k, r = row + (lane >> 2);
    if (k >= cols || n >= j.cols) return;
    const __half* in = j.in + t.z * j.step + (int64_t)r * j.ld + n + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 8 * i < j.rows) a.next[i] = *reinterpret_cast<const uint4*>(in + 8 * i * j.ld);
  }
  static __device__ __forceinline__ Ahead ahead(const Job& j, const Plan&, const ProductTile& t, int row,
                                                Share share, int cols, int lane) {
    Ahead a = {};
    ask(j, t, row, share.first, cols, lane, a);
    return a;
  }
  static __device__ __forceinline__ void finish(const Job& j, const Plan&, const ProductTile& t,
                                                const Accumulator& acc, int row, Share share, int cols,
                                                Ahead& a, const Out& o) {
    if (row >= j.rows) return;
    const int r4 = o.lane >> 2, c4 = o.lane & 3;
#pragma unroll 1
    for (int k = share.first; k < cols; k += share.step) {
      const int n = t.n * cols + k;
      if (n >= j.cols) break;
      o.room();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r4 + 8 * i;
        shared_store16(o.at + r * 64 + ((c4 ^ ((r >> 1) & 3)) << 4), a.next[i].x, a.next[i].y, a.next[i].z,
                       a.next[i].w);
      }
      __syncwarp();
      if (o.real) ask(j, t, row, k + share.step, cols, o.lane, a);
      float v[32];
      acc.load32(k, v);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 u = shared_load16(o.place(0, c));
        const __half* old = reinterpret_cast<const __half*>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& x = v[8 * c + i];
          x = fmaf(j.c * (1.f / kScale), x, j.b * __half2float(old[i]));
          if (row + o.lane == n + 8 * c + i) x += j.a * kScale;
        }
      }
      __syncwarp();
      send_symmetric(j, t, v, row, n, o);
    }
  }
};

template <bool kTall>
struct Update {
  using Job = OrthoJob;
  static constexpr bool kAMn = false, kBMn = !kTall, kFp16 = true, kCounted = false, kHeld = false;
  using Ahead = None;
  static __device__ __forceinline__ None ahead(const Job&, const Plan&, const ProductTile&, int, Share, int, int) {
    return {};
  }
  static __device__ __forceinline__ void finish(const Job& j, const Plan&, const ProductTile& t,
                                                const Accumulator& acc, int row, Share share, int cols, None,
                                                const Out& o) {
    const int rows = max(0, min(32, j.rows - row));
    if (rows == 0) return;
    if (j.boxes) {
#pragma unroll 1
      for (int k = share.first, box = 0; k < cols; k += share.step, box ^= 1) {
        if (t.n * cols + k >= j.cols) break;
        float v[32];
        acc.load32(k, v);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = j.last ? pack_bf16x2(v[2 * i] * j.factor * j.scale, v[2 * i + 1] * j.factor * j.scale)
                        : pack_half2(v[2 * i] * j.factor, v[2 * i + 1] * j.factor);
        if (box == 0) o.room();
        o.put(box, w);
        o.send(box, t.n * cols + k, row, t.z);
      }
      return;
    }
    if (!o.real) return;
    // the caller's matrix, off 16 bytes
    bf16* last = j.last + t.z * j.step_last + row * j.ld_last;
    // 16 columns at a time, both halves of each 32
#pragma unroll 1
    for (int k = share.first; k < cols; k += k & kCols ? share.step - kCols : kCols) {
      const int64_t n = (int64_t)t.n * cols + k;
      const int left = (int)min((int64_t)kCols, j.cols - n);
      if (left <= 0) break;
      float v[kCols];
      acc.load(k, v);
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = v[i] * j.factor * j.scale;
      store_rows(last + n, j.ld_last, false, v, rows, left, o.words, o.lane);
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------ the host's side
// Rows a power of two apart would meet in few of L2's slices.
int64_t ld_of(int64_t cols) {
  const int64_t n = up_to(cols, 64);
  return n % 2048 ? n : n + 64;
}

// Threads for a row of the first two kernels: eight values each, or more.
int lanes_of(int64_t cols) {
  int n = 8;
  while (n < 256 && n * 8 < cols) n *= 2;
  return n;
}

// Their CTAs for a matrix: four for each of 152 SMs in all, or more where there are
// more matrices.
int64_t parts_of(int64_t count, int64_t rows, int64_t cols) {
  const int64_t n = over(4 * 152, count), most = over(rows, 256 / lanes_of(cols));
  return n < most ? n : most;
}

// Parts of A's sum.  The tensor cores cut their sums off instead of rounding them: 16 terms
// at a time leave A low by 2^-26 of itself or more each, 2^18 terms by as much as rounding
// A to fp16 (in one part, A was 0.6 % low at 2^22 and five steps 2.4 % off, at 2^24 2.3 and
// 8.7 %).  Longer sums are made in parts of 2^16 terms, or of 2^18 where A has tiles enough
// by itself and its parts take memory.
int64_t gram_splits(int64_t rows, int64_t cols) {
  const int64_t k = rows > cols ? rows : cols, m = rows > cols ? cols : rows;
  return k <= 1 << 18 ? 1 : over(k, m <= 1024 ? 1 << 16 : 1 << 18);
}

struct Layout {
  size_t sums, x[2], a, b, gram, total;
  int64_t ld_x, rows_padded, m, ld_m, parts, splits, ld_gram;
};

Layout layout(int64_t count, int64_t rows, int64_t cols) {
  Layout l = {};
  size_t at = 256;  // the status word
  auto take = [&at](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  l.ld_x = ld_of(cols);
  l.rows_padded = up_to(rows, 64);
  l.m = rows < cols ? rows : cols;
  l.ld_m = ld_of(l.m);
  l.parts = parts_of(count > 0 ? count : 1, rows, cols);
  l.sums = take((size_t)(count * l.parts) * sizeof(double));
  for (size_t& x : l.x) x = take((size_t)(count * l.rows_padded) * l.ld_x * 2);
  l.a = take((size_t)(count * l.m) * l.ld_m * 2);
  l.b = take((size_t)(count * l.m) * l.ld_m * 2);
  l.splits = gram_splits(rows, cols);
  l.ld_gram = up_to(l.m, 4);
  if (l.splits > 1) l.gram = take((size_t)(l.splits * count * l.m) * l.ld_gram * 4);
  l.total = at;
  return l;
}

template <bool kTall>
zr_status steps(const OrthoArgs& a, const Input& in, bool f32, const Layout& l, char* ws,
                cudaStream_t stream) {
  const CUtensorMapDataType half = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  __half *sym_a = reinterpret_cast<__half*>(ws + l.a), *sym_b = reinterpret_cast<__half*>(ws + l.b);
  __half* x[2] = {in.x0, in.x1};
  const int64_t gram_blocks = kTall ? l.rows_padded / kDepth : over(a.cols, kDepth);
  const int64_t m_blocks = over(l.m, kDepth);
  OrthoJob sym = {};
  sym.count = (int)a.count;
  sym.status = reinterpret_cast<int32_t*>(ws);
  sym.ld = l.ld_m;
  sym.step = l.m * l.ld_m;
  sym.rows = sym.cols = (int)l.m;
  sym.symmetric = 1;
  OrthoJob gram = sym, square = sym, update = sym;
  Cut cut_gram = best_cut(l.m, l.m, over(gram_blocks, l.splits), a.count, true, 20, 0, l.splits == 1);
  cut_gram.splits = (int)l.splits;
  apply_cut(gram, cut_gram, l.m, l.m, gram_blocks);
  gram.a_rows = gram.b_rows = (int)l.rows_padded;
  const Cut cut_square = best_cut(l.m, l.m, m_blocks, a.count, true, 20, 0, true);
  apply_cut(square, cut_square, l.m, l.m, m_blocks);
  square.in = sym_a;
  square.a_rows = square.b_rows = (int)l.m;
  const Cut cut_update = best_cut(a.rows, a.cols, m_blocks, a.count, false, 14, 0, true);
  apply_cut(update, cut_update, a.rows, a.cols, m_blocks);
  update.symmetric = 0;
  update.boxes = 1;
  update.a_rows = (int)(kTall ? l.rows_padded : l.m);
  update.b_rows = (int)(kTall ? l.m : l.rows_padded);
  update.rows = (int)a.rows;
  update.cols = (int)a.cols;
  update.factor = 1.f / kScale;

  // X by its rows (k along them) and by its columns, A and B by their rows
  const int64_t x_rows = a.count * l.rows_padded, m_rows = a.count * l.m;
  ProductMaps of_gram[2] = {}, of_square = {}, of_update[2] = {};
  zr_status st = ZR_OK;
  auto rows = [&](CUtensorMap* map, const __half* p, int64_t n, int64_t cols, int64_t ld, int box) {
    if (st == ZR_OK) st = make_map(map, p, n, cols, ld, box, half);
  };
  auto columns = [&](CUtensorMap* map, const __half* p, int64_t n, int64_t cols, int64_t ld, int box) {
    if (st == ZR_OK) st = make_chunk_map(map, p, n, cols, ld, box / 64, half);
  };
  for (int i = 0; i < 2; ++i) {
    if (kTall) {
      columns(&of_gram[i].a, x[i], x_rows, a.cols, l.ld_x, 128);
      columns(&of_gram[i].b, x[i], x_rows, a.cols, l.ld_x, cut_gram.width);
      rows(&of_update[i].a, x[i], x_rows, a.cols, l.ld_x, 128);
      rows(&of_update[i].b, sym_b, m_rows, l.m, l.ld_m, cut_update.width);
    } else {
      rows(&of_gram[i].a, x[i], x_rows, a.cols, l.ld_x, 128);
      rows(&of_gram[i].b, x[i], x_rows, a.cols, l.ld_x, cut_gram.width);
      rows(&of_update[i].a, sym_b, m_rows, l.m, l.ld_m, 128);
      columns(&of_update[i].b, x[i], x_rows, a.cols, l.ld_x, cut_update.width);
    }
  }
  auto out = [&](CUtensorMap* map, const __half* p, int64_t n, int64_t cols, int64_t ld, int64_t step) {
    if (st == ZR_OK) st = make_store_map(map, p, n, cols, ld, a.count, step, half);
  };
  for (int i = 0; i < 2; ++i) {
    if (l.splits == 1) out(&of_gram[i].out, sym_a, l.m, l.m, l.ld_m, sym.step);
    else if (st == ZR_OK)
      st = make_store_map(&of_gram[i].out, ws + l.gram, l.m, l.m, l.ld_gram, l.splits * a.count,
                          l.m * l.ld_gram, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
    out(&of_update[i].out, x[i ^ 1], a.rows, a.cols, l.ld_x, l.rows_padded * l.ld_x);
  }
  out(&of_square.out, sym_b, l.m, l.m, l.ld_m, sym.step);
  bool last_boxes = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 &&
                    (a.rows == 1 || a.ld_out % 8 == 0) && (a.count == 1 || a.step_out % 8 == 0);
  CUtensorMap of_last = {};
  if (last_boxes)  // (rows or matrices too far apart for a map go one by one)
    last_boxes = make_store_map(&of_last, a.out, a.rows, a.cols, a.rows == 1 ? up_to(a.cols, 8) : a.ld_out,
                                a.count, a.step_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) == ZR_OK;
  rows(&of_square.a, sym_a, m_rows, l.m, l.ld_m, 128);
  rows(&of_square.b, sym_a, m_rows, l.m, l.ld_m, cut_square.width);
  if (st != ZR_OK) return st;

  const GramSum sum = {reinterpret_cast<const float*>(ws + l.gram), sym_a, a.count, l.m, l.ld_gram, l.ld_m,
                       cut_gram.splits, 128 * cut_gram.ctas};
  const unsigned grid = (unsigned)(a.count * in.parts);
  const bool chains = a.cols > kChain;
  const auto norm = f32      ? chains ? ortho_norm_kernel<float, true> : ortho_norm_kernel<float, false>
                    : chains ? ortho_norm_kernel<bf16, true>
                             : ortho_norm_kernel<bf16, false>;
  st = launched(launch_kernel(norm, grid, 256, 0, 1, stream, in));
  if (st == ZR_OK)
    st = f32 ? launched(launch_kernel(ortho_start_kernel<float>, grid, 256, 0, 1, stream, in))
             : launched(launch_kernel(ortho_start_kernel<bf16>, grid, 256, 0, 1, stream, in));
  for (int s = 0; s < a.steps && st == ZR_OK; ++s) {
    const float* k = a.coefficients + 3 * s;
    square.a = k[0];
    square.b = k[1];
    square.c = k[2];
    if (s == a.steps - 1) {
      update.last = static_cast<bf16*>(a.out);
      update.ld_last = a.ld_out;
      update.step_last = a.step_out;
      update.factor = 1.f / (kScale * kScale);
      update.scale = a.scale;
      update.boxes = last_boxes;
      if (last_boxes) of_update[s & 1].out = of_last;
    }
    st = product_launch<Gram<kTall>>(gram, of_gram[s & 1], cut_gram.ctas, l.m, l.m, stream);
    if (st == ZR_OK && l.splits > 1) {
      const int64_t ctas = over(a.count * l.m * l.m, 256);
      st = launched(launch_kernel(ortho_gram_kernel, (unsigned)(ctas < 152 * 16 ? ctas : 152 * 16), 256, 0, 1,
                                  stream, sum));
    }
    if (st == ZR_OK) st = product_launch<Square>(square, of_square, cut_square.ctas, l.m, l.m, stream);
    if (st == ZR_OK)
      st = product_launch<Update<kTall>>(update, of_update[s & 1], cut_update.ctas, a.rows, a.cols, stream);
  }
  return st;
}

}  // namespace

// Whether rows, tiles and CTAs of all matrices can be numbered in 32 bits.  (Then no
// product of a layout's sizes leaves 64.)
bool orthogonalise_fits(int64_t count, int64_t rows, int64_t cols) {
  if (count == 0) return true;
  const int64_t m = rows < cols ? rows : cols;
  return count * up_to(rows, 64) <= INT32_MAX - 512 && cols <= INT32_MAX - 512 &&
         over(rows, 128) * over(cols, 64) <= INT32_MAX / 2 / count &&
         over(m, 128) * over(m, 64) * count <= INT32_MAX / 2 / gram_splits(rows, cols) &&
         count * parts_of(count, rows, cols) <= INT32_MAX;
}

size_t orthogonalise_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
  return orthogonalise_fits(count, rows, cols) ? layout(count, rows, cols).total : 0;
}

zr_status orthogonalise_launch(const OrthoArgs& a, zr_dtype dt, void* ws, cudaStream_t stream) {
  char* w = static_cast<char*>(ws);
  const Layout l = layout(a.count, a.rows, a.cols);
  const size_t elem = dt == ZR_F32 ? 4 : 2;
  Input in = {};
  in.g = a.g;
  in.ld = a.ld_g;
  in.step = a.step_g;
  in.rows = a.rows;
  in.cols = a.cols;
  in.vectors = (reinterpret_cast<uintptr_t>(a.g) & 15) == 0 && a.cols * elem % 16 == 0 &&
               (a.rows == 1 || a.ld_g * elem % 16 == 0) && (a.count == 1 || a.step_g * elem % 16 == 0);
  in.parts = (int)l.parts;
  in.lanes = lanes_of(a.cols);
  in.sums = reinterpret_cast<double*>(w + l.sums);
  in.status = reinterpret_cast<int32_t*>(w);
  in.eps = a.eps;
  in.x0 = reinterpret_cast<__half*>(w + l.x[0]);
  in.x1 = reinterpret_cast<__half*>(w + l.x[1]);
  in.ld_x = l.ld_x;
  in.rows_padded = l.rows_padded;
  return a.rows > a.cols ? steps<true>(a, in, dt == ZR_F32, l, w, stream)
                         : steps<false>(a, in, dt == ZR_F32, l, w, stream);
}

}  // namespace zr
