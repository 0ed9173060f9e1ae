// Cross entropy of token states over a vocabulary, with the gradients of the states
// and of the vocabulary's weights (zr.h has the formulas).  The logits z = x W^T are in
// memory for gradients only, a piece of the rows at a time (up to 4096 + 2 d rows are one
// piece) and in 16 bits, the size of bf16 logits; a loss alone leaves none:
//
//   pack      the rows that have a target, one below the other (so that a row that
//             is left out costs nothing, and what it holds reaches no sum);
//   logits    z of a piece of those rows on the tensor cores.  Each half tile leaves
//             its rows' maxima and sums of exponentials, without the targets, whose
//             logits are kept in fp32, and, where gradients are wanted, the logits
//             themselves in 16 bits: their distances to the maximum, (max - z) log2(e),
//             in steps of 2^-10;
//   rows      log sum exp, the loss and the gradient's factors of each row;
//   weights   dz = w (softmax - one-hot) in bf16 over the 16-bit distances;
//   dx        dz W, over k = vocabulary, in parts that are then added up in order;
//   dw        dz^T x, over k = the piece's rows.
//
// Distances of 2^-10 in the power give each probability to 3.4e-4 of itself over 64
// octaves, whatever its size (16-bit floats of the logits would give 0.03, of the
// probabilities 0 below 2^-24); dz is then rounded to bf16, 3.9e-3 at most, because it
// is an operand of the tensor cores.  It is held in units of the largest weight, which
// is multiplied in with the fp32 sums: where all weights are alike (a mean over tokens),
// a target's p - 1 near -1 is then rounded by little, and not by the weight's own digits,
// the same in every row.  The target's own dz, where the difference to 1 counts, is made
// from its fp32 logit.  Three products for the flops of three; making the logits again,
// once the sums are known, would be a fourth.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "product.cuh"
#include "zr.h"

namespace zr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSteps = 1024.f;       // of the distances, to an octave
constexpr uint32_t kFarthest = 65535;  // a distance that stands for probability 0
constexpr float kMagic = 8388608.f;    // 2^23: an integer's bits in a float's

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's numbers for its gradient, in units of the largest weight.
struct RowInfo {
  float max, log2_sum;
  float weight;     // NaN where the row's logits are not numbers; 0: no gradient
  float of_target;  // the gradient of the target's logit
};

// The workspace's first words.
struct Head {
  int32_t status, packed;  // rows with a target
  float unit;              // the largest weight's size
};

// What all kernels of a call are given.
struct Ce {
  CeArgs a;
  Head* head;
  int32_t* map;      // [rows] packed row -> row
  int32_t* target;   // [rows] packed
  float* weight;     // [rows] packed
  bf16* xp;          // [rows up to 64, ld_xp: d up to 64] packed
  int64_t ld_xp;
  float* on;         // [piece] the target's logit
  RowInfo* info;     // [piece]
  float2* stats;     // [n_stats, piece] maxima and sums of half tiles: rows beside one
                     // another (the other way they met in few of L2's slices, and a tile
                     // took 13 us instead of 9, whatever its depth)
  int n_stats, half;  // columns of a half tile
  uint16_t* dist;    // [piece, ld_z]: distances, then dz
  int64_t ld_z;
  float* dx_parts;   // [splits, piece, ld_dxp]
  int64_t ld_dxp;
  float* dw_sum;     // [vocab, ld_dws], where there are several pieces
  int64_t ld_dws;
  int64_t first;     // packed rows before the piece
  int64_t piece;     // rows of a piece
  int splits;        // of dx
};

// Rows of the piece.
__device__ __forceinline__ int rows_here(const Ce& c) {
  const int64_t n = (int64_t)c.head->packed - c.first;
  return (int)(n < 0 ? 0 : n < c.piece ? n : c.piece);
}

// ------------------------------------------------------------ pack
constexpr int kPackThreads = 256;

__device__ __forceinline__ bool has_target(const CeArgs& a, int64_t r, bool* bad, float* unit) {
  const int32_t t = a.target[r];
  if (t >= a.vocab) *bad = true;
  if (t < 0 || t >= a.vocab) return false;
  const float w = a.weight ? fabsf(a.weight[r]) : 1.f;
  if (w < INFINITY) *unit = fmaxf(*unit, w);
  return w != 0.f;
}

// A row of d values to 128-byte boundaries, zeros up to ld.
__device__ __forceinline__ void copy_row(const uint16_t* in, uint16_t* out, int64_t d, int64_t ld,
                                         bool vectors, int lane) {
  if (vectors) {
    for (int64_t i = lane; i < ld / 8; i += 32) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (i < d / 8) v = reinterpret_cast<const uint4*>(in)[i];
      reinterpret_cast<uint4*>(out)[i] = v;
    }
    return;
  }
  int64_t i = lane;
  for (; i + 7 * 32 < d; i += 8 * 32) {  // all loads first: their latency is what this takes
    uint16_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = in[i + k * 32];
#pragma unroll
    for (int k = 0; k < 8; ++k) out[i + k * 32] = x[k];
  }
#pragma unroll 8
  for (; i < ld; i += 32) out[i] = i < d ? in[i] : (uint16_t)0;
}

// Each CTA counts the rows with a target before its own ones, and copies those that
// have one behind them.  (Counting reads 8 bytes a row out of L2: at 8192 rows 10 MB
// for all CTAs.)  The last one has seen all rows.  Latency bounds it: 2048 x 1024 take 9 us
// from cold caches.
__global__ void __launch_bounds__(kPackThreads) ce_pack_kernel(const Ce c, int64_t per_cta) {
  __shared__ int32_t sums[kPackThreads / 32], slot[kPackThreads];
  __shared__ float units[kPackThreads / 32];
  __shared__ int any_bad;
  const CeArgs& a = c.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_start();
  wait_for_kernels_before();
  const int64_t lo = blockIdx.x * per_cta;
  const int64_t hi = lo + per_cta < a.rows ? lo + per_cta : a.rows;
  if (tid == 0) any_bad = 0;
  __syncthreads();
  bool bad = false;
  float unit = 0.f;
  int32_t n = 0;
  for (int64_t r = tid; r < lo; r += kPackThreads) n += has_target(a, r, &bad, &unit);
  n = __reduce_add_sync(~0u, n);
  if (lane == 0) sums[warp] = n;
  __syncthreads();
  int32_t base = 0;
  for (int w = 0; w < kPackThreads / 32; ++w) base += sums[w];
  const bool vectors = a.d % 8 == 0 && on16(a.x, a.ld_x);
  for (int64_t r0 = lo; r0 < hi; r0 += kPackThreads) {
    const int64_t r = r0 + tid;
    const bool mine = r < hi && has_target(a, r, &bad, &unit);
    const uint32_t votes = __ballot_sync(~0u, mine);
    __syncthreads();
    if (lane == 0) sums[warp] = __popc(votes);
    __syncthreads();
    int32_t at = base;
    for (int w = 0; w < kPackThreads / 32; ++w) {
      if (w < warp) at += sums[w];
      base += sums[w];
    }
    at += __popc(votes & ((1u << lane) - 1));
    slot[tid] = mine ? at : -1;
    if (mine) {
      c.map[at] = (int32_t)r;
      c.target[at] = a.target[r];
      c.weight[at] = a.weight ? a.weight[r] : 1.f;
    } else if (r < hi) {
      if (a.loss) a.loss[r] = 0.f;
      if (a.lse) a.lse[r] = 0.f;
    }
    __syncthreads();
    const int here = (int)(hi - r0 < kPackThreads ? hi - r0 : kPackThreads);
    for (int i = warp; i < here; i += kPackThreads / 32) {
      const uint16_t* in = static_cast<const uint16_t*>(a.x) + (r0 + i) * a.ld_x;
      if (slot[i] >= 0) {
        copy_row(in, reinterpret_cast<uint16_t*>(c.xp) + slot[i] * c.ld_xp, a.d, c.ld_xp, vectors, lane);
      } else if (a.dx) {
        uint16_t* out = static_cast<uint16_t*>(a.dx) + (r0 + i) * a.ld_dx;
        for (int64_t k = lane; k < a.d; k += 32) out[k] = 0;
      }
    }
  }
  if (blockIdx.x != gridDim.x - 1) return;
  // rows up to a whole step of k are zeros
  for (int64_t r = base + warp; r < ((int64_t)base + 63) / 64 * 64; r += kPackThreads / 32)
    for (int64_t i = lane; i < c.ld_xp / 8; i += 32)
      reinterpret_cast<uint4*>(c.xp + r * c.ld_xp)[i] = make_uint4(0, 0, 0, 0);
  if (bad) any_bad = 1;
#pragma unroll
  for (int o = 16; o; o >>= 1) unit = fmaxf(unit, __shfl_xor_sync(~0u, unit, o));
  if (lane == 0) units[warp] = unit;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kPackThreads / 32; ++w) unit = fmaxf(unit, units[w]);
    c.head->status = any_bad ? ZR_ERR_INVALID_ARG : ZR_OK;
    c.head->packed = base;
    c.head->unit = unit > 0.f ? unit : 1.f;
  }
}

// ------------------------------------------------------------ logits
// Two fp32 at a time (one instruction on sm_103a).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Every thread has half a tile's columns of one row in registers: the maximum, then
// the powers (four a cycle and quarter of an SM; with the rest of the epilogue 2500 cycles
// and 13 a column, hidden behind the next tile's products from d = 600 on).  2048 x 65536
// at d = 1024: the whole call without gradients takes 148 us, the products alone 126 at
// the tensor cores' best rate.
struct Logits {
  struct Job : Product {
    Ce c;
  };
  static constexpr bool kAMn = false, kBMn = false, kFp16 = false, kCounted = true, kHeld = true;
  template <int kCtas>
  static __device__ __forceinline__ Plan plan(const Job& j) {
    const int rows = rows_here(j.c), m_tiles = (rows + kCtas * 128 - 1) / (kCtas * 128);
    return {m_tiles, j.k_blocks, m_tiles * j.n_tiles, rows};
  }
  using Ahead = int32_t;  // the row's target
  static __device__ __forceinline__ Ahead ahead(const Job& j, const Plan& p, const ProductTile&, int row,
                                                Share, int, int lane) {
    return row + lane < p.rows ? j.c.target[j.c.first + row + lane] : -1;
  }
  // Rows past the last one go along: what they leave in `dist` is either overwritten with
  // zeros or never read.
  static __device__ __forceinline__ void finish(const Job& j, const Plan& p, const ProductTile& t,
                                                float* v, int row, int part, int half,
                                                Ahead target, const Out& o) {
    const Ce& c = j.c;
    const int r = row + o.lane;
    const bool mine = r < p.rows;
    const int64_t n0 = ((int64_t)t.n * 2 + part) * half;
    const int64_t on = target - n0;
    if (row >= p.rows) return;  // the whole warp's
    if (on >= 0 && on < half) {
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (on == i) c.on[r] = v[i], v[i] = -INFINITY;  // (the rows' kernel adds it)
    }
    __syncwarp();
    if (n0 + half > c.a.vocab) {
      const int left = (int)(c.a.vocab - n0);  // columns that exist
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (i >= left) v[i] = -INFINITY;
    }
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < 128; k += 32) {
      if (k >= half) break;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = fmaxf(m, v[k + i]);
    }
    // nothing but -inf: any finite reference leaves the powers 0
    const float2 ref = both(m == -INFINITY ? 0.f : -m);
    float2 sum = both(0.f);
#pragma unroll
    for (int k = 0; k < 128; k += 32) {
      if (k >= half) break;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        // octaves below the maximum, as negative numbers
        const float2 d = mul2(add2(make_float2(v[k + i], v[k + i + 1]), ref), both(kLog2e));
        sum = add2(sum, make_float2(ex2(d.x), ex2(d.y)));
        const float2 q = fma2(d, both(-kSteps), both(kMagic));
        w[i / 2] = __byte_perm(__float_as_uint(fminf(q.x, kMagic + 65535.f)),
                               __float_as_uint(fminf(q.y, kMagic + 65535.f)), 0x5410);
      }
      if (c.dist && n0 + k < c.ld_z) {
        if (k % 64 == 0) o.room();
        o.put_half(k / 32 & 1, w);
        if (k % 64) o.send(0, (int)(n0 + k - 32), row, 0);
      }
    }
    if (mine) c.stats[(2 * t.n + part) * c.piece + r] = make_float2(m, sum.x + sum.y);
  }
};

// ------------------------------------------------------------ rows
// 32 rows a CTA: its warps take the half tiles in turn, a lane for each row.  8 bytes a half
// tile and row; latency bounds it (2048 rows of 512 half tiles 8.5 us from cold caches).
constexpr int kRowWarps = 32;

__global__ void __launch_bounds__(32 * kRowWarps) ce_rows_kernel(const Ce c) {
  __shared__ float words[kRowWarps][32];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = rows_here(c);
  const int64_t r = blockIdx.x * 32ll + lane;
  if (blockIdx.x * 32ll >= rows) return;
  const float2* s = c.stats + (r < rows ? r : rows - 1);
  // one pass, eight half tiles at a time: a running maximum and the sum below it
  float m = -INFINITY, sum = 0.f;
  for (int i = warp; i < c.n_stats; i += 8 * kRowWarps) {
    float2 x[8];
    float top = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = i + k * kRowWarps;
      x[k] = at < c.n_stats ? s[at * c.piece] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, x[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    sum = m == top ? sum : sum * exp2f((m - ref) * kLog2e);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(x[k].y, exp2f((x[k].x - ref) * kLog2e), sum);
    m = top;
  }
  words[warp][lane] = m;
  __syncthreads();
  const float own = m;
#pragma unroll
  for (int i = 0; i < kRowWarps; ++i) m = fmaxf(m, words[i][lane]);
  __syncthreads();
  const float ref = m == -INFINITY ? 0.f : m;
  if (own != m) sum *= exp2f((own - ref) * kLog2e);
  words[warp][lane] = sum;
  __syncthreads();
  if (warp || r >= rows) return;
#pragma unroll
  for (int i = 1; i < kRowWarps; ++i) sum += words[i][lane];
  const int64_t packed = c.first + r, row = c.map[packed];
  const float w = c.weight[packed];
  // The target is not among the sums so far: with it among them, what is left of 1 when
  // its probability is near 1 would be their rounding.
  const float on = c.on[r], top = fmaxf(m, on);
  RowInfo info = {top, 0.f, 0.f, 0.f};
  float loss = 0.f, lse = 0.f;
  if (sum != 0.f || on != -INFINITY) {  // (else all its logits are -inf: left out)
    const bool first = on >= m;
    const float others = first ? sum * expf(m - on) : sum;
    const float all = first ? 1.f + others : others + expf(on - m);
    const float log_sum = first ? log1pf(others) : logf(all);
    const float log_p = on - top - log_sum;
    info.log2_sum = log2f(all);
    info.weight = w / c.head->unit;
    info.of_target = info.weight * expm1f(log_p);
    lse = top + log_sum;
    loss = -w * log_p;
    if (isnan(lse) || lse == INFINITY) loss = lse = info.weight = info.of_target = NAN;
  }
  if (c.a.loss) c.a.loss[row] = loss;
  if (c.a.lse) c.a.lse[row] = lse;
  c.info[r] = info;
}

// ------------------------------------------------------------ weights
// dz over the distances, eight at a time.  4 bytes of memory traffic a logit bound it
// once its instructions are few: 2048 x 65536 take 82 us (6.5 TB/s), and took 100 when
// each power had its own subtraction, scale and look for the target, and the loads waited
// for the row's numbers.  So the power's constant goes in steps of the distances, which
// makes its argument one exact multiply-add with the integer still in the low bits of a
// float; the rest of the constant, under half a step, goes into the weight.
constexpr int kDzColumns = 8192;  // of a CTA

__global__ void __launch_bounds__(256) ce_dz_kernel(const Ce c, int chunks) {
  let_next_kernel_start();
  wait_for_kernels_before();
  const int r = (int)(blockIdx.x / (unsigned)chunks);
  const int64_t n0 = (int64_t)(blockIdx.x - (unsigned)r * (unsigned)chunks) * kDzColumns + threadIdx.x * 8;
  const int rows = rows_here(c);
  if (r >= (rows + 63) / 64 * 64) return;
  uint16_t* z = c.dist + r * c.ld_z;
  RowInfo info = {};
  if (r < rows) info = c.info[r];
  const int64_t on = r < rows ? c.target[c.first + r] : -1;
  const float2* stats = c.stats + r;
  const int half_bits = __ffs(c.half) - 1;  // (a power of two)
  constexpr int kUnits = kDzColumns / 2048;
  uint4 v[kUnits];
  float off[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {  // all loads first
    const int64_t n = n0 + u * 2048;
    v[u] = make_uint4(0, 0, 0, 0);
    off[u] = 0.f;
    if (r < rows && n < c.a.vocab) {
      v[u] = *reinterpret_cast<const uint4*>(z + n);
      off[u] = stats[(n >> half_bits) * c.piece].x;
    }
  }
  // (a row past the last, or one without any mass, is zeros)
  const bool any = info.weight != 0.f;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t n = n0 + u * 2048;
    if (n >= c.a.vocab) break;
    if (!any) v[u] = make_uint4(0, 0, 0, 0);
    else {
      // (octaves; what is 1000 or infinitely many below the maximum is 0 all the same)
      const float base = fmaxf((off[u] - info.max) * kLog2e - info.log2_sum, -1000.f);
      const float in_steps = rintf(base * kSteps) / kSteps;
      const float2 start = both(in_steps + kMagic / kSteps), scale = both(info.weight * ex2(base - in_steps));
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = make_float2(__uint_as_float(__byte_perm(w[i], 0x4B000000, 0x7610)),
                                     __uint_as_float(__byte_perm(w[i], 0x4B000000, 0x7632)));
        const float2 d = fma2(q, both(-1.f / kSteps), start);
        const float p0 = q.x == kMagic + kFarthest ? 0.f : ex2(d.x);
        const float p1 = q.y == kMagic + kFarthest ? 0.f : ex2(d.y);
        const float2 g = mul2(make_float2(p0, p1), scale);  // (NaN stays in a row that is NaN)
        w[i] = pack_bf16x2(g.x, g.y);
      }
      const int64_t at = on - n;
      if (at >= 0 && at < 8) {
        const uint32_t x = pack_bf16x2(info.of_target, info.of_target);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at >> 1 == i) w[i] = at & 1 ? __byte_perm(w[i], x, 0x7610) : __byte_perm(w[i], x, 0x3254);
      }
    }
    *reinterpret_cast<uint4*>(z + n) = v[u];
  }
  // A row all of whose logits are -inf may have got them from states that are infinite:
  // zeros of dz times those would be NaN in dW.
  if (!any && r < rows && c.a.dw && n0 < kDzColumns) {
    uint4* x = reinterpret_cast<uint4*>(c.xp + (c.first + r) * c.ld_xp);
    for (int64_t i = threadIdx.x; i < c.ld_xp / 8; i += 256) x[i] = make_uint4(0, 0, 0, 0);
  }
}

// ------------------------------------------------------------ gradients
// Both are bound by the tensor cores: 2048 x 65536 x 1024 takes 151 us for dx and 150 for
// dw, the tensor pipe active 84 and 85 % of them.  dx has few tiles and a long k, which is
// cut until the tiles fill the GPU; dw has many tiles and a short k.
struct StatesGradient {
  struct Job : Product {
    Ce c;
  };
  static constexpr bool kAMn = false, kBMn = true, kFp16 = false, kCounted = true, kHeld = false;
  using Ahead = None;
  static __device__ __forceinline__ None ahead(const Job&, const Plan&, const ProductTile&, int, Share, int, int) {
    return {};
  }
  template <int kCtas>
  static __device__ __forceinline__ Plan plan(const Job& j) {
    const int rows = rows_here(j.c), m_tiles = (rows + kCtas * 128 - 1) / (kCtas * 128);
    return {m_tiles, j.k_blocks, m_tiles * j.n_tiles * j.splits, rows};
  }
  static __device__ __forceinline__ void finish(const Job& j, const Plan& p, const ProductTile& t,
                                                const Accumulator& acc, int row, Share share, int cols, None,
                                                const Out& o) {
    if (row >= p.rows) return;
#pragma unroll 1
    for (int k = share.first; k < cols; k += share.step) {
      const int n = t.n * cols + k;
      if (n >= j.c.a.d) break;
      float v[32];
      acc.load32(k, v);
      o.room();
      o.put_wide(v);
      o.send(0, n, row, t.split);
    }
  }
};

// The parts of k in their order, to the rows that the packed ones came from.  Many
// parts (of few rows) are added up by the CTA's eight warps, an eighth each (kMany), few
// by the thread that stores them.
template <bool kMany>
__global__ void __launch_bounds__(256) ce_dx_kernel(const Ce c) {
  __shared__ float4 sums[kMany ? 8 : 1][32];
  let_next_kernel_start();
  wait_for_kernels_before();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per_row = c.ld_dxp / 4;
  const int64_t i = kMany ? blockIdx.x * 32ll + lane : blockIdx.x * 256ll + threadIdx.x;
  const int64_t r = i / per_row, n = (i - r * per_row) * 4;
  const bool there = r < rows_here(c);
  const float* p = c.dx_parts + r * c.ld_dxp + n;
  const int lo_part = kMany ? c.splits * warp / 8 : 0, hi_part = kMany ? c.splits * (warp + 1) / 8 : c.splits;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (there) {
    v = *reinterpret_cast<const float4*>(p + (int64_t)lo_part * c.piece * c.ld_dxp);
#pragma unroll 8
    for (int s = lo_part + 1; s < hi_part; ++s) {
      const float4 u = *reinterpret_cast<const float4*>(p + (int64_t)s * c.piece * c.ld_dxp);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
  }
  if (kMany) {
    sums[warp][lane] = v;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 u = sums[w][lane];
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
  }
  if (!there) return;
  // (a row without any mass, whatever W holds)
  if (c.info[r].weight == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
  const float unit = c.head->unit;
  const uint32_t lo = pack_bf16x2(v.x * unit, v.y * unit), hi = pack_bf16x2(v.z * unit, v.w * unit);
  uint16_t* out = static_cast<uint16_t*>(c.a.dx) + c.map[c.first + r] * c.a.ld_dx + n;
  if (c.a.ld_dx % 4 == 0 && (reinterpret_cast<uintptr_t>(c.a.dx) & 7) == 0 && n + 4 <= c.a.d) {
    *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    return;
  }
  const uint16_t x[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n + k < c.a.d) out[k] = x[k];
}

struct WeightsGradient {
  struct Job : Product {
    Ce c;
    int first_piece, last_piece;
    int boxes;  // dw goes as boxes: it is written, whole, and lies on 16 bytes
  };
  static constexpr bool kAMn = true, kBMn = true, kFp16 = false, kCounted = true, kHeld = false;
  using Ahead = None;
  static __device__ __forceinline__ None ahead(const Job&, const Plan&, const ProductTile&, int, Share, int, int) {
    return {};
  }
  template <int kCtas>
  static __device__ __forceinline__ Plan plan(const Job& j) {
    return {j.m_tiles, (rows_here(j.c) + kDepth - 1) / kDepth, j.m_tiles * j.n_tiles, 0};
  }
  static __device__ __forceinline__ void finish(const Job& j, const Plan&, const ProductTile& t,
                                                const Accumulator& acc, int row, Share share, int cols, None,
                                                const Out& o) {
    const Ce& c = j.c;
    const int rows = (int)max((int64_t)0, min((int64_t)32, c.a.vocab - row));
    if (rows == 0) return;
    const float unit = c.head->unit;
    if (j.boxes) {
#pragma unroll 1
      // (rows of 64 columns: 79992 x 2608 of 111 rows 122 us, in boxes of 32 columns 135)
      for (int k = 2 * share.first; k < cols; k += 2 * share.step) {
        if ((int64_t)t.n * cols + k >= c.a.d) break;
        o.room();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float v[32];
          acc.load32(k + 32 * half, v);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i] * unit, v[2 * i + 1] * unit);
          o.put_half(half, w);
        }
        o.send(0, t.n * cols + k, row, 0);
      }
      return;
    }
    if (!o.real) return;
    uint32_t* stage = o.words;
    const int lane = o.lane;
    bf16* out = static_cast<bf16*>(c.a.dw) + row * c.a.ld_dw;
    const bool fast = on16(c.a.dw, c.a.ld_dw);
    // 16 columns at a time, both halves of each 32
#pragma unroll 1
    for (int k = share.first; k < cols; k += k & kCols ? share.step - kCols : kCols) {
      const int64_t n = (int64_t)t.n * cols + k;
      const int left = (int)min((int64_t)kCols, c.a.d - n);
      if (left <= 0) break;
      float v[kCols];
      acc.load(k, v);
      if (c.dw_sum) {  // fp32 sums over the pieces
        float4* sum = reinterpret_cast<float4*>(c.dw_sum + (int64_t)(row + lane) * c.ld_dws + n);
        if (lane < rows) {
#pragma unroll
          for (int i = 0; i < kCols; i += 4) {
            if (n + i >= c.ld_dws) break;
            if (!j.first_piece) {
              const float4 u = sum[i / 4];
              v[i] += u.x, v[i + 1] += u.y, v[i + 2] += u.z, v[i + 3] += u.w;
            }
            if (!j.last_piece) sum[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
        __syncwarp();
        if (!j.last_piece) continue;
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] *= unit;
      if (c.a.accumulate) {
        float old[kCols];
        load_rows(out + n, c.a.ld_dw, fast, old, rows, left, stage, lane);
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] += old[i];
      }
      store_rows(out + n, c.a.ld_dw, fast, v, rows, left, stage, lane);
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------ the host's side
// Rows of a piece.  One piece holds all rows while that takes no more memory than
// pieces of 4096 rows, which need fp32 sums of dw between them: 2 rows vocab bytes of
// distances against (2 x 4096 + 4 d) vocab.  Without gradients only the half tiles'
// numbers grow with the rows.
constexpr int64_t kMostTerms = 1 << 18;  // of a sum of the tensor cores
int64_t piece_rows(int64_t rows, int64_t d, bool dw, bool grad) {
  int64_t most = !grad ? 16384 : dw ? 4096 + 2 * d : 4096;
  if (most > kMostTerms) most = kMostTerms;  // (dw's terms are a piece's rows)
  return rows <= most ? up_to(rows > 0 ? rows : 1, 256) : !grad ? 16384 : 4096;
}

// Rows of logits a power of two apart would meet in few of L2's slices.
int64_t ld_of_logits(int64_t vocab) {
  const int64_t n = up_to(vocab, 64);
  return n % 2048 ? n : n + 64;
}

struct Layout {
  size_t map, target, weight, xp, wp, on, info, stats, dist, dx_parts, dw_sum, total;
  int64_t ld_xp, ld_w, piece, pieces;
  Cut logits, dx, dw;
  int n_stats;
};

Layout make_layout(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w, bool dx, bool dw) {
  Layout l = {};
  size_t at = 256;  // Head
  auto take = [&at](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const bool grad = dx || dw;
  l.piece = piece_rows(rows, d, dw, grad);
  l.pieces = rows > 0 ? over(rows, l.piece) : 1;
  l.ld_xp = up_to(d, 64);
  l.ld_w = ld_w;
  const int64_t d_blocks = over(d, kDepth), v_blocks = over(vocab, kDepth);
  const int64_t one = rows < l.piece ? (rows > 0 ? rows : 1) : l.piece;
  l.logits = best_cut(one, vocab, d_blocks, 1, false, 13, 0);
  if (l.logits.ctas == 1 && l.logits.width == 64) l.logits.width = 128;  // (half a tile is a box's 64 columns)
  // a part of k of dx: its fp32 sums written and read, at 2800 bytes a cycle (loss and dx of
  // 1000 x 1000 x 50000: 4 parts 202 us, 9 parts 212, 1 part 367)
  l.dx = best_cut(one, d, v_blocks, 1, false, 26, (double)(one * d) * 8 / 2800 + 1);
  // Parts of at most 2^18 terms: the tensor cores cut their sums off, and leave them low by
  // 2^-26 or more for each 16 terms (a mean over 2^21 tokens in one part by 1 %).
  const int64_t parts = over(vocab, kMostTerms);
  if (l.dx.splits < parts) l.dx.splits = (int)parts;
  l.dw = best_cut(vocab, d, over(one, kDepth), 1, false, 26, 0);
  l.n_stats = (int)(2 * over(vocab, l.logits.ctas * l.logits.width));
  l.map = take((size_t)rows * 4);
  l.target = take((size_t)rows * 4);
  l.weight = take((size_t)rows * 4);
  l.xp = take((size_t)up_to(rows, 64) * l.ld_xp * 2);
  if (ld_w % 8) l.wp = take((size_t)vocab * (l.ld_w = up_to(d, 64)) * 2);
  l.on = take((size_t)l.piece * 4);
  l.info = take((size_t)l.piece * sizeof(RowInfo));
  l.stats = take((size_t)l.piece * l.n_stats * sizeof(float2));
  if (grad) l.dist = take((size_t)l.piece * ld_of_logits(vocab) * 2);
  if (dx) l.dx_parts = take((size_t)l.dx.splits * l.piece * up_to(d, 4) * 4);
  if (dw && l.pieces > 1) l.dw_sum = take((size_t)vocab * up_to(d, 4) * 4);
  l.total = at;
  return l;
}

// A training loop asks for the same sizes again and again, and the cut of dx is chosen
// among hundreds (10 of a call's 50 us on the host): the last answer is kept by its sizes.
Layout layout(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w, bool dx, bool dw) {
  struct Kept {
    int64_t rows, d, vocab, ld_w;
    int dx, dw, sms;
    Layout l;
  };
  static thread_local Kept kept = {-1, 0, 0, 0, 0, 0, 0, {}};
  const int sms = sm_count();
  if (kept.rows != rows || kept.d != d || kept.vocab != vocab || kept.ld_w != ld_w || kept.dx != dx ||
      kept.dw != dw || kept.sms != sms)
    kept = {rows, d, vocab, ld_w, dx, dw, sms, make_layout(rows, d, vocab, ld_w, dx, dw)};
  return kept.l;
}

// Of dx: an eighth of them goes to each warp of the kernel that adds them up.
bool many_parts(const Cut& dx) { return dx.splits >= 8; }

}  // namespace

// Whether all CTAs and tiles of a piece can be numbered in 32 bits.  (Then no product of a
// layout's sizes leaves 64.)
bool cross_entropy_fits(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w, int dx, int dw) {
  const Layout l = layout(rows, d, vocab, ld_w, dx, dw);
  const int64_t quads = l.piece * (up_to(d, 4) / 4);
  return l.piece * over(vocab, kDzColumns) <= INT32_MAX &&
         over(quads, many_parts(l.dx) ? 32 : 256) <= INT32_MAX &&
         over(vocab, 128) * over(d, 64) <= INT32_MAX / 2 &&
         over(l.piece, 128) * over(vocab, 64) <= INT32_MAX / 2 &&
         over(l.piece, 128) * over(d, 64) * l.dx.splits <= INT32_MAX / 2 &&
         (l.ld_w == ld_w || over(vocab * (l.ld_w / 8), 256) <= INT32_MAX);
}

size_t cross_entropy_workspace_bytes(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w, int dx,
                                     int dw) {
  return cross_entropy_fits(rows, d, vocab, ld_w, dx, dw) ? layout(rows, d, vocab, ld_w, dx, dw).total : 0;
}

zr_status cross_entropy_launch(const CeArgs& a, void* ws, cudaStream_t stream) {
  const Layout l = layout(a.rows, a.d, a.vocab, a.ld_w, a.dx, a.dw);
  char* w = static_cast<char*>(ws);
  const bool grad = a.dx || a.dw;
  Ce c = {};
  c.a = a;
  c.head = reinterpret_cast<Head*>(w);
  c.map = reinterpret_cast<int32_t*>(w + l.map);
  c.target = reinterpret_cast<int32_t*>(w + l.target);
  c.weight = reinterpret_cast<float*>(w + l.weight);
  c.xp = reinterpret_cast<bf16*>(w + l.xp);
  c.ld_xp = l.ld_xp;
  c.on = reinterpret_cast<float*>(w + l.on);
  c.info = reinterpret_cast<RowInfo*>(w + l.info);
  c.stats = reinterpret_cast<float2*>(w + l.stats);
  c.n_stats = l.n_stats;
  c.half = l.logits.ctas * l.logits.width / 2;
  c.dist = grad ? reinterpret_cast<uint16_t*>(w + l.dist) : nullptr;
  c.ld_z = ld_of_logits(a.vocab);
  c.dx_parts = a.dx ? reinterpret_cast<float*>(w + l.dx_parts) : nullptr;
  c.ld_dxp = up_to(a.d, 4);
  c.dw_sum = l.dw_sum ? reinterpret_cast<float*>(w + l.dw_sum) : nullptr;
  c.ld_dws = up_to(a.d, 4);
  c.piece = l.piece;
  c.splits = l.dx.splits;
  const void* wp = l.wp ? w + l.wp : a.w;
  const bool chunks_of_w = l.wp || a.d % 64 == 0;
  const int64_t d_blocks = over(a.d, kDepth), v_blocks = over(a.vocab, kDepth);
  const int64_t rows64 = up_to(a.rows > 0 ? a.rows : 1, 64);

  const bool many = many_parts(l.dx);
  const int64_t quads = l.piece * (c.ld_dxp / 4);

  const int64_t chunks = over(a.vocab, kDzColumns);
  Copies copies = {};
  copies.cols = a.d;
  copies.ld_out = up_to(a.d, 64);
  if (l.wp)
    copies.c[copies.n++] = {static_cast<const bf16*>(a.w), reinterpret_cast<bf16*>(w + l.wp), a.ld_w,
                            a.vocab};
  const int64_t copy_ctas = over(a.vocab * (copies.ld_out / 8), 256);
  ProductMaps logits = {}, dx = {}, dw = {};
  zr_status st = make_map(&logits.b, wp, a.vocab, a.d, l.ld_w, l.logits.width);
  if (st == ZR_OK && a.dx) {
    st = make_map(&dx.a, c.dist, l.piece, a.vocab, c.ld_z, 128);
    // W's rows by their columns: in one load where its memory goes on to a whole chunk
    if (st == ZR_OK)
      st = chunks_of_w ? make_chunk_map(&dx.b, wp, a.vocab, a.d, l.ld_w, l.dx.width / 64)
                       : make_map(&dx.b, wp, a.vocab, a.d, l.ld_w, 64);
  }
  if (st == ZR_OK && a.dw)
    st = make_chunk_map(&dw.a, c.dist, l.piece, a.vocab, c.ld_z, 2);
  if (st == ZR_OK && grad)
    st = make_store_map(&logits.out, c.dist, l.piece, c.ld_z, c.ld_z, 1, 0, CU_TENSOR_MAP_DATA_TYPE_UINT16, 64);
  if (st == ZR_OK && a.dx)
    st = make_store_map(&dx.out, c.dx_parts, l.piece, c.ld_dxp, c.ld_dxp, l.dx.splits, l.piece * c.ld_dxp,
                        CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
  bool dw_boxes = a.dw && !a.accumulate && l.pieces == 1 && a.ld_dw % 8 == 0 &&
                        (reinterpret_cast<uintptr_t>(a.dw) & 15) == 0;
  // (rows too far apart for a map go one by one)
  if (dw_boxes)
    dw_boxes = make_store_map(&dw.out, a.dw, a.vocab, a.d, a.ld_dw, 1, 0,
                              CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 64) == ZR_OK;
  if (st == ZR_OK) st = make_map(&logits.a, c.xp, rows64, a.d, c.ld_xp, 128);
  if (st == ZR_OK && a.dw) st = make_chunk_map(&dw.b, c.xp, rows64, a.d, c.ld_xp, l.dw.width / 64);
  if (st != ZR_OK) return st;

  const int64_t share = over(a.rows, 4 * (int64_t)sm_count());
  const int64_t per_cta = share < 8 ? 8 : share;
  const int64_t packers = a.rows > 0 ? over(a.rows, per_cta) : 1;
  st = launched(launch_kernel(ce_pack_kernel, (unsigned)packers, kPackThreads, 0, 1, stream, c, per_cta));
  if (st == ZR_OK && l.wp)
    st = launched(launch_kernel(layout_kernel, (unsigned)copy_ctas, 256, 0, 1, stream, copies));

  for (int64_t p = 0; st == ZR_OK && p < l.pieces; ++p) {
    c.first = p * l.piece;
    // the piece's packed rows; what lies past the last one's step reads as 0
    const int64_t rest = rows64 - c.first;
    const int64_t in_piece = rest < l.piece ? rest : l.piece;
    if (l.pieces > 1) st = make_map(&logits.a, c.xp + c.first * c.ld_xp, in_piece, a.d, c.ld_xp, 128);
    if (st == ZR_OK && l.pieces > 1 && a.dw)
      st = make_chunk_map(&dw.b, c.xp + c.first * c.ld_xp, in_piece, a.d, c.ld_xp, l.dw.width / 64);
    if (st == ZR_OK) {
      Logits::Job j = {};
      j.count = 1;
      apply_cut(j, l.logits, l.piece, a.vocab, d_blocks);
      j.c = c;
      j.status = &c.head->status;
      st = product_launch<Logits>(j, logits, l.logits.ctas, l.piece, a.vocab, stream);
    }
    if (st == ZR_OK)
      st = launched(launch_kernel(ce_rows_kernel, (unsigned)over(l.piece, 32), 32 * kRowWarps, 0, 1, stream, c));
    if (st == ZR_OK && grad)
      st = launched(launch_kernel(ce_dz_kernel, (unsigned)(l.piece * chunks), 256, 0, 1, stream, c,
                                  (int)chunks));
    if (st == ZR_OK && a.dx) {
      StatesGradient::Job j = {};
      j.count = 1;
      apply_cut(j, l.dx, l.piece, a.d, v_blocks);
      if (!chunks_of_w) j.b_boxes = l.dx.width / 64;
      j.c = c;
      j.status = &c.head->status;
      st = product_launch<StatesGradient>(j, dx, l.dx.ctas, l.piece, a.d, stream);
      if (st == ZR_OK)
        st = many ? launched(launch_kernel(ce_dx_kernel<true>, (unsigned)over(quads, 32), 256, 0, 1, stream, c))
                  : launched(launch_kernel(ce_dx_kernel<false>, (unsigned)over(quads, 256), 256, 0, 1, stream, c));
    }
    if (st == ZR_OK && a.dw) {
      WeightsGradient::Job j = {};
      j.count = 1;
      apply_cut(j, l.dw, a.vocab, a.d, over(l.piece, kDepth));
      j.c = c;
      j.status = &c.head->status;
      j.first_piece = p == 0;
      j.last_piece = p == l.pieces - 1;
      j.boxes = dw_boxes;
      st = product_launch<WeightsGradient>(j, dw, l.dw.ctas, a.vocab, a.d, stream);
    }
  }
  return st;
}

}  // namespace zr
