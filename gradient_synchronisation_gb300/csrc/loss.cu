// Losses over a vocabulary with their gradients: distillation from a
// teacher's top logits, the clipped policy loss with a KL term, and the
// preference loss over pairs of sequences (zr.h has the formulas).
//
// All three are the same pass over a row of logits z: with the row's maximum
// M, e_j = exp((z_j - M) / temperature) and Z = sum e_j, the probabilities
// are q_j = e_j / Z and the gradient of the row is
//     dz_j = k0 e_j   for every token j that the row does not list,
// and a value of its own on the tokens that it lists (the teacher's list, or
// the one action or target).  k0 is a number of the row that follows from Z
// and the listed tokens' logits.  What differs is how k0 and the loss follow.
//
// The maximum and the sums are fp32; e_j is 2^((z_j - M) log2(e) /
// temperature), subtracted first so that masks of the type's lowest value
// stay finite.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zr.h"
#include "zr_device.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum class Op { kDistill, kDistillRest, kPolicy, kTarget };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ rows as vectors
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kN = 4;
  using Store = float;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ uint32_t raw(float x) { return __float_as_uint(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kN = 8;
  using Store = __nv_bfloat16;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float x) {
    *p = __float2bfloat16_rn(x);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// A row cut at the 16-byte boundaries of its address: vector v holds the
// elements v*kN - shift .. v*kN - shift + kN - 1 that exist.  Rows may start
// at any element, so the first and last vectors may be partial; those are
// read and written element by element, never past the row.
template <typename T>
struct Row {
  static constexpr int kN = Elem<T>::kN;
  const T* z;
  T* dz;
  int vocab, shift, vectors;
  bool same;  // dz has z's alignment: whole vectors can be stored

  __device__ __forceinline__ Row(const void* z_, int64_t ld, void* dz_, int64_t ldd, int64_t t,
                                 int vocab_) {
    z = static_cast<const T*>(z_) + t * ld;
    dz = dz_ ? static_cast<T*>(dz_) + t * ldd : nullptr;
    vocab = vocab_;
    shift = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    vectors = (shift + vocab + kN - 1) / kN;
    same = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
  }
  __device__ __forceinline__ bool whole(int v) const {
    return v * kN >= shift && v * kN - shift + kN <= vocab;
  }
  // Elements that do not exist read as -inf: e = 0, and they are not stored.
  __device__ __forceinline__ void load(int v, float* x) const {
    const int j0 = v * kN - shift;
    if (whole(v)) {
      const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(z + j0));
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = Elem<T>::get(raw, i);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        x[i] = (unsigned)(j0 + i) < (unsigned)vocab ? Elem<T>::load(z + j0 + i) : -INFINITY;
    }
  }
  __device__ __forceinline__ void store(int v, const float* x) const {
    const int j0 = v * kN - shift;
    if (same && whole(v)) {
      __stcs(reinterpret_cast<uint4*>(dz + j0), Elem<T>::pack(x));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if ((unsigned)(j0 + i) < (unsigned)vocab) Elem<T>::store(dz + j0 + i, x[i]);
    }
  }
};

// ------------------------------------------------------------ sums of a row
// The row's maximum m and sums of 2^((z - m) c): `on` over the tokens of the
// teacher's list (kDistillRest only; 0 elsewhere), `off` over all others.
struct Sum {
  float m, off, on;
};

// m = -inf stands for "nothing yet": its sums are 0 (or NaN, which stays).
__device__ __forceinline__ float rescale(float m, float to, float c) {
  return m == to ? 1.f : ex2((m - to) * c);
}

__device__ __forceinline__ Sum join(Sum a, Sum b, float c) {
  Sum r;
  r.m = fmaxf(a.m, b.m);
  const float fa = rescale(a.m, r.m, c), fb = rescale(b.m, r.m, c);
  r.off = a.off * fa + b.off * fb;
  r.on = a.on * fa + b.on * fb;
  return r;
}

__device__ __forceinline__ Sum warp_join(Sum a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum b;
    b.m = __shfl_xor_sync(~0u, a.m, o);
    b.off = __shfl_xor_sync(~0u, a.off, o);
    b.on = __shfl_xor_sync(~0u, a.on, o);
    a = join(a, b, c);
  }
  return a;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  return x;
}

// ------------------------------------------------------------ the teacher's list
// Shared memory of a row's list: token (-1: padding), student's logit,
// teacher's probability.
struct List {
  int* idx;
  float* z;
  float* p;
  __device__ __forceinline__ List(void* smem, int k) {
    idx = static_cast<int*>(smem);
    z = reinterpret_cast<float*>(idx + k);
    p = z + k;
  }
};

// The teacher's side of a row, by one warp: fills the list and returns
// (sum p, sum p log2 p).  Without the rest class sum p is 1, or 0 where the
// list has no mass.
template <typename T, bool kRest>
__device__ __forceinline__ float2 teacher(const LossArgs& a, const Row<T>& row, int64_t t,
                                          List list, int lane) {
  const int32_t* idx = a.top_idx + t * a.ld_top;
  const float* logit = a.top_logit + t * a.ld_top;
  float most = -INFINITY;
  for (int i = lane; i < a.k; i += 32) {
    const int j = idx[i];
    const bool there = (unsigned)j < (unsigned)row.vocab;
    const float x = there ? logit[i] : -INFINITY;
    list.idx[i] = there ? j : -1;
    list.z[i] = there ? Elem<T>::load(row.z + j) : -INFINITY;
    list.p[i] = x;
    most = fmaxf(most, x);
  }
  float sum = 0.f, plogp = 0.f;
  if (kRest) {
    const float lse = a.teacher_lse[t];
    for (int i = lane; i < a.k; i += 32) {
      const float lp = (list.p[i] * a.inv_tau - lse) * kLog2e;
      const float p = list.idx[i] < 0 ? 0.f : ex2(lp);
      list.p[i] = p;
      sum += p;
      if (p != 0.f) plogp += p * lp;
    }
    return make_float2(warp_sum(sum), warp_sum(plogp));
  }
  most = warp_max(most);
  for (int i = lane; i < a.k; i += 32) {
    const float x = list.p[i];
    sum += x == -INFINITY ? 0.f : ex2((x - most) * a.c);
  }
  sum = warp_sum(sum);
  if (sum == 0.f) {
    for (int i = lane; i < a.k; i += 32) list.p[i] = 0.f;
    return make_float2(0.f, 0.f);
  }
  const float log2_sum = log2f(sum), inv = 1.f / sum;
  for (int i = lane; i < a.k; i += 32) {
    const float x = list.p[i];
    const float lp = (x - most) * a.c - log2_sum;
    const float p = x == -INFINITY ? 0.f : ex2((x - most) * a.c) * inv;
    list.p[i] = p;
    if (p != 0.f) plogp += p * lp;
  }
  return make_float2(isnan(sum) ? sum : 1.f, warp_sum(plogp));
}

// sum p log2 q over the list, by one warp.
__device__ __forceinline__ float cross(List list, int k, const Sum& s, float log2_z, float c,
                                       int lane) {
  float x = 0.f;
  for (int i = lane; i < k; i += 32)
    if (list.p[i] != 0.f) x += list.p[i] * ((list.z[i] - s.m) * c - log2_z);
  return warp_sum(x);
}

// ------------------------------------------------------------ a row's numbers
struct Coef {
  float k0;     // gradient per e off the list
  float scale;  // weight / temperature
  float inv_z;
  float log2_z;
  float rest;  // the rest's term of the loss
  bool none;   // no distribution: the row is left out
};

template <bool kRest>
__device__ __forceinline__ Coef distill_coef(const Sum& s, float sum_p, float weight,
                                             float inv_tau) {
  Coef r;
  const float z = s.off + s.on;
  r.scale = weight * inv_tau;
  r.inv_z = 1.f / z;
  r.log2_z = log2f(z);
  r.rest = 0.f;
  r.none = z == 0.f || (!kRest && sum_p == 0.f);
  r.k0 = r.scale * r.inv_z;
  if (kRest) {
    const float p_rest = 1.f - sum_p;  // NaN stays; at or under 0 there is no rest
    if (s.off == 0.f) {
      r.k0 = 0.f;
      if (p_rest > 0x1p-20f) r.rest = INFINITY;
    } else if (!(p_rest <= 0.f)) {
      r.k0 = r.scale * (r.inv_z - p_rest / s.off);
      // log p_rest - log q_rest, each as log1p of what is on the list: exact
      // to rounding where the list holds little of the mass
      r.rest = p_rest * (log1pf(-sum_p) + log1pf(s.on / s.off));
    }
  } else if (isnan(sum_p)) {
    r.k0 = sum_p;
  }
  return r;
}

// A listed token's gradient.
__device__ __forceinline__ float listed_grad(const Coef& r, float z, float p, const Sum& s,
                                             float c) {
  return r.scale * (ex2((z - s.m) * c) * r.inv_z - p);
}

// One action: its log probability, loss, KL term and g = d loss / d logp.
struct Action {
  float logp, loss, kl, g, q;
};

__device__ __forceinline__ Action policy_action(const LossArgs& a, int64_t t, float z,
                                                const Sum& s, float weight) {
  Action r;
  const float total = s.off;
  const float x = (z - s.m) * a.c;
  r.q = ex2(x) / total;
  r.logp = (x - log2f(total)) * kLn2;
  const float adv = a.advantage[t];
  const float ratio = a.old_logp ? expf(r.logp - a.old_logp[t]) : isnan(r.logp) ? r.logp : 1.f;
  const float clipped = fminf(fmaxf(ratio, a.clip_min), a.clip_max);
  const float free_ = ratio * adv, held = clipped * adv;
  r.kl = 0.f;
  float g = free_ <= held ? -free_ : 0.f;
  float loss = -fminf(free_, held);
  if (isnan(ratio) || isnan(adv)) g = loss = ratio * adv;
  if (a.ref_logp) {
    const float d = a.ref_logp[t] - r.logp;
    const float up = expm1f(d);  // exp(d) - 1
    r.kl = up - d;
    if (a.kl_coef != 0.f) {
      loss += a.kl_coef * r.kl;
      g -= a.kl_coef * up;
    }
  }
  r.loss = weight * loss;
  r.g = weight * g;
  return r;
}

// The rows that need no pass: 0 reads and writes as any other, 1 is left out
// (zeros), 2 has an action past the vocabulary (NaN).
template <Op kOp>
__device__ __forceinline__ int row_kind(const LossArgs& a, int64_t t, float* weight, int* act) {
  *weight = a.weight ? a.weight[t] : 1.f;
  *act = -1;
  if (kOp != Op::kTarget && *weight == 0.f) return 1;
  if (kOp == Op::kPolicy || kOp == Op::kTarget) {
    *act = a.action[t];
    if (*act < 0) return 1;
    if (*act >= a.vocab) return 2;
  }
  return 0;
}

// What one thread writes for a row that has no pass.
template <Op kOp>
__device__ __forceinline__ void row_without_pass(const LossArgs& a, int64_t t, float value) {
  if (kOp == Op::kTarget) {
    a.row_stat[t] = make_float2(0.f, 0.f);
    a.logp[t] = 0.f;
    if (value != 0.f) *a.status = ZR_ERR_INVALID_ARG;
    return;
  }
  if (a.loss) a.loss[t] = value;
  if (kOp == Op::kPolicy) {
    if (a.logp) a.logp[t] = value;
    if (a.kl) a.kl[t] = value;
  }
}

// ------------------------------------------------------------ one CTA per row
// Two passes over the row, the second from wherever it still is.  For rows of
// any length and alignment.
constexpr int kStreamThreads = 512;
constexpr int kChunk = 32768;  // elements that the list's bitmap covers at a time

template <typename T, Op kOp>
__global__ void __launch_bounds__(kStreamThreads) loss_stream_kernel(const LossArgs a) {
  constexpr int kN = Elem<T>::kN;
  constexpr bool kDist = kOp == Op::kDistill || kOp == Op::kDistillRest;
  constexpr bool kRest = kOp == Op::kDistillRest;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Sum part[kStreamThreads / 32];
  __shared__ float2 teach;
  __shared__ uint32_t bits[kRest ? kChunk / 32 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  List list(smem, a.k);

  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const Row<T> row(a.z, a.ld, a.dz, a.ldd, t, a.vocab);
    float weight;
    int act;
    const int kind = row_kind<kOp>(a, t, &weight, &act);
    bool none = kind != 0;
    float fill = kind == 2 ? NAN : 0.f;
    if (!none) {
      __syncthreads();  // the last row's list and sums are no longer read
      float za = 0.f;
      if (kDist && warp == 0) {
        const float2 tp = teacher<T, kRest>(a, row, t, list, lane);
        if (lane == 0) teach = tp;
      } else if (!kDist) {
        za = Elem<T>::load(row.z + act);
      }
      Sum s = {-INFINITY, 0.f, 0.f};
      for (int v0 = 0; v0 < row.vectors; v0 += kChunk / kN) {
        if (kRest) {
          for (int i = tid; i < kChunk / 32; i += kStreamThreads) bits[i] = 0;
          __syncthreads();
          for (int i = tid; i < a.k; i += kStreamThreads) {
            const int b = list.idx[i] + row.shift - v0 * kN;
            if (list.idx[i] >= 0 && b >= 0 && b < kChunk) atomicOr(&bits[b >> 5], 1u << (b & 31));
          }
          __syncthreads();
        }
        const int v1 = min(v0 + kChunk / kN, row.vectors);
        for (int v = v0 + tid; v < v1; v += kStreamThreads) {
          float x[kN];
          row.load(v, x);
          float m = s.m;
#pragma unroll
          for (int i = 0; i < kN; ++i) m = fmaxf(m, x[i]);
          const float f = rescale(s.m, m, a.c);
          const float from = m == -INFINITY ? 0.f : m;
          s.m = m;
          s.off *= f;
          s.on *= f;
          const int b = (v - v0) * kN;
          const uint32_t hit = kRest ? bits[b >> 5] >> (b & 31) : 0u;
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float e = ex2((x[i] - from) * a.c);
            if (kRest && (hit >> i & 1)) s.on += e;
            else s.off += e;
          }
        }
        if (kRest) __syncthreads();
      }
      s = warp_join(s, a.c);
      if (lane == 0) part[warp] = s;
      __syncthreads();
      s = part[0];
      for (int i = 1; i < kStreamThreads / 32; ++i) s = join(s, part[i], a.c);

      if (kDist) {
        const Coef r = distill_coef<kRest>(s, teach.x, weight, a.inv_tau);
        none = r.none;
        if (!none) {
          if (warp == 0 && a.loss) {
            const float x = cross(list, a.k, s, r.log2_z, a.c, lane);
            if (lane == 0) a.loss[t] = weight * ((teach.y - x) * kLn2 + r.rest);
          }
          if (row.dz) {
            for (int v = tid; v < row.vectors; v += kStreamThreads) {
              float x[kN];
              row.load(v, x);
#pragma unroll
              for (int i = 0; i < kN; ++i) x[i] = ex2((x[i] - s.m) * a.c) * r.k0;
              row.store(v, x);
            }
            __syncthreads();
            for (int i = tid; i < a.k; i += kStreamThreads)
              if (list.idx[i] >= 0)
                Elem<T>::store(row.dz + list.idx[i],
                               listed_grad(r, list.z[i], list.p[i], s, a.c));
          }
        }
      } else {
        none = s.off == 0.f;
        if (!none && kOp == Op::kTarget) {
          if (tid == 0) {
            a.row_stat[t] = make_float2(s.m, 1.f / s.off);
            a.logp[t] = ((za - s.m) * a.c - log2f(s.off)) * kLn2 - a.ref_logp[t];
          }
        } else if (!none) {
          const Action r = policy_action(a, t, za, s, weight);
          if (tid == 0) {
            if (a.loss) a.loss[t] = r.loss;
            if (a.logp) a.logp[t] = r.logp;
            if (a.kl) a.kl[t] = r.kl;
          }
          if (row.dz) {
            const float g = r.g * a.inv_tau, k0 = -g / s.off;
            for (int v = tid; v < row.vectors; v += kStreamThreads) {
              float x[kN];
              row.load(v, x);
              const int j0 = v * kN - row.shift;
#pragma unroll
              for (int i = 0; i < kN; ++i)
                x[i] = j0 + i == act ? g * (1.f - r.q) : ex2((x[i] - s.m) * a.c) * k0;
              row.store(v, x);
            }
          }
        }
      }
    }
    if (none) {
      if (tid == 0) row_without_pass<kOp>(a, t, fill);
      if (kOp != Op::kTarget && row.dz) {
        float x[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = fill;
        for (int v = tid; v < row.vectors; v += kStreamThreads) row.store(v, x);
      }
    }
  }
}

// ------------------------------------------------------------ preference
// One CTA per pair: both sequences' sums of (logp - ref_logp), in 64 bits and
// in a fixed order, the pair's loss and rewards, and every row's slope
// d loss / d logp.
constexpr int kPairThreads = 256;

__device__ __forceinline__ double block_sum(double x, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kPairThreads / 32; ++i) x += part[i];
  return x;
}

__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(const PairArgs a) {
  __shared__ double part[kPairThreads / 32];
  const int p = blockIdx.x, tid = threadIdx.x;
  const int64_t r0 = a.offsets[2 * p], r1 = a.offsets[2 * p + 1], r2 = a.offsets[2 * p + 2];
  if (r0 < 0 || r1 < r0 || r2 < r1 || r2 > a.rows) {
    if (tid == 0) {
      *a.status = ZR_ERR_INVALID_ARG;
      a.loss[p] = NAN;
      if (a.reward) a.reward[2 * p] = a.reward[2 * p + 1] = NAN;
    }
    return;
  }
  double chosen = 0.0, rejected = 0.0;
  for (int64_t t = r0 + tid; t < r1; t += kPairThreads) chosen += a.delta[t];
  for (int64_t t = r1 + tid; t < r2; t += kPairThreads) rejected += a.delta[t];
  chosen = block_sum(chosen, part);
  rejected = block_sum(rejected, part);
  const float win = (float)(a.beta * chosen), lose = (float)(a.beta * rejected);
  const float m = (float)(a.beta * (chosen - rejected));
  const float weight = a.weight ? a.weight[p] : 1.f;
  // -log sigma(x) = log(1 + exp(-|x|)) + max(-x, 0); sigma from the same power
  const float e = expf(-fabsf(m)), soft = log1pf(e), big = 1.f / (1.f + e), small = e * big;
  const float sig_pos = m >= 0.f ? big : small, sig_neg = m >= 0.f ? small : big;
  float loss = (1.f - a.eps) * (soft + fmaxf(-m, 0.f)) + a.eps * (soft + fmaxf(m, 0.f));
  float slope = a.beta * weight * (a.eps * sig_pos - (1.f - a.eps) * sig_neg);
  if (isnan(m)) loss = slope = m;
  loss *= weight;
  if (weight == 0.f) loss = slope = 0.f;
  if (tid == 0) {
    a.loss[p] = loss;
    if (a.reward) {
      a.reward[2 * p] = win;
      a.reward[2 * p + 1] = lose;
    }
  }
  for (int64_t t = r0 + tid; t < r2; t += kPairThreads) a.slope[t] = t < r1 ? slope : -slope;
}

// The gradient of rows whose maximum, 1 / Z and slope are known: one read and
// one write.
constexpr int kGradThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kGradThreads) preference_grad_kernel(const LossArgs a,
                                                                       const float* slope) {
  constexpr int kN = Elem<T>::kN;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const Row<T> row(a.z, a.ld, a.dz, a.ldd, t, a.vocab);
    const float2 stat = a.row_stat[t];
    const float g = stat.y == 0.f ? 0.f : slope[t];
    const int act = a.action[t];
    const float k0 = -g * stat.y;
    for (int v = threadIdx.x; v < row.vectors; v += kGradThreads) {
      float x[kN];
      if (g == 0.f) {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = 0.f;
      } else {
        row.load(v, x);
        const int j0 = v * kN - row.shift;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float e = ex2((x[i] - stat.x) * a.c);
          x[i] = j0 + i == act ? g * (1.f - e * stat.y) : e * k0;
        }
      }
      row.store(v, x);
    }
  }
}

// The status word and the slopes of rows outside every sequence.
__global__ void preference_clear_kernel(float* slope, int64_t rows, int32_t* status) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i == 0) *status = ZR_OK;
  for (int64_t t = i; t < rows; t += (int64_t)gridDim.x * blockDim.x) slope[t] = 0.f;
}

constexpr int64_t kMaxGrid = 1 << 20;

zr_status launched() { return cudaGetLastError() == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

template <typename T, Op kOp>
zr_status rows_launch(const LossArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t)a.k * 12;
  const unsigned grid = (unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid);
  loss_stream_kernel<T, kOp><<<grid, kStreamThreads, smem, stream>>>(a);
  return launched();
}

template <Op kOp>
zr_status by_type(const LossArgs& a, zr_dtype dt, cudaStream_t stream) {
  return dt == ZR_F32 ? rows_launch<float, kOp>(a, stream)
                      : rows_launch<__nv_bfloat16, kOp>(a, stream);
}

}  // namespace

zr_status distill_launch(const LossArgs& a, zr_dtype dt, cudaStream_t stream) {
  return a.teacher_lse ? by_type<Op::kDistillRest>(a, dt, stream)
                       : by_type<Op::kDistill>(a, dt, stream);
}

zr_status policy_launch(const LossArgs& a, zr_dtype dt, cudaStream_t stream) {
  return by_type<Op::kPolicy>(a, dt, stream);
}

// Workspace: 256 bytes (status word), then per row the maximum and 1 / Z,
// logp - ref_logp, and the slope.
size_t preference_workspace_bytes(int64_t rows) { return 256 + (size_t)rows * 16; }

zr_status preference_launch(LossArgs a, PairArgs p, zr_dtype dt, void* ws, cudaStream_t stream) {
  char* w = static_cast<char*>(ws);
  a.status = p.status = reinterpret_cast<int32_t*>(w);
  a.row_stat = reinterpret_cast<float2*>(w + 256);
  a.logp = reinterpret_cast<float*>(a.row_stat + a.rows);
  p.delta = a.logp;
  p.slope = a.logp + a.rows;
  const int64_t blocks = (a.rows + 255) / 256;
  preference_clear_kernel<<<(unsigned)(blocks < 1 ? 1 : blocks < 1024 ? blocks : 1024), 256, 0,
                            stream>>>(p.slope, a.rows, p.status);
  zr_status st = launched();
  if (st == ZR_OK && a.rows > 0) st = by_type<Op::kTarget>(a, dt, stream);
  if (st == ZR_OK && p.pairs > 0) {
    preference_pair_kernel<<<p.pairs, kPairThreads, 0, stream>>>(p);
    st = launched();
  }
  if (st == ZR_OK && a.rows > 0 && a.dz) {
    const unsigned grid = (unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid);
    if (dt == ZR_F32)
      preference_grad_kernel<float><<<grid, kGradThreads, 0, stream>>>(a, p.slope);
    else
      preference_grad_kernel<__nv_bfloat16><<<grid, kGradThreads, 0, stream>>>(a, p.slope);
    st = launched();
  }
  return st;
}

}  // namespace zr
