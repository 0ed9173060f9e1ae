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

#include "tcgen05.cuh"
#include "zr.h"
#include "zr_device.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kLn2Low = (float)(0.6931471805599453 - (double)kLn2);
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);
// ex2.approx is low by 5e-8 of its result in the mean for arguments from -1
// down (and by half of that above, where they are rounded less), which would move
// every row's log Z.  Sums are corrected for it: where they are rescaled by an
// exponent that is this much higher, and once for what a thread has summed.
constexpr float kEx2Mean = 7.1e-8f;

enum class Op { kDistill, kDistillRest, kPolicy, kTarget };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 2^((x - m) c) for two values; minus_m = (-m, -m).
__device__ __forceinline__ float2 power2(float2 x, float2 minus_m, float2 c) {
  const float2 y = mul2(add2(x, minus_m), c);
  return make_float2(ex2(y.x), ex2(y.y));
}

// ------------------------------------------------------------ rows as vectors
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNothing = 0xFF800000u;  // -inf
  static __device__ __forceinline__ float2 get2(const uint4& v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  // A load that is issued here, and its value, which may be asked for later.
  static __device__ __forceinline__ uint32_t start_load(const float* p) {
    uint32_t r;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
    return r;
  }
  static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r); }
  static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
  static __device__ __forceinline__ uint4 pack(const float2* x) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNothing = 0xFF80FF80u;
  static __device__ __forceinline__ float2 get2(const uint4& v, int i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ uint32_t start_load(const __nv_bfloat16* p) {
    uint16_t r;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(r) : "l"(p) : "memory");
    return r;
  }
  static __device__ __forceinline__ float value(uint32_t r) { return bf16_lo(r); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float x) {
    *p = __float2bfloat16_rn(x);
  }
  static __device__ __forceinline__ uint32_t pair(float2 x) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
    return r;
  }
  static __device__ __forceinline__ uint4 pack(const float2* x) {
    return make_uint4(pair(x[0]), pair(x[1]), pair(x[2]), pair(x[3]));
  }
};

// A row that may start at any element: `head` elements up to the first
// 16-byte boundary, `full` whole vectors, and a tail.  Head and tail (the
// edges, fewer than 2 kN elements) go element by element, by threads that
// each take one, so that the vectors need no checks and nothing outside the
// row is touched.
template <typename T>
struct Row {
  static constexpr int kN = Elem<T>::kN;
  static constexpr int kEdges = 2 * kN;
  const T* z;
  T* dz;
  int vocab, head, full;
  bool same;  // dz has z's alignment: whole vectors can be stored

  __device__ __forceinline__ Row(const void* z_, int64_t ld, void* dz_, int64_t ldd, int64_t t,
                                 int vocab_) {
    z = static_cast<const T*>(z_) + t * ld;
    dz = dz_ ? static_cast<T*>(dz_) + t * ldd : nullptr;
    vocab = vocab_;
    head = min(vocab, (int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(T)));
    full = (vocab - head) / kN;
    same = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
  }
  __device__ __forceinline__ int at(int v) const { return head + v * kN; }  // vector's first element
  // The element of edge i < kEdges, or -1.
  __device__ __forceinline__ int edge(int i) const {
    if (i < kN) return i < head ? i : -1;
    const int j = at(full) + i - kN;
    return i < kEdges && j < vocab ? j : -1;
  }
  __device__ __forceinline__ const uint4* vectors() const {
    return reinterpret_cast<const uint4*>(z + head);
  }
  template <bool kSame>
  __device__ __forceinline__ void store(int v, const float2* x) const {
    if (kSame) {
      __stcs(reinterpret_cast<uint4*>(dz + head) + v, Elem<T>::pack(x));
    } else {
      T* p = dz + at(v);
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        Elem<T>::store(p + 2 * i, x[i].x);
        Elem<T>::store(p + 2 * i + 1, x[i].y);
      }
    }
  }
};

// Notes that an edge's element is on the teacher's list.
template <typename T>
__device__ __forceinline__ void mark_edge(const Row<T>& row, int j, uint32_t* edge_bits) {
  atomicOr(edge_bits, 1u << (j < row.head ? j : Row<T>::kN + j - row.at(row.full)));
}

// Sets elements of a vector to -inf (bit i of hit: element i).
template <typename T>
__device__ __forceinline__ void blank(uint4& v, uint32_t hit) {
  if constexpr (Elem<T>::kN == 8) {
    auto word = [](uint32_t w, uint32_t h) {
      if (h & 1) w = (w & 0xFFFF0000u) | 0xFF80u;
      if (h & 2) w = (w & 0xFFFFu) | 0xFF800000u;
      return w;
    };
    v.x = word(v.x, hit);
    v.y = word(v.y, hit >> 2);
    v.z = word(v.z, hit >> 4);
    v.w = word(v.w, hit >> 6);
  } else {
    if (hit & 1) v.x = Elem<T>::kNothing;
    if (hit & 2) v.y = Elem<T>::kNothing;
    if (hit & 4) v.z = Elem<T>::kNothing;
    if (hit & 8) v.w = Elem<T>::kNothing;
  }
}

// ------------------------------------------------------------ sums of a row
// The row's maximum m and its sum of 2^((z - m) c); with the rest class both are
// of the tokens off the teacher's list (the list's part is summed from the list
// itself: the rest is never a difference of two sums, and keeps its digits however
// far the list is ahead of it).
struct Sum {
  float m, s;
};

// A thread's sum without that mean error, which its largest term, 1, has not.
// (In every exponent instead: 1.3 % more time for 8192 rows of 131072.)
__device__ __forceinline__ float even_out(float s) {
  return fmaf(fmaxf(s - 1.f, 0.f), kEx2Mean * kLn2, s);
}

// m = -inf stands for "nothing yet": its sum is 0 (or NaN, which stays).
// A thread's maximum moves by little from one vector to the next.
__device__ __forceinline__ float rescale(float m, float to, float c) {
  return m == to ? 1.f : ex2(fmaf(m - to, c, kEx2Mean));
}

// Most of a row's sum is rescaled by the distance of its thread's or warp's
// maximum from the row's: with c in both parts, as in add_vector.
__device__ __forceinline__ float rescale_far(float m, float to, const LossArgs& a) {
  const float x = m - to, more = x * a.c > -1.f ? kEx2Mean / 2 : kEx2Mean;
  return m == to ? 1.f : ex2(fmaf(x, a.c_high, fmaf(x, a.c_low, more)));
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

// One rescaling for all of a warp's sums; the maximum is taken by one
// instruction, on the floats in the order of signed integers (1 % less time than by
// shuffles, 8192 rows of 131072).
__device__ __forceinline__ Sum warp_join(Sum a, const LossArgs& args) {
  const int i = __float_as_int(a.m), most = __reduce_max_sync(~0u, i ^ (i >> 31 & 0x7FFFFFFF));
  const float m = __int_as_float(most ^ (most >> 31 & 0x7FFFFFFF));
  return {m, warp_sum(a.s * rescale_far(a.m, m, args))};
}

// A number in two parts, hi + lo.  A row's log Z is around 10, where one fp32
// is off by up to 5e-7: that would be most of the error of a sum of log ratios.
// (In fp64, a unit of which there is little, the scalars of a row cost 5 % of the
// time of 8192 rows of 131072.)
struct Wide {
  float hi, lo;  // lo says nothing where hi is not finite
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

__device__ __forceinline__ Wide add(Wide a, float b) {
  const float s = a.hi + b, t = s - a.hi;
  return {s, a.lo + ((a.hi - (s - t)) + (b - t))};
}

// a (c + low)
__device__ __forceinline__ Wide scale(Wide a, float c, float low) {
  const float s = a.hi * c;
  return {s, fmaf(a.hi, c, -s) + fmaf(a.hi, low, a.lo * c)};
}

// log2 x: the exponent is exact, and the rest, within 1/2 of zero, has log2f's
// rounding.
__device__ __forceinline__ Wide log2_wide(float x) {
  int e;
  float f = frexpf(x, &e);
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  const float rest = log2f(f);
  return isfinite(rest) ? Wide{(float)e, rest} : Wide{rest, 0.f};
}

// a - b
__device__ __forceinline__ Wide less(Wide a, Wide b) {
  a.lo -= b.lo;
  return add(a, -b.hi);
}

// lead ln 2 + (z - m) / temperature - log sum.  A distance like that of the type's
// lowest value stands alone: the others are less than its rounding, and in units of
// log2 it would pass fp32's range.
__device__ __forceinline__ Wide log_of(const LossArgs& a, Wide lead, float z, float m, float sum) {
  const Wide x = add({z, 0.f}, -m);
  const float far = x.hi * a.inv_tau;
  if (far < -1e30f && !isnan(sum)) return {far, 0.f};
  const Wide y = less(scale(x, a.c_high, a.c_low), log2_wide(sum));
  return scale(less(y, {-lead.hi, -lead.lo}), kLn2, kLn2Low);
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

// Entry i of a row's list: the teacher's part, then the student's logit.
struct Entry {
  int j;
  float x, z;
};

__device__ __forceinline__ Entry read_entry(const LossArgs& a, int64_t t, int i) {
  return {a.top_idx[t * a.ld_top + i], a.top_logit[t * a.ld_top + i], -INFINITY};
}

template <typename T>
__device__ __forceinline__ void gather_entry(const Row<T>& row, Entry& e) {
  if ((unsigned)e.j < (unsigned)row.vocab) {
    e.z = Elem<T>::load(row.z + e.j);
  } else {
    e.j = -1;
    e.x = -INFINITY;
  }
}

__device__ __forceinline__ void keep_entry(List list, int i, const Entry& e) {
  list.idx[i] = e.j;
  list.z[i] = e.z;
  list.p[i] = e.x;
}

// The teacher's side of a row, and what the loss needs of the student's listed
// logits.  log2 p = (x - x0) c - lead for a listed logit x, and log2 q = (z - z0) c
// + (z0 - M) c - log2 Z: the loss is cross / temperature - sum_p ln 2 (lead + (z0 - M)
// c - log2 Z), which leaves M and Z to be known later, and whose large terms meet in
// two fp32 parts.  (cross is in units of the logits: one of the type's lowest value,
// times log2(e) or over a temperature below 1, would pass fp32's range.)
struct Teacher {
  float mass;   // sum p; without the rest class 1, or 0 where the list has none
  float sum_p;  // over the entries that count (p > 0)
  float cross;  // sum p ((x - x0) - (z - z0))
  float z0;     // the largest listed z (0 where there is none)
  float on;     // sum of 2^((z - z0) c) over the list (rest class only)
  Wide lead;    // log2 of the list's sum of 2^((x - x0) c); with the rest class of all tokens'
};

// Makes it, and puts the teacher's probabilities in place of its logits; by one
// warp.
template <bool kRest>
__device__ __forceinline__ Teacher teacher(const LossArgs& a, float lse, List list, int lane) {
  Teacher r;
  float most = -INFINITY, inv = 1.f, sum = 0.f;
  r.z0 = -INFINITY;
  for (int i = lane; i < a.k; i += 32) {
    most = fmaxf(most, kRest && list.idx[i] < 0 ? -INFINITY : list.p[i]);
    r.z0 = fmaxf(r.z0, list.z[i]);
  }
  r.z0 = warp_max(r.z0);
  const float from = r.z0 == -INFINITY ? 0.f : r.z0;
  r.z0 = from;
  most = warp_max(most);
  if (kRest) {
    if (most == -INFINITY) most = 0.f;
    r.lead = less(scale({lse, 0.f}, kLog2e, kLog2eLow), scale({most, 0.f}, a.c_high, a.c_low));
  } else {
    for (int i = lane; i < a.k; i += 32) {
      const float x = list.p[i];
      sum += x == -INFINITY ? 0.f : ex2((x - most) * a.c);
    }
    sum = warp_sum(sum);
    r.lead = log2_wide(sum);
    inv = 1.f / sum;
  }
  const float lead = r.lead.value();
  float sum_p = 0.f, cross = 0.f, on = 0.f;
  for (int i = lane; i < a.k; i += 32) {
    const float x = list.p[i], z = list.z[i] - from, lx = (x - most) * a.c;
    const bool none = kRest ? list.idx[i] < 0 : x == -INFINITY || sum == 0.f;
    const float p = none ? 0.f : kRest ? ex2(lx - lead) : ex2(lx) * inv;
    list.p[i] = p;
    if (p != 0.f) {
      sum_p += p;
      cross += p * ((x - most) - z);
    }
    if (kRest) on += ex2(z * a.c);  // padding has z = -inf
  }
  r.sum_p = warp_sum(sum_p);
  r.cross = warp_sum(cross);
  r.on = kRest ? warp_sum(on) : 0.f;
  r.mass = kRest ? r.sum_p : sum == 0.f ? 0.f : isnan(sum) ? sum : 1.f;
  return r;
}

// ------------------------------------------------------------ a row's numbers
// 1 - sum p up to this may be the rounding of the sum: it is no mass where q has
// none either (less than 2^-126).
constexpr float kNoRest = 0x1p-20f;

struct Coef {
  float m;      // the maximum over all tokens
  float k0;     // gradient per e off the list, where e = 2^((z - Sum's m) c)
  float scale;  // weight / temperature
  float inv_z;
  float z;      // the sum over all tokens, from m
  bool rest;  // the rest class counts
  bool none;  // no distribution: the row is left out
};

template <bool kRest>
__device__ __forceinline__ Coef distill_coef(const LossArgs& a, const Sum& s, const Teacher& tc,
                                             float weight) {
  Coef r;
  r.m = s.m;
  r.z = s.s;
  r.scale = weight * a.inv_tau;
  r.rest = false;
  float off = 1.f;  // 2^((s.m - m) c)
  if (kRest && tc.on != 0.f) {
    r.m = fmaxf(s.m, tc.z0);
    off = s.s != 0.f ? rescale_far(s.m, r.m, a) : 0.f;
    r.z = s.s * off + tc.on * rescale_far(tc.z0, r.m, a);
  }
  r.inv_z = 1.f / r.z;
  r.none = r.z == 0.f || (!kRest && tc.mass == 0.f);
  r.k0 = r.scale * off * r.inv_z;
  if (kRest) {
    const float p_rest = 1.f - tc.mass;  // NaN stays; at or under 0 there is no rest
    if (s.s == 0.f) {
      r.k0 = 0.f;
      r.rest = p_rest > kNoRest;
    } else {
      const bool nothing = tc.on * ex2((tc.z0 - s.m) * a.c - 126.f) > s.s;  // of q
      r.rest = !(p_rest <= (nothing ? kNoRest : 0.f));
      if (r.rest) r.k0 -= r.scale * (p_rest / s.s);
    }
  } else if (isnan(tc.mass)) {
    r.k0 = tc.mass;
  }
  return r;
}

// The rest's term of the loss: log p_rest - log q_rest, each as log1p of what is on
// the list, exact to rounding where the list holds little of the mass.  Where the
// list is far ahead of the rest, log(on / off) is a distance and a logarithm.
__device__ __forceinline__ float rest_term(const LossArgs& a, const Sum& s, const Teacher& tc) {
  if (s.s == 0.f) return isnan(tc.on) ? tc.on : INFINITY;
  const float x = tc.on / s.s, up = x == 0.f ? 0.f : (tc.z0 - s.m) * a.c;
  const float ahead = up < 64.f ? log1pf(x * ex2(up)) : (tc.z0 - s.m) * a.inv_tau + logf(x);
  return (1.f - tc.mass) * (log1pf(-tc.mass) + ahead);
}

// A listed token's gradient.
__device__ __forceinline__ float listed_grad(const Coef& r, float z, float p, float c) {
  return r.scale * (ex2((z - r.m) * c) * r.inv_z - p);
}

__device__ __forceinline__ Wide action_logp(const LossArgs& a, float z, const Sum& s) {
  return log_of(a, {0.f, 0.f}, z, s.m, s.s);
}

// exp(d) - 1 - d; near 0, where that would be a difference of almost equal
// numbers, by its power series (the first term left out is under 2e-8 of it); +inf
// where the power is.
__device__ __forceinline__ float exp_past_line(float d, float up) {
  const float tail =
      1 / 6.f + d * (1 / 24.f + d * (1 / 120.f + d * (1 / 720.f + d * (1 / 5040.f))));
  return fabsf(d) < 0.25f ? d * d * (0.5f + d * tail) : up == INFINITY ? up : up - d;
}

// One action: its log probability, loss, KL term and g = d loss / d logp.
struct Action {
  float logp, loss, kl, g, q;
};

// What the policy loss reads of a token, ahead of its row's sums.
struct Token {
  float adv, old, ref;
};

template <Op kOp>
__device__ __forceinline__ Token read_token(const LossArgs& a, int64_t t) {
  Token k;
  k.adv = kOp == Op::kPolicy ? a.advantage[t] : 0.f;
  k.old = kOp == Op::kPolicy && a.old_logp ? a.old_logp[t] : 0.f;
  k.ref = a.ref_logp ? a.ref_logp[t] : 0.f;
  return k;
}

__device__ __forceinline__ Action policy_action(const LossArgs& a, const Token& k, float z,
                                                const Sum& s, float weight) {
  Action r;
  const float total = s.s;
  const float x = (z - s.m) * a.c;
  r.q = ex2(x) / total;
  const Wide logp = action_logp(a, z, s);
  r.logp = logp.value();
  const float adv = k.adv;
  const float ratio = a.old_logp ? expf(add(logp, -k.old).value()) : isnan(r.logp) ? r.logp : 1.f;
  const float clipped = fminf(fmaxf(ratio, a.clip_min), a.clip_max);
  const float free_ = ratio * adv, held = clipped * adv;
  r.kl = 0.f;
  float g = free_ <= held ? -free_ : 0.f;
  float loss = -fminf(free_, held);
  if (isnan(ratio) || isnan(adv)) g = loss = ratio * adv;
  if (a.ref_logp) {
    const float d = -add(logp, -k.ref).value();
    const float up = expm1f(d);  // exp(d) - 1
    r.kl = exp_past_line(d, up);
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
__device__ __forceinline__ int row_kind(const LossArgs& a, int64_t t, float* weight, int* act,
                                        bool first) {
  if (kOp == Op::kTarget && first) {
    a.slope[t] = 0.f;
    if (t == 0) *a.status = ZR_OK;
  }
  constexpr bool kAction = kOp == Op::kPolicy || kOp == Op::kTarget;
  *act = kAction ? a.action[t] : 0;
  *weight = kOp != Op::kTarget && a.weight ? a.weight[t] : 1.f;
  if (kOp != Op::kTarget && *weight == 0.f) return 1;
  if (*act < 0) return 1;
  return *act >= a.vocab ? 2 : 0;
}

// What one thread writes for a row that has no pass.
template <Op kOp>
__device__ __forceinline__ void row_without_pass(const LossArgs& a, int64_t t, float value) {
  if (kOp == Op::kTarget) {
    a.row_stat[t] = make_float2(0.f, 0.f);
    a.logp[t] = 0.f;
    return;
  }
  if (a.loss) a.loss[t] = value;
  if (kOp == Op::kPolicy) {
    if (a.logp) a.logp[t] = value;
    if (a.kl) a.kl[t] = value;
  }
}

// A row that is left out (or has an action past the vocabulary): its outputs
// and its gradient's vectors v0 .. v1 - 1, and with `edges` the rest.
template <typename T, Op kOp>
__device__ __forceinline__ void row_left_out(const LossArgs& a, const Row<T>& row, int64_t t,
                                             int kind, int v0, int v1, int threads, bool edges) {
  constexpr int kN = Elem<T>::kN;
  const float fill = kind == 2 ? NAN : 0.f;
  const int tid = threadIdx.x;
  if (edges && tid == 0) row_without_pass<kOp>(a, t, fill);
  if (kOp == Op::kTarget || !row.dz) return;
  float2 x[kN / 2];
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) x[i] = both(fill);
  if (row.same) {
    for (int v = v0 + tid; v < v1; v += threads) row.template store<true>(v, x);
  } else {
    for (int v = v0 + tid; v < v1; v += threads) row.template store<false>(v, x);
  }
  const int edge = edges ? row.edge(tid) : -1;
  if (edge >= 0) Elem<T>::store(row.dz + edge, fill);
}

// What the threads of a row need for its gradient, from one warp.
struct Plan {
  float m, k0;
  float listed;  // the action's gradient
  Coef r;
};

// By one warp, when the row's sums are known: the row's outputs (where `first`),
// and its plan.
template <Op kOp>
__device__ __forceinline__ Plan make_plan(const LossArgs& a, int64_t t, const Sum& s,
                                          const Teacher& tc, float za, const Token& token,
                                          float weight, int lane, bool first) {
  Plan p;
  p.m = s.m;
  if (kOp == Op::kDistill || kOp == Op::kDistillRest) {
    p.r = distill_coef<kOp == Op::kDistillRest>(a, s, tc, weight);
    p.k0 = p.r.k0;
    if (kOp == Op::kDistillRest && s.m == -INFINITY) p.m = 0.f;  // no token off the list
    if (first && lane == 0 && !p.r.none && a.loss) {
      const float over = log_of(a, tc.lead, tc.z0, p.r.m, p.r.z).value();
      const float on_list = tc.sum_p != 0.f ? tc.cross * a.inv_tau - tc.sum_p * over : 0.f;
      const float rest = p.r.rest ? rest_term(a, s, tc) : 0.f;
      a.loss[t] = weight * (on_list + rest);
    }
  } else {
    p.r.none = s.s == 0.f;
    if (kOp == Op::kTarget) {
      if (first && lane == 0 && !p.r.none) {
        a.row_stat[t] = make_float2(s.m, 1.f / s.s);
        a.logp[t] = add(action_logp(a, za, s), -token.ref).value();
      }
    } else {
      const Action x = policy_action(a, token, za, s, weight);
      if (first && lane == 0 && !p.r.none) {
        if (a.loss) a.loss[t] = x.loss;
        if (a.logp) a.logp[t] = x.logp;
        if (a.kl) a.kl[t] = x.kl;
      }
      const float g = x.g * a.inv_tau;
      p.k0 = -g / s.s;
      p.listed = g * (1.f - x.q);
    }
  }
  return p;
}

// Adds one vector to a sum.  The exponents here take log2(e) / temperature in
// two parts: its rounding alone would move every row's log Z the same way
// (5e-8), which the sums over a sequence's rows add up.
template <typename T>
__device__ __forceinline__ void add_vector(float& s, const uint4& v, float2 minus_m, float2 c_high,
                                           float2 c_low) {
#pragma unroll
  for (int i = 0; i < Elem<T>::kN / 2; ++i) {
    const float2 x = add2(Elem<T>::get2(v, i), minus_m);
    const float2 y = fma2(x, c_high, mul2(x, c_low));
    s += ex2(y.x) + ex2(y.y);
  }
}

__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest value of kCount vectors and m (NaN is passed over).
template <typename T, int kCount>
__device__ __forceinline__ float vectors_max(float m, const uint4* v) {
  if constexpr (Elem<T>::kN == 8) {
    uint32_t w = max_pair(max_pair(v[0].x, v[0].y), max_pair(v[0].z, v[0].w));
#pragma unroll
    for (int i = 1; i < kCount; ++i)
      w = max_pair(w, max_pair(max_pair(v[i].x, v[i].y), max_pair(v[i].z, v[i].w)));
    return fmaxf(m, fmaxf(bf16_lo(w), bf16_hi(w)));
  } else {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const float2 x = Elem<T>::get2(v[i], 0), y = Elem<T>::get2(v[i], 1);
      m = fmaxf(m, fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y)));
    }
    return m;
  }
}

template <bool kSame, typename T>
__device__ __forceinline__ void grad_vector(const Row<T>& row, int v, const uint4& raw,
                                            float2 minus_m, float2 c, float2 k0) {
  constexpr int kN = Elem<T>::kN;
  float2 x[kN / 2];
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) x[i] = mul2(power2(Elem<T>::get2(raw, i), minus_m, c), k0);
  row.template store<kSame>(v, x);
}

// ------------------------------------------------------------ one CTA per row
// Two passes over the row, the second from wherever it still is.  For rows
// that are too long to be held (below): over 16 CTAs' 64 KB.  Measured with it
// on rows that can be held, 4096 x 131072 bf16 (distillation): 531 us against 337.
constexpr int kStreamThreads = 512;
constexpr int kChunk = 32768;  // elements that the list's bitmap covers at a time

template <typename T, Op kOp>
__global__ void __launch_bounds__(kStreamThreads) loss_stream_kernel(const LossArgs a) {
  using E = Elem<T>;
  constexpr int kN = E::kN;
  constexpr bool kDist = kOp == Op::kDistill || kOp == Op::kDistillRest;
  constexpr bool kRest = kOp == Op::kDistillRest;
  constexpr int kStep = kChunk / kN;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Sum part[kStreamThreads / 32];
  __shared__ Plan plan;
  __shared__ uint32_t bits[kRest ? kChunk / 32 : 1], edge_bits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float2 c = both(a.c);
  List list(smem, a.k);
  let_next_kernel_start();
  wait_for_kernels_before();

  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const Row<T> row(a.z, a.ld, a.dz, a.ldd, t, a.vocab);
    float weight;
    int act;
    const int kind = row_kind<kOp>(a, t, &weight, &act, tid == 0);
    bool none = kind != 0;
    const int edge = row.edge(tid);
    if (!none) {
      __syncthreads();  // nothing of the last row is read any more
      float za = 0.f;
      Token token = {0.f, 0.f, 0.f};
      if (kDist) {
        for (int i = tid; i < a.k; i += kStreamThreads) {
          Entry e = read_entry(a, t, i);
          gather_entry(row, e);
          keep_entry(list, i, e);
        }
      } else if (warp == 0) {
        za = E::load(row.z + act);
        token = read_token<kOp>(a, t);
      }
      const float edge_z = edge >= 0 ? E::load(row.z + edge) : -INFINITY;
      Sum s = {kRest ? -INFINITY : edge_z, 0.f};
      if (kRest && tid == 0) edge_bits = 0;
      for (int v0 = 0; v0 < row.full || v0 == 0; v0 += kStep) {
        if (kRest) {
          for (int i = tid; i < kChunk / 32; i += kStreamThreads) bits[i] = 0;
          __syncthreads();
          for (int i = tid; i < a.k; i += kStreamThreads) {
            const int j = list.idx[i];
            if (j < 0) continue;
            const int v = (j - row.head) / kN - v0;
            if (j < row.head || j >= row.at(row.full)) mark_edge(row, j, &edge_bits);
            else if (v >= 0 && v < kStep)
              atomicOr(&bits[v * kN / 32], 1u << (v * kN % 32 + (j - row.head) % kN));
          }
          __syncthreads();
        }
        if (v0 == 0 && !(kRest && edge >= 0 && (edge_bits >> tid & 1))) {
          s.m = edge_z;
          s.s = ex2((edge_z - (edge_z == -INFINITY ? 0.f : edge_z)) * a.c);
        }
        const int v1 = min(v0 + kStep, row.full);
        for (int v = v0 + tid; v < v1; v += kStreamThreads) {
          uint4 raw = row.vectors()[v];
          if (kRest) {
            const int b = (v - v0) * kN;
            const uint32_t hit = bits[b >> 5] >> (b & 31) & ((1u << kN) - 1);
            if (hit) blank<T>(raw, hit);
          }
          const float m = vectors_max<T, 1>(s.m, &raw);
          s.s *= rescale(s.m, m, a.c);
          s.m = m;
          add_vector<T>(s.s, raw, both(m == -INFINITY ? 0.f : -m), both(a.c_high), both(a.c_low));
        }
        if (kRest) __syncthreads();
      }
      s.s = even_out(s.s);
      s = warp_join(s, a);
      if (lane == 0) part[warp] = s;
      __syncthreads();
      if (warp == 0) {
        s = lane < kStreamThreads / 32 ? part[lane] : Sum{-INFINITY, 0.f};
        s = warp_join(s, a);
        Teacher teach = {};
        if (kDist) teach = teacher<kRest>(a, kRest ? a.teacher_lse[t] : 0.f, list, lane);
        const Plan p = make_plan<kOp>(a, t, s, teach, za, token, weight, lane, true);
        if (lane == 0) plan = p;
      }
      __syncthreads();
      none = plan.r.none;
      if (!none && kOp != Op::kTarget && row.dz) {
        const float2 minus_m = both(-plan.m), k0 = both(plan.k0);
        if (row.same) {
          for (int v = tid; v < row.full; v += kStreamThreads)
            grad_vector<true>(row, v, row.vectors()[v], minus_m, c, k0);
        } else {
          for (int v = tid; v < row.full; v += kStreamThreads)
            grad_vector<false>(row, v, row.vectors()[v], minus_m, c, k0);
        }
        if (edge >= 0) E::store(row.dz + edge, ex2((edge_z - plan.m) * a.c) * plan.k0);
        __syncthreads();
        if (kDist) {
          for (int i = tid; i < a.k; i += kStreamThreads)
            if (list.idx[i] >= 0)
              E::store(row.dz + list.idx[i],
                       listed_grad(plan.r, list.z[i], list.p[i], a.c));
        } else if (tid == 0) {
          E::store(row.dz + act, plan.listed);
        }
      }
    }
    if (none) row_left_out<T, kOp>(a, row, t, kind, 0, row.full, kStreamThreads, true);
  }
}

// ------------------------------------------------------------ rows held in registers
// One pass over memory: a cluster of CTAs takes a row, every thread keeps its
// vectors of the row between the sums and the gradient (in registers, and in
// places of shared memory that only it uses), and the CTAs send one another
// their sums through distributed shared memory.
//
// Bound: memory.  8192 x 131072 bf16 (policy) takes 617 us, 6.5 TB/s of what has
// to be read and written (96 % of the copy rate); distillation with the rest
// class 337 us for 4096 rows (88 %), where the list's reads, its softmax and the
// second writing of its tokens are added to a CTA's some 11 us.  What keeps it
// there: as many bytes of rows resident as fit (256 KB an SM), reads of what
// decides a row ahead of its logits, bf16 maxima two at a time, sums and
// gradients on pairs of fp32, and one warp for the row's scalars while another
// does the teacher's.  1000 x 50001 takes 39 us (71 %): its 2000 CTAs are 3.3
// waves.
__device__ __forceinline__ uint4 load_vector(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The vectors are unpacked again in each pass: their fp32 values would take
// twice the registers.
template <int kVectors>
__device__ __forceinline__ void keep_packed(uint4 (&v)[kVectors]) {
#pragma unroll
  for (int i = 0; i < kVectors; ++i)
    asm volatile("" : "+r"(v[i].x), "+r"(v[i].y), "+r"(v[i].z), "+r"(v[i].w));
}

__device__ __forceinline__ void copy_async(uint32_t dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

constexpr int kMaxCluster = 16;
// 256 threads of 8 vectors in registers and, for rows longer than one CTA's
// registers, 8 more in shared memory: a CTA holds 64 KB of a row, four CTAs an
// SM.  Measured on 4096 x 131072 bf16, policy / distillation with the rest class:
// 314 / 337 us; without the shared memory, or with 4 vectors in it, 332 / 424 (8
// CTAs a row); with 12 334 / 367 (the row is cut in four as with 8); 3 CTAs an SM
// 352 / 368.
constexpr int kHeldThreads = 256, kHeldVectors = 8, kHeldMore = 8, kHeldBlocks = 4;

template <typename T, Op kOp, int kThreads, int kVectors, int kMore>
__global__ void __launch_bounds__(kThreads, kHeldBlocks)
    loss_rows_kernel(const __grid_constant__ LossArgs a, const int share) {
  using E = Elem<T>;
  constexpr int kN = E::kN;
  constexpr bool kDist = kOp == Op::kDistill || kOp == Op::kDistillRest;
  constexpr bool kRest = kOp == Op::kDistillRest;
  constexpr int kWarps = kThreads / 32;
  let_next_kernel_start();
  wait_for_kernels_before();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Sum part[kWarps];
  __shared__ __align__(16) float4 all[kMaxCluster];
  __shared__ __align__(8) uint64_t arrived;
  __shared__ Plan plan;
  __shared__ Teacher teach;
  // rest class: which elements of a thread's vectors are listed, a byte each
  constexpr int kWords = (kVectors + kMore) / 4;  // of hits, a thread
  __shared__ __align__(16) uint32_t hits[kRest ? kThreads * kWords : 1];
  __shared__ uint32_t edge_bits;
  static_assert(kVectors % 4 == 0 && kMore % 4 == 0, "whole words of hits");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
  const int64_t t = blockIdx.x / ctas;
  const Row<T> row(a.z, a.ld, a.dz, a.ldd, t, a.vocab);
  // this CTA's vectors of the row: `share` of them (what the threads hold at most), or
  // what is left
  const int first = rank * share, last = min(row.full, first + share);
  const float2 c = both(a.c);
  // This thread's vectors beyond the ones in registers: its own places in
  // shared memory, which no other thread touches.
  uint4* more = reinterpret_cast<uint4*>(smem) + tid;
  List list(smem + kThreads * kMore * 16, a.k);
  // Whether this CTA writes element j; the first one has the edges.
  auto ours = [&](int j) {
    return (j >= row.at(first) && j < row.at(last)) ||
           (rank == 0 && ((unsigned)j < (unsigned)row.head ||
                          (j >= row.at(row.full) && j < row.vocab)));
  };

  // What decides the row, and what hangs on nothing, is read first: behind the
  // row's own loads it would wait for all of them.
  float weight, lse = 0.f;
  int act;
  Entry entry = {-1, -INFINITY, -INFINITY};
  if (kDist && tid < a.k) entry = read_entry(a, t, tid);
  Token token = {0.f, 0.f, 0.f};
  if (!kDist && warp == 0) token = read_token<kOp>(a, t);
  if (kRest && warp == 1) lse = a.teacher_lse[t];
  const int kind = row_kind<kOp>(a, t, &weight, &act, rank == 0 && tid == 0);
  bool none = kind != 0;
  if (!none) {
    if (ctas > 1) {
      if (tid == 0) {
        mbar_init(smem_u32(&arrived), 1);
        mbar_init_fence();
        mbar_expect(smem_u32(&arrived), ctas * 16);
      }
      __syncwarp();
      cluster_arrive_relaxed();  // started, and ready to be sent to
    }
    float za = 0.f;
    if (!kDist && warp == 0 && ours(act)) za = E::load(row.z + act);
    const int edge = rank == 0 ? row.edge(tid) : -1;
    const float edge_z = edge >= 0 ? E::load(row.z + edge) : -INFINITY;
    if (kMore) {
#pragma unroll
      for (int i = 0; i < kMore; ++i) {
        const int v = first + (kVectors + i) * kThreads + tid;
        if (v < last) copy_async(smem_u32(more + i * kThreads), row.vectors() + v);
        else more[i * kThreads] = make_uint4(E::kNothing, E::kNothing, E::kNothing, E::kNothing);
      }
    }
    uint4 held[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int v = first + i * kThreads + tid;
      held[i] = make_uint4(E::kNothing, E::kNothing, E::kNothing, E::kNothing);
      if (v < last) held[i] = load_vector(row.vectors() + v);
    }
    auto mark = [&](int j) {
      if ((unsigned)j >= (unsigned)a.vocab) return;
      if (j < row.head || j >= row.at(row.full)) {
        mark_edge(row, j, &edge_bits);
      } else if (ours(j)) {
        const int v = (j - row.head) / kN - first, i = v / kThreads;
        atomicOr(&hits[v % kThreads * kWords + i / 4], 1u << (i % 4 * 8 + (j - row.head) % kN));
      }
    };
    if (kDist) {
      if (kRest) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) hits[tid * kWords + i] = 0;
        if (tid == 0) edge_bits = 0;
        __syncthreads();
        mark(entry.j);
      }
      for (int i = tid + kThreads; i < a.k; i += kThreads) {
        Entry e = read_entry(a, t, i);
        gather_entry(row, e);
        keep_entry(list, i, e);
        if (kRest) mark(e.j);
      }
      if (kRest) __syncthreads();
    }

    const bool off_list = !(kRest && edge >= 0 && (edge_bits >> tid & 1));
    Sum s = {off_list ? edge_z : -INFINITY, 0.f};
    s.m = vectors_max<T, kVectors>(s.m, held);
    keep_packed(held);
    // The listed logits only now: the row's loads have brought them to L2 (read
    // before, they cost a memory access each).
    uint32_t gathered = 0;
    if (kDist && tid < a.k)
      gathered = E::start_load(row.z + ((unsigned)entry.j < (unsigned)a.vocab ? entry.j : 0));
    if (kRest) {  // few threads have a listed token: it is stored as one below
      uint32_t h[kWords], any = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) any |= h[i] = hits[tid * kWords + i];
      if (any) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) blank<T>(held[i], h[i / 4] >> (i % 4 * 8) & 0xFF);
        s.m = vectors_max<T, kVectors>(off_list ? edge_z : -INFINITY, held);
      }
    }
    const float from = s.m == -INFINITY ? 0.f : s.m;
    if (off_list) s.s = ex2((edge_z - from) * a.c);
#pragma unroll
    for (int i = 0; i < kVectors; ++i) add_vector<T>(s.s, held[i], both(-from), both(a.c_high), both(a.c_low));
    if (kMore) {
      copy_async_wait();
      constexpr int kPart = 2;
#pragma unroll
      for (int i = 0; i < kMore; i += kPart) {
        uint4 x[kPart];
#pragma unroll
        for (int q = 0; q < kPart; ++q) x[q] = more[(i + q) * kThreads];
        if (kRest) {
          const uint32_t h = hits[tid * kWords + (kVectors + i) / 4] >> (i % 4 * 8) & 0xFFFF;
          if (h) {
#pragma unroll
            for (int q = 0; q < kPart; ++q) {
              blank<T>(x[q], h >> (8 * q) & 0xFF);
              more[(i + q) * kThreads] = x[q];
            }
          }
        }
        const float m = vectors_max<T, kPart>(s.m, x);
        s.s *= rescale(s.m, m, a.c);
        s.m = m;
#pragma unroll
        for (int q = 0; q < kPart; ++q)
          add_vector<T>(s.s, x[q], both(m == -INFINITY ? 0.f : -m), both(a.c_high), both(a.c_low));
      }
    }
    s.s = even_out(s.s);
    s = warp_join(s, a);
    if (lane == 0) part[warp] = s;
    if (kDist && tid < a.k) {
      if ((unsigned)entry.j < (unsigned)a.vocab) entry.z = E::value(gathered);
      else entry = {-1, -INFINITY, -INFINITY};
      keep_entry(list, tid, entry);
    }
    __syncthreads();
    if (kDist && warp == 1) {  // while the sums are exchanged
      const Teacher tc = teacher<kRest>(a, lse, list, lane);
      if (lane == 0) teach = tc;
      asm volatile("bar.sync 1, 64;" ::: "memory");
    }
    if (warp == 0) {
      s = lane < kWarps ? part[lane] : Sum{-INFINITY, 0.f};
      s = warp_join(s, a);
      if (ctas > 1) {
        cluster_wait();
        // Once a CTA has all sums it may store gradients over its logits (in place).
        // The others' reads of them are over by then: the list's logits are in
        // shared memory, and the action's is read by the CTA that stores there alone,
        // which sends it along.
        if (lane < ctas)
          send_cluster(map_to_cta(smem_u32(&all[rank]), lane), s.m, s.s, za,
                       map_to_cta(smem_u32(&arrived), lane));
        const bool ok = mbar_wait_cluster(smem_u32(&arrived), 0);
        const float4 x = lane < ctas ? all[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        s = warp_join(Sum{x.x, x.y}, a);
        if (!kDist) {
          const bool inside = act >= row.head && act < row.at(row.full);
          za = __shfl_sync(~0u, x.z, inside ? (act - row.head) / kN / share : 0);
        }
        if (!ok) s.s = NAN;  // a CTA of the cluster was not heard of: not a result
      }
      Teacher tc = {};
      if (kDist) {
        asm volatile("bar.sync 1, 64;" ::: "memory");
        tc = teach;
      }
      const Plan p = make_plan<kOp>(a, t, s, tc, za, token, weight, lane, rank == 0);
      if (lane == 0) plan = p;
    }
    __syncthreads();
    none = plan.r.none;
    if (!none && kOp != Op::kTarget && row.dz) {
      const float2 minus_m = both(-plan.m), k0 = both(plan.k0);
      keep_packed(held);
      if (row.same) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
          const int v = first + i * kThreads + tid;
          if (v < last) grad_vector<true>(row, v, held[i], minus_m, c, k0);
        }
#pragma unroll 2
        for (int i = 0; i < kMore; ++i) {
          const int v = first + (kVectors + i) * kThreads + tid;
          if (v < last) grad_vector<true>(row, v, more[i * kThreads], minus_m, c, k0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
          const int v = first + i * kThreads + tid;
          if (v < last) grad_vector<false>(row, v, held[i], minus_m, c, k0);
        }
#pragma unroll 2
        for (int i = 0; i < kMore; ++i) {
          const int v = first + (kVectors + i) * kThreads + tid;
          if (v < last) grad_vector<false>(row, v, more[i * kThreads], minus_m, c, k0);
        }
      }
      if (edge >= 0) E::store(row.dz + edge, ex2((edge_z - plan.m) * a.c) * plan.k0);
      __syncthreads();
      // the listed tokens that this CTA has just written
      if (kDist) {
        for (int i = tid; i < a.k; i += kThreads) {
          const int j = list.idx[i];
          if (ours(j))
            E::store(row.dz + j, listed_grad(plan.r, list.z[i], list.p[i], a.c));
        }
      } else if (tid == 0) {
        if (ours(act)) E::store(row.dz + act, plan.listed);
      }
    }
  }
  if (none)
    row_left_out<T, kOp>(a, row, t, kind, first, last, kThreads, rank == 0);
}

// ------------------------------------------------------------ preference
// The logits are read twice, for no gradient is known before both sequences'
// sums are.  8190 x 65536 fp32 takes 787 us: the target pass (as above, without
// the writing) 240, the pairs 9, the gradients 540; 5.4 GB in all, of which the
// last rows of the first pass still lie in L2 when the second begins with them.
//
// A pair: both sequences' sums of (logp - ref_logp), in 64 bits and in a fixed
// order, the pair's loss and rewards, and every row's slope d loss / d logp.
constexpr int kPairThreads = 256;

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

__device__ __forceinline__ double block_sum(double x, double* part) {
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kPairThreads / 32; ++i) x += part[i];
  return x;
}

struct Pair {
  int64_t r0, r1, r2;  // chosen rows r0 .. r1 - 1, rejected r1 .. r2 - 1
  __device__ __forceinline__ bool good(int64_t rows) const {
    return r0 >= 0 && r1 >= r0 && r2 >= r1 && r2 <= rows;
  }
};

__device__ __forceinline__ Pair read_pair(const PairArgs& a, int p) {
  return {a.offsets[2 * p], a.offsets[2 * p + 1], a.offsets[2 * p + 2]};
}

struct PairResult {
  float win, lose, loss, slope;
};

// By kThreads threads: all of kPairThreads, or the first warp (part: not used).
template <int kThreads>
__device__ __forceinline__ PairResult pair_result(const PairArgs& a, int p, const Pair& pair,
                                                  double* part) {
  const int tid = threadIdx.x;
  double chosen = 0.0, rejected = 0.0;
  for (int64_t t = pair.r0 + tid; t < pair.r1; t += kThreads) chosen += a.delta[t];
  for (int64_t t = pair.r1 + tid; t < pair.r2; t += kThreads) rejected += a.delta[t];
  chosen = kThreads == 32 ? warp_sum(chosen) : block_sum(chosen, part);
  rejected = kThreads == 32 ? warp_sum(rejected) : block_sum(rejected, part);
  PairResult r;
  r.win = (float)(a.beta * chosen);
  r.lose = (float)(a.beta * rejected);
  const float m = (float)(a.beta * (chosen - rejected));
  const float weight = a.weight ? a.weight[p] : 1.f;
  // -log sigma(x) = log(1 + exp(-|x|)) + max(-x, 0); sigma from the same power
  const float e = expf(-fabsf(m)), soft = log1pf(e), big = 1.f / (1.f + e), small = e * big;
  const float sig_pos = m >= 0.f ? big : small, sig_neg = m >= 0.f ? small : big;
  // a part without weight is none, also where m is infinite (a target of logit -inf)
  r.loss = (a.eps < 1.f ? (1.f - a.eps) * (soft + fmaxf(-m, 0.f)) : 0.f) +
           (a.eps > 0.f ? a.eps * (soft + fmaxf(m, 0.f)) : 0.f);
  r.slope = a.beta * weight * (a.eps * sig_pos - (1.f - a.eps) * sig_neg);
  if (isnan(m)) r.loss = r.slope = m;
  r.loss *= weight;
  if (weight == 0.f) r.loss = r.slope = 0.f;
  return r;
}

// Pair p by one of `blocks` CTAs, which look over the targets between them; the
// rows' slopes where they are wanted (kSlopes).
template <bool kSlopes>
__device__ __forceinline__ void do_pair(const PairArgs& a, int p, int blocks, double* part) {
  const int tid = threadIdx.x;
  Pair pair = {};
  if (p < a.pairs) pair = read_pair(a, p);
  for (int64_t t = (int64_t)p * kPairThreads + tid; t < a.rows; t += (int64_t)blocks * kPairThreads)
    if (a.target[t] >= a.vocab) *a.status = ZR_ERR_INVALID_ARG;
  if (p >= a.pairs) return;
  if (!pair.good(a.rows)) {
    if (tid == 0) {
      *a.status = ZR_ERR_INVALID_ARG;
      a.loss[p] = NAN;
      if (a.reward) a.reward[2 * p] = a.reward[2 * p + 1] = NAN;
    }
    return;
  }
  const PairResult r = pair_result<kPairThreads>(a, p, pair, part);
  if (tid == 0) {
    a.loss[p] = r.loss;
    if (a.reward) {
      a.reward[2 * p] = r.win;
      a.reward[2 * p + 1] = r.lose;
    }
  }
  if (kSlopes)
    for (int64_t t = pair.r0 + tid; t < pair.r2; t += kPairThreads)
      a.slope[t] = t < pair.r1 ? r.slope : -r.slope;
}

// One CTA per pair.  Bound by the latency of its few dependent reads.
__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(const PairArgs a) {
  __shared__ double part[kPairThreads / 32];
  let_next_kernel_start();
  wait_for_kernels_before();
  do_pair<true>(a, blockIdx.x, gridDim.x, part);
}

// A row's slope, from its pair's sums (0 outside all pairs), by the first warp.
__device__ __forceinline__ float row_slope(const PairArgs& a, int64_t t, int lane) {
  int p = -1;
  for (int i = lane; i < a.pairs; i += 32) {
    const Pair pair = read_pair(a, i);
    if (pair.good(a.rows) && pair.r0 <= t && t < pair.r2) p = i;
  }
  p = __reduce_max_sync(~0u, p);
  if (p < 0) return 0.f;
  const Pair pair = read_pair(a, p);
  const float slope = pair_result<32>(a, p, pair, nullptr).slope;
  return t < pair.r1 ? slope : -slope;
}

// The gradient of rows whose maximum, 1 / Z and slope are known: one read and
// one write, by CTAs of 8 vectors a thread; the first of a row has its edges.
// With kPairs the first CTAs do the pairs, and the others make their row's slope
// themselves while its logits come: one launch and one wait fewer for few rows.
// Four CTAs an SM, whose 64 registers spill 40 bytes with kPairs: 150 x 65537 takes
// 16.9 us, with three (80 registers, no spills) 18.4.
constexpr int kGradThreads = kPairThreads, kGradVectors = 8;

template <typename T, bool kPairs>
__global__ void __launch_bounds__(kGradThreads, 4)
    preference_grad_kernel(const LossArgs a, const PairArgs pairs, const int parts) {
  using E = Elem<T>;
  __shared__ double sums[kPairThreads / 32];
  __shared__ float made;
  const int tid = threadIdx.x;
  const float2 c = both(a.c);
  let_next_kernel_start();
  wait_for_kernels_before();
  int block = blockIdx.x;
  if (kPairs) {
    if (block < pairs.pairs) {
      do_pair<false>(pairs, block, pairs.pairs, sums);
      return;
    }
    block -= pairs.pairs;
  }
  // the rows that were summed last first: the L2 cache may still hold some
  const int64_t t = a.rows - 1 - block / parts;
  const int part = block % parts, v0 = part * kGradThreads * kGradVectors;
  const Row<T> row(a.z, a.ld, a.dz, a.ldd, t, a.vocab);
  const int last = min(row.full, v0 + kGradThreads * kGradVectors);
  const float2 stat = a.row_stat[t];
  const bool none = stat.y == 0.f;
  float g = kPairs || none ? 0.f : pairs.slope[t];
  const int edge = part == 0 ? row.edge(tid) : -1;
  const int act = a.action[t];
  const bool ours = (act >= row.at(v0) && act < row.at(max(v0, last))) ||
                    (part == 0 && (act < row.head || act >= row.at(row.full)));
  float za = 0.f, edge_z = 0.f;
  uint4 held[kGradVectors];
  if (kPairs ? !none : g != 0.f) {
    if (tid == 0 && ours) za = E::load(row.z + act);
    if (edge >= 0) edge_z = E::load(row.z + edge);
#pragma unroll
    for (int i = 0; i < kGradVectors; ++i) {
      const int v = v0 + i * kGradThreads + tid;
      if (v < last) held[i] = load_vector(row.vectors() + v);
    }
    if (kPairs) {
      if (tid < 32) g = row_slope(pairs, t, tid);
      if (tid == 0) made = g;
      __syncthreads();
      g = made;
    }
  }
  if (g == 0.f) {
    const float2 x[E::kN / 2] = {};
    if (row.same) {
      for (int v = v0 + tid; v < last; v += kGradThreads) row.template store<true>(v, x);
    } else {
      for (int v = v0 + tid; v < last; v += kGradThreads) row.template store<false>(v, x);
    }
    if (edge >= 0) E::store(row.dz + edge, 0.f);
    return;
  }
  // Where the gradient replaces the logits, the thread that owns the target's
  // vector stores over the logit that thread 0 reads: not before it has read it.
  // (With kPairs the barrier above, after the loads, orders them.)
  if (!kPairs) __syncthreads();
  const float2 minus_m = both(-stat.x), k0 = both(-g * stat.y);
  if (tid == 0) za = g * (1.f - ex2((za - stat.x) * a.c) * stat.y);
  if (row.same) {
#pragma unroll
    for (int i = 0; i < kGradVectors; ++i) {
      const int v = v0 + i * kGradThreads + tid;
      if (v < last) grad_vector<true>(row, v, held[i], minus_m, c, k0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGradVectors; ++i) {
      const int v = v0 + i * kGradThreads + tid;
      if (v < last) grad_vector<false>(row, v, held[i], minus_m, c, k0);
    }
  }
  if (edge >= 0) E::store(row.dz + edge, ex2((edge_z - stat.x) * a.c) * k0.x);
  __syncthreads();  // over what this CTA has stored
  if (tid == 0 && ours) E::store(row.dz + act, za);
}

__global__ void preference_clear_kernel(int32_t* status) { *status = ZR_OK; }

constexpr int64_t kMaxGrid = 1 << 20;

zr_status launched(cudaError_t e) { return e == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

template <typename T, Op kOp, int kMore>
zr_status held_launch(const LossArgs& a, int ctas, int64_t vectors, cudaStream_t stream) {
  auto kernel = loss_rows_kernel<T, kOp, kHeldThreads, kHeldVectors, kMore>;
  const size_t smem = (size_t)kHeldThreads * kMore * 16 + (size_t)a.k * 12;
  // over 48 KB with what is static only for long rows with long lists
  if (smem > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem) != cudaSuccess)
    return ZR_ERR_CUDA;
  if (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                      cudaSuccess)
    return ZR_ERR_CUDA;
  const int share = (int)((vectors + ctas - 1) / ctas);
  return launched(launch_kernel(kernel, (unsigned)(a.rows * ctas), kHeldThreads, smem,
                                (unsigned)ctas, stream, a, share));
}

template <typename T, Op kOp>
zr_status rows_launch(const LossArgs& a, cudaStream_t stream) {
  const int64_t vectors = a.vocab / Elem<T>::kN;  // at most, at any alignment
  constexpr int64_t kHold = kHeldThreads * kHeldVectors, kHoldMore = kHold + kHeldThreads * kHeldMore;
  int ctas = 1;
  while (ctas < kMaxCluster && ctas * kHoldMore < vectors) ctas *= 2;
  // Few rows: more CTAs for each, down to one vector a thread.
  while (ctas < 8 && a.rows * ctas < sm_count() && ctas * kHeldThreads < vectors) ctas *= 2;
  // Twice the CTAs, in registers alone, where these come out full: their last
  // wave is shorter, which counts up to some thousand CTAs.  bf16, twice / not, us:
  // 1000 x 65536 45.2 / 46.4, 1000 x 131072 85.1 / 85.8; but 2048 x 131072 167.5 / 164.8,
  // 4096 x 131072 331.8 / 315.4.
  // (The list's work would be doubled: 2000 x 32000 distillation 53.3 / 50.1.)
  if (kOp == Op::kPolicy && ctas <= 4 && ctas * kHold < vectors && 2 * ctas * kHold >= vectors &&
      4 * vectors >= 3 * 2 * ctas * kHold && a.rows * 2 * ctas <= 8192)
    ctas *= 2;
  if (ctas * kHoldMore >= vectors && a.rows * ctas <= INT32_MAX) {
    return ctas * kHold >= vectors ? held_launch<T, kOp, 0>(a, ctas, vectors, stream)
                                   : held_launch<T, kOp, kHeldMore>(a, ctas, vectors, stream);
  }
  const size_t smem = (size_t)a.k * 12;
  const unsigned grid = (unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid);
  return launched(
      launch_kernel(loss_stream_kernel<T, kOp>, grid, kStreamThreads, smem, 1, stream, a));
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
  a.slope = p.slope;
  p.target = a.action;
  p.vocab = a.vocab;
  const int64_t vectors = a.vocab / (dt == ZR_F32 ? 4 : 8);
  const int64_t each = kGradThreads * kGradVectors;
  const int parts = (int)(vectors < each ? 1 : (vectors + each - 1) / each);
  if (a.dz && a.rows * parts > INT32_MAX) return ZR_ERR_UNSUPPORTED;
  zr_status st;
  if (a.rows > 0) {
    st = by_type<Op::kTarget>(a, dt, stream);
  } else {
    preference_clear_kernel<<<1, 1, 0, stream>>>(a.status);
    st = launched(cudaGetLastError());
  }
  // Each CTA of the gradient reads its pair's rows, which costs less than a
  // launch where they are few and most CTAs run at once.  Inside / apart, in us:
  // 64 x 32000 fp32 13.4 / 15.1, 150 x 65537 bf16 16.7 / 19.0, 512 x 8192 bf16 in one
  // pair 13.5 / 15.4; past the limits 512 x 65537 40.3 / 37.3, 1024 x 8192 21.5 / 19.4.
  const bool pairs_inside = a.dz && a.rows > 0 && a.rows <= 512 && a.rows * parts <= 1024 &&
                            p.pairs > 0 && p.pairs <= 512;
  if (st == ZR_OK && !pairs_inside) {
    st = launched(launch_kernel(preference_pair_kernel, p.pairs > 0 ? p.pairs : 1, kPairThreads, 0,
                                1, stream, p));
  }
  if (st == ZR_OK && a.rows > 0 && a.dz) {
    auto kernel = dt == ZR_F32 ? (pairs_inside ? preference_grad_kernel<float, true>
                                               : preference_grad_kernel<float, false>)
                               : (pairs_inside ? preference_grad_kernel<__nv_bfloat16, true>
                                               : preference_grad_kernel<__nv_bfloat16, false>);
    const int64_t grid = a.rows * parts + (pairs_inside ? p.pairs : 0);
    st = launched(launch_kernel(kernel, (unsigned)grid, kGradThreads, 0, 1, stream, a, p, parts));
  }
  return st;
}

}  // namespace zr
