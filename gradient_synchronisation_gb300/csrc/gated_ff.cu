// Gated feed-forward block: h = a(x Wg^T) (x Wu^T), and its gradients (zr.h
// has the formulas).  Plain tiled products with fp32 accumulators.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zr.h"
#include "zr_device.cuh"
#include "zr_internal.h"

namespace zr {
namespace {

using bf16 = __nv_bfloat16;

struct Act {
  float a, da;  // a(g) and a'(g)
};

__device__ __forceinline__ Act activation(float g, int act) {
  Act r;
  if (act == ZR_ACT_SILU) {
    const float s = 1.f / (1.f + __expf(-g));
    r.a = g * s;
    r.da = s * (1.f + g * (1.f - s));
  } else if (act == ZR_ACT_GELU) {
    const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752f));
    r.a = g * cdf;
    r.da = cdf + g * expf(-0.5f * g * g) * 0.39894228040143268f;
  } else {
    const float c = 0.79788456080286536f;
    const float t = tanhf(c * (g + 0.044715f * g * g * g));
    r.a = 0.5f * g * (1.f + t);
    r.da = 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * c * (1.f + 0.134145f * g * g);
  }
  return r;
}

constexpr int kT = 64, kK = 16;

// C[m, n] = sum_k A(m, k) B(n, k) for two products at once (gate and up), or
// one whose k runs over two segments.  A(m, k) is at a + m am + k ak.
struct Operand {
  const bf16* p;
  int64_t outer, inner;
};

__device__ __forceinline__ void load_tile(float (*s)[kT + 1], Operand o, int64_t m0, int64_t m_end,
                                          int64_t k0, int64_t k_end) {
  for (int i = threadIdx.x; i < kT * kK; i += 256) {
    const int mm = o.inner == 1 ? i / kK : i % kT, kk = o.inner == 1 ? i % kK : i / kT;
    const int64_t m = m0 + mm, k = k0 + kk;
    s[kk][mm] = m < m_end && k < k_end ? __bfloat162float(o.p[m * o.outer + k * o.inner]) : 0.f;
  }
}

__device__ __forceinline__ void multiply(const float (*sa)[kT + 1], const float (*sb)[kT + 1],
                                         float acc[4][4]) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
  }
}

template <bool kBackward>
__global__ void __launch_bounds__(256) ff_projections_kernel(const FfArgs a, bf16* dg, bf16* du) {
  __shared__ float sx[kK][kT + 1], sg[kK][kT + 1], su[kK][kT + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
  float g[4][4] = {}, u[4][4] = {};
  const Operand x = {(const bf16*)a.x, a.ld_x, 1}, wg = {(const bf16*)a.w_gate, a.ld_w, 1},
                wu = {(const bf16*)a.w_up, a.ld_w, 1};
  for (int64_t k0 = 0; k0 < a.d; k0 += kK) {
    load_tile(sx, x, m0, a.rows, k0, a.d);
    load_tile(sg, wg, n0, a.f, k0, a.d);
    load_tile(su, wu, n0, a.f, k0, a.d);
    __syncthreads();
    multiply(sx, sg, g);
    multiply(sx, su, u);
    __syncthreads();
  }
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= a.rows || n >= a.f) continue;
      const Act t = activation(g[i][j], a.act);
      if (kBackward) {
        const float dh = __bfloat162float(((const bf16*)a.dh)[m * a.ld_dh + n]);
        dg[m * a.f + n] = __float2bfloat16_rn(dh * u[i][j] * t.da);
        du[m * a.f + n] = __float2bfloat16_rn(dh * t.a);
      } else {
        ((bf16*)a.h)[m * a.ld_h + n] = __float2bfloat16_rn(t.a * u[i][j]);
      }
    }
}

__global__ void __launch_bounds__(256) ff_product_kernel(Operand a0, Operand b0, Operand a1,
                                                         Operand b1, int64_t m_end, int64_t n_end,
                                                         int64_t k_end, int segments, bf16* out,
                                                         int64_t ld, int accumulate) {
  __shared__ float sa[kK][kT + 1], sb[kK][kT + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
  float acc[4][4] = {};
  for (int s = 0; s < segments; ++s)
    for (int64_t k0 = 0; k0 < k_end; k0 += kK) {
      load_tile(sa, s ? a1 : a0, m0, m_end, k0, k_end);
      load_tile(sb, s ? b1 : b0, n0, n_end, k0, k_end);
      __syncthreads();
      multiply(sa, sb, acc);
      __syncthreads();
    }
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= m_end || n >= n_end) continue;
      float v = acc[i][j];
      if (accumulate) v += __bfloat162float(out[m * ld + n]);
      out[m * ld + n] = __float2bfloat16_rn(v);
    }
}

zr_status launched() { return cudaGetLastError() == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

dim3 tiles(int64_t m, int64_t n) {
  return dim3((unsigned)((n + kT - 1) / kT), (unsigned)((m + kT - 1) / kT));
}

}  // namespace

size_t gated_ff_workspace_bytes(int64_t rows, int64_t, int64_t f, int64_t, int64_t, int backward) {
  return backward ? (size_t)rows * f * 4 : 0;
}

zr_status gated_ff_launch(const FfArgs& a, void*, cudaStream_t stream) {
  ff_projections_kernel<false><<<tiles(a.rows, a.f), 256, 0, stream>>>(a, nullptr, nullptr);
  return launched();
}

zr_status gated_ff_backward_launch(const FfArgs& a, void* ws, cudaStream_t stream) {
  bf16* dg = static_cast<bf16*>(ws);
  bf16* du = dg + a.rows * a.f;
  if (a.rows > 0) {
    ff_projections_kernel<true><<<tiles(a.rows, a.f), 256, 0, stream>>>(a, dg, du);
    if (launched() != ZR_OK) return ZR_ERR_CUDA;
  }
  const bf16* x = static_cast<const bf16*>(a.x);
  if (a.dx && a.rows > 0) {
    ff_product_kernel<<<tiles(a.rows, a.d), 256, 0, stream>>>(
        Operand{dg, a.f, 1}, Operand{(const bf16*)a.w_gate, 1, a.ld_w}, Operand{du, a.f, 1},
        Operand{(const bf16*)a.w_up, 1, a.ld_w}, a.rows, a.d, a.f, 2, (bf16*)a.dx, a.ld_dx, 0);
    if (launched() != ZR_OK) return ZR_ERR_CUDA;
  }
  if (a.dw_gate && !(a.rows == 0 && a.accumulate)) {
    const Operand xt = {x, 1, a.ld_x};
    for (int s = 0; s < 2; ++s) {
      const Operand dt = {s ? du : dg, 1, a.f};
      ff_product_kernel<<<tiles(a.f, a.d), 256, 0, stream>>>(
          dt, xt, dt, xt, a.f, a.d, a.rows, 1, (bf16*)(s ? a.dw_up : a.dw_gate), a.ld_dw,
          a.accumulate);
      if (launched() != ZR_OK) return ZR_ERR_CUDA;
    }
  }
  return ZR_OK;
}

}  // namespace zr
