// Gated feed-forward block: h = a(x Wg^T) (x Wu^T), and its gradients (zr.h
// has the formulas).
//
// Every product runs on the tensor cores (tcgen05, bf16 into fp32), in one
// kernel with four uses:
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
    const float flat = 1.f - t * t;  // 0 where g^2 may overflow
    r.da = 0.5f * (1.f + t) +
           (flat == 0.f ? 0.f : 0.5f * g * flat * c * (1.f + 0.134145f * g * g));
  }
  return r;
}

// ------------------------------------------------------------ the product
// A pair of CTAs makes one tile of 256 x 256: each CTA holds 128 of the rows
// (of A and of the accumulator) and loads 128 of B's 256.  One k-step is 64
// deep, 32 KB of shared memory in each CTA, loaded as four boxes of 64 x 64.
enum class Use { kForward, kProjections, kInput, kWeights };

constexpr int kTile = 256, kHalf = 128, kDepth = 64;
constexpr int kBox = 64 * 64 * 2;             // bytes of a 64 x 64 box
constexpr int kStageBytes = 4 * kBox;         // A half, then B half
constexpr int kStages = 6;
constexpr int kThreads = 192;                 // 4 epilogue warps, loader, multiplier
constexpr int kColumns = 512;                 // tensor memory: two accumulators of 256
constexpr int kSmem = kStages * kStageBytes + 1024;

struct Maps {
  CUtensorMap x, w_gate, w_up, grads;
};

struct Job {
  FfArgs a;
  bf16* grads;      // [rows, 2 padded]: dg, then du from column `padded`
  int64_t ld_grads;
  int padded;       // f, up to a multiple of 64; the columns between are 0
  int m_tiles, n_tiles, k_blocks;
  int32_t* status;
};

struct Tile {
  int m, n;
};

// Tiles in groups of 16 tile rows, down each group's columns: a wave of pairs
// shares few rows of A and few of B, which then come from L2.
__device__ __forceinline__ Tile tile_at(const Job& j, int i) {
  const int per = 16 * j.n_tiles, g = i / per, first = g * 16;
  const int high = min(16, j.m_tiles - first), r = i - g * per;
  return {first + r % high, r / high};
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ bool vector_at(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// 32 values of one row; `left` of them exist.
__device__ __forceinline__ void store32(bf16* p, const float* v, int left) {
  if (left >= 32 && vector_at(p)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(p)[i] = pack8(v + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < left) p[i] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ void load32(const bf16* p, float* v, int left) {
  if (left >= 32 && vector_at(p)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[i];
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * i + 2 * k] = bf16_lo(u[k]);
        v[8 * i + 2 * k + 1] = bf16_hi(u[k]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < left ? __bfloat162float(p[i]) : 0.f;
  }
}

// One row of the tile's accumulator (this thread's) to memory.
template <Use kUse>
__device__ __forceinline__ void epilogue(const Job& j, Tile t, int row, uint32_t tmem) {
  const FfArgs& a = j.a;
  if (kUse == Use::kForward || kUse == Use::kProjections) {
    const int64_t m = (int64_t)t.m * kTile + row;
    const int n0 = t.n * kHalf;
#pragma unroll 1
    for (int c = 0; c < kHalf; c += 32) {
      float g[32], u[32];
      __syncwarp();  // rows past the end skip the work, not the loads
      tmem_load32(tmem + c, g);
      tmem_load32(tmem + kHalf + c, u);
      const int64_t n = n0 + c;
      const int left = (int)min((int64_t)32, a.f - n);
      if (m < a.rows) {
        if (kUse == Use::kForward) {
          if (left > 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = activation(g[i], a.act).a * u[i];
            store32(static_cast<bf16*>(a.h) + m * a.ld_h + n, g, left);
          }
        } else if (n < j.padded) {
          float dh[32];
          load32(static_cast<const bf16*>(a.dh) + m * a.ld_dh + n, dh, left);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const Act act = activation(g[i], a.act);
            g[i] = i < left ? dh[i] * u[i] * act.da : 0.f;
            u[i] = i < left ? dh[i] * act.a : 0.f;
          }
          bf16* out = j.grads + m * j.ld_grads + n;
          store32(out, g, 32);
          store32(out + j.padded, u, 32);
        }
      }
    }
  } else {
    bf16* out;
    int64_t m, ld;
    bool there;
    if (kUse == Use::kInput) {
      m = (int64_t)t.m * kTile + row;
      there = m < a.rows;
      ld = a.ld_dx;
      out = static_cast<bf16*>(a.dx);
    } else {
      const int half = j.m_tiles / 2;
      m = (int64_t)(t.m < half ? t.m : t.m - half) * kTile + row;
      there = m < a.f;
      ld = a.ld_dw;
      out = static_cast<bf16*>(t.m < half ? a.dw_gate : a.dw_up);
    }
#pragma unroll 1
    for (int c = 0; c < kTile; c += 32) {
      float v[32];
      __syncwarp();
      tmem_load32(tmem + c, v);
      const int64_t n = (int64_t)t.n * kTile + c;
      const int left = (int)min((int64_t)32, a.d - n);
      if (there && left > 0) {
        bf16* p = out + m * ld + n;
        if (kUse == Use::kWeights && a.accumulate) {
          float old[32];
          load32(p, old, left);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += old[i];
        }
        store32(p, v, left);
      }
    }
  }
}

// The loader's boxes of one k-step: A's 128 rows of this CTA, then B's.
template <Use kUse>
__device__ __forceinline__ void load_step(const Job& j, const Maps& maps, Tile t, int k,
                                          uint32_t rank, uint32_t smem, uint32_t bar) {
  const int k0 = k * kDepth;
  const int m0 = t.m * kTile + rank * kHalf;
  if (kUse == Use::kForward || kUse == Use::kProjections) {
    const CUtensorMap* w = rank == 0 ? &maps.w_gate : &maps.w_up;
    const int n0 = t.n * kHalf;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.x, k0, m0 + 64 * b, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, w, k0, n0 + 64 * b, bar);
  } else if (kUse == Use::kInput) {
    const bool second = k0 >= j.padded;
    const CUtensorMap* w = second ? &maps.w_up : &maps.w_gate;
    const int n0 = t.n * kTile + rank * kHalf, f0 = second ? k0 - j.padded : k0;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.grads, k0, m0 + 64 * b, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, w, n0 + 64 * b, f0, bar);
  } else {
    const int half = j.m_tiles / 2;
    const int f0 = t.m < half ? m0 : m0 - half * kTile + j.padded;
    const int n0 = t.n * kTile + rank * kHalf;
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + b * kBox, &maps.grads, f0 + 64 * b, k0, bar);
#pragma unroll
    for (int b = 0; b < 2; ++b) tma_load_pair(smem + (2 + b) * kBox, &maps.x, n0 + 64 * b, k0, bar);
  }
}

template <Use kUse>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ff_mma_kernel(const __grid_constant__ Job j, const __grid_constant__ Maps maps) {
  constexpr bool kAMn = kUse == Use::kWeights;
  constexpr bool kBMn = kUse == Use::kInput || kUse == Use::kWeights;
  constexpr uint32_t kDesc = mma_descriptor(kTile, kTile, kAMn, kBMn);
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done[2], taken[2];
  __shared__ uint32_t tmem_slot;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int tiles = j.m_tiles * j.n_tiles;

  if ((kUse == Use::kForward || kUse == Use::kProjections) && blockIdx.x == 0 && threadIdx.x == 0)
    *j.status = ZR_OK;  // the first kernel of a call
  if (warp == 4) tmem_alloc<2>(smem_u32(&tmem_slot), kColumns);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&done[b]), 1);
      mbar_init(smem_u32(&taken[b]), 8);  // 4 epilogue warps of both CTAs
    }
    mbar_init_fence();
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;

  if (warp == 4) {
    if (lane == 0) {
      uint32_t step = 0;
      for (int i = pair; ok && i < tiles; i += pairs) {
        const Tile t = tile_at(j, i);
        for (int k = 0; k < j.k_blocks; ++k, ++step) {
          const uint32_t s = step % kStages, turn = step / kStages;
          ok = mbar_wait(smem_u32(&empty[s]), (turn & 1) ^ 1);
          if (!ok) break;
          if (rank == 0) mbar_expect(smem_u32(&full[s]), 2 * kStageBytes);
          load_step<kUse>(j, maps, t, k, rank, smem + s * kStageBytes,
                          map_to_cta(smem_u32(&full[s]), 0));
        }
      }
    }
  } else if (warp == 5) {
    if (rank == 0 && lane == 0) {
      uint32_t step = 0, n = 0;
      for (int i = pair; ok && i < tiles; i += pairs, ++n) {
        const uint32_t b = n & 1;
        ok = mbar_wait(smem_u32(&taken[b]), ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        tmem_fence_after();
        for (int k = 0; k < j.k_blocks; ++k, ++step) {
          const uint32_t s = step % kStages;
          ok = mbar_wait(smem_u32(&full[s]), (step / kStages) & 1);
          if (!ok) break;
          tmem_fence_after();
          const uint32_t base = smem + s * kStageBytes;
          const uint64_t da = tile_descriptor(base, kAMn ? kBox : 16);
          const uint64_t db = tile_descriptor(base + 2 * kBox, kBMn ? kBox : 16);
#pragma unroll
          for (int q = 0; q < kDepth / 16; ++q)
            mma_bf16<2>(tmem + b * kTile, da + q * (kAMn ? 2048 >> 4 : 32 >> 4),
                        db + q * (kBMn ? 2048 >> 4 : 32 >> 4), kDesc, k > 0 || q > 0);
          mma_commit<2>(smem_u32(&empty[s]));
        }
        if (ok) mma_commit<2>(smem_u32(&done[b]));
      }
    }
  } else {
    uint32_t n = 0;
    for (int i = pair; ok && i < tiles; i += pairs, ++n) {
      const uint32_t b = n & 1;
      ok = mbar_wait(smem_u32(&done[b]), (n >> 1) & 1);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tmem_fence_after();
      epilogue<kUse>(j, tile_at(j, i), (int)rank * kHalf + warp * 32 + lane,
                     tmem + b * kTile + ((uint32_t)(warp * 32) << 16));
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&taken[b]), 0));
    }
  }
  if (!ok) {
    // A wait gave up: report, and let the copies in flight land before the
    // shared memory is given back.
    *j.status = ZR_ERR_TIMEOUT;
    const uint64_t t0 = global_time_ns();
    while (global_time_ns() - t0 < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 4) tmem_free<2>(tmem, kColumns);
}

// ------------------------------------------------------------ layout
// A matrix whose rows do not start on 16 bytes, laid out again with rows that do.
__global__ void __launch_bounds__(256) ff_layout_kernel(const bf16* in, int64_t ld_in, bf16* out,
                                                        int64_t ld_out, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t c = blockIdx.x * 256 + threadIdx.x; c < cols; c += (int64_t)gridDim.x * 256)
      out[r * ld_out + c] = in[r * ld_in + c];
}

__global__ void ff_clear_status_kernel(int32_t* status) { *status = ZR_OK; }

zr_status launched() { return cudaGetLastError() == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

int64_t up_to(int64_t n, int64_t step) { return (n + step - 1) / step * step; }

// Workspace: status (256 bytes), the matrices laid out again, then [dg | du].
struct Layout {
  size_t x, w_gate, w_up, grads, total;
  int64_t ld_x, ld_w;  // as the product reads them
};

Layout layout(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w, int backward) {
  Layout l = {};
  size_t at = 256;
  auto take = [&at](int64_t r, int64_t ld) {
    const size_t p = at;
    at += ((size_t)r * ld * 2 + 255) / 256 * 256;
    return p;
  };
  l.ld_x = ld_x;
  l.ld_w = ld_w;
  if (ld_x % 8) l.x = take(rows, l.ld_x = up_to(d, 8));
  if (ld_w % 8) {
    l.ld_w = up_to(d, 8);
    l.w_gate = take(f, l.ld_w);
    l.w_up = take(f, l.ld_w);
  }
  if (backward) l.grads = take(rows, 2 * up_to(f, 64));
  l.total = at;
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

// A [rows, cols] matrix read in boxes of 64 x 64; what lies outside reads as 0.
zr_status make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  const Encode encode = encoder();
  if (!encode) return ZR_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
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
  if (cudaFuncSetAttribute(ff_mma_kernel<kUse>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmem) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sm_count() / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  if (cudaOccupancyMaxActiveClusters(&n, ff_mma_kernel<kUse>, &cfg) != cudaSuccess || n < 1)
    return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <Use kUse>
zr_status product(Job j, const Maps& maps, int64_t m_tiles, int64_t n_tiles, int64_t k_blocks,
                  cudaStream_t stream) {
  if (m_tiles * n_tiles > INT32_MAX - (1 << 20)) return ZR_ERR_UNSUPPORTED;
  const int pairs = resident_pairs<kUse>();
  if (pairs == 0) return ZR_ERR_CUDA;
  j.m_tiles = (int)m_tiles;
  j.n_tiles = (int)n_tiles;
  j.k_blocks = (int)k_blocks;
  const int tiles = j.m_tiles * j.n_tiles;
  ff_mma_kernel<kUse><<<2 * (tiles < pairs ? tiles : pairs), kThreads, kSmem, stream>>>(j, maps);
  return launched();
}

// Lays out what needs it, and makes the job and the maps.
zr_status begin(const FfArgs& a, const Layout& l, void* ws, Job* j, Maps* maps,
                cudaStream_t stream) {
  char* w = static_cast<char*>(ws);
  *j = Job{};
  j->a = a;
  j->padded = (int)up_to(a.f, 64);
  j->ld_grads = 2 * (int64_t)j->padded;
  j->grads = reinterpret_cast<bf16*>(w + l.grads);
  j->status = reinterpret_cast<int32_t*>(w);
  const void* x = l.x ? w + l.x : a.x;
  const void* wg = l.w_gate ? w + l.w_gate : a.w_gate;
  const void* wu = l.w_up ? w + l.w_up : a.w_up;
  zr_status st = make_map(&maps->x, x, a.rows, a.d, l.ld_x);
  if (st == ZR_OK) st = make_map(&maps->w_gate, wg, a.f, a.d, l.ld_w);
  if (st == ZR_OK) st = make_map(&maps->w_up, wu, a.f, a.d, l.ld_w);
  if (st == ZR_OK && l.grads) st = make_map(&maps->grads, j->grads, a.rows, j->ld_grads, j->ld_grads);
  if (st != ZR_OK) return st;
  auto lay = [&](const void* in, int64_t ld_in, size_t at, int64_t ld_out, int64_t rows) {
    const dim3 grid((unsigned)((a.d + 255) / 256 < 64 ? (a.d + 255) / 256 : 64),
                    (unsigned)(rows < 16384 ? rows : 16384));
    ff_layout_kernel<<<grid, 256, 0, stream>>>(static_cast<const bf16*>(in), ld_in,
                                               reinterpret_cast<bf16*>(w + at), ld_out, rows, a.d);
  };
  if (l.x) lay(a.x, a.ld_x, l.x, l.ld_x, a.rows);
  if (l.w_gate) {
    lay(a.w_gate, a.ld_w, l.w_gate, l.ld_w, a.f);
    lay(a.w_up, a.ld_w, l.w_up, l.ld_w, a.f);
  }
  return launched();
}

}  // namespace

size_t gated_ff_workspace_bytes(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w,
                                int backward) {
  return layout(rows, d, f, ld_x, ld_w, backward).total;
}

zr_status gated_ff_launch(const FfArgs& a, void* ws, cudaStream_t stream) {
  Job j;
  Maps maps = {};
  const zr_status st =
      begin(a, layout(a.rows, a.d, a.f, a.ld_x, a.ld_w, 0), ws, &j, &maps, stream);
  if (st != ZR_OK) return st;
  return product<Use::kForward>(j, maps, (a.rows + kTile - 1) / kTile, (a.f + kHalf - 1) / kHalf,
                                (a.d + kDepth - 1) / kDepth, stream);
}

zr_status gated_ff_backward_launch(const FfArgs& a, void* ws, cudaStream_t stream) {
  if (a.rows == 0) {
    ff_clear_status_kernel<<<1, 1, 0, stream>>>(static_cast<int32_t*>(ws));
    if (launched() != ZR_OK) return ZR_ERR_CUDA;
    if (a.dw_gate && !a.accumulate)
      for (void* p : {a.dw_gate, a.dw_up})
        if (cudaMemset2DAsync(p, (size_t)a.ld_dw * 2, 0, (size_t)a.d * 2, (size_t)a.f, stream) !=
            cudaSuccess)
          return ZR_ERR_CUDA;
    return ZR_OK;
  }
  Job j;
  Maps maps = {};
  zr_status st = begin(a, layout(a.rows, a.d, a.f, a.ld_x, a.ld_w, 1), ws, &j, &maps, stream);
  const int64_t row_tiles = (a.rows + kTile - 1) / kTile, d_tiles = (a.d + kTile - 1) / kTile;
  if (st == ZR_OK)
    st = product<Use::kProjections>(j, maps, row_tiles, (a.f + kHalf - 1) / kHalf,
                                    (a.d + kDepth - 1) / kDepth, stream);
  if (st == ZR_OK && a.dx)
    st = product<Use::kInput>(j, maps, row_tiles, d_tiles, 2 * (int64_t)j.padded / kDepth, stream);
  if (st == ZR_OK && a.dw_gate)
    st = product<Use::kWeights>(j, maps, 2 * ((a.f + kTile - 1) / kTile), d_tiles,
                                (a.rows + kDepth - 1) / kDepth, stream);
  return st;
}

}  // namespace zr
