// Internal declarations shared by the libzr translation units (not part of
// the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "zr.h"

namespace zr {

// Streaming multiprocessors on the current device (cached per device).
int sm_count();

// Dense ring all-reduce / SkipReduce launch; arguments already validated.
zr_status ring_launch(void* const* bufs, int n, int64_t m, zr_dtype dt, int k, int mode,
                      uint64_t seed, uint64_t step, int divisor, int rs_only, uint64_t drop_thr,
                      uint64_t drop_seed, uint64_t drop_step, cudaStream_t stream);

// Multi-bucket SkipReduce in one launch; arguments already validated.
zr_status ring_buckets_launch(const zr_bucket* buckets, int n_buckets, int n, zr_dtype dt,
                              cudaStream_t stream);

// Sparse aggregation; arguments already validated.
size_t sparse_workspace_bytes(int n, int64_t dense_size, int n_parts);
zr_status sparse_launch(const int32_t* const* idx, const float* const* val, const int64_t* nnz,
                        int n, int64_t dense_size, int n_parts, uint64_t part_seed, int average,
                        int32_t* out_idx, float* out_val, int64_t out_cap, int64_t* d_out_nnz,
                        int64_t* d_offsets, void* ws, cudaStream_t stream);

// Union sizes of groups of 2^L consecutive ranks; arguments already validated.
size_t densify_workspace_bytes(int n, int64_t dense_size);
zr_status densify_launch(const int32_t* const* idx, const int64_t* nnz, int n, int64_t dense_size,
                         int64_t* d_union_counts, void* ws, cudaStream_t stream);

// Zen's index sets I_p (the partition of [0, m) by h0); same workspace as a
// partition of m entries.
zr_status index_sets_launch(int64_t m, int n_parts, uint64_t part_seed, int32_t* out_sets,
                            int64_t* d_offsets, void* ws, cudaStream_t stream);

// Zen's directory of index-set counts and the hash bitmap encode / decode;
// arguments already validated.
size_t hash_directory_bytes(int64_t m, int n_parts);
zr_status hash_directory_launch(int64_t m, int n_parts, uint64_t part_seed, int32_t* d_dir,
                                cudaStream_t stream);
size_t hash_bitmap_workspace_bytes(int64_t m, int n_parts);
zr_status hash_bitmap_encode_launch(const int32_t* d_dir, int64_t m, int n_parts,
                                    uint64_t part_seed, const int32_t* keys, int64_t n_keys,
                                    uint32_t* out_bits, int64_t out_cap_words,
                                    int64_t* d_word_offsets, void* ws, cudaStream_t stream);
zr_status hash_bitmap_decode_launch(const int32_t* d_dir, int64_t m, int n_parts,
                                    uint64_t part_seed, const uint32_t* bits, int32_t* out_keys,
                                    int64_t out_cap, int64_t* d_key_offsets, void* ws,
                                    cudaStream_t stream);

// Push-side partition; arguments already validated.
size_t partition_workspace_bytes(int64_t nnz, int n_parts);
zr_status partition_launch(const int32_t* idx, const float* val, int64_t nnz, int n_parts,
                           uint64_t part_seed, int32_t* out_idx, float* out_val,
                           int64_t* d_offsets, void* ws, cudaStream_t stream);

// Losses over a vocabulary; arguments already validated.
struct LossArgs {
  const void* z;  // logits
  int64_t ld;
  void* dz;  // gradient, or null
  int64_t ldd;
  int64_t rows;
  int vocab;
  float inv_tau;        // 1 / temperature
  float c;              // log2(e) / temperature
  float c_high, c_low;  // the same in two parts, c_low > 0
  const float* weight;  // per row, or null
  float* loss;          // per row, or null
  // distillation
  const int32_t* top_idx;
  const float* top_logit;
  const float* teacher_lse;
  int64_t ld_top;
  int k;
  // policy; preference's targets, reference and logp - ref_logp
  const int32_t* action;
  const float* advantage;
  const float* old_logp;
  const float* ref_logp;
  float clip_min, clip_max, kl_coef;
  float* logp;
  float* kl;
  // preference: the row's maximum and 1 / Z, and its slope (cleared)
  float2* row_stat;
  float* slope;
  int32_t* status;
};

struct PairArgs {
  const int64_t* offsets;
  const float* weight;
  float* loss;
  float* reward;
  float beta, eps;
  int32_t pairs;
  int64_t rows;
  const int32_t* target;
  int vocab;
  const float* delta;
  float* slope;
  int32_t* status;
};

zr_status distill_launch(const LossArgs& a, zr_dtype dt, cudaStream_t stream);
zr_status policy_launch(const LossArgs& a, zr_dtype dt, cudaStream_t stream);
size_t preference_workspace_bytes(int64_t rows);
zr_status preference_launch(LossArgs a, PairArgs p, zr_dtype dt, void* ws, cudaStream_t stream);

// Gated feed-forward block; arguments already validated.
struct FfArgs {
  const void *x, *w_gate, *w_up;
  int64_t ld_x, ld_w;
  int64_t rows, d, f;
  int act;
  void* h;  // forward
  int64_t ld_h;
  const void* dh;  // backward
  int64_t ld_dh;
  void *dx, *dw_gate, *dw_up;
  int64_t ld_dx, ld_dw;
  int accumulate;
};

// The kernels' tile coordinates are 32 bits: a dimension rounded up to whole tiles
// must fit them, and in the backward pass, whose input gradient sums over [dg | du]
// and whose weight gradients lie one below the other, twice f.
constexpr int64_t kFfMostDim = INT32_MAX - 512;
constexpr int64_t kFfMostBackward = INT32_MAX / 2 - 512;  // f

size_t gated_ff_workspace_bytes(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w,
                                int backward);
zr_status gated_ff_launch(const FfArgs& a, void* ws, cudaStream_t stream);
zr_status gated_ff_backward_launch(const FfArgs& a, void* ws, cudaStream_t stream);

}  // namespace zr
