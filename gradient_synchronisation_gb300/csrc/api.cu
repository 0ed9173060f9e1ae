// libzr C ABI: argument validation, status mapping and dispatch to the
// kernels in ring.cu, sparse.cu, partition.cu, hashbitmap.cu, loss.cu, gated_ff.cu,
// rms_norm.cu, cross_entropy.cu and orthogonalise.cu.  Every check here runs on the host before anything is enqueued;
// a failed check returns without touching any buffer.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <utility>
#include <atomic>
#include <vector>

#include "zr.h"
#include "zr_internal.h"

namespace zr {

int sm_count() {
  static std::atomic<int> cached[64];  // 0 until first asked; any thread may fill it
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  const int c = cached[dev].load(std::memory_order_relaxed);
  if (c > 0) return c;
  int s = 0;
  if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || s <= 0)
    s = 148;
  cached[dev].store(s, std::memory_order_relaxed);
  return s;
}

namespace {

size_t elem_size(zr_dtype dt) { return dt == ZR_F32 ? 4 : 2; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Dense rank buffers: present, aligned, pairwise disjoint.
zr_status check_dense(void* const* bufs, int32_t n, int64_t m, zr_dtype dt) {
  if (!bufs || n < 1 || n > ZR_MAX_RANKS || m < 0) return ZR_ERR_INVALID_ARG;
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (m > (INT64_MAX / 16)) return ZR_ERR_INVALID_ARG;
  if (m == 0) return ZR_OK;
  const uint64_t bytes = (uint64_t)m * elem_size(dt);
  std::vector<std::pair<uintptr_t, int>> spans;
  for (int r = 0; r < n; ++r) {
    if (!bufs[r]) return ZR_ERR_INVALID_ARG;
    if (!aligned16(bufs[r])) return ZR_ERR_ALIGNMENT;
    spans.emplace_back(reinterpret_cast<uintptr_t>(bufs[r]), r);
  }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first - spans[i - 1].first < bytes) return ZR_ERR_INVALID_ARG;  // overlap
  return ZR_OK;
}

zr_status check_cfg(const zr_skip_cfg* cfg, int32_t n) {
  if (!cfg) return ZR_ERR_INVALID_ARG;
  if (cfg->mode != ZR_SKIP_STATIC && cfg->mode != ZR_SKIP_RANDOM) return ZR_ERR_INVALID_ARG;
  if (cfg->k < 0 || cfg->k > n - 1) return ZR_ERR_INVALID_ARG;
  if (cfg->divisor != ZR_DIV_N && cfg->divisor != ZR_DIV_N_MINUS_K && cfg->divisor != ZR_DIV_NONE)
    return ZR_ERR_INVALID_ARG;
  if ((cfg->flags & ~ZR_SKIP_RS_ONLY) != 0) return ZR_ERR_INVALID_ARG;
  return ZR_OK;
}

zr_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return ZR_ERR_INVALID_ARG;
  if (!aligned16(ws)) return ZR_ERR_ALIGNMENT;
  return ws_bytes >= need ? ZR_OK : ZR_ERR_CAPACITY;
}

// A row-major matrix of the step's calls.
struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
  size_t elem;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const {
    return rows == 0 ? begin() : begin() + ((uintptr_t)(rows - 1) * ld + cols) * elem;
  }
};

// Present, a leading dimension that holds a row, aligned to its element, offsets
// that fit 63 bits, and an end that is an address.
zr_status check_matrix(const Matrix& m) {
  if (m.ld < m.cols || m.ld > (int64_t)1 << 40) return ZR_ERR_INVALID_ARG;
  if (m.rows == 0) return ZR_OK;
  if (!m.p) return ZR_ERR_INVALID_ARG;
  const int64_t most = INT64_MAX / (int64_t)m.elem - m.cols;  // cols: at most 2^31 - 1
  if (m.rows - 1 > most / m.ld || m.begin() > UINTPTR_MAX - (m.end() - m.begin()))
    return ZR_ERR_INVALID_ARG;
  if (m.begin() % m.elem) return ZR_ERR_ALIGNMENT;
  return ZR_OK;
}

// Whether two matrices share an element; two that lie beside one another in the
// same rows (equal strides) do not.
bool overlap(const Matrix& a, const Matrix& b) {
  if (!a.p || !b.p || a.begin() >= b.end() || b.begin() >= a.end()) return false;
  if (a.ld != b.ld || a.elem != b.elem) return true;
  const uintptr_t row = (uintptr_t)a.ld * a.elem;
  const uintptr_t off = a.begin() <= b.begin() ? (b.begin() - a.begin()) % row
                                               : (row - (a.begin() - b.begin()) % row) % row;
  return !(off >= (uintptr_t)a.cols * a.elem && off + (uintptr_t)b.cols * b.elem <= row);
}

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kMaxVocab = INT32_MAX - 65535;

bool finite_positive(float x) { return isfinite(x) && x > 0.f; }

// The arguments that the losses share, into a.
zr_status check_loss(LossArgs& a, const void* logits, int64_t ld, zr_dtype dt, int64_t rows,
                     int64_t vocab, float temperature, const float* weight, float* loss,
                     void* dlogits, int64_t ld_d) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (rows < 0 || rows > kMaxDim || vocab < 1 || vocab > kMaxVocab) return ZR_ERR_INVALID_ARG;
  if (!finite_positive(temperature)) return ZR_ERR_INVALID_ARG;
  a.inv_tau = 1.f / temperature;
  const double c = 1.4426950408889634 / (double)temperature;
  a.c = (float)c;
  a.c_high = nextafterf(a.c, 0.f);  // below c, so that -inf times either part is -inf
  a.c_low = (float)(c - (double)a.c_high);
  if (!isfinite(a.inv_tau) || !isfinite(a.c) || !(a.c_high > 0.f && a.c_low > 0.f))
    return ZR_ERR_INVALID_ARG;
  const Matrix z = {logits, rows, vocab, ld, elem_size(dt)};
  zr_status st = check_matrix(z);
  if (st != ZR_OK) return st;
  if (dlogits) {
    const Matrix dz = {dlogits, rows, vocab, ld_d, elem_size(dt)};
    st = check_matrix(dz);
    if (st != ZR_OK) return st;
    if (overlap(z, dz) && !(logits == dlogits && ld == ld_d)) return ZR_ERR_INVALID_ARG;
  }
  a.z = logits;
  a.ld = ld;
  a.dz = dlogits;
  a.ldd = ld_d;
  a.rows = rows;
  a.vocab = (int)vocab;
  a.weight = weight;
  a.loss = loss;
  return ZR_OK;
}

zr_status check_ff(const FfArgs& a, zr_dtype dt, bool backward) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (a.rows < 0 || a.rows > kMaxDim || a.d < 1 || a.d > kMaxDim || a.f < 1 || a.f > kMaxDim)
    return ZR_ERR_INVALID_ARG;
  if (a.act != ZR_ACT_SILU && a.act != ZR_ACT_GELU && a.act != ZR_ACT_GELU_TANH)
    return ZR_ERR_INVALID_ARG;
  if (dt != ZR_BF16) return ZR_ERR_UNSUPPORTED;
  if (a.rows > kFfMostDim || a.d > kFfMostDim || a.f > (backward ? kFfMostBackward : kFfMostDim))
    return ZR_ERR_UNSUPPORTED;
  const Matrix x = {a.x, a.rows, a.d, a.ld_x, 2}, wg = {a.w_gate, a.f, a.d, a.ld_w, 2},
               wu = {a.w_up, a.f, a.d, a.ld_w, 2};
  for (const Matrix& m : {x, wg, wu}) {
    const zr_status st = check_matrix(m);
    if (st != ZR_OK) return st;
    if (m.rows > 0 && m.ld % 8 == 0 && !aligned16(m.p)) return ZR_ERR_ALIGNMENT;
  }
  return ZR_OK;
}

// The block's workspace: none where nothing is needed, or one that holds the
// status word at least.
zr_status check_ff_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0 && !ws) return ZR_OK;
  const zr_status st = check_ws(ws, ws_bytes, need > 4 ? need : 4);
  if (st != ZR_OK) return st;
  return (reinterpret_cast<uintptr_t>(ws) & 255u) ? ZR_ERR_ALIGNMENT : ZR_OK;
}

// An output of the block: a matrix of its own, apart from the inputs.
zr_status check_ff_output(const FfArgs& a, const Matrix& out) {
  const zr_status st = check_matrix(out);
  if (st != ZR_OK) return st;
  const Matrix in[] = {{a.x, a.rows, a.d, a.ld_x, 2},
                       {a.w_gate, a.f, a.d, a.ld_w, 2},
                       {a.w_up, a.f, a.d, a.ld_w, 2},
                       {a.dh, a.rows, a.f, a.ld_dh, 2}};
  for (const Matrix& m : in)
    if (overlap(m, out)) return ZR_ERR_INVALID_ARG;
  return ZR_OK;
}

// An output that may replace an input (the same place and stride) but not overlap it
// otherwise.
bool clash(const Matrix& in, const Matrix& out) {
  return overlap(in, out) && !(in.p == out.p && (in.ld == out.ld || out.rows <= 1));
}

// Matrices of a batch, `step` elements apart: where they end, or an error.  An
// output's matrices lie one behind the other, or beside one another in the same rows.
zr_status check_batch(const Matrix& m, int64_t count, int64_t step, bool output, uintptr_t* end) {
  const zr_status st = check_matrix(m);
  if (st != ZR_OK) return st;
  const unsigned __int128 one = (unsigned __int128)(m.rows - 1) * m.ld + m.cols;
  unsigned __int128 all = one;
  if (count > 1) {
    if (step < 0 || step > (int64_t)1 << 50) return ZR_ERR_INVALID_ARG;
    const unsigned __int128 last = (unsigned __int128)(count - 1) * (uint64_t)step;
    const bool beside = step >= m.cols && last + m.cols <= (uint64_t)m.ld;
    if (output && (uint64_t)step < one && !beside) return ZR_ERR_INVALID_ARG;
    all += last;
  }
  all *= m.elem;
  if (all > (unsigned __int128)INT64_MAX || m.begin() > UINTPTR_MAX - (uintptr_t)all)
    return ZR_ERR_INVALID_ARG;
  *end = m.begin() + (uintptr_t)all;
  return ZR_OK;
}

// A workspace of 256-byte alignment.
zr_status check_ws256(const void* ws, size_t ws_bytes, size_t need) {
  const zr_status st = check_ws(ws, ws_bytes, need);
  if (st != ZR_OK) return st;
  return (reinterpret_cast<uintptr_t>(ws) & 255u) ? ZR_ERR_ALIGNMENT : ZR_OK;
}

}  // namespace
}  // namespace zr

extern "C" {

zr_status zr_ring_allreduce(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                            int32_t average, void* stream) {
  zr_status st = zr::check_dense(bufs, n, m, dt);
  if (st != ZR_OK) return st;
  if (average != 0 && average != 1) return ZR_ERR_INVALID_ARG;
  if (m == 0) return ZR_OK;
  return zr::ring_launch(bufs, n, m, dt, 0, ZR_SKIP_STATIC, 0, 0,
                         average ? ZR_DIV_N : ZR_DIV_NONE, 0, 0, 0, 0,
                         static_cast<cudaStream_t>(stream));
}

zr_status zr_skipreduce(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                        const zr_skip_cfg* cfg, void* stream) {
  zr_status st = zr::check_dense(bufs, n, m, dt);
  if (st != ZR_OK) return st;
  st = zr::check_cfg(cfg, n);
  if (st != ZR_OK) return st;
  if (m == 0) return ZR_OK;
  return zr::ring_launch(bufs, n, m, dt, cfg->k, cfg->mode, cfg->seed, cfg->step, cfg->divisor,
                         (cfg->flags & ZR_SKIP_RS_ONLY) ? 1 : 0, 0, 0, 0,
                         static_cast<cudaStream_t>(stream));
}

zr_status zr_skipreduce_buckets(const zr_bucket* buckets, int32_t n_buckets, int32_t n,
                                zr_dtype dt, void* stream) {
  if (!buckets || n_buckets < 1 || n_buckets > ZR_MAX_BUCKETS) return ZR_ERR_INVALID_ARG;
  if (n < 1 || n > ZR_MAX_RANKS || (int64_t)n_buckets * n > ZR_MAX_BUCKET_BUFS)
    return ZR_ERR_INVALID_ARG;
  // Every bucket as zr_skipreduce would check it, then no overlap between
  // the buffers of different buckets (one launch writes them all).
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  for (int b = 0; b < n_buckets; ++b) {
    const zr_bucket& B = buckets[b];
    zr_status st = zr::check_dense(B.bufs, n, B.m, dt);
    if (st != ZR_OK) return st;
    st = zr::check_cfg(&B.cfg, n);
    if (st != ZR_OK) return st;
    if (B.m == 0) continue;
    const uintptr_t bytes = (uintptr_t)B.m * zr::elem_size(dt);
    for (int r = 0; r < n; ++r) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(B.bufs[r]);
      spans.emplace_back(a, a + bytes);
    }
  }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second) return ZR_ERR_INVALID_ARG;  // overlap
  return zr::ring_buckets_launch(buckets, n_buckets, n, dt, static_cast<cudaStream_t>(stream));
}

zr_status zr_allreduce_dropout(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                               uint64_t threshold, uint64_t seed, uint64_t step,
                               int32_t average, void* stream) {
  zr_status st = zr::check_dense(bufs, n, m, dt);
  if (st != ZR_OK) return st;
  if (average != 0 && average != 1) return ZR_ERR_INVALID_ARG;
  if (threshold > (1ull << 32)) return ZR_ERR_INVALID_ARG;
  if (m == 0) return ZR_OK;
  return zr::ring_launch(bufs, n, m, dt, 0, ZR_SKIP_STATIC, 0, 0,
                         average ? ZR_DIV_N : ZR_DIV_NONE, 0, threshold, seed, step,
                         static_cast<cudaStream_t>(stream));
}

zr_status zr_hash_index_sets(int64_t dense_size, int32_t n_parts, uint64_t part_seed,
                             int32_t* out_sets, int64_t* d_offsets, void* ws, size_t ws_bytes,
                             void* stream) {
  if (dense_size < 1 || dense_size > INT32_MAX) return ZR_ERR_INVALID_ARG;
  if (n_parts < 1 || n_parts > ZR_MAX_PARTS || !out_sets || !d_offsets) return ZR_ERR_INVALID_ARG;
  zr_status st = zr::check_ws(ws, ws_bytes, zr::partition_workspace_bytes(dense_size, n_parts));
  if (st != ZR_OK) return st;
  return zr::index_sets_launch(dense_size, n_parts, part_seed, out_sets, d_offsets, ws,
                               static_cast<cudaStream_t>(stream));
}

size_t zr_hash_directory_size(int64_t dense_size, int32_t n_parts) {
  if (dense_size < 1 || dense_size > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS) return 0;
  return zr::hash_directory_bytes(dense_size, n_parts);
}

zr_status zr_hash_directory(int64_t dense_size, int32_t n_parts, uint64_t part_seed,
                            int32_t* d_dir, size_t dir_bytes, void* stream) {
  if (dense_size < 1 || dense_size > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS || !d_dir)
    return ZR_ERR_INVALID_ARG;
  zr_status st = zr::check_ws(d_dir, dir_bytes, zr::hash_directory_bytes(dense_size, n_parts));
  if (st != ZR_OK) return st;
  return zr::hash_directory_launch(dense_size, n_parts, part_seed, d_dir,
                                   static_cast<cudaStream_t>(stream));
}

size_t zr_hash_bitmap_workspace_size(int64_t dense_size, int32_t n_parts) {
  if (dense_size < 1 || dense_size > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS) return 0;
  return zr::hash_bitmap_workspace_bytes(dense_size, n_parts);
}

zr_status zr_hash_bitmap_encode(const int32_t* d_dir, int64_t dense_size, int32_t n_parts,
                                uint64_t part_seed, const int32_t* keys, int64_t n_keys,
                                uint32_t* out_bits, int64_t out_cap_words,
                                int64_t* d_word_offsets, void* ws, size_t ws_bytes, void* stream) {
  if (dense_size < 1 || dense_size > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS)
    return ZR_ERR_INVALID_ARG;
  if (!d_dir || !out_bits || !d_word_offsets || n_keys < 0 || (n_keys > 0 && !keys))
    return ZR_ERR_INVALID_ARG;
  if (out_cap_words < (dense_size + 31) / 32 + n_parts) return ZR_ERR_CAPACITY;
  zr_status st = zr::check_ws(ws, ws_bytes, zr::hash_bitmap_workspace_bytes(dense_size, n_parts));
  if (st != ZR_OK) return st;
  return zr::hash_bitmap_encode_launch(d_dir, dense_size, n_parts, part_seed, keys, n_keys,
                                       out_bits, out_cap_words, d_word_offsets, ws,
                                       static_cast<cudaStream_t>(stream));
}

zr_status zr_hash_bitmap_decode(const int32_t* d_dir, int64_t dense_size, int32_t n_parts,
                                uint64_t part_seed, const uint32_t* bits, int32_t* out_keys,
                                int64_t out_cap, int64_t* d_key_offsets, void* ws,
                                size_t ws_bytes, void* stream) {
  if (dense_size < 1 || dense_size > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS)
    return ZR_ERR_INVALID_ARG;
  if (!d_dir || !bits || !d_key_offsets || out_cap < 0 || (out_cap > 0 && !out_keys))
    return ZR_ERR_INVALID_ARG;
  zr_status st = zr::check_ws(ws, ws_bytes, zr::hash_bitmap_workspace_bytes(dense_size, n_parts));
  if (st != ZR_OK) return st;
  return zr::hash_bitmap_decode_launch(d_dir, dense_size, n_parts, part_seed, bits, out_keys,
                                       out_cap, d_key_offsets, ws,
                                       static_cast<cudaStream_t>(stream));
}

size_t zr_densification_workspace_size(int32_t n, int64_t dense_size) {
  if (n < 1 || n > ZR_MAX_RANKS || (n & (n - 1)) != 0 || dense_size < 1 || dense_size > INT32_MAX)
    return 0;
  return zr::densify_workspace_bytes(n, dense_size);
}

zr_status zr_densification(const int32_t* const* idx, const int64_t* nnz, int32_t n,
                           int64_t dense_size, int64_t* d_union_counts, void* ws,
                           size_t ws_bytes, void* stream) {
  if (!idx || !nnz || !d_union_counts) return ZR_ERR_INVALID_ARG;
  if (n < 1 || n > ZR_MAX_RANKS || (n & (n - 1)) != 0) return ZR_ERR_INVALID_ARG;
  if (dense_size < 1 || dense_size > INT32_MAX) return ZR_ERR_INVALID_ARG;
  for (int r = 0; r < n; ++r) {
    if (nnz[r] < 0 || nnz[r] > dense_size) return ZR_ERR_INVALID_ARG;
    if (nnz[r] > 0 && !idx[r]) return ZR_ERR_INVALID_ARG;
  }
  zr_status st = zr::check_ws(ws, ws_bytes, zr::densify_workspace_bytes(n, dense_size));
  if (st != ZR_OK) return st;
  return zr::densify_launch(idx, nnz, n, dense_size, d_union_counts, ws,
                            static_cast<cudaStream_t>(stream));
}

int32_t zr_choose_scheme(const int64_t* union_counts, int32_t n, double* gammas, double* t_bp,
                         double* t_hc) {
  if (!union_counts || n < 2 || n > ZR_MAX_RANKS || (n & (n - 1)) != 0) return -1;
  int logn = 0;
  while ((1 << logn) < n) ++logn;
  if (union_counts[0] <= 0) return -1;
  double g[7];
  for (int level = 0; level <= logn; ++level) {
    if (union_counts[level] < 0) return -1;
    g[level] = (double)union_counts[level] * (double)(1 << level) / (double)union_counts[0];
    if (gammas) gammas[level] = g[level];
  }
  const double bp = 2.0 * (n - 1) * (g[logn] + 1.0) / n;
  double hc = 0.0;
  for (int i = 1; i <= logn; ++i) hc += g[i - 1];
  hc *= 2.0;
  if (t_bp) *t_bp = bp;
  if (t_hc) *t_hc = hc;
  return bp <= hc ? ZR_SCHEME_BALANCED : ZR_SCHEME_HIERARCHICAL;
}

size_t zr_sparse_workspace_size(int32_t n, int64_t dense_size, int32_t n_parts) {
  if (n < 1 || n > ZR_MAX_RANKS || dense_size < 1 || dense_size > INT32_MAX || n_parts < 0 ||
      n_parts > ZR_MAX_PARTS)
    return 0;
  return zr::sparse_workspace_bytes(n, dense_size, n_parts);
}

zr_status zr_sparse_aggregate(const int32_t* const* idx, const float* const* val,
                              const int64_t* nnz, int32_t n, int64_t dense_size,
                              int32_t n_parts, uint64_t part_seed, int32_t average,
                              int32_t* out_idx, float* out_val, int64_t out_cap,
                              int64_t* d_out_nnz, int64_t* d_offsets, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!idx || !val || !nnz || n < 1 || n > ZR_MAX_RANKS) return ZR_ERR_INVALID_ARG;
  if (dense_size < 1 || dense_size > INT32_MAX) return ZR_ERR_INVALID_ARG;
  if (n_parts < 0 || n_parts > ZR_MAX_PARTS) return ZR_ERR_INVALID_ARG;
  if (average != 0 && average != 1) return ZR_ERR_INVALID_ARG;
  if (!d_out_nnz || (n_parts > 0 && !d_offsets)) return ZR_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int r = 0; r < n; ++r) {
    if (nnz[r] < 0 || nnz[r] > INT32_MAX - 1) return ZR_ERR_INVALID_ARG;
    if (nnz[r] > 0 && (!idx[r] || !val[r])) return ZR_ERR_INVALID_ARG;
    total += nnz[r];
  }
  if (total > 0 && (!out_idx || !out_val)) return ZR_ERR_INVALID_ARG;
  if (out_cap < total) return ZR_ERR_CAPACITY;
  zr_status st = zr::check_ws(ws, ws_bytes, zr::sparse_workspace_bytes(n, dense_size, n_parts));
  if (st != ZR_OK) return st;
  return zr::sparse_launch(idx, val, nnz, n, dense_size, n_parts, part_seed, average, out_idx,
                           out_val, out_cap, d_out_nnz, d_offsets, ws,
                           static_cast<cudaStream_t>(stream));
}

size_t zr_partition_workspace_size(int64_t nnz, int32_t n_parts) {
  if (nnz < 0 || nnz > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS) return 0;
  return zr::partition_workspace_bytes(nnz, n_parts);
}

zr_status zr_partition(const int32_t* idx, const float* val, int64_t nnz, int32_t n_parts,
                       uint64_t part_seed, int32_t* out_idx, float* out_val, int64_t* d_offsets,
                       void* ws, size_t ws_bytes, void* stream) {
  if (nnz < 0 || nnz > INT32_MAX || n_parts < 1 || n_parts > ZR_MAX_PARTS || !d_offsets)
    return ZR_ERR_INVALID_ARG;
  if (nnz > 0 && (!idx || !val || !out_idx || !out_val)) return ZR_ERR_INVALID_ARG;
  zr_status st = zr::check_ws(ws, ws_bytes, zr::partition_workspace_bytes(nnz, n_parts));
  if (st != ZR_OK) return st;
  return zr::partition_launch(idx, val, nnz, n_parts, part_seed, out_idx, out_val, d_offsets, ws,
                              static_cast<cudaStream_t>(stream));
}

zr_status zr_distill_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                          int64_t vocab, const int32_t* top_idx, const float* top_logit, int32_t k,
                          int64_t ld_top, const float* teacher_lse, float temperature,
                          const float* weight, float* loss, void* dlogits, int64_t ld_dlogits,
                          void* stream) {
  zr::LossArgs a = {};
  zr_status st = zr::check_loss(a, logits, ld_logits, dt, rows, vocab, temperature, weight, loss,
                                dlogits, ld_dlogits);
  if (st != ZR_OK) return st;
  if (k < 0 || k > ZR_MAX_TOP) return ZR_ERR_INVALID_ARG;
  if (rows == 0) return ZR_OK;
  if (!loss && !dlogits) return ZR_ERR_INVALID_ARG;
  if (k > 0) {
    st = zr::check_matrix({top_idx, rows, k, ld_top, 4});
    if (st == ZR_OK) st = zr::check_matrix({top_logit, rows, k, ld_top, 4});
    if (st != ZR_OK) return st;
  }
  a.top_idx = top_idx;
  a.top_logit = top_logit;
  a.k = k;
  a.ld_top = ld_top;
  a.teacher_lse = teacher_lse;
  return zr::distill_launch(a, dt, static_cast<cudaStream_t>(stream));
}

zr_status zr_policy_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                         int64_t vocab, const int32_t* action, const float* advantage,
                         const float* old_logp, const float* ref_logp, float clip_low,
                         float clip_high, float kl_coef, float temperature, const float* weight,
                         float* loss, float* logp, float* kl, void* dlogits, int64_t ld_dlogits,
                         void* stream) {
  zr::LossArgs a = {};
  zr_status st = zr::check_loss(a, logits, ld_logits, dt, rows, vocab, temperature, weight, loss,
                                dlogits, ld_dlogits);
  if (st != ZR_OK) return st;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f && isfinite(clip_high)) ||
      !(kl_coef >= 0.f && isfinite(kl_coef)) || (kl_coef != 0.f && !ref_logp))
    return ZR_ERR_INVALID_ARG;
  if (rows == 0) return ZR_OK;
  if (!loss && !logp && !kl && !dlogits) return ZR_ERR_INVALID_ARG;
  if (!action || !advantage) return ZR_ERR_INVALID_ARG;
  a.action = action;
  a.advantage = advantage;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.clip_min = 1.f - clip_low;
  a.clip_max = 1.f + clip_high;
  a.kl_coef = kl_coef;
  a.logp = logp;
  a.kl = kl;
  return zr::policy_launch(a, dt, static_cast<cudaStream_t>(stream));
}

size_t zr_preference_workspace_size(int64_t rows) {
  return rows < 0 || rows > zr::kMaxDim ? 0 : zr::preference_workspace_bytes(rows);
}

zr_status zr_preference_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                             int64_t vocab, const int32_t* target, const int64_t* offsets,
                             int32_t pairs, const float* ref_logp, float beta,
                             float label_smoothing, const float* weight, float* loss,
                             float* reward, void* dlogits, int64_t ld_dlogits, void* ws,
                             size_t ws_bytes, void* stream) {
  zr::LossArgs a = {};
  zr_status st = zr::check_loss(a, logits, ld_logits, dt, rows, vocab, 1.f, nullptr, nullptr,
                                dlogits, ld_dlogits);
  if (st != ZR_OK) return st;
  if (pairs < 0 || pairs > (1 << 24) || !zr::finite_positive(beta) ||
      !(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return ZR_ERR_INVALID_ARG;
  if (rows > 0 && (!target || !ref_logp)) return ZR_ERR_INVALID_ARG;
  if (pairs > 0 && (!offsets || !loss)) return ZR_ERR_INVALID_ARG;
  st = zr::check_ws(ws, ws_bytes, zr::preference_workspace_bytes(rows));
  if (st != ZR_OK) return st;
  a.action = target;
  a.ref_logp = ref_logp;
  zr::PairArgs p = {};
  p.offsets = offsets;
  p.weight = weight;
  p.loss = loss;
  p.reward = reward;
  p.beta = beta;
  p.eps = label_smoothing;
  p.pairs = pairs;
  p.rows = rows;
  return zr::preference_launch(a, p, dt, ws, static_cast<cudaStream_t>(stream));
}

size_t zr_gated_ff_workspace_size(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w,
                                  int32_t backward) {
  if (rows < 0 || rows > zr::kMaxDim || d < 1 || d > zr::kMaxDim || f < 1 || f > zr::kMaxDim ||
      ld_x < d || ld_w < d || (backward != 0 && backward != 1))
    return 0;
  return zr::gated_ff_workspace_bytes(rows, d, f, ld_x, ld_w, backward);
}

zr_status zr_gated_ff(const void* x, int64_t ld_x, const void* w_gate, const void* w_up,
                      int64_t ld_w, int64_t rows, int64_t d, int64_t f, zr_dtype dt, int32_t act,
                      void* h, int64_t ld_h, void* ws, size_t ws_bytes, void* stream) {
  zr::FfArgs a = {};
  a.x = x;
  a.ld_x = ld_x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.ld_w = ld_w;
  a.rows = rows;
  a.d = d;
  a.f = f;
  a.act = act;
  a.h = h;
  a.ld_h = ld_h;
  zr_status st = zr::check_ff(a, dt, false);
  if (st != ZR_OK) return st;
  st = zr::check_ff_output(a, {h, rows, f, ld_h, 2});
  if (st != ZR_OK || rows == 0) return st;
  st = zr::check_ff_ws(ws, ws_bytes, zr::gated_ff_workspace_bytes(rows, d, f, ld_x, ld_w, 0));
  if (st != ZR_OK) return st;
  return zr::gated_ff_launch(a, ws, static_cast<cudaStream_t>(stream));
}

zr_status zr_gated_ff_backward(const void* x, int64_t ld_x, const void* w_gate, const void* w_up,
                               int64_t ld_w, const void* dh, int64_t ld_dh, int64_t rows,
                               int64_t d, int64_t f, zr_dtype dt, int32_t act, int32_t accumulate,
                               void* dx, int64_t ld_dx, void* dw_gate, void* dw_up, int64_t ld_dw,
                               void* ws, size_t ws_bytes, void* stream) {
  zr::FfArgs a = {};
  a.x = x;
  a.ld_x = ld_x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.ld_w = ld_w;
  a.rows = rows;
  a.d = d;
  a.f = f;
  a.act = act;
  a.dh = dh;
  a.ld_dh = ld_dh;
  a.dx = dx;
  a.ld_dx = ld_dx;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  a.ld_dw = ld_dw;
  a.accumulate = accumulate;
  zr_status st = zr::check_ff(a, dt, true);
  if (st == ZR_OK) st = zr::check_matrix({dh, rows, f, ld_dh, 2});
  if (st != ZR_OK) return st;
  if (accumulate != 0 && accumulate != 1) return ZR_ERR_INVALID_ARG;
  if ((dw_gate == nullptr) != (dw_up == nullptr) || (!dx && !dw_gate)) return ZR_ERR_INVALID_ARG;
  const zr::Matrix gate = {dw_gate, f, d, ld_dw, 2}, up = {dw_up, f, d, ld_dw, 2},
                   in = {dx, rows, d, ld_dx, 2};
  if (dw_gate) {
    st = zr::check_ff_output(a, gate);
    if (st == ZR_OK) st = zr::check_ff_output(a, up);
    if (st != ZR_OK) return st;
    if (zr::overlap(gate, up)) return ZR_ERR_INVALID_ARG;
  }
  if (dx) {
    st = zr::check_ff_output(a, in);
    if (st != ZR_OK) return st;
    if (zr::overlap(in, gate) || zr::overlap(in, up)) return ZR_ERR_INVALID_ARG;
  }
  st = zr::check_ff_ws(ws, ws_bytes, zr::gated_ff_workspace_bytes(rows, d, f, ld_x, ld_w, 1));
  if (st != ZR_OK) return st;
  return zr::gated_ff_backward_launch(a, ws, static_cast<cudaStream_t>(stream));
}

zr_status zr_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                      const void* weight, int64_t rows, int64_t d, zr_dtype dt, float eps, void* y,
                      int64_t ld_y, void* sum, int64_t ld_sum, float* rstd, void* stream) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (rows < 0 || rows > zr::kMaxDim || d < 1 || d > zr::kMaxDim || !zr::finite_positive(eps))
    return ZR_ERR_INVALID_ARG;
  if (rows > 0 && (residual == nullptr) != (sum == nullptr)) return ZR_ERR_INVALID_ARG;
  const size_t e = zr::elem_size(dt);
  const zr::Matrix mx = {x, rows, d, ld_x, e}, mr = {residual, rows, d, ld_residual, e},
                   mw = {weight, 1, d, d, e}, my = {y, rows, d, ld_y, e},
                   ms = {sum, rows, d, ld_sum, e};
  for (const zr::Matrix* m : {&mx, &mw, &my, &mr, &ms}) {
    if ((m == &mr || m == &ms) && !residual) continue;
    const zr_status st = zr::check_matrix(*m);
    if (st != ZR_OK) return st;
  }
  if (rows == 0) return ZR_OK;
  for (const zr::Matrix* out : {&my, &ms})
    if (zr::clash(mx, *out) || zr::clash(mr, *out) || zr::overlap(mw, *out)) return ZR_ERR_INVALID_ARG;
  if (zr::overlap(my, ms)) return ZR_ERR_INVALID_ARG;
  zr::NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.ld_x = ld_x;
  a.ld_res = ld_residual;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.y = y;
  a.sum = sum;
  a.ld_y = ld_y;
  a.ld_sum = ld_sum;
  a.rstd = rstd;
  return zr::norm_launch(a, dt, static_cast<cudaStream_t>(stream));
}

size_t zr_rms_norm_workspace_size(int64_t rows, int64_t d) {
  if (rows < 0 || rows > zr::kMaxDim || d < 1 || d > zr::kMaxDim) return 0;
  return zr::norm_backward_workspace_bytes(rows, d);
}

zr_status zr_rms_norm_backward(const void* s, int64_t ld_s, const void* weight, const float* rstd,
                               const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds,
                               int64_t rows, int64_t d, zr_dtype dt, int32_t accumulate, void* dx,
                               int64_t ld_dx, void* dweight, void* ws, size_t ws_bytes,
                               void* stream) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (rows < 0 || rows > zr::kMaxDim || d < 1 || d > zr::kMaxDim) return ZR_ERR_INVALID_ARG;
  if ((accumulate != 0 && accumulate != 1) || (!dx && !dweight)) return ZR_ERR_INVALID_ARG;
  const size_t e = zr::elem_size(dt);
  const zr::Matrix ms = {s, rows, d, ld_s, e}, mw = {weight, 1, d, d, e},
                   my = {dy, rows, d, ld_dy, e}, md = {ds, rows, d, ld_ds, e},
                   mx = {dx, rows, d, ld_dx, e}, mg = {dweight, 1, d, d, e};
  for (const zr::Matrix* m : {&ms, &mw, &my, &md, &mx, &mg}) {
    if ((m == &md && !ds) || (m == &mx && !dx) || (m == &mg && !dweight)) continue;
    const zr_status st = zr::check_matrix(*m);
    if (st != ZR_OK) return st;
  }
  if (rows > 0 && !rstd) return ZR_ERR_INVALID_ARG;
  for (const zr::Matrix* in : {&ms, &my, &md}) {
    if (in == &md && !ds) continue;
    if (dx && rows > 0 && zr::clash(*in, mx)) return ZR_ERR_INVALID_ARG;
    if (zr::overlap(*in, mg)) return ZR_ERR_INVALID_ARG;
  }
  if (zr::overlap(mw, mg) || zr::overlap(mw, mx) || zr::overlap(mx, mg)) return ZR_ERR_INVALID_ARG;
  if (dweight) {
    const zr_status st = zr::check_ws(ws, ws_bytes, zr::norm_backward_workspace_bytes(rows, d));
    if (st != ZR_OK) return st;
  }
  zr::NormBackArgs a = {};
  a.s = s;
  a.weight = weight;
  a.dy = dy;
  a.ds = ds;
  a.ld_s = ld_s;
  a.ld_dy = ld_dy;
  a.ld_ds = ld_ds;
  a.rstd = rstd;
  a.rows = rows;
  a.d = d;
  a.dx = dx;
  a.dweight = dweight;
  a.ld_dx = ld_dx;
  a.accumulate = accumulate;
  return zr::norm_backward_launch(a, dt, ws, static_cast<cudaStream_t>(stream));
}

size_t zr_cross_entropy_workspace_size(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w,
                                       int32_t dx, int32_t dw) {
  if (rows < 0 || rows > zr::kFfMostDim || d < 1 || d > zr::kFfMostDim || vocab < 1 ||
      vocab > zr::kFfMostDim || ld_w < d || (dx != 0 && dx != 1) || (dw != 0 && dw != 1))
    return 0;
  return zr::cross_entropy_workspace_bytes(rows, d, vocab, ld_w, dx, dw);
}

zr_status zr_cross_entropy_loss(const void* x, int64_t ld_x, const void* w_vocab, int64_t ld_w,
                                int64_t rows, int64_t d, int64_t vocab, zr_dtype dt,
                                const int32_t* target, const float* weight, float* loss,
                                float* lse, int32_t accumulate, void* dx, int64_t ld_dx, void* dw,
                                int64_t ld_dw, void* ws, size_t ws_bytes, void* stream) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (rows < 0 || rows > zr::kMaxDim || d < 1 || d > zr::kMaxDim || vocab < 1 || vocab > zr::kMaxDim)
    return ZR_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return ZR_ERR_INVALID_ARG;
  if (dt != ZR_BF16) return ZR_ERR_UNSUPPORTED;
  if (rows > zr::kFfMostDim || d > zr::kFfMostDim || vocab > zr::kFfMostDim) return ZR_ERR_UNSUPPORTED;
  const zr::Matrix mx = {x, rows, d, ld_x, 2}, mw = {w_vocab, vocab, d, ld_w, 2},
                   gx = {dx, rows, d, ld_dx, 2}, gw = {dw, vocab, d, ld_dw, 2};
  for (const zr::Matrix* m : {&mx, &mw, &gx, &gw}) {
    if ((m == &gx && !dx) || (m == &gw && !dw)) continue;
    const zr_status st = zr::check_matrix(*m);
    if (st != ZR_OK) return st;
  }
  if (ld_w % 8 == 0 && !zr::aligned16(w_vocab)) return ZR_ERR_ALIGNMENT;
  if (rows > 0 && !target) return ZR_ERR_INVALID_ARG;
  if (!loss && !lse && !dx && !dw) return ZR_ERR_INVALID_ARG;
  if (rows > 0 && (zr::overlap(mw, gx) || zr::clash(mx, gx) || zr::overlap(mx, gw) || zr::overlap(gx, gw)))
    return ZR_ERR_INVALID_ARG;
  if (zr::overlap(mw, gw)) return ZR_ERR_INVALID_ARG;
  if (!zr::cross_entropy_fits(rows, d, vocab, ld_w, dx != nullptr, dw != nullptr))
    return ZR_ERR_UNSUPPORTED;
  const zr_status st = zr::check_ws256(
      ws, ws_bytes, zr::cross_entropy_workspace_bytes(rows, d, vocab, ld_w, dx != nullptr, dw != nullptr));
  if (st != ZR_OK) return st;
  zr::CeArgs a = {};
  a.x = x;
  a.w = w_vocab;
  a.ld_x = ld_x;
  a.ld_w = ld_w;
  a.rows = rows;
  a.d = d;
  a.vocab = vocab;
  a.target = target;
  a.weight = weight;
  a.loss = loss;
  a.lse = lse;
  a.dx = dx;
  a.dw = dw;
  a.ld_dx = ld_dx;
  a.ld_dw = ld_dw;
  a.accumulate = accumulate;
  return zr::cross_entropy_launch(a, ws, static_cast<cudaStream_t>(stream));
}

size_t zr_orthogonalise_workspace_size(int64_t count, int64_t rows, int64_t cols) {
  if (count < 0 || count > zr::kMaxDim || rows < 1 || rows > zr::kMaxDim || cols < 1 || cols > zr::kMaxDim)
    return 0;
  return zr::orthogonalise_workspace_bytes(count, rows, cols);
}

zr_status zr_orthogonalise(const void* g, int64_t ld_g, int64_t step_g, int64_t count,
                           int64_t rows, int64_t cols, zr_dtype dt, const float* coefficients,
                           int32_t steps, float scale, float eps, void* out, int64_t ld_out,
                           int64_t step_out, void* ws, size_t ws_bytes, void* stream) {
  if (dt != ZR_F32 && dt != ZR_BF16) return ZR_ERR_INVALID_ARG;
  if (count < 0 || count > zr::kMaxDim || rows < 1 || rows > zr::kMaxDim || cols < 1 || cols > zr::kMaxDim)
    return ZR_ERR_INVALID_ARG;
  if (steps < 1 || steps > ZR_MAX_STEPS || !coefficients) return ZR_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * steps; ++i)
    if (!isfinite(coefficients[i])) return ZR_ERR_INVALID_ARG;
  if (!isfinite(scale) || !(eps >= 0.f && isfinite(eps))) return ZR_ERR_INVALID_ARG;
  if (count == 0) {  // (a status word from an earlier call is not this one's)
    if (!ws || ws_bytes < sizeof(int32_t)) return ZR_OK;
    return cudaMemsetAsync(ws, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ZR_OK
               : ZR_ERR_CUDA;
  }
  const zr::Matrix mg = {g, rows, cols, ld_g, zr::elem_size(dt)}, mo = {out, rows, cols, ld_out, 2};
  uintptr_t end_g = 0, end_o = 0;
  zr_status st = zr::check_batch(mg, count, step_g, false, &end_g);
  if (st == ZR_OK) st = zr::check_batch(mo, count, step_out, true, &end_o);
  if (st != ZR_OK) return st;
  const bool same = dt == ZR_BF16 && g == out && (rows == 1 || ld_g == ld_out) &&
                    (count == 1 || step_g == step_out);
  if (mg.begin() < end_o && mo.begin() < end_g && !same) return ZR_ERR_INVALID_ARG;
  if (!zr::orthogonalise_fits(count, rows, cols)) return ZR_ERR_UNSUPPORTED;
  st = zr::check_ws256(ws, ws_bytes, zr::orthogonalise_workspace_bytes(count, rows, cols));
  if (st != ZR_OK) return st;
  zr::OrthoArgs a = {};
  a.g = g;
  a.ld_g = ld_g;
  a.step_g = step_g;
  a.count = count;
  a.rows = rows;
  a.cols = cols;
  a.coefficients = coefficients;
  a.steps = steps;
  a.scale = scale;
  a.eps = eps;
  a.out = out;
  a.ld_out = ld_out;
  a.step_out = step_out;
  return zr::orthogonalise_launch(a, dt, ws, static_cast<cudaStream_t>(stream));
}

zr_status zr_query_status(const void* ws, void* stream, int32_t* status) {
  if (!ws || !status) return ZR_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(status, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return ZR_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return ZR_ERR_CUDA;
  return ZR_OK;
}

const char* zr_status_string(zr_status s) {
  switch (s) {
    case ZR_OK: return "ok";
    case ZR_ERR_INVALID_ARG: return "invalid argument";
    case ZR_ERR_UNSUPPORTED: return "unsupported";
    case ZR_ERR_ALIGNMENT: return "buffer not 16-byte aligned";
    case ZR_ERR_CAPACITY: return "output or workspace too small";
    case ZR_ERR_INPUT_UNSORTED: return "sparse indices not strictly ascending or out of range";
    case ZR_ERR_TIMEOUT: return "device wait timed out";
    case ZR_ERR_CUDA: return "CUDA error";
    case ZR_ERR_INTERNAL: return "internal consistency check failed on the device";
  }
  return "unknown status";
}

const char* zr_version(void) { return "zr 0.1.0 sm_103a"; }

}  // extern "C"
