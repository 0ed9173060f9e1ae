/*
 * zr.h -- C ABI of libzr: gradient aggregation across N data-parallel ranks
 * whose buffers all live in one GPU's memory, and operators of the training
 * step that makes those gradients.
 *
 * Pages the operations follow (cited by title and section):
 *   [SR]  "SkipReduce: (Interconnection) Network Sparsity to Accelerate
 *         Distributed Machine Learning" (MICRO'25 digest)
 *   [ZEN] "Zen: Empowering Distributed Training with Sparsity-driven Data
 *         Synchronization" (OSDI'25 digest)
 *   [CMU] "15642 Machine Learning Systems: Distributed Training and
 *         Parallelization" (CMU course notes)
 *
 * Conventions for every entry point:
 *   - Pointers named d_* / device buffers are CUDA device pointers; arrays of
 *     pointers (bufs, idx, val) and count arrays (nnz) are HOST arrays.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Every call is stream-ordered and asynchronous: it validates
 *     its arguments on the host, enqueues its kernels and returns.  Nothing
 *     is copied back to the host and nothing synchronises.
 *   - The caller owns every buffer, including the workspace `ws`; the library
 *     allocates no device or host memory.
 *   - The return value reports argument errors (checked before anything is
 *     enqueued; on error nothing is enqueued and no buffer is touched) and
 *     launch errors (ZR_ERR_CUDA).  Errors found by a kernel on the device
 *     (an unsorted or out-of-range sparse index) are written to a status
 *     word inside `ws`; read it with zr_query_status after the stream work.
 *   - zr_partition, zr_partition_static and zr_hash_index_sets are each one
 *     cooperative launch whose CTAs wait for one another once.  That wait is
 *     bounded: if the CTAs cannot all run at once (for example while another
 *     cooperative grid holds the device from a stream that is not ordered
 *     with this one) it gives up after about a second, the status word
 *     becomes ZR_ERR_TIMEOUT and the outputs are unspecified.  Order such
 *     calls on one stream, or with events.  Besides these, CTAs of one
 *     cluster, which the hardware runs together, wait for one another inside
 *     zr_gated_ff, zr_gated_ff_backward, zr_cross_entropy_loss, zr_orthogonalise
 *     and the losses over logits (zr_distill_loss,
 *     zr_policy_loss, zr_preference_loss); those waits give up after two
 *     seconds (a product's, whose length grows with its sum, after two seconds
 *     and 2 us for each 64 terms of it), and what they leave unknown is NaN.
 *   - No C++ exception crosses this interface.
 */
#ifndef ZR_H
#define ZR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zr_status {
  ZR_OK = 0,
  ZR_ERR_INVALID_ARG = 1,    /* a size, count, pointer or flag is out of range */
  ZR_ERR_UNSUPPORTED = 2,    /* a valid request this build does not implement */
  ZR_ERR_ALIGNMENT = 3,      /* a dense rank buffer or a workspace is not
                                16-byte aligned */
  ZR_ERR_CAPACITY = 4,       /* an output or workspace buffer is too small */
  ZR_ERR_INPUT_UNSORTED = 5, /* device-detected: sparse indices not strictly
                                ascending or outside [0, dense_size) */
  ZR_ERR_TIMEOUT = 6,        /* device-detected: a bounded wait gave up */
  ZR_ERR_CUDA = 7,           /* a CUDA runtime call or launch failed */
  ZR_ERR_INTERNAL = 8        /* device-detected: an internal consistency check
                                failed (the access was skipped) */
} zr_status;

typedef enum zr_dtype {
  ZR_F32 = 0,  /* IEEE binary32 */
  ZR_BF16 = 1  /* bfloat16: widened exactly to fp32, accumulated in fp32,
                  rounded once (round-to-nearest-even) on output */
} zr_dtype;

#define ZR_MAX_RANKS 64
#define ZR_MAX_PARTS 256

/* SkipReduce slice choice [SR section 4.2 (Static), section 4.3 (Random)]. */
typedef enum zr_skip_mode {
  ZR_SKIP_STATIC = 0, /* offset o = 0: slice c omits ranks c .. c+k-1 */
  ZR_SKIP_RANDOM = 1  /* offset o drawn from (seed, step), see zr_skip_cfg */
} zr_skip_mode;

/* What the reduced slice is divided by [SR section 4.1, and section 5's
 * SkipReduce vs DropReduce comparison]. */
typedef enum zr_divisor {
  ZR_DIV_N = 0,         /* SkipReduce average: skipped slices count as zero */
  ZR_DIV_N_MINUS_K = 1, /* DropReduce: skipped slices are removed */
  ZR_DIV_NONE = 2       /* plain sum */
} zr_divisor;

/*
 * SkipReduce configuration.
 *   mode     ZR_SKIP_STATIC or ZR_SKIP_RANDOM.
 *   k        Reduce-Scatter steps skipped, 0 <= k <= n-1 [SR Algorithm 2:
 *            the loop runs s = k .. N-2].  A skip fraction p maps to k = p*N.
 *   seed     Random mode: generator seed shared by every rank.
 *   step     Random mode: the iteration count [SR section 4.3].
 *   divisor  a zr_divisor value.
 * Random offset: o = floor(hi32(x) * n / 2^32), where x is output number
 * `step` (0-based) of SplitMix64 seeded with `seed` (Steele, Lea and Flood,
 * OOPSLA 2014): x = mix(seed + (step + 1) * 0x9E3779B97F4A7C15 mod 2^64),
 * mix(z) = z ^= z>>30; z *= 0xBF58476D1CE4E5B9; z ^= z>>27;
 *          z *= 0x94D049BB133111EB; z ^= z>>31.
 * With k = 0 the offset is 0 in both modes (p = 0 is exactly the plain ring).
 *   flags    0, or ZR_SKIP_RS_ONLY: run the Reduce-Scatter only [15-642
 *            notes, "ZeRO Stage 2": Reduce-Scatter replaces AllReduce and
 *            each GPU keeps only its own partition].  Slice c is then written
 *            only to its holder, rank (c - 1 - o) mod n, the rank where the
 *            Reduce-Scatter ends; every other element of every buffer keeps
 *            its input value.
 */
#define ZR_SKIP_RS_ONLY 1

typedef struct zr_skip_cfg {
  int32_t mode;
  int32_t k;
  uint64_t seed;
  uint64_t step;
  int32_t divisor;
  int32_t flags; /* 0 or ZR_SKIP_RS_ONLY */
} zr_skip_cfg;

/*
 * Ring all-reduce, in place [CMU "Ring AllReduce"; SR section 2 and
 * Algorithm 1 with p = 0].
 *
 * bufs     host array of n device pointers; bufs[r] is rank r's buffer of m
 *          elements of type dt, 16-byte aligned, pairwise non-overlapping.
 * n        ranks, 1 <= n <= ZR_MAX_RANKS.   m: elements per rank, >= 0.
 * average  0: every rank ends with the sum; 1: with the sum / n.
 *
 * Result, bit for bit: the tensor is cut into n slices of C = ceil(m/n)
 * elements (the last ones may be short or empty).  Element e of slice c ends,
 * on every rank, as fl(...fl(fl(g_c[e] + g_{c+1}[e]) + g_{c+2}[e]) ... +
 * g_{c+n-1}[e]) (ranks mod n; each + one fp32 RNE addition) -- the order in
 * which the Reduce-Scatter accumulates slice c, starting at the rank that
 * first sends it -- then divided by n with one fp32 RNE division when
 * average = 1, then (bf16) rounded once to bf16.  AllGather copies it to all
 * ranks.  m = 0 or n = 1 with average = 0 changes nothing.
 */
zr_status zr_ring_allreduce(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                            int32_t average, void* stream);

/*
 * SkipReduce all-reduce, in place [SR section 4.2 Algorithm 2, section 4.3].
 *
 * Arguments as zr_ring_allreduce, plus cfg (host pointer, see zr_skip_cfg).
 * Result: slice c is folded as above but starting at rank
 * s_c = (c + k - o) mod n and over the n - k ranks s_c .. s_c+n-k-1 only;
 * the k skipped ranks' values are not read.  The divisor is n, n - k or none.
 * With k = 0 and divisor ZR_DIV_N the result equals
 * zr_ring_allreduce(average = 1) bit for bit.
 */
zr_status zr_skipreduce(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                        const zr_skip_cfg* cfg, void* stream);

/*
 * Selective SkipReduce: several gradient buckets in one launch [SR section
 * 4.4: gradients are communicated in buckets, each its own AllReduce, so
 * each bucket can take its own skip rate -- aggressive for unimportant
 * layers, k = 0 for protected ones].
 *
 * buckets    host array of n_buckets entries, 1 <= n_buckets <=
 *            ZR_MAX_BUCKETS and n_buckets * n <= ZR_MAX_BUCKET_BUFS.
 *            Bucket b is bufs (host array of n device pointers, each
 *            16-byte aligned), m elements per rank buffer (>= 0) and its own
 *            zr_skip_cfg (mode, k, seed, step, divisor, flags), validated as
 *            for zr_skipreduce.  No two buffers of any buckets may overlap.
 * n, dt      ranks and element type, shared by every bucket.
 * Result: every bucket ends exactly as zr_skipreduce(bucket.bufs, n,
 * bucket.m, dt, &bucket.cfg) would leave it, bit for bit.  The caller gives
 * each bucket its own seed or step when buckets should skip different
 * slices.
 */
#define ZR_MAX_BUCKETS 128
#define ZR_MAX_BUCKET_BUFS 2048

typedef struct zr_bucket {
  void* const* bufs;
  int64_t m;
  zr_skip_cfg cfg;
} zr_bucket;

zr_status zr_skipreduce_buckets(const zr_bucket* buckets, int32_t n_buckets, int32_t n,
                                zr_dtype dt, void* stream);

/*
 * AllReduce_Dropout, in place [SR section 4.2, Algorithm 1 "AllReduce with
 * Fine-Grained Skipping": at every Reduce-Scatter step the receiving rank
 * skips its local gradient element with probability p, forwarding what it
 * received unchanged; the AllGather is the baseline one].
 *
 * Arguments as zr_ring_allreduce, plus:
 * threshold  T in [0, 2^32]: an element is skipped when its 32-bit draw is
 *            below T; T = ceil(p * 2^32) gives skip probability p (T = 0
 *            never skips, T = 2^32 always does).
 * seed, step generator seed shared by every rank, and the iteration count.
 * Draw of receiving rank r for element e (its index in the buffer): one
 * 32-bit half of output number floor(e / 2) of SplitMix64 seeded with
 * s_r = (output number step * 64 + r of SplitMix64 seeded with seed), the
 * high half for even e and the low half for odd e.
 * Result: slice c (as in zr_ring_allreduce) is folded from its first sender,
 * rank c, whose value is always kept; rank c + t (t = 1 .. n-1, mod n) adds
 * its value unless its draw for e is below T.  Then divided by n when
 * average = 1, (bf16) rounded once, and written to every rank.  Every rank's
 * element is read (skipping saves no traffic, as the pages note).
 */
zr_status zr_allreduce_dropout(void* const* bufs, int32_t n, int64_t m, zr_dtype dt,
                               uint64_t threshold, uint64_t seed, uint64_t step,
                               int32_t average, void* stream);

/*
 * Sparse (COO) aggregation with partitioning [ZEN section 2.1 (COO), Problem
 * 1, section 3.2 Technique #3 and Algorithm 1's first-level hash h0].
 *
 * idx, val, nnz  host arrays of n entries: rank r's list is nnz[r] entries at
 *                device pointers idx[r] (int32, strictly ascending, each in
 *                [0, dense_size)) and val[r] (fp32).  nnz[r] may be 0 (its
 *                pointers are then ignored).
 * n              ranks, 1 <= n <= ZR_MAX_RANKS.
 * dense_size     M, the dense tensor size, 1 <= M <= 2^31 - 1.
 * n_parts        partitions (servers), 0 <= n_parts <= ZR_MAX_PARTS;
 *                0 = no partitioning (plain ascending union).
 * part_seed      seed of h0.
 * average        0: sums; 1: sums divided once by n (fp32 RNE).
 * out_idx, out_val  device outputs of out_cap entries; out_cap must be at
 *                least sum(nnz) (checked here, so the kernels cannot write
 *                past it).
 * d_out_nnz      device int64: receives U, the union size.
 * d_offsets      device int64[n_parts + 1]: partition j is
 *                [d_offsets[j], d_offsets[j+1]); may be NULL if n_parts = 0.
 * ws, ws_bytes   device workspace of at least
 *                zr_sparse_workspace_size(n, dense_size, n_parts) bytes,
 *                16-byte aligned.  Its first 4 bytes are the status word.
 *
 * Result: one entry per index in the union of the n lists.  Its value is the
 * left fold, in ascending rank order, of the values of the ranks that hold
 * the index, starting from the first holder's value (fp32 RNE additions).
 * Partition of index x: h(x) = ((a*x + b) mod 2^64) >> 32,
 * p(x) = (h(x) * n_parts) >> 32, with a = (SplitMix64(part_seed) output 0) | 1
 * and b = output 1.  Entries are written partition-major, ascending index
 * inside each partition.
 * If an input list is not strictly ascending or holds an index outside
 * [0, dense_size), the status word becomes ZR_ERR_INPUT_UNSORTED and the
 * outputs are unspecified (every access still stays inside the buffers).
 */
zr_status zr_sparse_aggregate(const int32_t* const* idx, const float* const* val,
                              const int64_t* nnz, int32_t n, int64_t dense_size,
                              int32_t n_parts, uint64_t part_seed, int32_t average,
                              int32_t* out_idx, float* out_val, int64_t out_cap,
                              int64_t* d_out_nnz, int64_t* d_offsets,
                              void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes zr_sparse_aggregate needs (0 on invalid arguments).  The
 * kernels keep per-bin tables over the key range (bins of 1024 keys, wider
 * for very large dense sizes): bin starts per rank and per-bin counts and
 * positions per partition, so the size grows with dense_size * (n +
 * n_parts), not with the entry count. */
size_t zr_sparse_workspace_size(int32_t n, int64_t dense_size, int32_t n_parts);

/*
 * Push-side partition of one rank's COO list [ZEN Problem 1, requirement 1:
 * each worker splits its nonzeros into n parts with the shared h0].
 *
 * idx, val   device inputs of nnz entries (any order; indices need not be
 *            unique).  out_idx, out_val: device outputs of nnz entries.
 * d_offsets  device int64[n_parts + 1].   1 <= n_parts <= ZR_MAX_PARTS.
 * ws         device workspace of zr_partition_workspace_size(nnz, n_parts)
 *            bytes, 16-byte aligned.
 * Result: entries grouped by p(idx) (same h0 as above), partition-major; inside
 * a partition entries keep their input order (a stable split).
 */
zr_status zr_partition(const int32_t* idx, const float* val, int64_t nnz,
                       int32_t n_parts, uint64_t part_seed, int32_t* out_idx,
                       float* out_val, int64_t* d_offsets, void* ws,
                       size_t ws_bytes, void* stream);

/* Workspace bytes zr_partition needs (0 on invalid arguments); like the
 * union's, it does not grow with nnz (about 4 KB per partition). */
size_t zr_partition_workspace_size(int64_t nnz, int32_t n_parts);

/*
 * Zen's index sets [ZEN section 3.3.2 "Hash bitmap": the indices a worker
 * pushes to server p are I_p = {x in [0, M) : h0(x) = p}, computed once,
 * offline, and sorted].
 *
 * dense_size M, 1 <= M <= 2^31 - 1.   n_parts: 1 <= n_parts <= ZR_MAX_PARTS.
 * out_sets   device int32[M]: every I_p, ascending, concatenated in
 *            partition order (a permutation of 0 .. M-1).
 * d_offsets  device int64[n_parts + 1]: I_p = out_sets[d_offsets[p] ..
 *            d_offsets[p+1]).
 * ws         device workspace of zr_partition_workspace_size(M, n_parts)
 *            bytes, 16-byte aligned.
 * h0 is the partition hash of zr_sparse_aggregate (same part_seed).
 */
zr_status zr_hash_index_sets(int64_t dense_size, int32_t n_parts, uint64_t part_seed,
                             int32_t* out_sets, int64_t* d_offsets, void* ws, size_t ws_bytes,
                             void* stream);

/*
 * Zen's index sets as a directory [ZEN section 3.3.2 "Hash bitmap":
 * I_p = {x in [0, M) : h0(x) = p}, ascending, fixed for the whole run].  The
 * hash bitmap calls below use this directory instead of the index sets; it
 * is built once per (M, n_parts, part_seed), in two launches, and holds
 * NB = ceil(log2 n_parts) bits per index instead of the index sets' 32.
 *
 * dense_size M, 1 <= M <= 2^31 - 1.   n_parts: 1 <= n_parts <= ZR_MAX_PARTS.
 * d_dir      device buffer of zr_hash_directory_size(M, n_parts) bytes,
 *            16-byte aligned.  With R = ceil(M / ZR_HASH_RANGE) and S = R + 1
 *            rounded up to a multiple of 4, it holds
 *            header  256 bytes: int64 magic, M, n_parts, part_seed;
 *            counts  int32, from byte 256: entry [p S + r], r <= R, is
 *                    |{x < min(r ZR_HASH_RANGE, M) : h0(x) = p}|, so entry
 *                    [p S + R] is |I_p|;
 *            slices  uint64, from byte 256 + ceil(n_parts S 4 / 256) 256:
 *                    word [(r NB + b) 32 + l] has bit k set iff bit b of
 *                    h0(r ZR_HASH_RANGE + 64 l + k) is set (bits of indices
 *                    at or past M unspecified).
 *            The encode and decode calls read it; they report
 *            ZR_ERR_INVALID_ARG, and write nothing, for a directory built
 *            for another (M, n_parts, part_seed), and they check every
 *            range's counts against the slices.
 * h0 is the partition hash of zr_sparse_aggregate (same part_seed).
 */
#define ZR_HASH_RANGE 2048
size_t zr_hash_directory_size(int64_t dense_size, int32_t n_parts);
zr_status zr_hash_directory(int64_t dense_size, int32_t n_parts, uint64_t part_seed,
                            int32_t* d_dir, size_t dir_bytes, void* stream);

/*
 * Hash bitmap encode [ZEN section 3.3.2, Figure 10, Algorithm 2
 * hash_bitmap_encode: a server marks which elements of I_p are nonzero,
 * one bit each, so that all servers' bitmaps total |G| bits].
 *
 * d_dir                 the directory of (dense_size, n_parts, part_seed).
 * keys, n_keys   device int32: the nonzero indices (any order, each in
 *                [0, M)), e.g. the out_idx of zr_sparse_aggregate.
 * out_bits       device uint32[out_cap_words], out_cap_words >=
 *                ceil(M / 32) + n_parts.  Partition p's bitmap is
 *                ceil(|I_p| / 32) words from word d_word_offsets[p]; bit j
 *                (bit j mod 32 of word j / 32, least significant first) is 1
 *                iff I_p[j] is one of the keys; padding bits are 0.
 * d_word_offsets device int64[n_parts + 1] (output).
 * ws             device workspace of zr_hash_bitmap_workspace_size(M,
 *                n_parts) bytes, 16-byte aligned; its first 4 bytes are the
 *                status word (ZR_ERR_INPUT_UNSORTED: a key outside [0, M);
 *                ZR_ERR_INVALID_ARG: a directory that does not match h0).
 * Four launches: two memsets, the membership marks, the encode.
 */
zr_status zr_hash_bitmap_encode(const int32_t* d_dir, int64_t dense_size, int32_t n_parts,
                                uint64_t part_seed, const int32_t* keys, int64_t n_keys,
                                uint32_t* out_bits, int64_t out_cap_words,
                                int64_t* d_word_offsets, void* ws, size_t ws_bytes, void* stream);

/*
 * Hash bitmap decode [ZEN section 3.3.2, Algorithm 2 hash_bitmap_decode: a
 * worker maps the set bits j of server p's bitmap back to the indices
 * I_p[j]].
 *
 * d_dir          the directory of (dense_size, n_parts, part_seed).
 * bits           device uint32 bitmaps laid out as zr_hash_bitmap_encode
 *                writes them (partition p from word sum_{q<p} ceil(|I_q|/32));
 *                the buffer holds at least the sum_q ceil(|I_q|/32) words the
 *                directory gives (ceil(M / 32) + n_parts always suffices).
 * out_keys       device int32[out_cap]: partition-major, ascending inside a
 *                partition (the indices I_p[j] of the set bits j).
 * d_key_offsets  device int64[n_parts + 1] (output): partition p's keys are
 *                out_keys[d_key_offsets[p] .. d_key_offsets[p+1]).
 * ws             as for encode.  Status: ZR_ERR_CAPACITY if more keys than
 *                out_cap (nothing is written past it), ZR_ERR_INVALID_ARG if a
 *                padding bit is set or the directory does not match h0.
 * Four launches: the status memset, the segment counts, their scan, the
 * decode.
 */
zr_status zr_hash_bitmap_decode(const int32_t* d_dir, int64_t dense_size, int32_t n_parts,
                                uint64_t part_seed, const uint32_t* bits, int32_t* out_keys,
                                int64_t out_cap, int64_t* d_key_offsets, void* ws,
                                size_t ws_bytes, void* stream);

/* Workspace bytes zr_hash_bitmap_encode / _decode need (0 on invalid
 * arguments): the status word, an M-bit membership map and 4 bytes per
 * partition per ZR_HASH_RANGE indices. */
size_t zr_hash_bitmap_workspace_size(int64_t dense_size, int32_t n_parts);

/*
 * Densification of rank groups, measured on the device [ZEN Definition 4
 * and section 2.3: the densification ratio gamma_k of aggregating k sparse
 * tensors decides between the two optimal schemes].
 *
 * idx, nnz, n, dense_size  as zr_sparse_aggregate (values are not needed);
 *                n must be a power of two, 1 <= n <= ZR_MAX_RANKS.
 * d_union_counts device int64[log2(n) + 1] (output): entry L is the sum,
 *                over the n / 2^L groups of 2^L consecutive ranks
 *                (ranks i*2^L .. (i+1)*2^L - 1), of the size of the union of
 *                the group's index lists.  Entry 0 is sum(nnz); entry log2(n)
 *                is the size of the whole union.
 * ws, ws_bytes   device workspace of zr_densification_workspace_size(n,
 *                dense_size) bytes, 16-byte aligned; status word first
 *                (ZR_ERR_INPUT_UNSORTED as for zr_sparse_aggregate).
 */
zr_status zr_densification(const int32_t* const* idx, const int64_t* nnz, int32_t n,
                           int64_t dense_size, int64_t* d_union_counts, void* ws,
                           size_t ws_bytes, void* stream);

size_t zr_densification_workspace_size(int32_t n, int64_t dense_size);

/*
 * Zen's scheme choice [ZEN Theorem 1 and Equations (1), (2)], on the host.
 *
 * union_counts  host int64[log2(n) + 1], as zr_densification writes them.
 * gamma_k = union_counts[L] * k / union_counts[0] for k = 2^L (the mean
 * union of a k-group over the mean per-rank count).  Balanced parallelism
 * costs t_bp = 2 (n-1) (gamma_n + 1) / n, hierarchical centralisation
 * t_hc = 2 sum_{i=1}^{log2 n} gamma_{2^(i-1)} (both in units of d_G M / b).
 * gammas, t_bp, t_hc  optional host outputs (gammas has log2(n) + 1 slots).
 * Returns ZR_SCHEME_BALANCED (also on a tie) or ZR_SCHEME_HIERARCHICAL, or
 * -1 on invalid arguments (n not a power of two in [2, 64], a count < 0, or
 * union_counts[0] = 0).
 */
#define ZR_SCHEME_BALANCED 0
#define ZR_SCHEME_HIERARCHICAL 1

int32_t zr_choose_scheme(const int64_t* union_counts, int32_t n, double* gammas, double* t_bp,
                         double* t_hc);

/*
 * zr_partition without a workspace argument, for callers that cannot
 * allocate device memory (for example a gradient hook running inside a
 * framework whose caching allocator owns the device, or a service that
 * reserves all device memory at start-up).  The pages have no counterpart:
 * it exists only for such callers.
 *
 * Arguments and result are those of zr_partition minus ws / ws_bytes.  The
 * scratch is a fixed array of ZR_STATIC_SCRATCH_BYTES inside the library on
 * every device that loads it.  It holds what zr_partition_workspace_size
 * asks for at every valid nnz and n_parts (at most about 1 MiB), so every
 * valid request fits; a request that did not would return ZR_ERR_CAPACITY
 * and enqueue nothing.  The library never calls cudaMalloc or cudaFree
 * here.  The first call on a device (with that device current) looks up the
 * array's device address and keeps it for the process; make that first call
 * before any stream capture, and do not call this entry point on a device
 * after cudaDeviceReset, which can move the array.  All calls on a device
 * share the array (each call clears what must start at zero), so calls that
 * overlap on the GPU race.
 */
#define ZR_STATIC_SCRATCH_BYTES (2u << 20)
zr_status zr_partition_static(const int32_t* idx, const float* val, int64_t nnz,
                              int32_t n_parts, uint64_t part_seed, int32_t* out_idx,
                              float* out_val, int64_t* d_offsets, void* stream);

/*
 * Testing only: makes the CTA with index `cta` skip its arrival at the grid
 * wait of the next cooperative launches (zr_partition, zr_partition_static,
 * zr_hash_index_sets), so that every other CTA's
 * bounded wait runs out and the status word becomes ZR_ERR_TIMEOUT; -1 (the
 * default) turns it off.  A process-wide setting, for tests of the timeout
 * path; no GPU faults or hangs because of it.
 */
void zr_test_barrier_skip(int32_t cta);

/*
 * ---------------------------------------------------------------------------
 * The training step before the aggregation: one gated feed-forward block
 * with its gradients, and three losses over a vocabulary with theirs.  The
 * weight gradients can be written into (or added to) a rank's buffer, from
 * where the calls above average them.
 *
 * Conventions of these calls, on top of the ones at the top of this file:
 *   - Matrices are row-major with a leading dimension ld (elements between
 *     the starts of two rows, at least the row's length).
 *   - Inputs and outputs must not overlap, except where a call says so.
 *   - Every result depends on the inputs alone: repeating a call repeats its
 *     bits.
 * ---------------------------------------------------------------------------
 */

/* Activations a(g) of the gated block. */
typedef enum zr_act {
  ZR_ACT_SILU = 0,     /* g / (1 + exp(-g)) */
  ZR_ACT_GELU = 1,     /* g (1 + erf(g / sqrt 2)) / 2 */
  ZR_ACT_GELU_TANH = 2 /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
} zr_act;

/*
 * Gated feed-forward block: both projections, the activation and the product
 * in one kernel.
 *   g = x Wg^T,  u = x Wu^T,  h = a(g) u   (elementwise)
 *
 * x        [rows, d], ld_x.        w_gate, w_up  [f, d], both with ld_w.
 * h        [rows, f], ld_h: the result.
 * rows >= 0; d, f >= 1; each at most 2^31 - 513 (past that, up to 2^31 - 1,
 * ZR_ERR_UNSUPPORTED).   dt must be ZR_BF16 (ZR_ERR_UNSUPPORTED otherwise):
 * products and sums in fp32, g and u are not rounded, h is rounded once.
 * x, w_gate and w_up must be 16-byte aligned, except that a matrix whose ld
 * is not a multiple of 8 may start anywhere (it is laid out again in the
 * workspace first).  h may start anywhere.
 * ws       workspace of zr_gated_ff_workspace_size(rows, d, f, ld_x, ld_w, 0)
 *          bytes, 256-byte aligned; may be NULL when that is 0 (both strides
 *          are multiples of 8).  Where one is given (of at least 4 bytes), its
 *          first 4 bytes become the status word: ZR_ERR_TIMEOUT if a wait
 *          inside a kernel gave up.  Outputs that such a wait leaves unknown
 *          are NaN, with or without a workspace.
 * rows = 0 does nothing.
 */
zr_status zr_gated_ff(const void* x, int64_t ld_x, const void* w_gate, const void* w_up,
                      int64_t ld_w, int64_t rows, int64_t d, int64_t f, zr_dtype dt, int32_t act,
                      void* h, int64_t ld_h, void* ws, size_t ws_bytes, void* stream);

/*
 * Its gradients, from the inputs and dh alone (g and u are computed again,
 * nothing is kept from the forward call):
 *   dg = dh u a'(g),  du = dh a(g)
 *   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
 *
 * dh       [rows, f], ld_dh.   dx  [rows, d], ld_dx.
 * dw_gate, dw_up  [f, d], both with ld_dw.
 * accumulate  0: the weight gradients are written; 1: they are added to what
 *          dw_gate and dw_up hold (the sum in fp32, rounded once), for
 *          several micro-batches into one rank buffer.
 * dx may be NULL (not wanted), and dw_gate and dw_up may both be NULL.
 * f at most 2^30 - 513 (ZR_ERR_UNSUPPORTED past that); rows and d as above.
 * dg and du are rounded to bf16 once, before the products that use them; all
 * sums are fp32.  Alignment as for zr_gated_ff; dh, dx, dw_gate and dw_up
 * may start anywhere (a weight gradient can be a slice of a flat rank
 * buffer).
 * rows = 0: the weight gradients become 0 (accumulate = 0) or stay as they
 * are (accumulate = 1).
 * ws       workspace of zr_gated_ff_workspace_size(rows, d, f, ld_x, ld_w, 1)
 *          bytes, as for zr_gated_ff.
 */
zr_status zr_gated_ff_backward(const void* x, int64_t ld_x, const void* w_gate, const void* w_up,
                               int64_t ld_w, const void* dh, int64_t ld_dh, int64_t rows,
                               int64_t d, int64_t f, zr_dtype dt, int32_t act, int32_t accumulate,
                               void* dx, int64_t ld_dx, void* dw_gate, void* dw_up, int64_t ld_dw,
                               void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of the two calls above (backward: 0 or 1); 0 where none is
 * needed, and on invalid arguments. */
size_t zr_gated_ff_workspace_size(int64_t rows, int64_t d, int64_t f, int64_t ld_x, int64_t ld_w,
                                  int32_t backward);

/*
 * The three losses below share these arguments:
 *
 * logits   [rows, vocab], ld_logits, of type dt (ZR_F32 or ZR_BF16), aligned
 *          to its element only; rows >= 0, 1 <= vocab <= 2^31 - 65536.
 * dlogits  [rows, vocab], ld_dlogits, of type dt: the gradient of the sum of
 *          all losses; NULL when only the losses are wanted.  It may be
 *          logits itself with the same ld (the gradient replaces them).
 * q        denotes softmax(logits[t, :] / temperature), computed in fp32; the
 *          gradient is rounded once.
 * A row that is left out (its weight is 0, its target is negative, or all its
 * logits are -inf) has loss 0 and a gradient of zeros; the logits of a row
 * left out by its weight or target are not read, so they may hold anything.
 * A NaN or +inf logit makes the row's loss and gradient NaN.
 * weight   fp32 per row (or pair): multiplies loss and gradient (a mean over
 *          tokens is a weight of 1 / tokens); NULL for ones.
 */

/*
 * Distillation from a teacher's top logits: KL(p || q) per row.
 *
 * top_idx    int32 [rows, k], ld_top: the tokens of the teacher's list.  An
 *            entry outside [0, vocab) is padding and not read further; the
 *            others of a row must be distinct (the row's result is
 *            unspecified if not).   0 <= k <= ZR_MAX_TOP.
 * top_logit  fp32 [rows, k], ld_top: the teacher's logits of those tokens
 *            (-inf: probability 0).
 * teacher_lse  NULL: p = softmax(top_logit / temperature) over the list, and
 *            0 elsewhere.  Otherwise fp32 [rows], log sum exp of the
 *            teacher's whole row of logits / temperature:
 *            p_i = exp(top_logit_i / temperature - lse), and the rest of the
 *            mass, p_rest = max(0, 1 - sum p_i), is one more class whose
 *            student probability is the sum of q outside the list.
 * loss       fp32 [rows]: weight * sum_i p_i (log p_i - log q_i), over the
 *            classes with p_i > 0.  NULL when only the gradient is wanted.
 * Gradient of a row, times weight / temperature: q_j - p_j on the list; off
 * the list q_j, or q_j (1 - p_rest / q_rest) with teacher_lse.
 * A row with an empty list (or whose list has no mass) is left out when
 * teacher_lse is NULL.  With teacher_lse, a p_rest <= 2^-20 (the rounding of
 * its sum) is none where q has less than 2^-126 outside the list; a larger one
 * gives +inf where q has nothing there at all (every other logit is -inf).
 */
#define ZR_MAX_TOP 1024
zr_status zr_distill_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                          int64_t vocab, const int32_t* top_idx, const float* top_logit, int32_t k,
                          int64_t ld_top, const float* teacher_lse, float temperature,
                          const float* weight, float* loss, void* dlogits, int64_t ld_dlogits,
                          void* stream);

/*
 * Clipped policy loss with a KL term, per token (row).
 *
 * action     int32 [rows]: the token taken; negative: the row is left out; at
 *            or past vocab: an error, the row's outputs become NaN.
 * advantage  fp32 [rows] (A).
 * old_logp   fp32 [rows]: log q of the action under the policy that took it;
 *            NULL: the present one (ratio 1).
 * ref_logp   fp32 [rows]: under the reference policy; may be NULL if kl_coef
 *            is 0 (kl is then 0).
 * With logp = log q[action], r = exp(logp - old_logp), c = r clamped to
 * [1 - clip_low, 1 + clip_high], x = ref_logp - logp:
 *   kl = exp(x) - x - 1   (+inf where exp(x) is)
 *   loss = weight (kl_coef kl - min(r A, c A))
 *   gradient = weight (kl_coef (1 - exp(x)) - [r A <= c A] r A)
 *              (1{j = action} - q_j) / temperature
 * loss, logp, kl  fp32 [rows] each, or NULL.  A row that is left out has 0 in
 * all three.
 * clip_low in [0, 1], clip_high >= 0, kl_coef >= 0, temperature > 0, finite.
 */
zr_status zr_policy_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                         int64_t vocab, const int32_t* action, const float* advantage,
                         const float* old_logp, const float* ref_logp, float clip_low,
                         float clip_high, float kl_coef, float temperature, const float* weight,
                         float* loss, float* logp, float* kl, void* dlogits, int64_t ld_dlogits,
                         void* stream);

/*
 * Preference loss over pairs of sequences, by the log ratios to a reference.
 *
 * target     int32 [rows]: the row's next token; negative: the row is left
 *            out (a prompt); at or past vocab: an error, the status word
 *            becomes ZR_ERR_INVALID_ARG and the row is left out.
 * offsets    device int64 [2 pairs + 1], ascending (equal is an empty
 *            sequence), within [0, rows]: sequence s has the rows offsets[s]
 *            .. offsets[s+1] - 1; sequence 2p is pair p's chosen one and
 *            2p + 1 its rejected one.  Rows outside every sequence are left
 *            out.  A pair whose offsets are not such gets the status
 *            ZR_ERR_INVALID_ARG, a NaN loss and no gradient; a row that two other
 *            pairs then share gets the gradient of one of them.
 * ref_logp   fp32 [rows]: log probability of the target under the reference.
 * D_s = sum over the rows of s of (log q[target] - ref_logp); the temperature
 * is 1.  With m = beta (D_chosen - D_rejected):
 *   loss = weight (-(1 - eps) log sigma(m) - eps log sigma(-m)),
 *   eps = label_smoothing   (a part of weight 0 is 0, also where m is infinite)
 * loss       fp32 [pairs].   reward  fp32 [2 pairs] or NULL: beta D_s.
 * weight     fp32 [pairs] or NULL; a pair of weight 0 has loss 0 and no
 *            gradient (its logits are read).
 * beta > 0, finite; eps in [0, 1]; pairs >= 0, at most 2^24.
 * With dlogits, rows times the row's parts of 32 KB must be at most 2^31 - 1
 * (ZR_ERR_UNSUPPORTED).
 * ws         workspace of zr_preference_workspace_size(rows) bytes, 16-byte
 *            aligned; its first 4 bytes are the status word.
 */
zr_status zr_preference_loss(const void* logits, int64_t ld_logits, zr_dtype dt, int64_t rows,
                             int64_t vocab, const int32_t* target, const int64_t* offsets,
                             int32_t pairs, const float* ref_logp, float beta,
                             float label_smoothing, const float* weight, float* loss,
                             float* reward, void* dlogits, int64_t ld_dlogits, void* ws,
                             size_t ws_bytes, void* stream);

/* Workspace bytes of zr_preference_loss (0 on invalid arguments). */
size_t zr_preference_workspace_size(int64_t rows);

/*
 * ---------------------------------------------------------------------------
 * The rest of the step, with the conventions above: the norm that a block reads, the
 * next token's cross entropy from the states themselves, and the update that an
 * averaged weight gradient becomes.
 * ---------------------------------------------------------------------------
 */

/*
 * Root-mean-square norm with the residual's addition, per row.
 *   s = x + residual   (rounded to the type; s = x without a residual)
 *   rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd weight
 *
 * x, residual, y, sum  [rows, d], each with its ld, of type dt (ZR_F32 or ZR_BF16).
 * weight   [d], of the same type.
 * sum      s, for the next block and the backward pass; with a residual only (both or
 *          neither is NULL).
 * rstd     fp32 [rows] or NULL.
 * y and sum may each replace x or the residual (the same address and ld); apart from
 * that no output overlaps anything.  All matrices may start at any element.
 * rows >= 0, d >= 1, both at most 2^31 - 1; eps > 0, finite.  Sums in fp32; a row whose
 * squares leave fp32's range is summed again from values of 2^-80 their size.
 */
zr_status zr_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                      const void* weight, int64_t rows, int64_t d, zr_dtype dt, float eps, void* y,
                      int64_t ld_y, void* sum, int64_t ld_sum, float* rstd, void* stream);

/*
 * Its gradients.  With h = s rstd:
 *   dx = rstd (dy weight - h mean(dy weight h)) + ds,   dweight = sum over rows of dy h
 *
 * s, dy, ds, dx  [rows, d], each with its ld.   weight, dweight  [d].
 * rstd     fp32 [rows], as zr_rms_norm gave it.
 * ds       the gradient that reaches s along the residual; NULL for none.  dx is the
 *          gradient of x and of the residual alike.
 * dx or dweight may be NULL (not wanted).  dx may replace s, dy or ds (the same address
 * and ld).
 * accumulate  1: dweight is added to (the sum in fp32, rounded once).
 * rows = 0: dweight becomes 0 (accumulate = 0) or stays as it is.
 * ws       workspace of zr_rms_norm_workspace_size(rows, d) bytes, 16-byte aligned;
 *          may be NULL without dweight.  It holds no status word.
 */
zr_status zr_rms_norm_backward(const void* s, int64_t ld_s, const void* weight, const float* rstd,
                               const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds,
                               int64_t rows, int64_t d, zr_dtype dt, int32_t accumulate, void* dx,
                               int64_t ld_dx, void* dweight, void* ws, size_t ws_bytes,
                               void* stream);

/* Workspace bytes of zr_rms_norm_backward (0 on invalid arguments). */
size_t zr_rms_norm_workspace_size(int64_t rows, int64_t d);

/*
 * Softmax cross entropy of token states over a vocabulary, per row, with the gradients
 * of the states and of the vocabulary's weights.  The logits are not given out; for the
 * gradients a piece of them is held in the workspace, in 16 bits.
 *   z = x W^T,   lse = log sum_j exp(z_j),   loss = weight (lse - z[target])
 *   dz = weight (softmax(z) - one-hot(target)),   dx = dz W,   dW = dz^T x
 *
 * x        [rows, d], ld_x: may start at any element.
 * w_vocab  [vocab, d], ld_w: 16-byte aligned, except where ld_w is not a multiple of 8
 *          (it is then laid out again in the workspace first).
 * dt must be ZR_BF16 (ZR_ERR_UNSUPPORTED otherwise): products, sums and softmax in
 * fp32.  rows >= 0; d, vocab >= 1; each at most 2^31 - 513.
 * target   int32 [rows]; negative: the row is left out; at or past vocab: an error, the
 *          status word becomes ZR_ERR_INVALID_ARG and the row is left out.
 * weight   fp32 [rows] or NULL for ones.
 * loss, lse  fp32 [rows], each or NULL.
 * dx       [rows, d], ld_dx, or NULL: the gradient of the sum of all losses.  It may be
 *          x itself with the same ld.
 * dw       [vocab, d], ld_dw, or NULL.   accumulate  1: dw is added to (the sum in
 *          fp32, rounded once), for several micro-batches into one rank buffer.  dx and
 *          dw may start at any element.
 * A row that is left out (its target is negative, its weight 0, or all its logits are
 * -inf) has loss 0 and a zero dx, and adds nothing to dw; the states of one left out by
 * its target or weight are not read, so they may hold anything.  Its lse is 0.  A NaN
 * or +inf logit makes the row's loss and dx NaN, and dw.
 * For the gradients the logits of a piece of the rows are held in 16 bits, as distances
 * to a maximum in steps of 2^-10 octaves (0 past 64 octaves), and dz, in units of the
 * largest finite weight, is rounded to bf16 once before its products.  A piece is all
 * rows, or 4096 where there are more than 4096 + 2 d (than 4096 without dw) or than 2^18.
 * ws       workspace of zr_cross_entropy_workspace_size(rows, d, vocab, ld_w, dx is
 *          wanted, dw is wanted) bytes, 256-byte aligned; its first 4 bytes are the
 *          status word (ZR_ERR_TIMEOUT too, as for zr_gated_ff).
 * rows = 0: dw becomes 0 (accumulate = 0) or stays as it is.
 */
zr_status zr_cross_entropy_loss(const void* x, int64_t ld_x, const void* w_vocab, int64_t ld_w,
                                int64_t rows, int64_t d, int64_t vocab, zr_dtype dt,
                                const int32_t* target, const float* weight, float* loss,
                                float* lse, int32_t accumulate, void* dx, int64_t ld_dx, void* dw,
                                int64_t ld_dw, void* ws, size_t ws_bytes, void* stream);

/* Its workspace bytes on the current device (dx, dw: 0 or 1); 0 on invalid arguments and
 * for sizes that the call does not take (ZR_ERR_UNSUPPORTED). */
size_t zr_cross_entropy_workspace_size(int64_t rows, int64_t d, int64_t vocab, int64_t ld_w,
                                       int32_t dx, int32_t dw);

/*
 * Orthogonalised matrices by Newton-Schulz steps: what a momentum update of a weight
 * matrix becomes in the Muon optimiser.  For each matrix of a batch:
 *   X = G / (|G|_F + eps), then for each step, with its a, b, c:
 *   A = X X^T,  X <- a X + (b A + c A A) X     (on the shorter side: with X^T X where
 *                                               there are more rows than columns)
 *   out = scale X
 *
 * g        count matrices [rows, cols] with ld_g, step_g elements from one to the next;
 *          type dt (ZR_F32 or ZR_BF16); may start at any element.
 * out      bf16, the same with ld_out and step_out: one behind the other, or beside one
 *          another in the same rows.  It may be g itself (dt ZR_BF16, the same strides),
 *          and overlaps it in no other way.
 * coefficients  HOST array of 3 steps floats: a, b, c of each step.
 * 1 <= steps <= ZR_MAX_STEPS; eps >= 0; scale and coefficients finite.  count >= 0;
 * rows, cols >= 1; count times rows (up to a multiple of 64), and cols, at most
 * 2^31 - 513 (ZR_ERR_UNSUPPORTED past that).
 * X between the steps, A and the polynomial are held in fp16 times 2^11, with fp32 sums.
 * So a step may be given singular values of X up to 5.6 (A has their squares, up to 31.9)
 * and may have a polynomial of up to 31.9 over them (at 0 too, which is a, where X has
 * directions of 0); coefficients that lead past that may overflow: infinities or NaN.
 * The last step's X has bf16's range.  Values under 2^-25 have fewer bits than the others,
 * and those under 2^-36 are 0: coefficients that shrink X or the polynomial that far lose it.
 * A matrix of zeros gives zeros; one with a NaN or an infinity gives NaN, and leaves
 * the batch's others as they are.
 * ws       workspace of zr_orthogonalise_workspace_size(count, rows, cols) bytes,
 *          256-byte aligned; its first 4 bytes are the status word (ZR_ERR_TIMEOUT, as
 *          for zr_gated_ff).
 */
#define ZR_MAX_STEPS 32
zr_status zr_orthogonalise(const void* g, int64_t ld_g, int64_t step_g, int64_t count,
                           int64_t rows, int64_t cols, zr_dtype dt, const float* coefficients,
                           int32_t steps, float scale, float eps, void* out, int64_t ld_out,
                           int64_t step_out, void* ws, size_t ws_bytes, void* stream);

/* Its workspace bytes; 0 on invalid arguments and for sizes that the call does not take
 * (ZR_ERR_UNSUPPORTED). */
size_t zr_orthogonalise_workspace_size(int64_t count, int64_t rows, int64_t cols);

/*
 * Read the device status word at the start of a workspace: waits for
 * `stream`, copies the word to *status.  Returns ZR_ERR_CUDA if the copy
 * fails, ZR_ERR_INVALID_ARG for NULL pointers, else ZR_OK.
 */
zr_status zr_query_status(const void* ws, void* stream, int32_t* status);

/* Static English description of a status code (never NULL). */
const char* zr_status_string(zr_status s);

/* Library version string, e.g. "zr 0.1.0 sm_103a". */
const char* zr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZR_H */
