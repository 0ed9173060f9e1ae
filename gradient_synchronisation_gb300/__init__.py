"""gradient_synchronisation_gb300 -- Python binding of libzr (``include/zr.h``).

Gradient aggregation across N data-parallel ranks whose buffers all live in
one GPU's memory: the ring all-reduce with SkipReduce slice skipping and the
fused average (dense), and the Zen-style COO union with rank-ordered sums and
the h0 partition (sparse).  Before the aggregation stand the operators of a
worker's training step: the gated feed-forward block with its gradients, and
the distillation, policy and preference losses over a vocabulary with theirs;
around them the root-mean-square norm, the cross entropy from token states with
the vocabulary's weights, and, behind the average, the orthogonalised update.
Every step runs in the library's CUDA kernels;
this module only marshals arguments (pointers, sizes, the stream handle) into
the C ABI.  There is no CPU fallback: the library is loaded on the first call,
and if ``libzr.so`` has not been built that call raises ImportError.  (Loading
lazily lets ``gradient_synchronisation_gb300._build`` run before the library
exists.)

Two layers:

* ``zr_ring_allreduce``, ``zr_skipreduce``, ``zr_skipreduce_buckets``,
  ``zr_allreduce_dropout``, ``zr_sparse_aggregate``, ``zr_partition``,
  ``zr_query_status`` ... -- the C entry points under their own names, taking
  integers for pointers and streams; they return the ``zr_status`` code.
* ``ring_allreduce``, ``skipreduce``, ``skipreduce_buckets``,
  ``allreduce_dropout``, ``sparse_aggregate``, ``partition``, ``gated_ff``,
  ``gated_ff_backward``, ``distill_loss``, ``policy_loss``,
  ``preference_loss``, ``rms_norm``, ``rms_norm_backward``,
  ``cross_entropy_loss``, ``orthogonalise`` -- the same calls taking torch CUDA
  tensors, raising ``ZrError`` on a non-OK status.  PyTorch supplies device
  memory and the current stream only.
"""

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzr.so")

ZR_OK = 0
ZR_ERR_INVALID_ARG = 1
ZR_ERR_UNSUPPORTED = 2
ZR_ERR_ALIGNMENT = 3
ZR_ERR_CAPACITY = 4
ZR_ERR_INPUT_UNSORTED = 5
ZR_ERR_TIMEOUT = 6
ZR_ERR_CUDA = 7
ZR_ERR_INTERNAL = 8

ZR_F32 = 0
ZR_BF16 = 1
ZR_SKIP_STATIC = 0
ZR_SKIP_RANDOM = 1
ZR_DIV_N = 0
ZR_DIV_N_MINUS_K = 1
ZR_DIV_NONE = 2
ZR_MAX_RANKS = 64
ZR_MAX_PARTS = 256
ZR_HASH_RANGE = 2048
ZR_SKIP_RS_ONLY = 1
ZR_MAX_BUCKETS = 128
ZR_MAX_BUCKET_BUFS = 2048
ZR_ACT_SILU = 0
ZR_ACT_GELU = 1
ZR_ACT_GELU_TANH = 2
ZR_MAX_TOP = 1024
ZR_MAX_STEPS = 32

EXPORTS = (
    "zr_ring_allreduce", "zr_skipreduce", "zr_sparse_aggregate", "zr_sparse_workspace_size",
    "zr_partition", "zr_partition_workspace_size", "zr_query_status", "zr_status_string",
    "zr_version", "zr_partition_static", "zr_skipreduce_buckets", "zr_allreduce_dropout",
    "zr_hash_index_sets", "zr_hash_directory", "zr_hash_directory_size",
    "zr_hash_bitmap_encode", "zr_hash_bitmap_decode",
    "zr_hash_bitmap_workspace_size", "zr_densification", "zr_densification_workspace_size",
    "zr_choose_scheme", "zr_test_barrier_skip", "zr_gated_ff", "zr_gated_ff_backward",
    "zr_gated_ff_workspace_size", "zr_distill_loss", "zr_policy_loss", "zr_preference_loss",
    "zr_preference_workspace_size", "zr_rms_norm", "zr_rms_norm_backward",
    "zr_rms_norm_workspace_size", "zr_cross_entropy_loss", "zr_cross_entropy_workspace_size",
    "zr_orthogonalise", "zr_orthogonalise_workspace_size",
)
ZR_SCHEME_BALANCED = 0
ZR_SCHEME_HIERARCHICAL = 1
ZR_STATIC_SCRATCH_BYTES = 2 << 20


class ZrError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


class SkipCfg(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("k", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("step", ctypes.c_uint64), ("divisor", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class Bucket(ctypes.Structure):
    _fields_ = [("bufs", ctypes.POINTER(ctypes.c_void_p)), ("m", ctypes.c_int64),
                ("cfg", SkipCfg)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libzr.so is not built (%s); run gradient_synchronisation_gb300._build.build()"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    i32, i64, u64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    f32 = ctypes.c_float
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "zr_ring_allreduce": (i32, [PP, i32, i64, i32, i32, P]),
        "zr_skipreduce": (i32, [PP, i32, i64, i32, ctypes.POINTER(SkipCfg), P]),
        "zr_sparse_aggregate": (i32, [PP, PP, ctypes.POINTER(i64), i32, i64, i32, u64, i32, P, P,
                                      i64, P, P, P, sz, P]),
        "zr_sparse_workspace_size": (sz, [i32, i64, i32]),
        "zr_partition": (i32, [P, P, i64, i32, u64, P, P, P, P, sz, P]),
        "zr_partition_workspace_size": (sz, [i64, i32]),
        "zr_query_status": (i32, [P, P, ctypes.POINTER(i32)]),
        "zr_status_string": (ctypes.c_char_p, [i32]),
        "zr_version": (ctypes.c_char_p, []),
        "zr_partition_static": (i32, [P, P, i64, i32, u64, P, P, P, P]),
        "zr_skipreduce_buckets": (i32, [ctypes.POINTER(Bucket), i32, i32, i32, P]),
        "zr_allreduce_dropout": (i32, [PP, i32, i64, i32, u64, u64, u64, i32, P]),
        "zr_hash_index_sets": (i32, [i64, i32, u64, P, P, P, sz, P]),
        "zr_hash_directory": (i32, [i64, i32, u64, P, sz, P]),
        "zr_hash_directory_size": (sz, [i64, i32]),
        "zr_hash_bitmap_encode": (i32, [P, i64, i32, u64, P, i64, P, i64, P, P, sz, P]),
        "zr_hash_bitmap_decode": (i32, [P, i64, i32, u64, P, P, i64, P, P, sz, P]),
        "zr_hash_bitmap_workspace_size": (sz, [i64, i32]),
        "zr_densification": (i32, [PP, ctypes.POINTER(i64), i32, i64, P, P, sz, P]),
        "zr_densification_workspace_size": (sz, [i32, i64]),
        "zr_test_barrier_skip": (None, [i32]),
        "zr_gated_ff": (i32, [P, i64, P, P, i64, i64, i64, i64, i32, i32, P, i64, P, sz, P]),
        "zr_gated_ff_backward": (i32, [P, i64, P, P, i64, P, i64, i64, i64, i64, i32, i32, i32, P,
                                       i64, P, P, i64, P, sz, P]),
        "zr_gated_ff_workspace_size": (sz, [i64, i64, i64, i64, i64, i32]),
        "zr_distill_loss": (i32, [P, i64, i32, i64, i64, P, P, i32, i64, P, f32, P, P, P, i64, P]),
        "zr_policy_loss": (i32, [P, i64, i32, i64, i64, P, P, P, P, f32, f32, f32, f32, P, P, P, P,
                                 P, i64, P]),
        "zr_preference_loss": (i32, [P, i64, i32, i64, i64, P, P, i32, P, f32, f32, P, P, P, P, i64,
                                     P, sz, P]),
        "zr_preference_workspace_size": (sz, [i64]),
        "zr_rms_norm": (i32, [P, i64, P, i64, P, i64, i64, i32, f32, P, i64, P, i64, P, P]),
        "zr_rms_norm_backward": (i32, [P, i64, P, P, P, i64, P, i64, i64, i64, i32, i32, P, i64, P, P,
                                       sz, P]),
        "zr_rms_norm_workspace_size": (sz, [i64, i64]),
        "zr_cross_entropy_loss": (i32, [P, i64, P, i64, i64, i64, i64, i32, P, P, P, P, i32, P, i64,
                                        P, i64, P, sz, P]),
        "zr_cross_entropy_workspace_size": (sz, [i64, i64, i64, i64, i32, i32]),
        "zr_orthogonalise": (i32, [P, i64, i64, i64, i64, i64, i32, ctypes.POINTER(f32), i32, f32,
                                   f32, P, i64, i64, P, sz, P]),
        "zr_orthogonalise_workspace_size": (sz, [i64, i64, i64]),
        "zr_choose_scheme": (i32, [ctypes.POINTER(i64), i32, ctypes.POINTER(ctypes.c_double),
                                   ctypes.POINTER(ctypes.c_double),
                                   ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib_handle = None


def lib():
    """The loaded libzr (ctypes.CDLL); loads it on first use."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load()
    return _lib_handle


def _ptrs(values):
    arr = (ctypes.c_void_p * max(1, len(values)))()
    for i, v in enumerate(values):
        arr[i] = v
    return arr


# ------------------------------------------------------------ C entry points
def zr_ring_allreduce(bufs, n, m, dtype, average, stream):
    return lib().zr_ring_allreduce(_ptrs(bufs), n, m, dtype, average, stream)


def zr_skipreduce(bufs, n, m, dtype, cfg, stream):
    return lib().zr_skipreduce(_ptrs(bufs), n, m, dtype, ctypes.byref(cfg), stream)


def zr_skipreduce_buckets(buckets, n, dtype, stream):
    """``buckets``: list of (list of n pointers, m, SkipCfg)."""
    arr = (Bucket * max(1, len(buckets)))()
    keep = []
    for i, (bufs, m, cfg) in enumerate(buckets):
        p = _ptrs(bufs)
        keep.append(p)
        arr[i].bufs = ctypes.cast(p, ctypes.POINTER(ctypes.c_void_p))
        arr[i].m = m
        arr[i].cfg = cfg
    return lib().zr_skipreduce_buckets(arr, len(buckets), n, dtype, stream)


def zr_allreduce_dropout(bufs, n, m, dtype, threshold, seed, step, average, stream):
    return lib().zr_allreduce_dropout(_ptrs(bufs), n, m, dtype, threshold, seed, step, average,
                                      stream)


def zr_hash_index_sets(dense_size, n_parts, part_seed, out_sets, d_offsets, ws, ws_bytes, stream):
    return lib().zr_hash_index_sets(dense_size, n_parts, part_seed, out_sets, d_offsets, ws,
                                    ws_bytes, stream)


def zr_hash_directory_size(dense_size, n_parts):
    return lib().zr_hash_directory_size(dense_size, n_parts)


def zr_hash_directory(dense_size, n_parts, part_seed, d_dir, dir_bytes, stream):
    return lib().zr_hash_directory(dense_size, n_parts, part_seed, d_dir, dir_bytes, stream)


def zr_hash_bitmap_workspace_size(dense_size, n_parts):
    return lib().zr_hash_bitmap_workspace_size(dense_size, n_parts)


def zr_hash_bitmap_encode(d_dir, dense_size, n_parts, part_seed, keys, n_keys, out_bits,
                          out_cap_words, d_word_offsets, ws, ws_bytes, stream):
    return lib().zr_hash_bitmap_encode(d_dir, dense_size, n_parts, part_seed, keys, n_keys,
                                       out_bits, out_cap_words, d_word_offsets, ws, ws_bytes,
                                       stream)


def zr_hash_bitmap_decode(d_dir, dense_size, n_parts, part_seed, bits, out_keys, out_cap,
                          d_key_offsets, ws, ws_bytes, stream):
    return lib().zr_hash_bitmap_decode(d_dir, dense_size, n_parts, part_seed, bits, out_keys,
                                       out_cap, d_key_offsets, ws, ws_bytes, stream)


def zr_densification(idx, nnz, n, dense_size, d_union_counts, ws, ws_bytes, stream):
    nnz_arr = (ctypes.c_int64 * max(1, len(nnz)))(*nnz)
    return lib().zr_densification(_ptrs(idx), nnz_arr, n, dense_size, d_union_counts, ws,
                                  ws_bytes, stream)


def zr_densification_workspace_size(n, dense_size):
    return lib().zr_densification_workspace_size(n, dense_size)


def zr_choose_scheme(union_counts, n):
    """Host call: returns (choice, gammas, t_bp, t_hc); choice -1 on invalid
    arguments."""
    levels = max(1, len(union_counts))
    uc = (ctypes.c_int64 * levels)(*union_counts)
    g = (ctypes.c_double * 8)()
    bp, hc = ctypes.c_double(0), ctypes.c_double(0)
    choice = lib().zr_choose_scheme(uc, n, g, ctypes.byref(bp), ctypes.byref(hc))
    return choice, list(g)[:len(union_counts)], bp.value, hc.value


def zr_sparse_aggregate(idx, val, nnz, n, dense_size, n_parts, part_seed, average, out_idx,
                        out_val, out_cap, d_out_nnz, d_offsets, ws, ws_bytes, stream):
    nnz_arr = (ctypes.c_int64 * max(1, len(nnz)))(*nnz)
    return lib().zr_sparse_aggregate(_ptrs(idx), _ptrs(val), nnz_arr, n, dense_size, n_parts,
                                    part_seed, average, out_idx, out_val, out_cap, d_out_nnz,
                                    d_offsets, ws, ws_bytes, stream)


def zr_sparse_workspace_size(n, dense_size, n_parts):
    return lib().zr_sparse_workspace_size(n, dense_size, n_parts)


def zr_test_barrier_skip(cta):
    """Testing only: the CTA ``cta`` skips its grid-wait arrival (-1: off)."""
    lib().zr_test_barrier_skip(cta)


def zr_partition(idx, val, nnz, n_parts, part_seed, out_idx, out_val, d_offsets, ws, ws_bytes,
                 stream):
    return lib().zr_partition(idx, val, nnz, n_parts, part_seed, out_idx, out_val, d_offsets, ws,
                             ws_bytes, stream)


def zr_partition_static(idx, val, nnz, n_parts, part_seed, out_idx, out_val, d_offsets, stream):
    """zr_partition with the library's own fixed scratch (no workspace)."""
    return lib().zr_partition_static(idx, val, nnz, n_parts, part_seed, out_idx, out_val,
                                     d_offsets, stream)


def zr_partition_workspace_size(nnz, n_parts):
    return lib().zr_partition_workspace_size(nnz, n_parts)


def zr_gated_ff(x, ld_x, w_gate, w_up, ld_w, rows, d, f, dtype, act, h, ld_h, ws, ws_bytes, stream):
    return lib().zr_gated_ff(x, ld_x, w_gate, w_up, ld_w, rows, d, f, dtype, act, h, ld_h, ws,
                             ws_bytes, stream)


def zr_gated_ff_backward(x, ld_x, w_gate, w_up, ld_w, dh, ld_dh, rows, d, f, dtype, act, accumulate,
                         dx, ld_dx, dw_gate, dw_up, ld_dw, ws, ws_bytes, stream):
    return lib().zr_gated_ff_backward(x, ld_x, w_gate, w_up, ld_w, dh, ld_dh, rows, d, f, dtype,
                                      act, accumulate, dx, ld_dx, dw_gate, dw_up, ld_dw, ws,
                                      ws_bytes, stream)


def zr_gated_ff_workspace_size(rows, d, f, ld_x, ld_w, backward):
    return lib().zr_gated_ff_workspace_size(rows, d, f, ld_x, ld_w, backward)


def zr_distill_loss(logits, ld_logits, dtype, rows, vocab, top_idx, top_logit, k, ld_top,
                    teacher_lse, temperature, weight, loss, dlogits, ld_dlogits, stream):
    return lib().zr_distill_loss(logits, ld_logits, dtype, rows, vocab, top_idx, top_logit, k,
                                 ld_top, teacher_lse, temperature, weight, loss, dlogits,
                                 ld_dlogits, stream)


def zr_policy_loss(logits, ld_logits, dtype, rows, vocab, action, advantage, old_logp, ref_logp,
                   clip_low, clip_high, kl_coef, temperature, weight, loss, logp, kl, dlogits,
                   ld_dlogits, stream):
    return lib().zr_policy_loss(logits, ld_logits, dtype, rows, vocab, action, advantage, old_logp,
                                ref_logp, clip_low, clip_high, kl_coef, temperature, weight, loss,
                                logp, kl, dlogits, ld_dlogits, stream)


def zr_preference_loss(logits, ld_logits, dtype, rows, vocab, target, offsets, pairs, ref_logp,
                       beta, label_smoothing, weight, loss, reward, dlogits, ld_dlogits, ws,
                       ws_bytes, stream):
    return lib().zr_preference_loss(logits, ld_logits, dtype, rows, vocab, target, offsets, pairs,
                                    ref_logp, beta, label_smoothing, weight, loss, reward, dlogits,
                                    ld_dlogits, ws, ws_bytes, stream)


def zr_preference_workspace_size(rows):
    return lib().zr_preference_workspace_size(rows)


def zr_rms_norm(x, ld_x, residual, ld_residual, weight, rows, d, dtype, eps, y, ld_y, sum, ld_sum,
                rstd, stream):
    return lib().zr_rms_norm(x, ld_x, residual, ld_residual, weight, rows, d, dtype, eps, y, ld_y,
                             sum, ld_sum, rstd, stream)


def zr_rms_norm_backward(s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, rows, d, dtype, accumulate,
                         dx, ld_dx, dweight, ws, ws_bytes, stream):
    return lib().zr_rms_norm_backward(s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, rows, d, dtype,
                                      accumulate, dx, ld_dx, dweight, ws, ws_bytes, stream)


def zr_rms_norm_workspace_size(rows, d):
    return lib().zr_rms_norm_workspace_size(rows, d)


def zr_cross_entropy_loss(x, ld_x, w_vocab, ld_w, rows, d, vocab, dtype, target, weight, loss, lse,
                          accumulate, dx, ld_dx, dw, ld_dw, ws, ws_bytes, stream):
    return lib().zr_cross_entropy_loss(x, ld_x, w_vocab, ld_w, rows, d, vocab, dtype, target, weight,
                                       loss, lse, accumulate, dx, ld_dx, dw, ld_dw, ws, ws_bytes,
                                       stream)


def zr_cross_entropy_workspace_size(rows, d, vocab, ld_w, dx, dw):
    return lib().zr_cross_entropy_workspace_size(rows, d, vocab, ld_w, dx, dw)


def zr_orthogonalise(g, ld_g, step_g, count, rows, cols, dtype, coefficients, scale, eps, out,
                     ld_out, step_out, ws, ws_bytes, stream):
    """``coefficients``: a sequence of three floats for each step."""
    c = (ctypes.c_float * max(1, len(coefficients)))(*coefficients)
    return lib().zr_orthogonalise(g, ld_g, step_g, count, rows, cols, dtype, c,
                                  len(coefficients) // 3, scale, eps, out, ld_out, step_out, ws,
                                  ws_bytes, stream)


def zr_orthogonalise_workspace_size(count, rows, cols):
    return lib().zr_orthogonalise_workspace_size(count, rows, cols)


def zr_query_status(ws, stream):
    out = ctypes.c_int32(-1)
    st = lib().zr_query_status(ws, stream, ctypes.byref(out))
    if st != ZR_OK:
        raise ZrError(st, "zr_query_status")
    return out.value


def status_string(status):
    return lib().zr_status_string(status).decode()


def version():
    return lib().zr_version().decode()


# ------------------------------------------------------------ torch wrappers
def _stream(stream):
    import torch

    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return ZR_F32
    if t.dtype == torch.bfloat16:
        return ZR_BF16
    raise TypeError("dense buffers must be float32 or bfloat16, got %s" % t.dtype)


def _check(st, where):
    if st != ZR_OK:
        raise ZrError(st, where)


def _dense_args(bufs):
    if len(bufs) == 0:
        raise ValueError("need at least one rank buffer")
    m = bufs[0].numel()
    dt = _dtype_code(bufs[0])
    for b in bufs:
        if not b.is_cuda or not b.is_contiguous() or b.numel() != m or _dtype_code(b) != dt:
            raise ValueError("rank buffers must be contiguous CUDA tensors of one size and dtype")
    return [b.data_ptr() for b in bufs], len(bufs), m, dt


def ring_allreduce(bufs, average=True, stream=None):
    """In-place ring all-reduce of the rank buffers ``bufs`` (list of tensors)."""
    ptrs, n, m, dt = _dense_args(bufs)
    _check(zr_ring_allreduce(ptrs, n, m, dt, 1 if average else 0, _stream(stream)),
           "zr_ring_allreduce")


def skipreduce(bufs, k, mode=ZR_SKIP_RANDOM, seed=0, step=0, divisor=ZR_DIV_N, rs_only=False,
               stream=None):
    """In-place SkipReduce all-reduce skipping ``k`` Reduce-Scatter steps
    (``rs_only``: Reduce-Scatter only, each slice written to its holder)."""
    ptrs, n, m, dt = _dense_args(bufs)
    cfg = SkipCfg(mode, k, seed, step, divisor, ZR_SKIP_RS_ONLY if rs_only else 0)
    _check(zr_skipreduce(ptrs, n, m, dt, cfg, _stream(stream)), "zr_skipreduce")


def skipreduce_buckets(buckets, stream=None):
    """Selective SkipReduce over several buckets in one launch.

    ``buckets``: list of dicts with ``bufs`` (list of rank tensors) and the
    ``skipreduce`` keywords ``k``, ``mode``, ``seed``, ``step``, ``divisor``,
    ``rs_only`` (k = 0 protects a bucket).  All buckets share N and dtype.
    """
    args, n, dt = [], None, None
    for b in buckets:
        ptrs, bn, m, bdt = _dense_args(b["bufs"])
        if n is None:
            n, dt = bn, bdt
        elif bn != n or bdt != dt:
            raise ValueError("every bucket needs the same number of ranks and dtype")
        cfg = SkipCfg(b.get("mode", ZR_SKIP_RANDOM), b.get("k", 0), b.get("seed", 0),
                      b.get("step", 0), b.get("divisor", ZR_DIV_N),
                      ZR_SKIP_RS_ONLY if b.get("rs_only", False) else 0)
        args.append((ptrs, m, cfg))
    _check(zr_skipreduce_buckets(args, n, dt, _stream(stream)), "zr_skipreduce_buckets")


def dropout_threshold(p):
    """Integer threshold T = ceil(p * 2^32) for skip probability p in [0, 1]."""
    from fractions import Fraction

    q = Fraction(p)
    if not (0 <= q <= 1):
        raise ValueError("p must be in [0, 1]")
    t = q * (1 << 32)
    return -(-t.numerator // t.denominator)


def allreduce_dropout(bufs, p, seed=0, step=0, average=True, stream=None):
    """In-place AllReduce_Dropout: each receiving rank skips its local element
    with probability ``p`` (SkipReduce's ReduceOrSkip)."""
    ptrs, n, m, dt = _dense_args(bufs)
    _check(zr_allreduce_dropout(ptrs, n, m, dt, dropout_threshold(p), seed, step,
                                1 if average else 0, _stream(stream)), "zr_allreduce_dropout")


def skip_fraction_to_k(p, n):
    """SkipReduce skip fraction p -> number of skipped steps k = p*N (the pages:
    skipping k Reduce-Scatter steps skips k/N of the gradients)."""
    k = p * n
    if abs(k - round(k)) > 1e-9 or not (0 <= round(k) <= n - 1):
        raise ValueError("skip fraction %r needs p*N to be an integer in [0, N-1]" % (p,))
    return int(round(k))


class SparseWorkspace:
    """Device workspace and outputs for ``sparse_aggregate`` (torch-allocated)."""

    def __init__(self, n, dense_size, n_parts, capacity, device):
        import torch

        ws_bytes = zr_sparse_workspace_size(n, dense_size, n_parts)
        if ws_bytes == 0:
            raise ValueError("invalid sparse workspace request")
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        self.out_idx = torch.empty(max(1, capacity), dtype=torch.int32, device=device)
        self.out_val = torch.empty(max(1, capacity), dtype=torch.float32, device=device)
        self.out_nnz = torch.zeros(1, dtype=torch.int64, device=device)
        self.offsets = torch.zeros(max(n_parts, 1) + 1, dtype=torch.int64, device=device)
        self.capacity = capacity
        self.n_parts = n_parts


def sparse_aggregate(idx_list, val_list, dense_size, n_parts, part_seed=0, average=False,
                     work=None, stream=None):
    """Union with rank-ordered sums, partitioned by h0.  Returns the workspace
    object whose ``out_idx``/``out_val``/``out_nnz``/``offsets`` hold the result
    (device tensors; nothing is copied to the host)."""
    n = len(idx_list)
    nnz = [int(a.numel()) for a in idx_list]
    for a, v in zip(idx_list, val_list):
        if a.dtype.itemsize != 4 or not a.is_cuda or not v.is_cuda or a.numel() != v.numel():
            raise ValueError("idx must be int32 and val float32 CUDA tensors of equal length")
    if work is None:
        work = SparseWorkspace(n, dense_size, n_parts, sum(nnz), idx_list[0].device)
    st = zr_sparse_aggregate([a.data_ptr() for a in idx_list], [v.data_ptr() for v in val_list],
                             nnz, n, dense_size, n_parts, part_seed, 1 if average else 0,
                             work.out_idx.data_ptr(), work.out_val.data_ptr(), work.capacity,
                             work.out_nnz.data_ptr(), work.offsets.data_ptr(), work.ws.data_ptr(),
                             work.ws.numel(), _stream(stream))
    _check(st, "zr_sparse_aggregate")
    return work


def partition(idx, val, n_parts, part_seed=0, out_idx=None, out_val=None, offsets=None, ws=None,
              stream=None):
    """Stable h0 partition of one COO list; returns (out_idx, out_val, offsets)."""
    import torch

    nnz = int(idx.numel())
    dev = idx.device
    out_idx = torch.empty(max(1, nnz), dtype=torch.int32, device=dev) if out_idx is None else out_idx
    out_val = torch.empty(max(1, nnz), dtype=torch.float32, device=dev) if out_val is None else out_val
    offsets = torch.empty(n_parts + 1, dtype=torch.int64, device=dev) if offsets is None else offsets
    if ws is None:
        ws = torch.empty(max(16, zr_partition_workspace_size(nnz, n_parts)), dtype=torch.uint8,
                         device=dev)
    st = zr_partition(idx.data_ptr(), val.data_ptr(), nnz, n_parts, part_seed, out_idx.data_ptr(),
                      out_val.data_ptr(), offsets.data_ptr(), ws.data_ptr(), ws.numel(),
                      _stream(stream))
    _check(st, "zr_partition")
    return out_idx, out_val, offsets


# ------------------------------------------------------------ hash bitmap
class HashBitmap:
    """Zen's hash bitmaps of a dense size, partition count and h0 seed: the
    directory of index-set counts built once on the device, and the encode /
    decode calls that use it.  ``bits`` and ``keys`` results are torch
    tensors (bitmap words stored as int32)."""

    def __init__(self, dense_size, n_parts, part_seed=0, device="cuda", stream=None):
        import torch

        self.m, self.parts, self.seed = dense_size, n_parts, part_seed
        n_dir = zr_hash_directory_size(dense_size, n_parts)
        n_ws = zr_hash_bitmap_workspace_size(dense_size, n_parts)
        if n_dir == 0 or n_ws == 0:
            raise ValueError("invalid hash bitmap request")
        self.directory = torch.empty(n_dir // 4, dtype=torch.int32, device=device)
        _check(zr_hash_directory(dense_size, n_parts, part_seed, self.directory.data_ptr(), n_dir,
                                 _stream(stream)), "zr_hash_directory")
        self.ws = torch.empty(n_ws, dtype=torch.uint8, device=device)
        self.cap_words = (dense_size + 31) // 32 + n_parts
        self.bits = torch.empty(self.cap_words, dtype=torch.int32, device=device)
        self.word_offsets = torch.empty(n_parts + 1, dtype=torch.int64, device=device)

    def encode(self, keys, stream=None):
        """Bitmaps of the nonzero indices ``keys`` (int32 CUDA tensor)."""
        _check(zr_hash_bitmap_encode(self.directory.data_ptr(), self.m, self.parts, self.seed,
                                     keys.data_ptr() if keys.numel() else None, keys.numel(),
                                     self.bits.data_ptr(), self.cap_words,
                                     self.word_offsets.data_ptr(), self.ws.data_ptr(),
                                     self.ws.numel(), _stream(stream)), "zr_hash_bitmap_encode")
        return self.bits, self.word_offsets

    def decode(self, bits, out_keys, key_offsets, stream=None):
        """Indices of the set bits of ``bits`` (laid out as ``encode``
        writes them) into ``out_keys``; partition offsets into
        ``key_offsets``."""
        _check(zr_hash_bitmap_decode(self.directory.data_ptr(), self.m, self.parts, self.seed,
                                     bits.data_ptr(), out_keys.data_ptr(), out_keys.numel(),
                                     key_offsets.data_ptr(), self.ws.data_ptr(), self.ws.numel(),
                                     _stream(stream)), "zr_hash_bitmap_decode")
        return out_keys, key_offsets

    def status(self, stream=None):
        return zr_query_status(self.ws.data_ptr(), _stream(stream))


def hash_index_sets(dense_size, n_parts, part_seed=0, device="cuda", stream=None):
    """Zen's index sets I_p of [0, dense_size) on the device: (sets, offsets)
    with I_p = sets[offsets[p]:offsets[p+1]], each ascending."""
    import torch

    sets = torch.empty(dense_size, dtype=torch.int32, device=device)
    offsets = torch.empty(n_parts + 1, dtype=torch.int64, device=device)
    ws = torch.empty(max(16, zr_partition_workspace_size(dense_size, n_parts)),
                     dtype=torch.uint8, device=device)
    _check(zr_hash_index_sets(dense_size, n_parts, part_seed, sets.data_ptr(), offsets.data_ptr(),
                              ws.data_ptr(), ws.numel(), _stream(stream)), "zr_hash_index_sets")
    torch.cuda.synchronize()  # one-time build; the workspace is freed on return
    return sets, offsets


def densification(idx_list, dense_size, stream=None):
    """Union sizes of groups of 2^L consecutive ranks (int64 CUDA tensor of
    log2(n) + 1 entries), measured on the device."""
    import torch

    n = len(idx_list)
    nnz = [int(a.numel()) for a in idx_list]
    dev = idx_list[0].device
    ws_bytes = zr_densification_workspace_size(n, dense_size)
    if ws_bytes == 0:
        raise ValueError("densification needs a power-of-two rank count and a valid dense size")
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    out = torch.empty(n.bit_length(), dtype=torch.int64, device=dev)
    _check(zr_densification([a.data_ptr() for a in idx_list], nnz, n, dense_size, out.data_ptr(),
                            ws.data_ptr(), ws_bytes, _stream(stream)), "zr_densification")
    return out, ws


def choose_scheme(union_counts, n):
    """Zen's choice between balanced parallelism and hierarchical
    centralisation from measured union sizes (host)."""
    choice, g, bp, hc = zr_choose_scheme([int(v) for v in union_counts], n)
    if choice < 0:
        raise ValueError("invalid union counts or rank count")
    return choice, g, bp, hc


# ------------------------------------------------------------ the training step
# These calls may be as short as a few microseconds on the device, so their
# wrappers look up what they need once and build no stream objects.
_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch

        _torch = torch
    return _torch


def _run_on(stream, call, first, *args):
    """The call with ``stream`` (a torch stream or a handle) as torch's current stream on
    the device of its first tensor, so that the memory it allocates belongs to the stream
    that uses it."""
    torch = _t()
    here = first.device
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=here if here.type == "cuda" else None)
    elif here.type == "cuda" and stream.device != here:
        raise ValueError("a stream of %s for a tensor on %s" % (stream.device, here))
    with torch.cuda.stream(stream):
        return call(first, *args)


def _current(t):
    """Handle of the current stream of a tensor's device."""
    return _torch._C._cuda_getCurrentRawStream(t.get_device())


def _type(t):
    dt = t.dtype
    if dt == _torch.bfloat16:
        return ZR_BF16
    if dt == _torch.float32:
        return ZR_F32
    raise TypeError("tensors must be float32 or bfloat16, got %s" % dt)


class _Scratch:
    """A workspace for one call: the caller's tensor, or bytes of torch's caching
    allocator that go back to the call's stream when it has been enqueued
    (a tensor of its own costs several microseconds more)."""

    __slots__ = ("ptr", "size", "mine")

    def __init__(self, ws, need, stream):
        if ws is not None:
            if not ws.is_cuda or not ws.is_contiguous():
                raise ValueError("ws must be a contiguous CUDA tensor, got one on %s" % ws.device)
            self.ptr, self.size, self.mine = ws.data_ptr(), ws.numel() * ws.element_size(), False
        else:
            self.ptr = _torch._C._cuda_cudaCachingAllocator_raw_alloc(need, stream) if need else 0
            self.size, self.mine = need, bool(need)

    def done(self):
        if self.mine:
            _torch._C._cuda_cudaCachingAllocator_raw_delete(self.ptr)


# The workspace sizes are functions of these numbers alone.
@functools.lru_cache(maxsize=1024)
def _ff_workspace(rows, d, f, ld_x, ld_w, backward):
    return lib().zr_gated_ff_workspace_size(rows, d, f, ld_x, ld_w, backward)


@functools.lru_cache(maxsize=1024)
def _preference_workspace(rows):
    return lib().zr_preference_workspace_size(rows)


def _matrix(t, what, dtype, shape):
    """Pointer and leading dimension of a 2-D CUDA tensor with contiguous rows."""
    if t.shape != shape or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor of shape %s, got %s on %s"
                         % (what, tuple(shape), tuple(t.shape), t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    ld, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError("%s must have contiguous rows" % what)
    # one row has no second one to step to: any stride is its length
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1])


def _vector(t, what, dtype, n):
    """Pointer of a contiguous 1-D CUDA tensor of n entries (None: NULL)."""
    if t is None:
        return None
    if t.shape != (n,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor of %d entries" % (what, n))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    return t.data_ptr()


def _rows_cols(t, what):
    if t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % what)
    return t.shape


def _ff_args(x, w_gate, w_up):
    rows, d = _rows_cols(x, "x")
    f = _rows_cols(w_gate, "w_gate")[0]
    dt = _type(x)
    xp, ld_x = _matrix(x, "x", x.dtype, (rows, d))
    gp, ld_w = _matrix(w_gate, "w_gate", x.dtype, (f, d))
    up, ld_u = _matrix(w_up, "w_up", x.dtype, (f, d))
    if ld_w != ld_u:
        raise ValueError("w_gate and w_up must have the same row stride")
    return rows, d, f, dt, xp, ld_x, gp, up, ld_w


def gated_ff(x, w_gate, w_up, activation=ZR_ACT_SILU, out=None, ws=None, stream=None):
    """h = a(x w_gate^T) * (x w_up^T) for x [rows, d] and weights [f, d] (bfloat16)."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, gated_ff, x, w_gate, w_up, activation, out, ws)
    rows, d, f, dt, xp, ld_x, gp, up, ld_w = _ff_args(x, w_gate, w_up)
    if out is None:
        out = torch.empty((rows, f), dtype=x.dtype, device=x.device)
    hp, ld_h = _matrix(out, "out", x.dtype, (rows, f))
    s = _current(x)
    w = _Scratch(ws, _ff_workspace(rows, d, f, ld_x, ld_w, 0), s)
    try:
        st = lib().zr_gated_ff(xp, ld_x, gp, up, ld_w, rows, d, f, dt, activation, hp, ld_h, w.ptr,
                               w.size, s)
    finally:
        w.done()
    _check(st, "zr_gated_ff")
    return out


def gated_ff_backward(x, w_gate, w_up, dh, activation=ZR_ACT_SILU, dx=None, dw_gate=None,
                      dw_up=None, accumulate=False, ws=None, stream=None):
    """Gradients of ``gated_ff`` from its inputs and dh: (dx, dw_gate, dw_up).
    ``dw_gate`` and ``dw_up`` may be views into a rank's flat buffer; with
    ``accumulate`` the gradients are added to what they hold."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, gated_ff_backward, x, w_gate, w_up, dh, activation, dx, dw_gate,
                       dw_up, accumulate, ws)
    rows, d, f, dt, xp, ld_x, gp, up, ld_w = _ff_args(x, w_gate, w_up)
    hp, ld_h = _matrix(dh, "dh", x.dtype, (rows, f))
    if accumulate and (dw_gate is None or dw_up is None):
        raise ValueError("accumulate needs the weight gradients' buffers")
    if dx is None:
        dx = torch.empty((rows, d), dtype=x.dtype, device=x.device)
    if dw_gate is None:
        dw_gate = torch.empty((f, d), dtype=x.dtype, device=x.device)
    if dw_up is None:
        dw_up = torch.empty((f, d), dtype=x.dtype, device=x.device)
    dxp, ld_dx = _matrix(dx, "dx", x.dtype, (rows, d))
    dgp, ld_dg = _matrix(dw_gate, "dw_gate", x.dtype, (f, d))
    dup, ld_du = _matrix(dw_up, "dw_up", x.dtype, (f, d))
    if ld_dg != ld_du:
        raise ValueError("dw_gate and dw_up must have the same row stride")
    s = _current(x)
    w = _Scratch(ws, _ff_workspace(rows, d, f, ld_x, ld_w, 1), s)
    try:
        st = lib().zr_gated_ff_backward(xp, ld_x, gp, up, ld_w, hp, ld_h, rows, d, f, dt,
                                        activation, 1 if accumulate else 0, dxp, ld_dx, dgp, dup,
                                        ld_dg, w.ptr, w.size, s)
    finally:
        w.done()
    _check(st, "zr_gated_ff_backward")
    return dx, dw_gate, dw_up


def _loss_args(logits, loss, n_loss, dlogits, grad):
    """Pointers that the losses share; the outputs are made where not given."""
    torch = _torch
    shape = _rows_cols(logits, "logits")
    dt = _type(logits)
    zp, ld = _matrix(logits, "logits", logits.dtype, shape)
    if loss is None:
        loss = torch.empty(n_loss, dtype=torch.float32, device=logits.device)
    lp = _vector(loss, "loss", torch.float32, n_loss)
    if dlogits is None and grad:
        dlogits = torch.empty(shape, dtype=logits.dtype, device=logits.device)
    dp, ldd = None, 0
    if dlogits is not None:
        dp, ldd = _matrix(dlogits, "dlogits", logits.dtype, shape)
    return dt, zp, ld, loss, lp, dlogits, dp, ldd


def distill_loss(logits, top_idx, top_logits, teacher_lse=None, temperature=1.0, weight=None,
                 loss=None, dlogits=None, grad=True, stream=None):
    """KL from a teacher's top logits (int32 tokens and float32 logits [rows, k])
    to the student's ``logits``, per row, with its gradient: (loss, dlogits).
    ``teacher_lse`` makes the rest of the teacher's mass one more class."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, distill_loss, logits, top_idx, top_logits, teacher_lse, temperature,
                       weight, loss, dlogits, grad)
    rows, vocab = _rows_cols(logits, "logits")
    k = _rows_cols(top_idx, "top_idx")[1]
    dt, zp, ld, loss, lp, dlogits, dp, ldd = _loss_args(logits, loss, rows, dlogits, grad)
    ip, ld_i = _matrix(top_idx, "top_idx", torch.int32, (rows, k))
    tp, ld_t = _matrix(top_logits, "top_logits", torch.float32, (rows, k))
    if ld_i != ld_t:
        raise ValueError("top_idx and top_logits must have the same row stride")
    f32 = torch.float32
    _check(lib().zr_distill_loss(zp, ld, dt, rows, vocab, ip, tp, k, ld_i,
                                 _vector(teacher_lse, "teacher_lse", f32, rows), temperature,
                                 _vector(weight, "weight", f32, rows), lp, dp, ldd,
                                 _current(logits)), "zr_distill_loss")
    return loss, dlogits


def policy_loss(logits, action, advantage, old_logp=None, ref_logp=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, temperature=1.0, weight=None, loss=None, logp=None,
                kl=None, dlogits=None, grad=True, stream=None):
    """Clipped policy loss with a KL term, per token, with its gradient:
    (loss, logp, kl, dlogits)."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, policy_loss, logits, action, advantage, old_logp, ref_logp, clip_low,
                       clip_high, kl_coef, temperature, weight, loss, logp, kl, dlogits, grad)
    rows, vocab = _rows_cols(logits, "logits")
    f32 = torch.float32
    dt, zp, ld, loss, lp, dlogits, dp, ldd = _loss_args(logits, loss, rows, dlogits, grad)
    if logp is None:
        logp = torch.empty(rows, dtype=f32, device=logits.device)
    if kl is None:
        kl = torch.empty(rows, dtype=f32, device=logits.device)
    _check(lib().zr_policy_loss(zp, ld, dt, rows, vocab,
                                _vector(action, "action", torch.int32, rows),
                                _vector(advantage, "advantage", f32, rows),
                                _vector(old_logp, "old_logp", f32, rows),
                                _vector(ref_logp, "ref_logp", f32, rows), clip_low, clip_high,
                                kl_coef, temperature, _vector(weight, "weight", f32, rows), lp,
                                _vector(logp, "logp", f32, rows), _vector(kl, "kl", f32, rows), dp,
                                ldd, _current(logits)), "zr_policy_loss")
    return loss, logp, kl, dlogits


def preference_loss(logits, target, offsets, ref_logp, beta=0.1, label_smoothing=0.0, weight=None,
                    loss=None, reward=None, dlogits=None, grad=True, ws=None, stream=None):
    """Preference loss over pairs of sequences (rows offsets[2p] .. offsets[2p+1]
    chosen, .. offsets[2p+2] rejected), with its gradient: (loss, reward, dlogits).
    A bad target or bad offsets are reported in ``ws`` (``zr_query_status``)."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, preference_loss, logits, target, offsets, ref_logp, beta,
                       label_smoothing, weight, loss, reward, dlogits, grad, ws)
    rows, vocab = _rows_cols(logits, "logits")
    if offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets must have 2 pairs + 1 entries")
    pairs = offsets.shape[0] // 2
    f32 = torch.float32
    dt, zp, ld, loss, lp, dlogits, dp, ldd = _loss_args(logits, loss, pairs, dlogits, grad)
    if reward is None:
        reward = torch.empty(2 * pairs, dtype=f32, device=logits.device)
    s = _current(logits)
    args = (_vector(target, "target", torch.int32, rows),
            _vector(offsets, "offsets", torch.int64, 2 * pairs + 1), pairs,
            _vector(ref_logp, "ref_logp", f32, rows), beta, label_smoothing,
            _vector(weight, "weight", f32, pairs), lp,
            _vector(reward, "reward", f32, 2 * pairs), dp, ldd)
    w = _Scratch(ws, _preference_workspace(rows), s)
    try:
        st = lib().zr_preference_loss(zp, ld, dt, rows, vocab, *args, w.ptr, w.size, s)
    finally:
        w.done()
    _check(st, "zr_preference_loss")
    return loss, reward, dlogits


# ------------------------------------------------------------ around the step
def _on_device(call, t, *others):
    """``call()`` with the first tensor's device as the current one; every other
    tensor given has to be there too."""
    at = t.get_device()
    for o in others:
        if o is not None and o.get_device() != at:
            raise ValueError("tensors on different devices: %s and %s" % (t.device, o.device))
    if at < 0 or at == _torch._C._cuda_getDevice():
        return call()
    with _torch.cuda.device(at):
        return call()


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, d):
    return lib().zr_rms_norm_workspace_size(rows, d)


@functools.lru_cache(maxsize=1024)
def _cross_entropy_workspace(device, rows, d, vocab, ld_w, dx, dw):
    return lib().zr_cross_entropy_workspace_size(rows, d, vocab, ld_w, dx, dw)


@functools.lru_cache(maxsize=1024)
def _orthogonalise_workspace(count, rows, cols):
    return lib().zr_orthogonalise_workspace_size(count, rows, cols)


def rms_norm(x, weight, residual=None, eps=1e-6, out=None, sum_out=None, rstd=None, stream=None):
    """y = s * rstd * weight with s = x + residual and rstd = 1 / sqrt(mean(s^2) + eps),
    per row of x [rows, d] (float32 or bfloat16): (y, s, rstd).  Without a residual s is
    x itself.  ``out`` and ``sum_out`` may be x or the residual."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, rms_norm, x, weight, residual, eps, out, sum_out, rstd)
    shape = _rows_cols(x, "x")
    rows, d = shape
    dt = _type(x)
    xp, ld_x = _matrix(x, "x", x.dtype, shape)
    wp = _vector(weight, "weight", x.dtype, d)
    rp, ld_r, sp, ld_s = None, d, None, d
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
    else:
        rp, ld_r = _matrix(residual, "residual", x.dtype, shape)
        if sum_out is None:
            sum_out = torch.empty(shape, dtype=x.dtype, device=x.device)
        sp, ld_s = _matrix(sum_out, "sum_out", x.dtype, shape)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    yp, ld_y = _matrix(out, "out", x.dtype, shape)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    qp = _vector(rstd, "rstd", torch.float32, rows)
    st = _on_device(lambda: lib().zr_rms_norm(xp, ld_x, rp, ld_r, wp, rows, d, dt, eps, yp, ld_y, sp,
                                              ld_s, qp, _current(x)),
                    x, weight, residual, out, sum_out, rstd)
    _check(st, "zr_rms_norm")
    return out, x if residual is None else sum_out, rstd


def rms_norm_backward(s, weight, rstd, dy, ds=None, dx=None, dweight=None, accumulate=False, ws=None,
                      stream=None):
    """Gradients of ``rms_norm`` from s and rstd: (dx, dweight).  ``ds`` is the gradient
    that reaches s along the residual; dx, which includes it, is that of x and of the
    residual.  With ``accumulate`` dweight is added to what it holds."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, rms_norm_backward, s, weight, rstd, dy, ds, dx, dweight, accumulate, ws)
    shape = _rows_cols(s, "s")
    rows, d = shape
    dt = _type(s)
    sp, ld_s = _matrix(s, "s", s.dtype, shape)
    wp = _vector(weight, "weight", s.dtype, d)
    qp = _vector(rstd, "rstd", torch.float32, rows)
    yp, ld_y = _matrix(dy, "dy", s.dtype, shape)
    rp, ld_r = (None, d) if ds is None else _matrix(ds, "ds", s.dtype, shape)
    if accumulate and dweight is None:
        raise ValueError("accumulate needs the weight gradient's buffer")
    if dx is None:
        dx = torch.empty(shape, dtype=s.dtype, device=s.device)
    if dweight is None:
        dweight = torch.empty(d, dtype=s.dtype, device=s.device)
    xp, ld_x = _matrix(dx, "dx", s.dtype, shape)
    gp = _vector(dweight, "dweight", s.dtype, d)

    def call():
        stream = _current(s)
        w = _Scratch(ws, _norm_workspace(rows, d), stream)
        try:
            return lib().zr_rms_norm_backward(sp, ld_s, wp, qp, yp, ld_y, rp, ld_r, rows, d, dt,
                                              1 if accumulate else 0, xp, ld_x, gp, w.ptr, w.size,
                                              stream)
        finally:
            w.done()

    _check(_on_device(call, s, weight, rstd, dy, ds, dx, dweight, ws), "zr_rms_norm_backward")
    return dx, dweight


def cross_entropy_loss(x, w_vocab, target, weight=None, loss=None, lse=None, dx=None, dw_vocab=None,
                       grad=True, accumulate=False, ws=None, stream=None):
    """Softmax cross entropy of the states x [rows, d] over the vocabulary whose weights
    are w_vocab [vocab, d] (bfloat16), per row, with its gradients, for which the logits
    are held in 16 bits at most: (loss, lse, dx, dw_vocab).  Rows of a negative ``target``
    (int32) are left out.  ``dw_vocab`` may be a view into a rank's flat buffer; with
    ``accumulate`` it is added to.  A target past the vocabulary is reported in ``ws``
    (``zr_query_status``)."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, cross_entropy_loss, x, w_vocab, target, weight, loss, lse, dx, dw_vocab,
                       grad, accumulate, ws)
    rows, d = _rows_cols(x, "x")
    vocab = _rows_cols(w_vocab, "w_vocab")[0]
    dt = _type(x)
    f32 = torch.float32
    xp, ld_x = _matrix(x, "x", x.dtype, (rows, d))
    wp, ld_w = _matrix(w_vocab, "w_vocab", x.dtype, (vocab, d))
    tp = _vector(target, "target", torch.int32, rows)
    kp = _vector(weight, "weight", f32, rows)
    if accumulate and dw_vocab is None:
        raise ValueError("accumulate needs the weight gradient's buffer")
    if loss is None:
        loss = torch.empty(rows, dtype=f32, device=x.device)
    if lse is None:
        lse = torch.empty(rows, dtype=f32, device=x.device)
    if grad and dx is None:
        dx = torch.empty((rows, d), dtype=x.dtype, device=x.device)
    if grad and dw_vocab is None:
        dw_vocab = torch.empty((vocab, d), dtype=x.dtype, device=x.device)
    lp, ep = _vector(loss, "loss", f32, rows), _vector(lse, "lse", f32, rows)
    dxp, ld_dx = (None, d) if dx is None else _matrix(dx, "dx", x.dtype, (rows, d))
    dwp, ld_dw = (None, d) if dw_vocab is None else _matrix(dw_vocab, "dw_vocab", x.dtype, (vocab, d))

    def call():
        s = _current(x)
        w = _Scratch(ws, _cross_entropy_workspace(x.get_device(), rows, d, vocab, ld_w,
                                                  0 if dx is None else 1,
                                                  0 if dw_vocab is None else 1), s)
        try:
            return lib().zr_cross_entropy_loss(xp, ld_x, wp, ld_w, rows, d, vocab, dt, tp, kp, lp, ep,
                                               1 if accumulate else 0, dxp, ld_dx, dwp, ld_dw, w.ptr,
                                               w.size, s)
        finally:
            w.done()

    _check(_on_device(call, x, w_vocab, target, weight, loss, lse, dx, dw_vocab, ws),
           "zr_cross_entropy_loss")
    return loss, lse, dx, dw_vocab


MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=256)
def _steps(coefficients, steps):
    """The C array of all steps' a, b, c."""
    if not 1 <= steps <= ZR_MAX_STEPS:  # (the library takes 32 bits of them, and no array as long)
        raise ZrError(ZR_ERR_INVALID_ARG, "zr_orthogonalise")
    if len(coefficients) == 3 and not hasattr(coefficients[0], "__len__"):
        coefficients = (coefficients,) * steps
    if len(coefficients) != steps or any(len(c) != 3 for c in coefficients):
        raise ValueError("coefficients must be a, b, c, or one such triple for each step")
    flat = [float(v) for c in coefficients for v in c]
    return (ctypes.c_float * max(1, len(flat)))(*flat)


def _batch(t, what, dtype, shape):
    """Pointer, leading dimension and step of a 2-D matrix or a 3-D batch of them."""
    if t.shape != shape or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor of shape %s, got %s on %s"
                         % (what, tuple(shape), tuple(t.shape), t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    rows, cols = shape[-2:]
    if t.stride(-1) != 1 and cols > 1:
        raise ValueError("%s must have contiguous rows" % what)
    ld = t.stride(-2) if rows > 1 else cols
    return t.data_ptr(), ld, (t.stride(0) if len(shape) == 3 and shape[0] > 1 else rows * ld)


def orthogonalise(g, steps=5, coefficients=MUON_COEFFICIENTS, scale=1.0, eps=1e-7, out=None, ws=None,
                  stream=None):
    """scale times the matrix g [rows, cols] (or each of a batch [n, rows, cols]; float32
    or bfloat16) after Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T, from
    g / (|g| + eps): its singular values pushed towards 1.  bfloat16 out.
    ``coefficients``: a, b, c, or such a triple for each step."""
    torch = _t()
    if stream is not None:
        return _run_on(stream, orthogonalise, g, steps, coefficients, scale, eps, out, ws)
    if g.dim() not in (2, 3):
        raise ValueError("g must be a 2-D or 3-D tensor")
    shape = g.shape
    rows, cols = shape[-2:]
    count = shape[0] if len(shape) == 3 else 1
    dt = _type(g)
    gp, ld_g, step_g = _batch(g, "g", g.dtype, shape)
    if type(coefficients) is not tuple or any(type(c) is list for c in coefficients):
        coefficients = tuple(tuple(c) if hasattr(c, "__len__") else c for c in coefficients)
    c = _steps(coefficients, steps)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=g.device)
    op, ld_o, step_o = _batch(out, "out", torch.bfloat16, shape)

    def call():
        s = _current(g)
        w = _Scratch(ws, _orthogonalise_workspace(count, rows, cols), s)
        try:
            return lib().zr_orthogonalise(gp, ld_g, step_g, count, rows, cols, dt, c, steps, scale, eps,
                                          op, ld_o, step_o, w.ptr, w.size, s)
        finally:
            w.done()

    _check(_on_device(call, g, out, ws), "zr_orthogonalise")
    return out
