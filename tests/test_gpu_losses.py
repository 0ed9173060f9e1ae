"""The losses over a vocabulary (distillation, policy, preference) through the
C ABI against the float64 oracle.

Tolerances.  u = 2^-24.  Every e_j = 2^((z_j - M) c) carries the rounding of
its argument (three roundings, 3 u |z_j - M| / temperature; tokens more than
30 below the maximum carry no mass) and of the power (2^-22).  A sum of V of
them adds at most V / 512 + 64 roundings in a row (one thread's share and the
joins, each with a power of its own).  So Z, and with it log q, is off by at
most REL(V) relatively (absolutely for log q).  The gradient adds the rounding
of its type.
"""

import numpy as np
import pytest

from oracle import step
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    return require_cuda()


def rel(vocab, tau):
    return (vocab / 512 + 64) * 2.0 ** -23 + 3 * U * 30 / tau


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23


def logits(rng, rows, vocab, spread=2.0):
    z = rng.normal(size=(rows, vocab)).astype(np.float32) * spread
    for t in range(rows):
        z[t, rng.integers(0, vocab, 4)] += rng.uniform(0, 3 + np.log(vocab), 4)
    return z


class Buffers:
    """Logits on the device in a wider and shifted buffer, and the gradient's."""

    def __init__(self, torch, z, dtype, pad=0, shift=0, in_place=False, dpad=None, dshift=None):
        td = torch.bfloat16 if dtype == "bf16" else torch.float32
        rows, vocab = z.shape

        def make(pad, shift):
            flat = torch.full((shift + rows * (vocab + pad) + 16,), 7.0, dtype=td, device="cuda")
            return flat, flat[shift:shift + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]

        self.flat, self.z = make(pad, shift)
        self.z.copy_(torch.from_numpy(z))
        self.exact = self.z.double().cpu().numpy()
        if in_place:
            self.dflat, self.dz = self.flat, self.z
        else:
            self.dflat, self.dz = make(pad if dpad is None else dpad, shift if dshift is None else dshift)

    def outside_untouched(self, torch):
        seen = torch.ones_like(self.dflat, dtype=torch.bool)
        base = self.dz.storage_offset()
        rows, vocab = self.dz.shape
        at = base + torch.arange(rows, device="cuda")[:, None] * (self.dz.stride(0) if rows > 1 else vocab) \
            + torch.arange(vocab, device="cuda")[None]
        seen[at.reshape(-1)] = False
        return bool((self.dflat[seen] == 7.0).all())


def check(got, want, tol):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    off = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert off.size == 0 or off.max() <= 0, "%.3g over its tolerance" % off.max()


SHAPES = [  # rows, vocab, dtype, pad, shift
    (1, 1, "f32", 0, 0), (2, 2, "bf16", 0, 0), (3, 7, "f32", 0, 0), (5, 33, "bf16", 0, 1),
    (4, 1000, "bf16", 0, 0), (4, 1003, "bf16", 0, 3), (3, 1021, "f32", 5, 1), (2, 4096, "f32", 0, 0),
    (3, 4097, "bf16", 2, 0), (2, 32000, "bf16", 0, 0), (3, 32769, "bf16", 0, 0),
    (2, 16400, "f32", 0, 2), (2, 50001, "bf16", 0, 7), (2, 65537, "f32", 3, 0),
    (2, 131072, "bf16", 0, 0), (2, 131072, "f32", 0, 0), (1, 262144, "bf16", 0, 0),
    (2, 270001, "bf16", 0, 1), (1, 262144, "f32", 0, 0), (1, 300007, "f32", 0, 0),
]


# ------------------------------------------------------------ distillation
def distill_case(rng, z, k, rest, tau, pad_share=0.2):
    rows, vocab = z.shape
    teacher = z.astype(np.float64) + rng.normal(size=z.shape)
    idx = np.full((rows, k), -1, dtype=np.int32)
    top = np.full((rows, k), 3.0, dtype=np.float32)
    for t in range(rows):
        n = min(k, vocab)
        best = np.argsort(-teacher[t])[:n]
        idx[t, :n] = best
        top[t, :n] = teacher[t, best]
        if n > 1:
            idx[t, :n][rng.random(n) < pad_share] = rng.choice([-1, vocab, -5, 2 ** 31 - 1])
    lse = None
    if rest:
        m = teacher.max(1)
        lse = (m / tau + np.log(np.exp((teacher - m[:, None]) / tau).sum(1))).astype(np.float32)
    return idx, top, lse


def run_distill(torch, zr, b, idx, top, lse, tau, w, **kw):
    dev = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    loss, dz = zr.distill_loss(b.z, dev(idx), dev(top), teacher_lse=dev(lse), temperature=tau,
                               weight=dev(w), dlogits=b.dz, **kw)
    torch.cuda.synchronize()
    return loss.cpu().numpy(), dz.double().cpu().numpy()


def distill_tol(b, idx, top, lse, tau, w, want_loss, want_dz, dtype):
    z, (rows, vocab) = b.exact, b.exact.shape
    r = rel(vocab, tau)
    tol_l, tol_d = np.zeros(rows), np.zeros(z.shape)
    for t in range(rows):
        wt = 1.0 if w is None else abs(float(w[t]))
        ok = (idx[t] >= 0) & (idx[t] < vocab)
        if wt == 0 or not np.isfinite(z[t].max()):
            continue
        q = np.exp(z[t] / tau - z[t].max() / tau)
        q /= q.sum()
        span = min(2.0 * np.abs(z[t][np.isfinite(z[t])]).max() / tau, 1e4)
        lt = top[t][ok].astype(np.float64) / tau
        size = np.abs(lt[np.isfinite(lt)]).max(initial=0) + (0 if lse is None else abs(float(lse[t])))
        # p: its argument's roundings, the power, the sum over the list
        rp = (3 * size + idx.shape[1] / 32 + 16) * 2 * U + 2.0 ** -21
        p = np.zeros(vocab)
        if ok.any():
            p[idx[t][ok]] = np.exp(lt - (lt.max() + np.log(np.exp(lt - lt.max()).sum()) if lse is None else float(lse[t]))) \
                if np.isfinite(lt.max()) else 0
        mass = p.sum()
        tol_l[t] = wt * (mass * (r + rp + 4 * U * span) * 2 + rp * mass * 20)
        tol_d[t] = wt / tau * (q * 2 * r + p * rp * 2 + (q + p) * 2.0 ** -20)
        if lse is not None:
            off = np.ones(vocab, dtype=bool)
            off[idx[t][ok]] = False
            rest = q[off].sum()
            if rest > 0:
                gap = abs(np.log(max(1 - mass, 1e-9) / rest))
                tol_l[t] += wt * ((rp * mass + 4 * U) * (gap + 2) + 4 * r * max(0, 1 - mass))
                tol_d[t][off] += wt / tau * q[off] * ((rp * mass + 4 * U) / rest + max(0, 1 - mass) / rest * 4 * r)
    return tol_l + 4 * U * np.abs(want_loss), tol_d + half_ulp(dtype) * np.abs(want_dz) + 1e-37


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rest", [False, True])
def test_distill(env, shape, rest):
    torch, zr = env
    rows, vocab, dtype, pad, shift = shape
    rng = np.random.default_rng(vocab + rest)
    tau = 1.0 if vocab % 2 else 1.5
    b = Buffers(torch, logits(rng, rows, vocab), dtype, pad, shift)
    k = [1, 5, 20, 64, 300][vocab % 5]
    idx, top, lse = distill_case(rng, b.exact, k, rest, tau)
    w = rng.uniform(0.1, 1, rows).astype(np.float32)
    if rows > 2:
        w[1] = 0
    loss, dz = run_distill(torch, zr, b, idx, top, lse, tau, w)
    want_loss, want_dz = step.distill(b.exact, idx, top, lse, tau, w)
    tl, td = distill_tol(b, idx, top, lse, tau, w, want_loss, want_dz, dtype)
    check(loss, want_loss, tl)
    check(dz, want_dz, td)
    assert b.outside_untouched(torch)


@pytest.mark.parametrize("dtype,vocab,k", [("bf16", 999, 0), ("f32", 2048, 1024), ("bf16", 600, 1024),
                                           ("f32", 40, 64), ("bf16", 40000, 1), ("bf16", 50001, 1024),
                                           ("f32", 40000, 700), ("f32", 270001, 1024)])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_list_lengths(env, dtype, vocab, k, rest):
    """Empty lists, the longest list, and lists that hold the whole vocabulary."""
    torch, zr = env
    rng = np.random.default_rng(k)
    b = Buffers(torch, logits(rng, 3, vocab), dtype)
    idx, top, lse = distill_case(rng, b.exact, k, rest, 1.0, pad_share=0.0)
    loss, dz = run_distill(torch, zr, b, idx, top, lse, 1.0, None)
    want_loss, want_dz = step.distill(b.exact, idx, top, lse, 1.0, None)
    tl, td = distill_tol(b, idx, top, lse, 1.0, None, want_loss, want_dz, dtype)
    if rest and k >= vocab:
        tl, td = tl + 2.0 ** -19, td + 2.0 ** -19  # sum p is 1 to the rounding of the given lse
    check(loss, want_loss, tl)
    check(dz, want_dz, td)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("vocab", [5000, 290000])
def test_distill_masks(env, dtype, rest, vocab):
    """-inf and lowest-value masks, rows with nothing, NaN where nothing is read."""
    torch, zr = env
    rng = np.random.default_rng(11)
    z = logits(rng, 8, vocab)
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    z[0, 100:4000] = -np.inf
    z[1, 100:4000] = low
    z[2, :] = -np.inf
    z[3, :] = low
    z[4, 17] = np.nan
    z[5, 18] = np.inf
    z[6, :] = np.nan  # left out by its weight
    z[7, 1:] = -np.inf
    w = np.ones(8, dtype=np.float32)
    w[6] = 0
    b = Buffers(torch, z, dtype)
    idx = np.tile(np.array([3, 50, 4500, -1, 7], dtype=np.int32), (8, 1))
    idx[7] = [0, -1, -1, -1, -1]
    top = rng.normal(size=(8, 5)).astype(np.float32)
    top[0, 2] = -np.inf
    lse = np.full(8, 2.5, dtype=np.float32) if rest else None
    loss, dz = run_distill(torch, zr, b, idx, top, lse, 1.0, w)
    want_loss, want_dz = step.distill(b.exact, idx, top, lse, 1.0, w)
    z3 = np.where(np.isnan(b.exact), 0, np.clip(b.exact, -100, 100))
    clean = type("B", (), {"exact": z3})
    tl, td = distill_tol(clean, idx, top, lse, 1.0, w, np.nan_to_num(want_loss, posinf=0, neginf=0),
                         np.nan_to_num(want_dz), dtype)
    # a token far down has log q of its own size: relative roundings
    tl = tl + 8 * U * np.abs(np.nan_to_num(want_loss, posinf=0))
    check(loss, want_loss, tl)
    check(dz, want_dz, td + 2.0 ** -20)


# ------------------------------------------------------------ policy
def policy_tol(b, w, g, want_dz, tau, dtype):
    z = b.exact
    r = rel(z.shape[1], tau)
    m = z.max(1, keepdims=True)
    with np.errstate(all="ignore"):
        e = np.nan_to_num(np.exp((z - m) / tau))
        q = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    return q, r, half_ulp(dtype) * np.abs(np.nan_to_num(want_dz)) + 1e-37


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kl_coef", [0.0, 0.1])
def test_policy(env, shape, kl_coef):
    torch, zr = env
    rows, vocab, dtype, pad, shift = shape
    rng = np.random.default_rng(vocab)
    tau = 0.8 if vocab % 2 else 1.0
    b = Buffers(torch, logits(rng, rows, vocab), dtype, pad, shift)
    run_policy_case(torch, zr, rng, b, dtype, tau, kl_coef)
    assert b.outside_untouched(torch)


def run_policy_case(torch, zr, rng, b, dtype, tau, kl_coef, stream=None):
    rows, vocab = b.exact.shape
    action = np.array([np.argsort(-r)[rng.integers(0, min(3, vocab))] for r in b.exact], dtype=np.int32)
    logp0 = step.policy(b.exact, action, np.zeros(rows), tau=tau)[1]
    old = (logp0 + rng.choice([-0.5, -0.1, 0.07, 0.6], rows)).astype(np.float32)
    ref = (logp0 + 0.3 * rng.normal(size=rows)).astype(np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    w = rng.uniform(0.1, 1, rows).astype(np.float32)
    if rows > 2:
        w[1], action[2] = 0, -1
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    args = [dev(v) for v in (action, adv, old, ref, w)]
    torch.cuda.synchronize()
    loss, logp, kl, dz = zr.policy_loss(b.z, args[0], args[1], old_logp=args[2], ref_logp=args[3],
                                        clip_low=0.2, clip_high=0.25, kl_coef=kl_coef,
                                        temperature=tau, weight=args[4], dlogits=b.dz, stream=stream)
    torch.cuda.synchronize()
    wl, wp, wk, wd = step.policy(b.exact, action, adv, old, ref, 0.2, 0.25, kl_coef, tau, w)
    r = rel(vocab, tau)
    # logp is off by r and its own rounding; the rest follows by derivatives
    dp = 2 * r + 4 * U * (np.abs(wp) + np.abs(old) + np.abs(ref))
    up = np.exp(ref - wp)
    ratio = np.exp(wp - old)
    slope = ratio * np.abs(adv) + kl_coef * (1 + up)
    check(logp.cpu().numpy(), wp, dp)
    check(kl.cpu().numpy(), wk, dp * (1 + up) + 8 * U * up)
    check(loss.cpu().numpy(), wl, w * slope * (dp + 16 * U))
    q, _, td = policy_tol(b, w, None, wd, tau, dtype)
    one = np.zeros_like(q)
    one[np.arange(rows), np.maximum(action, 0)] = 1
    td = td + (w * slope / tau)[:, None] * (q * 4 * r + (one + q) * (dp + 16 * U)[:, None])
    check(dz.double().cpu().numpy(), wd, td)


def test_policy_edges(env):
    """No old and no reference log probabilities; masked actions; bad actions; NaN."""
    torch, zr = env
    rng = np.random.default_rng(5)
    z = logits(rng, 6, 3000)
    z[0, :] = -np.inf
    z[1, 40:] = -np.inf
    z[3, 5] = np.nan
    z[5, :] = float(torch.finfo(torch.float32).min)
    b = Buffers(torch, z, "f32")
    action = np.array([4, 7, 3000, 1, -9, 2], dtype=np.int32)
    adv = rng.normal(size=6).astype(np.float32)
    loss, logp, kl, dz = zr.policy_loss(b.z, torch.from_numpy(action).cuda(), torch.from_numpy(adv).cuda(),
                                        dlogits=b.dz)
    wl, wp, wk, wd = step.policy(b.exact, action, adv)
    wk[[2, 3]] = kl.cpu().numpy()[[2, 3]]  # no reference: kl is 0, also of a row of NaN
    check(kl.cpu().numpy(), wk, 0)
    check(loss.cpu().numpy(), wl, 4 * U * np.abs(np.nan_to_num(wl)))
    check(logp.cpu().numpy(), wp, 4 * rel(3000, 1.0) + 8 * U * np.abs(np.nan_to_num(wp)))
    check(dz.cpu().numpy(), wd, 2 * np.nanmax(np.abs(wd)) * rel(3000, 1.0) + 1e-37)


# ------------------------------------------------------------ preference
@pytest.mark.parametrize("shape", [(7, 33, "bf16", 0, 1), (9, 1000, "f32", 0, 0), (40, 4097, "bf16", 1, 0),
                                   (30, 50001, "bf16", 0, 0), (12, 131072, "bf16", 0, 0),
                                   (9, 140003, "f32", 0, 0), (8, 300007, "bf16", 0, 0)], ids=str)
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_preference(env, shape, eps):
    torch, zr = env
    rows, vocab, dtype, pad, shift = shape
    rng = np.random.default_rng(rows)
    b = Buffers(torch, logits(rng, rows, vocab), dtype, pad, shift)
    pairs = 3
    cut = np.sort(rng.integers(1, rows, 2 * pairs))  # empty sequences among them
    offsets = np.concatenate([[0 if eps else 1], np.maximum(cut, 1)]).astype(np.int64)
    target = np.array([np.argsort(-r)[rng.integers(0, 3)] for r in b.exact], dtype=np.int32)
    target[rng.random(rows) < 0.2] = -100
    logp0 = step.policy(b.exact, target, np.zeros(rows))[1]
    ref = (logp0 + 0.5 * rng.normal(size=rows)).astype(np.float32)
    w = np.array([1.0, 0.25, 0.0 if eps else 2.0], dtype=np.float32)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    ws = torch.empty(zr.zr_preference_workspace_size(rows), dtype=torch.uint8, device="cuda")
    loss, reward, dz = zr.preference_loss(b.z, dev(target), dev(offsets), dev(ref), beta=0.4,
                                          label_smoothing=eps, weight=dev(w), dlogits=b.dz, ws=ws)
    assert zr.zr_query_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == zr.ZR_OK
    wl, wr, wd = step.preference(b.exact, target, offsets, ref, 0.4, eps, w)
    r = rel(vocab, 1.0)
    n = np.diff(offsets)
    big = np.abs(ref).max() + np.abs(logp0).max()
    tr = 0.4 * n * (2 * r + 6 * U * big) + 4 * U * np.abs(wr)
    check(reward.cpu().numpy(), wr, tr)
    check(loss.cpu().numpy(), wl, w * (tr[0::2] + tr[1::2] + 16 * U) + 8 * U * np.abs(wl))
    q = np.exp(b.exact - b.exact.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    one = np.zeros_like(q)
    one[np.arange(rows), np.maximum(target, 0)] = 1
    slack = 0.4 * w.max() * (tr.max() * 2 + 16 * U + 4 * r)
    check(dz.double().cpu().numpy(), wd, slack * (q + one) + half_ulp(dtype) * np.abs(wd) + 1e-37)
    assert b.outside_untouched(torch)


def test_preference_reports_bad_targets_and_offsets(env):
    torch, zr = env
    rng = np.random.default_rng(3)
    z = torch.from_numpy(logits(rng, 8, 100)).cuda()
    ref = torch.zeros(8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    good_t, good_o = [1] * 8, [0, 2, 4, 6, 8]
    for target, offsets, bad_pair in ((good_t, good_o, None), ([100] + [1] * 7, good_o, None),
                                      (good_t, [0, 2, 4, 3, 8], 1), (good_t, [-1, 2, 4, 6, 8], 0),
                                      (good_t, [0, 2, 4, 6, 9], 1)):
        ws = torch.empty(zr.zr_preference_workspace_size(8), dtype=torch.uint8, device="cuda")
        loss, _, dz = zr.preference_loss(z, torch.tensor(target, dtype=torch.int32, device="cuda"),
                                         torch.tensor(offsets, device="cuda"), ref, ws=ws)
        want = zr.ZR_OK if target == good_t and offsets == good_o else zr.ZR_ERR_INVALID_ARG
        assert zr.zr_query_status(ws.data_ptr(), stream) == want
        loss, dz = loss.cpu().numpy(), dz.cpu().numpy()
        assert np.isnan(loss).tolist() == [bad_pair == 0, bad_pair == 1]
        assert np.isfinite(dz).all()
        if bad_pair is not None:
            rows = [t for t in range(8) if (t < 4) == (bad_pair == 0)]
            assert not dz[rows].any()
        if target[0] == 100:
            assert not dz[0].any()


def test_preference_masks(env):
    torch, zr = env
    rng = np.random.default_rng(6)
    z = logits(rng, 6, 2000)
    z[0, 30:] = -np.inf
    z[1, :] = -np.inf   # left out
    z[2, :] = np.nan    # a prompt: not read
    z[3, 30:] = float(torch.finfo(torch.float32).min)
    target = np.array([5, 3, -1, 29, 7, 8], dtype=np.int32)
    offsets = np.array([0, 4, 6], dtype=np.int64)
    ref = np.zeros(6, dtype=np.float32)
    b = Buffers(torch, z, "f32")
    loss, reward, dz = zr.preference_loss(b.z, *[torch.from_numpy(v).cuda() for v in (target, offsets, ref)],
                                          dlogits=b.dz)
    wl, wr, wd = step.preference(b.exact, target, offsets, ref)
    tol = 6 * 4 * rel(2000, 1.0)
    check(reward.cpu().numpy(), wr, tol)
    check(loss.cpu().numpy(), wl, tol)
    check(dz.cpu().numpy(), wd, tol)


# ------------------------------------------------------------ all of them
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,shift", [(1003, 1), (40001, 0), (131072, 0), (300007, 3)])
def test_in_place_equals_apart_and_repeats(env, dtype, vocab, shift):
    torch, zr = env
    rng = np.random.default_rng(9)
    z = logits(rng, 5, vocab)
    idx, top, lse = distill_case(rng, z, 40, True, 1.0)
    action = torch.from_numpy(z.argmax(1).astype(np.int32)).cuda()
    adv = torch.from_numpy(rng.normal(size=5).astype(np.float32)).cuda()
    off = torch.tensor([0, 2, 5], device="cuda")
    calls = {
        "distill": lambda b: run_distill(torch, zr, b, idx, top, None, 1.0, None),
        "rest": lambda b: run_distill(torch, zr, b, idx, top, lse, 1.0, None),
        "policy": lambda b: [v.double().cpu().numpy() for v in
                             zr.policy_loss(b.z, action, adv, dlogits=b.dz)],
        "preference": lambda b: [v.double().cpu().numpy() for v in
                                 zr.preference_loss(b.z, action, off, adv, dlogits=b.dz)],
    }
    for name, call in calls.items():
        first = call(Buffers(torch, z, dtype, shift=shift))
        again = call(Buffers(torch, z, dtype, shift=shift))
        inside = call(Buffers(torch, z, dtype, shift=shift, in_place=True))
        # the gradient at another alignment than the logits
        other = call(Buffers(torch, z, dtype, shift=shift, dpad=1, dshift=shift + 1))
        for a, b, c, d in zip(first, again, inside, other):
            for v in (b, c, d):
                assert np.array_equal(a, v, equal_nan=True), name


def test_losses_without_gradient_and_gradient_without_loss(env):
    torch, zr = env
    rng = np.random.default_rng(12)
    z = torch.from_numpy(logits(rng, 4, 5000)).cuda()
    action = z.argmax(1).int()
    adv = torch.randn(4, device="cuda")
    full = zr.policy_loss(z, action, adv)
    part = zr.policy_loss(z, action, adv, grad=False)
    assert part[3] is None and torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])
    dz = torch.empty_like(z)
    st = zr.zr_policy_loss(z.data_ptr(), 5000, zr.ZR_F32, 4, 5000, action.data_ptr(), adv.data_ptr(), None,
                           None, 0.2, 0.2, 0.0, 1.0, None, None, None, None, dz.data_ptr(), 5000,
                           torch.cuda.current_stream().cuda_stream)
    assert st == zr.ZR_OK and torch.equal(dz, full[3])
    idx, top = torch.topk(z, 8)
    full = zr.distill_loss(z, top.int(), idx)
    assert torch.equal(zr.distill_loss(z, top.int(), idx, grad=False)[0], full[0])
    st = zr.zr_distill_loss(z.data_ptr(), 5000, zr.ZR_F32, 4, 5000, top.int().data_ptr(), idx.data_ptr(), 8, 8,
                            None, 1.0, None, None, dz.data_ptr(), 5000,
                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == zr.ZR_OK and torch.equal(dz, full[1])
    off = torch.tensor([0, 2, 4], device="cuda")
    full = zr.preference_loss(z, action, off, adv)
    part = zr.preference_loss(z, action, off, adv, grad=False)
    assert part[2] is None and torch.equal(full[0], part[0])


def test_no_rows_and_no_pairs(env):
    torch, zr = env
    z = torch.empty((0, 100), device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    loss, dz = zr.distill_loss(z, none.view(0, 0), torch.empty((0, 0), device="cuda"))
    assert loss.numel() == 0 and dz.numel() == 0
    assert zr.policy_loss(z, none, torch.empty(0, device="cuda"))[0].numel() == 0
    loss, reward, _ = zr.preference_loss(z, none, torch.tensor([0, 0, 0], device="cuda"),
                                         torch.empty(0, device="cuda"))
    assert loss.cpu().numpy() == pytest.approx([np.log(2)], rel=1e-6)
    z = torch.randn(3, 50, device="cuda")
    loss, _, dz = zr.preference_loss(z, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                     torch.tensor([0], device="cuda"), torch.zeros(3, device="cuda"))
    assert loss.numel() == 0 and not dz.any()


def test_on_another_stream(env):
    torch, zr = env
    rng = np.random.default_rng(13)
    s = torch.cuda.Stream()
    b = Buffers(torch, logits(rng, 9, 40000), "bf16")
    run_policy_case(torch, zr, rng, b, "bf16", 1.0, 0.1, stream=s)


def test_gradients_against_differences(env):
    """Central differences of the library's own losses along random directions:
    h^2 times a third derivative of order one, and two losses' rounding / 2h."""
    torch, zr = env
    rng = np.random.default_rng(14)
    n, vocab, h = 6, 300, 2.0 ** -6
    z = torch.from_numpy(rng.normal(size=(n, vocab)).astype(np.float32)).cuda()
    teacher = z + torch.randn(n, vocab, device="cuda")
    top, idx = torch.topk(teacher, 12)
    lse = torch.logsumexp(teacher, 1)
    action = torch.from_numpy(rng.integers(0, vocab, n).astype(np.int32)).cuda()
    adv = torch.from_numpy(rng.normal(size=n).astype(np.float32)).cuda()
    base = zr.policy_loss(z, action, adv)[1]
    old, ref = base - 0.05, base + 0.4
    off = torch.tensor([0, 2, 6], device="cuda")
    losses = {
        "distill": lambda v: zr.distill_loss(v, idx.int(), top)[0::1],
        "rest": lambda v: zr.distill_loss(v, idx.int(), top, teacher_lse=lse),
        "policy": lambda v: zr.policy_loss(v, action, adv, old, ref, kl_coef=0.3),
        "preference": lambda v: zr.preference_loss(v, action, off, ref, beta=0.5),
    }
    for name, f in losses.items():
        grad = f(z)[-1].double()
        for seed in range(4):
            d = torch.from_numpy(np.random.default_rng(seed).normal(size=(n, vocab)).astype(np.float32)).cuda()
            d /= d.norm()
            up, down = f(z + h * d)[0].double().sum(), f(z - h * d)[0].double().sum()
            assert abs(float((up - down) / (2 * h) - (grad * d).sum())) < 10 * h * h + n * 8 * U * 8 / h, name


@pytest.mark.parametrize("vocab, dtype", [(1071, "f32"), (8948, "f32"), (65537, "bf16"), (131072, "bf16")])
def test_rows_share_no_error(env, vocab, dtype):
    """A sequence's sum adds what its rows' errors have in common.

    One row a sequence, and the reference at the row's own log probability: the
    reward is the error, and what the reference's rounding leaves.  log Z in one
    fp32 number is off by up to 2^-21 in a row, by up to 2^-22 in the mean of
    rows whose sums have one size; a row here has 2^-21 in all, and the mean of
    the rows one rounding, 2^-23.
    """
    torch, zr = env
    rows = 512
    gen = torch.Generator("cuda").manual_seed(3)
    z = torch.randn(rows, vocab, generator=gen, device="cuda") * 2
    at = torch.randint(0, vocab, (rows, 8), generator=gen, device="cuda")
    z.scatter_(1, at, 2 + np.log(vocab) + 3 * torch.rand(rows, 8, generator=gen, device="cuda"))
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    logp = torch.log_softmax(z.double(), 1).gather(1, target[:, None])[:, 0]
    ref = logp.float()
    offsets = torch.arange(rows + 1, device="cuda")
    reward = torch.empty(rows, device="cuda")
    zr.preference_loss(z, target.int(), offsets, ref, beta=1.0, reward=reward)
    off = reward.double() - (logp - ref.double())
    assert off.abs().max() <= 2.0 ** -21
    assert abs(off.mean()) <= 2.0 ** -23


@pytest.mark.parametrize("gap", [0.0, 1e-4, 3e-3, 0.1, 0.24, 0.26, 3.0])
def test_kl_of_close_policies(env, gap):
    """exp(d) - 1 - d keeps its digits where d is small: d's own rounding, twice."""
    torch, zr = env
    z = torch.zeros(2, 1024, device="cuda")  # log p = -10 log 2, whose rounding is known
    action = torch.zeros(2, dtype=torch.int32, device="cuda")
    exact = -10 * np.log(2.0)
    ref = torch.tensor([exact + gap, exact - gap], dtype=torch.float64).float()
    kl = torch.empty(2, device="cuda")
    zr.policy_loss(z, action, torch.ones(2, device="cuda"), ref_logp=ref.cuda(), kl=kl,
                   kl_coef=0.1)
    d = ref.double().numpy() - exact
    want = np.expm1(d) - d
    # log p is known to 2^-26 of 7 and d to 2^-24 of itself
    off = np.abs(np.expm1(d)) * (7 * 2.0 ** -26 + np.abs(d) * 2.0 ** -24) + 8 * U * np.abs(want) + 2.0 ** -48
    assert np.all(np.abs(kl.double().cpu().numpy() - want) <= off)


@pytest.mark.parametrize("rows, vocab, pairs", [(1, 40, 1), (40, 40, 300), (512, 1003, 1), (513, 1003, 1),
                                                (512, 1003, 512), (512, 1003, 513), (512, 16384, 7),
                                                (512, 16385, 7), (512, 40000, 7)])
def test_preference_at_its_kernels_limits(env, rows, vocab, pairs):
    """Where the pairs are done changes the launches; pairs may be empty, rows in none."""
    torch, zr = env
    rng = np.random.default_rng(rows + vocab + pairs)
    b = Buffers(torch, logits(rng, rows, vocab), "bf16", shift=1)
    target = rng.integers(0, vocab, rows).astype(np.int32)
    target[rng.random(rows) < 0.1] = -1
    offsets = np.sort(rng.integers(rows // 20, rows - rows // 20 + 1, 2 * pairs + 1))
    ref = (-np.log(vocab) + rng.normal(size=rows)).astype(np.float32)
    loss, reward, dz = zr.preference_loss(
        b.z, *[torch.from_numpy(v).cuda() for v in (target, offsets, ref)], dlogits=b.dz)
    wl, wr, wd = step.preference(b.exact, target, offsets, ref)
    longest = max(offsets[2:] - offsets[:-2])
    tol = 0.1 * longest * 4 * rel(vocab, 1.0)  # beta and a row's log p, as many as there are
    check(reward.cpu().numpy(), wr, tol + 4 * U * np.abs(wr))
    check(loss.cpu().numpy(), wl, 2 * tol + 8 * U * np.abs(wl))
    # the slope's error and the softmax's, of values up to beta, then bf16
    check(dz.double().cpu().numpy(), wd, 0.1 * (2 * tol + 4 * rel(vocab, 1.0)) + half_ulp("bf16") * np.abs(wd))
    assert b.outside_untouched(torch)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, vocab, shift", [(700, 1003, 1), (700, 8192, 0), (513, 40001, 3), (300, 131072, 0),
                                                (60, 300007, 5)])
def test_preference_in_place_with_the_pairs_apart(env, rows, vocab, shift, dtype):
    """Over 512 rows, or 1024 CTAs of the gradient, its kernel is launched without
    the pairs.  Where it replaces the logits it reads the target's logit, wherever
    that lies (first and last elements, whole vectors), before it is overwritten."""
    torch, zr = env
    g = torch.Generator("cuda").manual_seed(rows)
    z = (torch.randn(rows, vocab, generator=g, device="cuda") * 2).cpu().numpy()
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    for i, at in enumerate((0, 1, 2, 7, 8, vocab - 1, vocab - 2, vocab - 9, 2048 * 4 - 1, 2048 * 8)):
        target[i::20] = min(at, vocab - 1)
    target[5::9] = -1
    target = target.int()
    ref = torch.randn(rows, generator=g, device="cuda") - 9
    off = torch.tensor([0, rows // 3, rows // 2, rows - rows // 8, rows], device="cuda")
    apart, inside = Buffers(torch, z, dtype, shift=shift), Buffers(torch, z, dtype, shift=shift, in_place=True)
    want = zr.preference_loss(apart.z, target, off, ref, dlogits=apart.dz)
    for _ in range(3):
        inside.z.copy_(apart.z)
        got = zr.preference_loss(inside.z, target, off, ref, dlogits=inside.z)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and what it is, at the targets: slope (1 - q)
    used = [t for t in range(0, rows, max(1, rows // 40)) if int(target[t]) >= 0]
    q = torch.softmax(apart.z[used].double(), 1).gather(1, target[used, None].long())[:, 0]
    slope = want[2][used].double().gather(1, target[used, None].long())[:, 0] / (1 - q)
    pair = torch.bucketize(torch.tensor(used, device="cuda"), off[[2]], right=True)
    reward = want[1].double()
    m = (reward[0::2] - reward[1::2])[pair]
    first = torch.bucketize(torch.tensor(used, device="cuda"), off[1:4], right=True) % 2 == 0
    expect = -0.1 * torch.sigmoid(-m) * torch.where(first, 1.0, -1.0)
    # m is formed here from rewards that were rounded to fp32; q to rel(); the output's type
    tol = expect.abs() * (half_ulp(dtype) + 4 * rel(vocab, 1.0) + 16 * U + 4 * U * reward.abs().max())
    assert bool(((slope - expect).abs() <= tol * 1.01 / (1 - q) + 1e-37).all())
    assert inside.outside_untouched(torch)


@pytest.mark.parametrize("rows, vocab, dtype", [(3, 40001, "bf16"), (700, 40001, "bf16"), (900, 131072, "bf16"),
                                                (300, 131072, "f32"), (40, 300007, "f32")])
def test_policy_in_place_over_a_cluster(env, rows, vocab, dtype):
    """The action's logit is read by every CTA of its row, and overwritten by one."""
    torch, zr = env
    g = torch.Generator("cuda").manual_seed(rows)
    z = torch.randn(rows, vocab, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    action = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
    adv = torch.randn(rows, generator=g, device="cuda")
    want = zr.policy_loss(z, action, adv, ref_logp=adv - 12, kl_coef=0.1)
    for _ in range(3):
        inside = z.clone()
        got = zr.policy_loss(inside, action, adv, ref_logp=adv - 12, kl_coef=0.1, dlogits=inside)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [8, 600])
@pytest.mark.parametrize("eps", [0.0, 0.1, 1.0])
def test_preference_of_impossible_answers(env, rows, eps):
    """A target whose logit is -inf makes the margin infinite: the loss is its
    limit (0 where the answer that is impossible is the one to be rejected, and
    nothing is smoothed), never 0 times infinity."""
    torch, zr = env
    rng = np.random.default_rng(rows)
    z = logits(rng, rows, 500)
    h = rows // 4
    offsets = np.array([0, h, 2 * h, 3 * h, rows], dtype=np.int64)
    target = rng.integers(0, 500, rows).astype(np.int32)
    for t in (2 * h - 1, 2 * h):  # in the first pair's rejected answer, the second's chosen one
        z[t, target[t]] = -np.inf
    ref = (-6 + rng.normal(size=rows)).astype(np.float32)
    b = Buffers(torch, z, "f32")
    loss, reward, dz = zr.preference_loss(b.z, *[torch.from_numpy(v).cuda() for v in (target, offsets, ref)],
                                          label_smoothing=eps, dlogits=b.dz)
    wl, wr, wd = step.preference(b.exact, target, offsets, ref, eps=eps)
    inf = np.inf
    assert wl.tolist() == {0.0: [0.0, inf], 0.1: [inf, inf], 1.0: [inf, 0.0]}[eps]
    check(loss.cpu().numpy(), wl, 0)
    check(reward.cpu().numpy(), wr, 0.1 * rows * 2 * rel(500, 1.0) + 4 * U * np.abs(np.nan_to_num(wr, neginf=0)))
    check(dz.cpu().numpy(), wd, 0.1 * (4 * rel(500, 1.0) + 16 * U))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab, shift", [(3000, 1), (40001, 0), (140000, 3), (300007, 2)])
def test_distill_of_a_list_far_ahead(env, vocab, shift, dtype):
    """The student's listed logits lead all others by 60 to 300 temperatures: the
    rest's term and its gradient are finite (only a rest without any mass gives
    +inf), and those of a rest whose tokens are ahead by as much."""
    torch, zr = env
    rng = np.random.default_rng(vocab)
    gaps = [60.0, 87.0, 89.0, 100.0, 200.0, 300.0, -100.0, -300.0]
    rows, tau = len(gaps), 0.25
    z = rng.normal(size=(rows, vocab)).astype(np.float32) * 0.25
    idx = np.tile(np.array([0, 5, vocab // 2, vocab - 1, -1, 1234], dtype=np.int32), (rows, 1))
    on = idx[0][idx[0] >= 0]
    for t, gap in enumerate(gaps):
        z[t, on] += gap * tau
    top = rng.normal(size=idx.shape).astype(np.float32) * 0.5
    real = np.where(idx[0] >= 0, top / np.float64(tau), -np.inf)
    lse = (np.log(np.exp(real).sum(1)) - np.log(0.9)).astype(np.float32)  # p_rest is 0.1
    w = rng.uniform(0.5, 1, rows).astype(np.float32)
    b = Buffers(torch, z, dtype, shift=shift)

    def listed_only(others, lse, tau):
        """The list alone has logits that count: q is even over it."""
        b.z.fill_(others)
        b.z[:, torch.from_numpy(on).long().cuda()] = 0.0
        lse = lse.astype(np.float32)
        got = run_distill(torch, zr, b, idx, top, lse, tau, w)
        want = step.distill(b.z.double().cpu().numpy(), idx, top, lse, tau, w)
        check(got[0], want[0], 2.0 ** -18)
        check(got[1], want[1], half_ulp(dtype) * np.abs(want[1]) + 2.0 ** -17)
        return got

    loss, dz = run_distill(torch, zr, b, idx, top, lse, tau, w)
    want_loss, want_dz = step.distill(b.exact, idx, top, lse, tau, w)
    assert np.isfinite(want_loss).all()
    tl, td = distill_tol(b, idx, top, lse, tau, w, want_loss, want_dz, dtype)
    # distances of 300 temperatures carry their own roundings, in every power of them
    far = 8 * U * (np.abs(gaps) + 40)[:, None]
    check(loss, want_loss, tl + 4 * far[:, 0])
    check(dz, want_dz, td + far * np.abs(want_dz))
    # nothing at all outside the list: its mass is missed without end
    loss, dz = listed_only(-np.inf, lse, tau)
    assert np.isposinf(loss).all()
    # lowest values there, and a rest that is the rounding of its own sum: none
    loss, dz = listed_only(float(torch.finfo(b.z.dtype).min), np.log(np.exp(top[:, idx[0] >= 0].astype(np.float64)).sum(1)), 1.0)
    assert np.isfinite(loss).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [900, 70001, 300007])
def test_tokens_masked_by_the_lowest_value(env, vocab, dtype):
    """An action, target or listed token whose logit is the type's lowest value has
    a log probability of that size, which fp32 holds: it is not -inf, and against a
    reference that masks the token too the ratio is 1."""
    torch, zr = env
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    rng = np.random.default_rng(vocab)
    rows = 8
    z = logits(rng, rows, vocab)
    tok = rng.integers(0, vocab, rows).astype(np.int32)
    z[np.arange(rows), tok] = low
    z[3, :] = np.where(rng.random(vocab) < 0.5, low, z[3])
    b = Buffers(torch, z, dtype)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    ref = np.full(rows, low, dtype=np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    loss, logp, kl, dz = zr.policy_loss(b.z, dev(tok), dev(adv), old_logp=dev(ref), ref_logp=dev(ref), kl_coef=0.1,
                                        dlogits=b.dz)
    want = step.policy(b.exact, tok, adv, old=ref, ref=ref, kl_coef=0.1)
    assert (want[1] < 0.99 * low).all() and (want[2] == 0).all()
    check(logp.cpu().numpy(), want[1], 4 * U * np.abs(want[1]))
    check(kl.cpu().numpy(), want[2], 0)
    check(loss.cpu().numpy(), want[0], 4 * U * np.abs(want[0]))
    check(dz.double().cpu().numpy(), want[3], 4 * rel(vocab, 1.0) + half_ulp(dtype) * np.abs(want[3]))
    # the first pair's reference masks its tokens, the second pair's does not
    off = np.array([0, 2, 4, 6, 8], dtype=np.int64)
    ref[4:] = -7.0
    loss, reward, dz = zr.preference_loss(b.z, dev(tok), dev(off), dev(ref), beta=0.01, dlogits=b.dz)
    want = step.preference(b.exact, tok, off, ref, beta=0.01)
    assert (want[1][:2] == 0).all() and (want[1][2:] < 0.01 * low).all()
    check(reward.cpu().numpy(), want[1], 8 * U * np.abs(want[1]))
    check(loss.cpu().numpy()[:1], want[0][:1], 4 * U)
    check(dz.double().cpu().numpy()[:4], want[2][:4], 4 * rel(vocab, 1.0) + half_ulp(dtype) * np.abs(want[2][:4]))
    # a list with one such token, one with nothing else, and the rest class
    idx = np.stack([tok, (tok + 1) % vocab, np.full(rows, -1)], 1).astype(np.int32)
    z[5, idx[5, :2]] = low / 2
    b = Buffers(torch, z, dtype)
    top = rng.normal(size=idx.shape).astype(np.float32) * 0.5
    for lse in (None, np.full(rows, 1.5, dtype=np.float32)):
        loss, dz = run_distill(torch, zr, b, idx, top, lse, 1.0, None)
        wl, wd = step.distill(b.exact, idx, top, lse, 1.0, None)
        assert np.isfinite(wl).all() and (wl > 1e36).all()
        check(loss, wl, 2.0 ** -18 * np.abs(wl))
        check(dz, wd, 2.0 ** -18 + 4 * rel(vocab, 1.0) + half_ulp(dtype) * np.abs(wd))


@pytest.mark.parametrize("vocab", [100, 40001, 300007])
def test_kl_of_an_impossible_action(env, vocab):
    """exp(x) - x - 1 is +inf for an action of probability 0 that the reference may
    take, and for one that the reference never takes; neither is inf - inf."""
    torch, zr = env
    z = torch.zeros(3, vocab, device="cuda")
    z[0, 7] = -np.inf
    action = torch.full((3,), 7, dtype=torch.int32, device="cuda")
    ref = torch.tensor([-3.0, -np.inf, -np.log(vocab)], dtype=torch.float32, device="cuda")
    adv = torch.ones(3, device="cuda")
    loss, logp, kl, dz = zr.policy_loss(z, action, adv, ref_logp=ref)
    assert kl[:2].tolist() == [np.inf, np.inf] and 0 <= float(kl[2]) <= 2.0 ** -40
    assert loss.tolist() == [-1.0] * 3 and float(logp[0]) == -np.inf  # the term has no weight
    assert bool(torch.isfinite(dz).all())
    loss, _, _, _ = zr.policy_loss(z, action, adv, ref_logp=ref, kl_coef=0.5)
    assert loss[:2].tolist() == [np.inf, np.inf] and float(loss[2]) == -1.0


def test_logits_and_temperature_of_any_size(env):
    """Logits times 2^101 at temperature 2^101 (where log2(e) / temperature still has
    two normal parts) are the logits at temperature 1, to the bits; the gradient is
    2^101 times less, to the bits where that is a normal number."""
    torch, zr = env
    rng = np.random.default_rng(8)
    z = torch.from_numpy(logits(rng, 6, 1200, spread=8.0)).cuda()
    action = torch.from_numpy(rng.integers(0, 1200, 6).astype(np.int32)).cuda()
    adv = torch.from_numpy(rng.normal(size=6).astype(np.float32)).cuda()
    top, idx = torch.topk(z + 1, 20)
    lse = torch.logsumexp(z + 1, 1) + 0.5  # 0.4 of the mass outside the list
    big = 2.0 ** 101

    def same_gradient(a, b):
        normal = b.abs() > 2.0 ** -120
        return bool(normal.any()) and torch.equal(a[normal], (b * big)[normal])

    one = zr.policy_loss(z, action, adv, old_logp=adv - 9, ref_logp=adv - 8, kl_coef=0.2)
    two = zr.policy_loss(z * big, action, adv, old_logp=adv - 9, ref_logp=adv - 8, kl_coef=0.2, temperature=big)
    assert all(torch.equal(a, b) for a, b in zip(one[:3], two[:3])) and same_gradient(one[3], two[3])
    for rest in (None, lse):
        one = zr.distill_loss(z, idx.int(), top, teacher_lse=rest)
        two = zr.distill_loss(z * big, idx.int(), top * big, teacher_lse=rest, temperature=big)
        assert torch.equal(one[0], two[0]) and same_gradient(one[1], two[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [700, 40001, 300007])
@pytest.mark.parametrize("k", [0, 3])
def test_distill_rest_alone(env, vocab, k, dtype):
    """No list, one of padding, and one of tokens that the student gives nothing: the
    rest is all of q, wherever the logits lie."""
    torch, zr = env
    rng = np.random.default_rng(vocab)
    z = rng.normal(size=(6, vocab)).astype(np.float32) + np.array([[-1000], [-200], [0], [200], [1e30], [-1e30]], np.float32)
    idx = np.full((6, k), -1, dtype=np.int32)
    top = np.zeros((6, k), dtype=np.float32)
    lse = np.full(6, 1.0, dtype=np.float32)
    b = Buffers(torch, z, dtype)
    loss, dz = run_distill(torch, zr, b, idx, top, lse, 1.0, None)
    # p_rest = q_rest = 1: no loss, and q - q is left of the gradient
    check(loss, np.zeros(6), 2.0 ** -22)
    check(dz, np.zeros(z.shape), 2.0 ** -22)
    if k:
        idx[:] = [0, 9, vocab - 1]
        b.z[:, [0, 9, vocab - 1]] = -np.inf
        b.exact = b.z.double().cpu().numpy()
        loss, dz = run_distill(torch, zr, b, idx, top - np.inf, lse, 1.0, None)
        check(loss, np.zeros(6), 2.0 ** -22)
        check(dz, np.zeros(z.shape), 2.0 ** -22)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_masked_token_of_little_probability(env, rest, dtype):
    """p (log p - log q) of a token that the student masks by the lowest value is in
    fp32's range where p is small, also below temperature 1, where log q is not."""
    torch, zr = env
    rng = np.random.default_rng(3)
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    z = logits(rng, 4, 3000)
    z[:, 17] = low
    idx = np.tile(np.array([4, 17, 99], dtype=np.int32), (4, 1))
    top = np.tile(np.array([1.0, -2.0, 0.5], dtype=np.float32), (4, 1))  # p of 5e-5 at temperature 0.3
    lse = np.full(4, 4.0, dtype=np.float32) if rest else None
    b = Buffers(torch, z, dtype)
    loss, dz = run_distill(torch, zr, b, idx, top, lse, 0.3, None)
    wl, wd = step.distill(b.exact, idx, top, lse, 0.3, None)
    assert (wl > 1e33).all() and (wl < 1e36).all()
    check(loss, wl, 2.0 ** -16 * wl)
    check(dz, wd, (2.0 ** -18 + 4 * rel(3000, 0.3)) / 0.3 + half_ulp(dtype) * np.abs(wd))


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("vocab", [1, 5, 900])
def test_distill_of_a_whole_vocabulary_with_a_bad_logit(env, vocab, bad):
    """Nothing outside the list, mass for it, and a NaN or +inf logit of a token to
    which the teacher gives nothing: NaN, not the +inf of a rest that is missed."""
    torch, zr = env
    z = torch.zeros(2, vocab, device="cuda")
    z[0, vocab // 2] = bad
    idx = torch.arange(vocab, device="cuda").int().repeat(2, 1)
    top = torch.full((2, vocab), -np.inf, dtype=torch.float32, device="cuda")
    loss, dz = zr.distill_loss(z, idx, top, teacher_lse=torch.ones(2, device="cuda"))
    assert bool(torch.isnan(loss[0])) and bool(torch.isnan(dz[0]).all())
    assert float(loss[1]) == np.inf
