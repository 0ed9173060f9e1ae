"""The operators of a training step in float64 numpy, from their definitions:
the gated feed-forward block, and the distillation, policy and preference
losses, each with its gradient.  Rows are handled one at a time; nothing is
shared with the CUDA path."""

import math

import numpy as np

SQRT_HALF = math.sqrt(0.5)


# ------------------------------------------------------------ activations
def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def activation(g, act):
    """a(g) and a'(g); act: 'silu', 'gelu' or 'gelu_tanh'."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s + g * s * (1.0 - s)
    if act == "gelu":
        cdf = 0.5 * (1.0 + _erf(g * SQRT_HALF))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    inner = k * (g + 0.044715 * g ** 3)
    t = np.tanh(inner)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def gated_ff(x, wg, wu, act):
    x, wg, wu = (np.asarray(v, dtype=np.float64) for v in (x, wg, wu))
    a, _ = activation(x @ wg.T, act)
    return a * (x @ wu.T)


def gated_ff_backward(x, wg, wu, dh, act):
    x, wg, wu, dh = (np.asarray(v, dtype=np.float64) for v in (x, wg, wu, dh))
    a, da = activation(x @ wg.T, act)
    dg, du = dh * (x @ wu.T) * da, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


# ------------------------------------------------------------ losses
def _log_softmax(z):
    """log softmax of one row; None when nothing has any mass."""
    m = z.max()
    if m == -np.inf:
        return None
    d = z - m
    return d - math.log(np.exp(d).sum())


def distill(z, idx, top, lse=None, tau=1.0, weight=None):
    """(loss [rows], dlogits [rows, vocab])."""
    z = np.asarray(z, dtype=np.float64)
    rows, vocab = z.shape
    loss, dz = np.zeros(rows), np.zeros((rows, vocab))
    for t in range(rows):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0.0:
            continue
        if np.isnan(z[t]).any() or (z[t] == np.inf).any():
            loss[t], dz[t] = np.nan, np.nan
            continue
        logq = _log_softmax(z[t] / tau)
        if logq is None:
            continue
        q = np.exp(logq)
        there = [i for i in range(len(idx[t])) if 0 <= idx[t][i] < vocab]
        tok = np.array([idx[t][i] for i in there], dtype=np.int64)
        lt = np.array([top[t][i] for i in there], dtype=np.float64) / tau
        if lse is None:
            if len(tok) == 0 or lt.max() == -np.inf:
                continue
            logp = lt - lt.max()
            logp = logp - math.log(np.exp(logp).sum())
        else:
            logp = lt - float(lse[t])
        p = np.exp(logp)
        total = 0.0
        for j, lp, pj in zip(tok, logp, p):
            if pj > 0:
                total += pj * (lp - logq[j])
        grad = q.copy()
        grad[tok] -= p
        if lse is not None:
            off = np.ones(vocab, dtype=bool)
            off[tok] = False
            rest_p, rest_q = max(0.0, 1.0 - p.sum()), q[off].sum()
            if rest_q == 0.0:
                total += np.inf if rest_p > 2.0 ** -20 else 0.0
            elif rest_p > 0:
                total += rest_p * math.log(rest_p / rest_q)
                grad[off] *= 1.0 - rest_p / rest_q
        loss[t], dz[t] = w * total, grad * w / tau
    return loss, dz


def policy(z, action, adv, old=None, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, tau=1.0,
           weight=None):
    """(loss, logp, kl [rows], dlogits [rows, vocab])."""
    z = np.asarray(z, dtype=np.float64)
    rows, vocab = z.shape
    loss, logps, kls, dz = np.zeros(rows), np.zeros(rows), np.zeros(rows), np.zeros((rows, vocab))
    for t in range(rows):
        w = 1.0 if weight is None else float(weight[t])
        a = int(action[t])
        if w == 0.0 or a < 0:
            continue
        if a >= vocab or np.isnan(z[t]).any() or (z[t] == np.inf).any():
            loss[t] = logps[t] = kls[t] = np.nan
            dz[t] = np.nan
            continue
        logq = _log_softmax(z[t] / tau)
        if logq is None:
            continue
        lp = logq[a]
        r = 1.0 if old is None else math.exp(lp - float(old[t]))
        adv_t = float(adv[t])
        free = r * adv_t
        held = min(max(r, 1.0 - clip_low), 1.0 + clip_high) * adv_t
        g = -free if free <= held else 0.0
        value = -min(free, held)
        if ref is not None:
            x = float(ref[t]) - lp
            kls[t] = math.exp(x) - x - 1.0
            value += kl_coef * kls[t]
            g += kl_coef * (1.0 - math.exp(x))
        loss[t], logps[t] = w * value, lp
        one = np.zeros(vocab)
        one[a] = 1.0
        dz[t] = w * g * (one - np.exp(logq)) / tau
    return loss, logps, kls, dz


def preference(z, target, offsets, ref, beta=0.1, eps=0.0, weight=None):
    """(loss [pairs], reward [2 pairs], dlogits [rows, vocab])."""
    z = np.asarray(z, dtype=np.float64)
    rows, vocab = z.shape
    pairs = len(offsets) // 2
    logq = [_log_softmax(z[t]) if target[t] >= 0 else None for t in range(rows)]
    used = [logq[t] is not None for t in range(rows)]
    reward = np.array([beta * math.fsum(logq[t][target[t]] - float(ref[t])
                                        for t in range(offsets[s], offsets[s + 1]) if used[t])
                       for s in range(2 * pairs)]).reshape(2 * pairs)
    loss, dz = np.zeros(pairs), np.zeros((rows, vocab))
    for p in range(pairs):
        w = 1.0 if weight is None else float(weight[p])
        m = reward[2 * p] - reward[2 * p + 1]
        log_sig = lambda x: -math.log1p(math.exp(-x)) if x > -30 else x - math.exp(x)  # noqa: E731
        # a part without weight is none, also where its logarithm is infinite
        loss[p] = w * sum(-c * log_sig(x) for c, x in ((1 - eps, m), (eps, -m)) if c > 0)
        slope = w * beta * (eps * math.exp(log_sig(m)) - (1 - eps) * math.exp(log_sig(-m)))
        for s, sign in ((2 * p, 1.0), (2 * p + 1, -1.0)):
            for t in range(offsets[s], offsets[s + 1]):
                if used[t]:
                    dz[t] = -sign * slope * np.exp(logq[t])
                    dz[t, target[t]] += sign * slope
    return loss, reward, dz


# ------------------------------------------------------------ norm
def rms_norm(s, weight, eps):
    """(y, rstd) of rows s (with their residual already added)."""
    s, weight = np.asarray(s, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    rstd = np.array([1.0 / math.sqrt(math.fsum(v * v for v in row) / len(row) + eps) for row in s])
    return s * rstd.reshape(-1, 1) * weight, rstd


def rms_norm_backward(s, weight, rstd, dy, ds=None):
    """(dx, dweight) with the given rstd."""
    s, weight, dy = (np.asarray(v, dtype=np.float64) for v in (s, weight, dy))
    h = s * np.asarray(rstd, dtype=np.float64).reshape(-1, 1)
    g = dy * weight
    c = (g * h).mean(axis=1, keepdims=True)
    dx = np.asarray(rstd, dtype=np.float64).reshape(-1, 1) * (g - h * c)
    if ds is not None:
        dx = dx + np.asarray(ds, dtype=np.float64)
    return dx, (dy * h).sum(axis=0)


# ------------------------------------------------------------ cross entropy over a vocabulary
def cross_entropy(x, w, target, weight=None):
    """(loss, lse [rows], dx, dw, dz [rows, vocab]) of states x over a vocabulary w."""
    w = np.asarray(w, dtype=np.float64)
    rows, vocab = len(target), w.shape[0]
    loss, lse = np.zeros(rows), np.zeros(rows)
    dz, dx, dw = np.zeros((rows, vocab)), np.zeros((rows, w.shape[1])), np.zeros(w.shape)
    for t in range(rows):
        k = 1.0 if weight is None else float(weight[t])
        if not 0 <= target[t] < vocab or k == 0.0:
            continue
        row = np.asarray(x[t], dtype=np.float64)
        z = w @ row
        if np.isnan(z).any() or (z == np.inf).any():
            loss[t] = lse[t] = np.nan
            dz[t] = dx[t] = np.nan
            dw += np.nan
            continue
        logp = _log_softmax(z)
        if logp is None:
            continue
        lse[t] = z.max() - logp.max()
        loss[t] = -k * logp[target[t]]
        dz[t] = k * np.exp(logp)
        dz[t, target[t]] = k * math.expm1(logp[target[t]])
        dx[t] = dz[t] @ w
        dw += np.outer(dz[t], row)
    return loss, lse, dx, dw, dz


# ------------------------------------------------------------ orthogonalised matrices
def orthogonalise(g, coefficients, eps=1e-7, rounded=None):
    """X after the steps of ``coefficients`` (a, b, c each), from g / (|g| + eps).
    ``rounded``: what X, A and the polynomial of each step are rounded by."""
    cut = rounded or (lambda v: v)
    x = np.asarray(g, dtype=np.float64)
    size = math.sqrt(math.fsum(float(v) ** 2 for v in x.ravel())) + eps
    x = cut(x / size if size > 0 else x)
    tall = x.shape[0] > x.shape[1]
    for n, (a, b, c) in enumerate(coefficients):
        s = cut(x.T @ x if tall else x @ x.T)
        p = cut(a * np.eye(len(s)) + b * s + c * (s @ s))
        x = x @ p if tall else p @ x
        if n + 1 < len(coefficients):
            x = cut(x)
    return x
