"""The operators of a data-parallel worker's training step, as measured cases.

Four operators stand before the gradient aggregation of this library: the
gated feed-forward block with its backward pass (the weight gradients go to
the rank's buffer), and three losses over a vocabulary with their gradients:
distillation from a teacher's top logits, the clipped policy loss with a KL
term, and the preference loss over pairs of sequences.

``own = False`` computes them in plain torch operations in 32 bits;
``own = True`` calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decoded token through a block of the size that the sparse
        # benchmark's gradient tensor has (4096 x 11008): weights are streamed.
        dict(name="ff_token", op="ff", rows=1, d=4096, f=11008, act="silu"),
        # A batch of sequences decoding together: still bound by the weights.
        dict(name="ff_batch", op="ff", rows=48, d=4096, f=11008, act="gelu_tanh"),
        # A long prompt, or one micro-batch going forward: bound by the tensor cores.
        dict(name="ff_prompt", op="ff", rows=4096, d=4096, f=11008, act="silu"),
        # The micro-batch's backward pass: input and weight gradients.
        dict(name="ff_train", op="ff_backward", rows=4096, d=4096, f=11008, act="silu"),
        # A small model of odd widths, a ragged batch.
        dict(name="ff_train_odd", op="ff_backward", rows=777, d=1001, f=2731, act="gelu"),
        # A few rows: latency.
        dict(name="distill_small", op="distill", rows=8, vocab=32000, k=8, dtype="f32",
             tail=False, ragged=False, tau=1.0),
        # An odd vocabulary (rows start at every alignment), ragged teacher lists.
        dict(name="distill_odd", op="distill", rows=1000, vocab=50001, k=20, dtype="bf16",
             tail=False, ragged=True, tau=1.5),
        # A micro-batch over a large vocabulary, the rest of the teacher's mass as one class.
        dict(name="distill_large", op="distill", rows=4096, vocab=131072, k=64, dtype="bf16",
             tail=True, ragged=False, tau=2.0),
        # A short answer's tokens.
        dict(name="policy_small", op="policy", rows=16, vocab=32000, dtype="bf16", kl=0.05, tau=1.0),
        # The tokens of a batch of long answers.
        dict(name="policy_large", op="policy", rows=8192, vocab=131072, dtype="bf16", kl=0.02,
             tau=0.8),
        # Three short pairs, an odd vocabulary.
        dict(name="preference_odd", op="preference", rows=150, pairs=3, vocab=65537, dtype="bf16",
             smoothing=0.1),
        # Sixteen pairs of long answers in fp32 logits.
        dict(name="preference_large", op="preference", rows=8190, pairs=16, vocab=65536, dtype="f32",
             smoothing=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["ff", "ff_backward", "distill", "policy", "preference"])
    if op in ("ff", "ff_backward"):
        d, f = _log(rng, 64, 4096), _log(rng, 64, 11008)
        if rng.random() < 0.6:  # most widths are multiples of 8
            d, f = max(64, d // 8 * 8), max(64, f // 8 * 8)
        return dict(op=op, rows=_log(rng, 1, 4096), d=d, f=f,
                    act=rng.choice(["silu", "gelu", "gelu_tanh"]))
    dtype = rng.choice(["f32", "bf16"])
    most = (1 << 31) // (4 if dtype == "f32" else 2)  # elements of 2 GiB of logits
    vocab = _log(rng, 1000, 262144)
    if rng.random() < 0.6:
        vocab = max(1000, vocab // 64 * 64)
    rows = _log(rng, 1, min(8192, most // vocab))
    if op == "distill":
        return dict(op=op, rows=rows, vocab=vocab, k=_log(rng, 1, 256), dtype=dtype,
                    tail=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    tau=rng.choice([1.0, 1.5, 2.0]))
    if op == "policy":
        return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, kl=rng.choice([0.0, 0.02, 0.1]),
                    tau=rng.choice([0.7, 1.0, 1.2]))
    rows = max(8, rows)
    return dict(op=op, rows=rows, pairs=_log(rng, 1, max(1, min(32, rows // 4))), vocab=vocab,
                dtype=dtype, smoothing=rng.choice([0.0, 0.1]))


def work(case):
    op = case["op"]
    if op in ("ff", "ff_backward"):
        t, d, f = case["rows"], case["d"], case["f"]
        if op == "ff":  # x, both weights in; h out
            return {"bytes": 2 * (t * d + 2 * f * d + t * f), "flops": 4 * t * d * f}
        # x, dh, both weights in; dx and both weight gradients out; the two
        # projections again, the input gradient, the weight gradients
        return {"bytes": 2 * (2 * t * d + t * f + 4 * f * d), "flops": 12 * t * d * f}
    t, v = case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    read = t - _left_out(case)  # rows that count; every row's gradient is written
    more = {"distill": 8 * t * case.get("k", 0) + 12 * t, "policy": 32 * t, "preference": 8 * t}[op]
    return {"bytes": size * v * (read + t) + more, "flops": 8 * v * read}


def _left_out(case):
    """Rows that the mask leaves out: padding, or the prompts of the pairs."""
    return case["rows"] // (4 if case["op"] == "preference" else 8)


# ------------------------------------------------------------------ the inputs
def _logits(case, gen):
    """Logits as a trained model gives them: most of the mass on a few tokens
    (one in each eighth of the vocabulary), a few percent on all the others.
    The token of a row is one of the likely ones."""
    t, v = case["rows"], case["vocab"]
    z = torch.randn(t, v, generator=gen, device=DEV, dtype=DTYPES[case["dtype"]])
    z.mul_(2.0)
    eighth = v // 8
    likely = torch.randint(0, eighth, (t, 8), generator=gen, device=DEV)
    likely += torch.arange(8, device=DEV) * eighth
    bump = math.log(v) + 2 + 3 * torch.rand(t, 8, generator=gen, device=DEV)
    z.scatter_(1, likely, (bump * case.get("tau", 1.0)).to(z.dtype))
    one = torch.randint(0, 8, (t, 1), generator=gen, device=DEV)
    return z, likely.gather(1, one)[:, 0].contiguous()


def _mask(case, gen):
    keep = torch.ones(case["rows"], device=DEV)
    keep[torch.randperm(case["rows"], generator=gen, device=DEV)[:_left_out(case)]] = 0
    return keep


def _token_logp(z, token, tau):
    """log softmax(z / tau)[token], a band of rows at a time."""
    out = torch.empty(z.shape[0], device=DEV)
    for lo in range(0, z.shape[0], 1024):
        s = z[lo:lo + 1024].float() / tau
        out[lo:lo + 1024] = s.gather(1, token[lo:lo + 1024, None])[:, 0] - torch.logsumexp(s, 1)
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if op in ("ff", "ff_backward"):
        t, d, f = case["rows"], case["d"], case["f"]
        b = torch.bfloat16
        st = dict(case=case, x=randn(t, d).to(b), wg=(randn(f, d) / math.sqrt(d)).to(b),
                  wu=(randn(f, d) / math.sqrt(d)).to(b))
        if op == "ff":
            st["h"] = torch.empty(t, f, device=DEV, dtype=b)
        else:
            st["dh"] = (randn(t, f) * 1e-2).to(b)
            st["dx"] = torch.empty_like(st["x"])
            st["dwg"], st["dwu"] = torch.empty_like(st["wg"]), torch.empty_like(st["wu"])
        return st

    t, v = case["rows"], case["vocab"]
    z, token = _logits(case, gen)
    keep = _mask(case, gen)
    st = dict(case=case, z=z, dz=torch.empty_like(z), loss=torch.empty(t, device=DEV))
    if op == "distill":
        k, tau = case["k"], case["tau"]
        idx = torch.empty(t, k, dtype=torch.int32, device=DEV)
        top, lse = torch.empty(t, k, device=DEV), torch.empty(t, device=DEV)
        for lo in range(0, t, 512):  # the teacher agrees with the student up to noise
            s = z[lo:lo + 512].float()
            s = s + torch.randn(s.shape, generator=gen, device=DEV)
            top[lo:lo + 512], at = torch.topk(s, k, dim=1)
            idx[lo:lo + 512] = at.int()
            lse[lo:lo + 512] = torch.logsumexp(s / tau, 1)
        if case["ragged"]:  # lists of different lengths, padded with -1
            length = torch.randint(1, k + 1, (t, 1), generator=gen, device=DEV)
            idx.masked_fill_(torch.arange(k, device=DEV)[None] >= length, -1)
        st.update(idx=idx, top=top, lse=lse if case["tail"] else None,
                  weight=keep / max(1, t - _left_out(case)))
    elif op == "policy":
        logp = _token_logp(z, token, case["tau"])
        old = logp + 0.15 * randn(t)
        for edge in (0.8, 1.25):  # no ratio on the edge of the clip range
            old = torch.where((torch.exp(logp - old) - edge).abs() < 1e-4, old + 1e-2, old)
        st.update(action=token.int(), old=old, ref=logp + 0.3 * randn(t), adv=randn(t),
                  weight=keep / max(1, t - _left_out(case)), logp=torch.empty(t, device=DEV),
                  kl=torch.empty(t, device=DEV))
    else:
        p = case["pairs"]
        cut = torch.randperm(t - 1, generator=gen, device=DEV)[:2 * p - 1] + 1
        off = torch.zeros(2 * p + 1, dtype=torch.int64, device=DEV)
        off[1:2 * p] = torch.sort(cut)[0]
        off[2 * p] = t
        ref = _token_logp(z, token, 1.0) + 0.5 * randn(t)
        st.update(target=torch.where(keep > 0, token, -1).int(), off=off, ref=ref,
                  weight=torch.full((p,), 1.0 / p, device=DEV), loss=torch.empty(p, device=DEV),
                  reward=torch.empty(2 * p, device=DEV))
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)(state)


def _own(st):
    import gradient_synchronisation_gb300 as zr

    case = st["case"]
    op = case["op"]
    if op == "ff":
        return zr.gated_ff(st["x"], st["wg"], st["wu"], activation=_code(zr, case), out=st["h"])
    if op == "ff_backward":
        return zr.gated_ff_backward(st["x"], st["wg"], st["wu"], st["dh"],
                                    activation=_code(zr, case), dx=st["dx"], dw_gate=st["dwg"],
                                    dw_up=st["dwu"])
    if op == "distill":
        return zr.distill_loss(st["z"], st["idx"], st["top"], teacher_lse=st["lse"],
                               temperature=case["tau"], weight=st["weight"], loss=st["loss"],
                               dlogits=st["dz"])
    if op == "policy":
        return zr.policy_loss(st["z"], st["action"], st["adv"], old_logp=st["old"],
                              ref_logp=st["ref"], clip_low=0.2, clip_high=0.25,
                              kl_coef=case["kl"], temperature=case["tau"], weight=st["weight"],
                              loss=st["loss"], logp=st["logp"], kl=st["kl"], dlogits=st["dz"])
    return zr.preference_loss(st["z"], st["target"], st["off"], st["ref"], beta=0.1,
                              label_smoothing=case["smoothing"], weight=st["weight"],
                              loss=st["loss"], reward=st["reward"], dlogits=st["dz"])


def _code(zr, case):
    return {"silu": zr.ZR_ACT_SILU, "gelu": zr.ZR_ACT_GELU, "gelu_tanh": zr.ZR_ACT_GELU_TANH}[case["act"]]


C_TANH = math.sqrt(2 / math.pi)


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(C_TANH * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * C_TANH * (1 + 0.134145 * g * g)


def _softmax(s):
    """exp(s - max), its sum, the maximum and the logarithm of the sum."""
    m = s.max(1, keepdim=True)[0]
    e = torch.exp(s - m)
    total = e.sum(1, keepdim=True)
    return e, total, m, torch.log(total)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("ff", "ff_backward"):
        x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, case["act"])
        if op == "ff":
            return (a * u).bfloat16()
        dh = st["dh"].float()
        dg, du = dh * u * da, dh * a
        return (dg @ wg + du @ wu).bfloat16(), (dg.t() @ x).bfloat16(), (du.t() @ x).bfloat16()
    z = st["z"]
    rows = torch.arange(z.shape[0], device=z.device)
    if op == "distill":
        tau = case["tau"]
        used = st["weight"] != 0
        s = z.float() / tau
        e, total, m, logsum = _softmax(s)
        there = st["idx"] >= 0
        at = st["idx"].clamp(min=0).long()
        top = (st["top"] / tau).masked_fill(~there, -math.inf)
        if case["tail"]:
            logt = top - st["lse"][:, None]
        else:
            _, _, most, logtop = _softmax(top)
            logt = top - most - logtop
        p = torch.exp(logt)
        logq = s.gather(1, at) - m - logsum
        loss = torch.where(p > 0, p * (logt - logq), 0.0).sum(1)
        if case["tail"]:
            listed_ = torch.zeros_like(s).scatter_add_(1, at, there.float()) > 0
            rest = torch.where(listed_, 0.0, e).sum(1, keepdim=True)
            on = torch.where(listed_, e, 0.0).sum(1, keepdim=True)
            pr = (1 - p.sum(1, keepdim=True)).clamp(min=0)
            qr = rest / (rest + on)
            gap = torch.log1p(-p.sum(1, keepdim=True)) + torch.log1p(on / rest)
            loss = loss + torch.where(pr > 0, pr * gap, 0.0)[:, 0]
            dz = e / total * torch.where(listed_, 1.0, 1 - pr / qr)
        else:
            dz = e / total
        dz.scatter_add_(1, at, -p)
        dz = torch.where(used[:, None], dz * (st["weight"] / tau)[:, None], 0.0)
        return torch.where(used, loss * st["weight"], 0.0), dz.to(z.dtype)
    if op == "policy":
        tau, beta, w = case["tau"], case["kl"], st["weight"]
        used = w != 0
        s = z.float() / tau
        e, total, m, logsum = _softmax(s)
        a = st["action"].long()
        logp = torch.where(used, s[rows, a] - m[:, 0] - logsum[:, 0], 0.0)
        r = torch.exp(logp - st["old"])
        free, clipped = r * st["adv"], r.clamp(0.8, 1.25) * st["adv"]
        back = torch.exp(st["ref"] - logp)
        kl = torch.where(used, back - (st["ref"] - logp) - 1, 0.0)
        loss = torch.where(used, w * (beta * kl - torch.minimum(free, clipped)), 0.0)
        g = torch.where(used, w * (beta * (1 - back) - torch.where(free <= clipped, free, 0.0)) / tau, 0.0)
        dz = e / total * -g[:, None]
        dz[rows, a] += g
        return loss, logp, kl, dz.to(z.dtype)
    p, eps, beta = case["pairs"], case["smoothing"], 0.1
    used = st["target"] >= 0
    a = st["target"].clamp(min=0).long()
    s = z.float()
    e, total, m, logsum = _softmax(s)
    delta = torch.where(used, s[rows, a] - m[:, 0] - logsum[:, 0] - st["ref"], 0.0)
    which = torch.searchsorted(st["off"], rows, right=True) - 1
    member = (torch.arange(2 * p, device=z.device)[:, None] == which[None]).float()
    reward = beta * (member * delta[None]).sum(1)
    m = reward[0::2] - reward[1::2]
    soft = torch.log1p(torch.exp(-m.abs()))
    lose, win = soft + (-m).clamp(min=0), soft + m.clamp(min=0)
    loss = st["weight"] * ((1 - eps) * lose + eps * win)
    slope = beta * st["weight"] * (eps / (1 + torch.exp(-m)) - (1 - eps) / (1 + torch.exp(m)))
    c = torch.stack([slope, -slope], 1).reshape(-1)[which]
    c = torch.where(used, c, 0.0)
    dz = e / total * -c[:, None]
    dz[rows, a] += c
    return loss, reward, dz.to(z.dtype)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("ff", "ff_backward"):
        t, d, f = case["rows"], case["d"], case["f"]
        if 12 * t * d * f > 4e12:
            return None
        st = prepare(case, seed)
        x, wg, wu = (st[n].double() for n in ("x", "wg", "wu"))
        g = torch.einsum("td,fd->tf", x, wg).requires_grad_()
        u = torch.einsum("td,fd->tf", x, wu)
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            a = g * torch.special.ndtr(g)
        else:
            a = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        if op == "ff":
            return (a * u).detach()
        (slope,) = torch.autograd.grad(a.sum(), g)
        dh = st["dh"].double()
        dg, du = dh * u * slope, dh * a.detach()
        return (torch.einsum("tf,fd->td", dg, wg) + torch.einsum("tf,fd->td", du, wu),
                torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x))
    st = prepare(case, seed)
    z, t = st["z"], case["rows"]
    out = torch.zeros(z.shape, dtype=torch.float64, device=DEV)
    if op == "preference":
        beta, eps = 0.1, case["smoothing"]
        logp = torch.zeros(t, dtype=torch.float64, device=DEV)
        target = st["target"].tolist()
        use = [i for i in range(t) if target[i] >= 0]
        for lo in range(0, t, 256):
            ls = torch.log_softmax(z[lo:lo + 256].double(), 1)
            tg = st["target"][lo:lo + 256].long()
            logp[lo:lo + 256] = torch.where(tg >= 0, ls.gather(1, tg.clamp(min=0)[:, None])[:, 0], 0.0)
        diff = (logp - st["ref"].double()).cpu()
        off = st["off"].tolist()
        usable = set(use)
        sums = torch.tensor([math.fsum(float(diff[i]) for i in range(a, b) if i in usable)
                             for a, b in zip(off, off[1:])], dtype=torch.float64)
        reward = (beta * sums).requires_grad_()
        m = reward[0::2] - reward[1::2]
        ls = torch.nn.functional.logsigmoid
        loss = st["weight"].double().cpu() * (-(1 - eps) * ls(m) - eps * ls(-m))
        (by_reward,) = torch.autograd.grad(loss.sum(), reward)
        row_slope = torch.zeros(t, dtype=torch.float64)
        for s, (a, b) in enumerate(zip(off, off[1:])):
            row_slope[a:b] = beta * by_reward[s]
        row_slope = torch.where(st["target"] >= 0, row_slope.to(DEV), 0.0)
        for lo in range(0, t, 256):
            q = torch.softmax(z[lo:lo + 256].double(), 1)
            tg = st["target"][lo:lo + 256].clamp(min=0).long()
            one = torch.zeros_like(q).scatter_(1, tg[:, None], 1.0)
            out[lo:lo + 256] = row_slope[lo:lo + 256, None] * (one - q)
        return loss.detach().to(DEV), reward.detach().to(DEV), out
    w, tau = st["weight"].double(), case["tau"]
    loss = torch.zeros(t, dtype=torch.float64, device=DEV)
    logps, kls = torch.zeros_like(loss), torch.zeros_like(loss)
    for lo in range(0, t, 256):
        b = slice(lo, lo + 256)
        live = w[b] != 0
        ls = torch.log_softmax(z[b].double() / tau, 1)
        q = torch.exp(ls)
        if op == "policy":
            a = st["action"][b].long()[:, None]
            lp = ls.gather(1, a)[:, 0]
            old, ref, adv = (st[n][b].double() for n in ("old", "ref", "adv"))
            leaf = lp.clone().requires_grad_()
            r = torch.exp(leaf - old)
            # the clip range's ends as the 32-bit arithmetic has them are off by under 1e-7
            surrogate = torch.where(adv >= 0, r.clamp(max=1.25), r.clamp(min=0.8)) * adv
            k3 = torch.exp(ref - leaf) - (ref - leaf) - 1
            each = w[b] * (case["kl"] * k3 - surrogate)
            (slope,) = torch.autograd.grad(each.sum(), leaf)
            loss[b] = torch.where(live, each.detach(), 0.0)
            logps[b], kls[b] = torch.where(live, lp, 0.0), torch.where(live, k3.detach(), 0.0)
            one = torch.zeros_like(q).scatter_(1, a, 1.0)
            dz = slope[:, None] * (one - q) / tau
        else:
            there = st["idx"][b] >= 0
            at = st["idx"][b].clamp(min=0).long()
            top = torch.where(there, st["top"][b].double() / tau, -math.inf)
            lt = st["lse"][b].double()[:, None] if case["tail"] else torch.logsumexp(top, 1, keepdim=True)
            p = torch.zeros_like(q).scatter_add_(1, at, torch.exp(top - lt))
            on = torch.zeros_like(q).scatter_add_(1, at, there.double()) > 0
            each = torch.where(on & (p > 0), p * (torch.log(p) - ls), 0.0).sum(1)
            dz = q - p
            if case["tail"]:
                rest = (1 - p.sum(1, keepdim=True)).clamp(min=0)
                qr = torch.where(on, 0.0, q).sum(1, keepdim=True)
                each = each + torch.special.xlogy(rest, rest / qr)[:, 0]
                dz = torch.where(on, dz, q - rest * q / qr)
            loss[b] = torch.where(live, w[b] * each, 0.0)
            dz = dz * (w[b] / tau)[:, None]
        out[b] = torch.where(live[:, None], dz, 0.0)
    return (loss, out) if op == "distill" else (loss, logps, kls, out)
