"""The rest of a data-parallel worker's step, as measured cases.

Four operators stand around the ones that perf/operators.py measures: the
root-mean-square norm with the residual's addition and its backward pass (what
a block reads), the cross entropy of token states over a vocabulary with the
gradients of the states and of the vocabulary's weights (the logits are not
kept), and the orthogonalised update that a weight matrix's averaged gradient
becomes.

``own = False`` computes them in plain torch operations in 32 bits;
``own = True`` calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token's state between two blocks while decoding: latency.
        dict(name="norm_token", op="norm", rows=1, d=4096, dtype="bf16", residual=True),
        # A small model of odd width in fp32, a ragged batch, the first norm (no residual yet).
        dict(name="norm_odd", op="norm", rows=777, d=1001, dtype="f32", residual=False),
        # A batch of long sequences: streams from memory.
        dict(name="norm_large", op="norm", rows=16384, d=4096, dtype="bf16", residual=True),
        # The odd model's backward pass.
        dict(name="norm_back_odd", op="norm_backward", rows=777, d=1001, dtype="bf16", residual=False),
        # The batch's backward pass, with the gradient that comes along the residual.
        dict(name="norm_back_large", op="norm_backward", rows=16384, d=4096, dtype="bf16", residual=True),
        # A few tokens of a small model over a small vocabulary: latency.
        dict(name="ce_small", op="ce", rows=16, d=512, vocab=32000, grad=True),
        # Held-out text: the loss alone.
        dict(name="ce_eval", op="ce", rows=2048, d=1024, vocab=65536, grad=False),
        # The odd model's step: rows off 16 bytes, an odd vocabulary.
        dict(name="ce_odd", op="ce", rows=1000, d=1001, vocab=50001, grad=True),
        # A micro-batch of a large model over a large vocabulary.
        dict(name="ce_large", op="ce", rows=8192, d=4096, vocab=131072, grad=True),
        # One shape's matrices of all the blocks of a small model, in one call.
        dict(name="ortho_batch", op="ortho", count=16, rows=704, cols=256, dtype="bf16"),
        # The odd model's projection, its gradient averaged in fp32.
        dict(name="ortho_odd", op="ortho", count=1, rows=2731, cols=1001, dtype="f32"),
        # A large model's projection.
        dict(name="ortho_large", op="ortho", count=1, rows=4096, cols=11008, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "ce", "ce", "ortho", "ortho"])
    even = rng.random() < 0.6  # most widths are multiples of 8

    def width(lo, hi):
        n = _log(rng, lo, hi)
        return max(lo, n // 8 * 8) if even else n

    if op in ("norm", "norm_backward"):
        d = width(64, 16384)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 26) // d)), d=d,
                    dtype=rng.choice(["f32", "bf16"]), residual=rng.random() < 0.5)
    if op == "ce":
        return dict(op=op, rows=_log(rng, 1, 8192), d=width(64, 4096), vocab=width(1000, 131072),
                    grad=rng.random() < 0.7)
    small, large = width(64, 4096), width(64, 11008)
    if rng.random() < 0.5:
        small, large = large, small
    one = (min(small, large) ** 2) * (small + large)
    return dict(op=op, count=_log(rng, 1, max(1, min(24, (1 << 37) // one))), rows=small, cols=large,
                dtype=rng.choice(["f32", "bf16"]))


def _left_out(case):
    """Rows without a target: padding, prompts."""
    return case["rows"] // 8


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        t, d = case["rows"], case["d"]
        size = 4 if case["dtype"] == "f32" else 2
        extra = 1 if case["residual"] else 0
        if op == "norm":  # x (and the residual) in; y (and the sum) out
            return {"bytes": size * d * (t * (2 + 2 * extra) + 1) + 4 * t, "flops": 5 * t * d}
        # s, dy (and the residual's gradient) in; dx out; the weight in, its gradient out
        return {"bytes": size * d * (t * (3 + extra) + 2) + 4 * t, "flops": 10 * t * d}
    if op == "ce":
        t, d, v = case["rows"], case["d"], case["vocab"]
        read = t - _left_out(case)
        moved = 2 * (read * d + v * d) + 16 * t
        if case["grad"]:  # both gradients out; logits, states' and weights' gradients
            return {"bytes": moved + 2 * (t * d + v * d), "flops": 6 * read * d * v}
        return {"bytes": moved, "flops": 2 * read * d * v}
    n, m, k = case["count"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    size = 4 if case["dtype"] == "f32" else 2
    # a step: the symmetric X X^T and A A, half of each; then B X
    return {"bytes": n * m * k * (size + 2), "flops": STEPS * n * (m * (m + 1) * (m + k) + 2 * m * m * k)}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if op in ("norm", "norm_backward"):
        t, d, dt = case["rows"], case["d"], DTYPES[case["dtype"]]
        # a residual stream: rows of different size, a few channels that are far larger
        channel = torch.exp(0.3 * randn(d))
        channel[torch.randint(0, d, (max(1, d // 512),), generator=gen, device=DEV)] *= 20
        stream = randn(t, d) * torch.exp(0.5 * randn(t, 1)) * channel
        st = dict(case=case, weight=(1 + 0.2 * randn(d)).to(dt))
        if op == "norm":
            st.update(x=(randn(t, d) if case["residual"] else stream).to(dt), y=torch.empty(t, d, device=DEV, dtype=dt),
                      rstd=torch.empty(t, device=DEV), res=None, s=None)
            if case["residual"]:
                st.update(res=stream.to(dt), s=torch.empty(t, d, device=DEV, dtype=dt))
        else:
            s = stream.to(dt)
            st.update(s=s, rstd=1 / torch.sqrt((s.float() ** 2).mean(1) + 1e-6), dy=(1e-2 * randn(t, d)).to(dt),
                      ds=(1e-2 * randn(t, d)).to(dt) if case["residual"] else None,
                      dx=torch.empty(t, d, device=DEV, dtype=dt), dweight=torch.empty(d, device=DEV, dtype=dt))
        return st

    if op == "ce":
        t, d, v = case["rows"], case["d"], case["vocab"]
        b = torch.bfloat16
        w = (randn(v, d) * (2 / math.sqrt(d))).to(b)  # logits spread by 2
        token = torch.randint(0, v, (t,), generator=gen, device=DEV)
        # states of a trained model: the next token is among the likely ones
        ahead = (math.log(v) + 5 * torch.rand(t, 1, generator=gen, device=DEV) - 1) / 4
        x = (randn(t, d) + ahead * w[token].float()).to(b)
        token[torch.randperm(t, generator=gen, device=DEV)[:_left_out(case)]] = -1
        st = dict(case=case, x=x, w=w, target=token.int(), loss=torch.empty(t, device=DEV),
                  lse=torch.empty(t, device=DEV),
                  weight=torch.full((t,), 1.0 / max(1, t - _left_out(case)), device=DEV))
        if case["grad"]:
            st.update(dx=torch.empty_like(x), dw=torch.empty_like(w))
        return st

    n, r, c = case["count"], case["rows"], case["cols"]
    # a gradient: a few strong directions over many weak ones
    low = torch.bmm(randn(n, r, 8), randn(n, 8, c))
    g = (1e-4 * (randn(n, r, c) + low)).to(DTYPES[case["dtype"]])
    return dict(case=case, g=g, out=torch.empty(n, r, c, device=DEV, dtype=torch.bfloat16))


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)(state)


def _own(st):
    import gradient_synchronisation_gb300 as zr

    op = st["case"]["op"]
    if op == "norm":
        y, s, rstd = zr.rms_norm(st["x"], st["weight"], residual=st["res"], eps=1e-6, out=st["y"], sum_out=st["s"],
                                 rstd=st["rstd"])
        return (y, s, rstd) if st["res"] is not None else (y, rstd)
    if op == "norm_backward":
        return zr.rms_norm_backward(st["s"], st["weight"], st["rstd"], st["dy"], ds=st["ds"], dx=st["dx"],
                                    dweight=st["dweight"])
    if op == "ce":
        if not st["case"]["grad"]:
            return zr.cross_entropy_loss(st["x"], st["w"], st["target"], weight=st["weight"], loss=st["loss"],
                                         lse=st["lse"], grad=False)[:2]
        return zr.cross_entropy_loss(st["x"], st["w"], st["target"], weight=st["weight"], loss=st["loss"],
                                     lse=st["lse"], dx=st["dx"], dw_vocab=st["dw"])
    return zr.orthogonalise(st["g"], steps=STEPS, coefficients=COEFFICIENTS, out=st["out"])


def _plain(st):
    op = st["case"]["op"]
    if op == "norm":
        s = st["x"]
        if st["res"] is not None:
            s = (s.float() + st["res"].float()).to(s.dtype)
        f = s.float()
        rstd = 1 / torch.sqrt((f * f).mean(1) + 1e-6)
        y = (f * rstd[:, None] * st["weight"].float()).to(s.dtype)
        return (y, s, rstd) if st["res"] is not None else (y, rstd)
    if op == "norm_backward":
        dt = st["s"].dtype
        hat = st["s"].float() * st["rstd"][:, None]
        dy = st["dy"].float()
        scaled = dy * st["weight"].float()
        dx = st["rstd"][:, None] * (scaled - hat * (scaled * hat).mean(1, keepdim=True))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        return dx.to(dt), (dy * hat).sum(0).to(dt)
    if op == "ce":
        x, w, weight = st["x"].float(), st["w"].float(), st["weight"]
        used = st["target"] >= 0
        at = st["target"].clamp(min=0).long()[:, None]
        z = x @ w.t()
        m = z.max(1, keepdim=True)[0]
        on = (z.gather(1, at) - m)[:, 0]
        e = torch.exp(z.sub_(m))
        total = e.sum(1, keepdim=True)
        log_total = torch.log(total)[:, 0]
        loss = torch.where(used, weight * (log_total - on), 0.0)
        lse = torch.where(used, m[:, 0] + log_total, 0.0)
        if not st["case"]["grad"]:
            return loss, lse
        scale = torch.where(used, weight, 0.0)[:, None]
        g = e.mul_(scale / total)
        # the target's own: p - 1 without the difference of near ones
        g.scatter_(1, at, scale * torch.expm1(on - log_total)[:, None])
        return loss, lse, (g @ w).bfloat16(), (g.t() @ x).bfloat16()
    a, b, c = COEFFICIENTS
    x = st["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + 1e-7)
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return (x.transpose(1, 2) if tall else x).bfloat16().contiguous()


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        st = prepare(case, seed)
        weight = st["weight"].double()
        if op == "norm":
            s = st["x"].double()
            if st["res"] is not None:
                # the sum is handed on as it is stored, and the norm is of that
                s = (s + st["res"].double()).to(st["x"].dtype).double()
            size = torch.linalg.vector_norm(s, dim=1) / math.sqrt(case["d"])
            rstd = torch.hypot(size, torch.full_like(size, 1e-3)).reciprocal()
            y = torch.einsum("td,t,d->td", s, rstd, weight)
            return (y, s, rstd) if st["res"] is not None else (y, rstd)
        # the norm's derivative, with the given 1 / size
        s, r, dy = st["s"].double(), st["rstd"].double(), st["dy"].double()
        inner = torch.einsum("td,td,d->t", dy, s, weight)
        dx = torch.einsum("td,d,t->td", dy, weight, r) - s * (inner * r ** 3 / case["d"])[:, None]
        if st["ds"] is not None:
            dx = dx + st["ds"].double()
        return dx, torch.einsum("td,td,t->d", dy, s, r)
    if op == "ce":
        t, d, v = case["rows"], case["d"], case["vocab"]
        if 6 * t * d * v > 6e12:
            return None
        st = prepare(case, seed)
        x, w = st["x"].double(), st["w"].double()
        loss = torch.zeros(t, dtype=torch.float64, device=DEV)
        lse, dx, dw = torch.zeros_like(loss), torch.zeros_like(x), torch.zeros_like(w)
        for lo in range(0, t, 512):
            rows = torch.nonzero(st["target"][lo:lo + 512] >= 0)[:, 0] + lo
            z = torch.einsum("td,vd->tv", x[rows], w)
            lse[rows] = torch.logsumexp(z, 1)
            at, weight = st["target"][rows].long(), st["weight"][rows].double()
            loss[rows] = -weight * torch.log_softmax(z, 1)[torch.arange(len(rows), device=DEV), at]
            if case["grad"]:
                dz = torch.softmax(z, 1) - torch.nn.functional.one_hot(at, v)
                dz *= weight[:, None]
                dx[rows] = torch.einsum("tv,vd->td", dz, w)
                dw += torch.einsum("tv,td->vd", dz, x[rows])
        return (loss, lse, dx, dw) if case["grad"] else (loss, lse)
    a, b, c = COEFFICIENTS
    st = prepare(case, seed)
    out = []
    for g in st["g"].double():
        x = g / (torch.linalg.matrix_norm(g) + 1e-7)
        one = torch.eye(min(g.shape), dtype=torch.float64, device=DEV)
        for _ in range(STEPS):  # on the shorter side: a + s (b + c s)
            if g.shape[0] <= g.shape[1]:
                s = torch.einsum("ik,jk->ij", x, x)
                x = (a * one + s @ (b * one + c * s)) @ x
            else:
                s = torch.einsum("ki,kj->ij", x, x)
                x = x @ (a * one + s @ (b * one + c * s))
        out.append(x)
    return torch.stack(out)
