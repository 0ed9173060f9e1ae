"""One data-parallel pre-training step with the library's operators, from the states to
the update.

N ranks, simulated as N rank buffers on one GPU, hold the same small model: a norm, a
gated feed-forward block with its down projection and a residual, a second norm (which
adds the residual), and a head over a vocabulary whose logits are never whole in fp32.  Each rank
takes its own micro-batches; the gradients are written and added straight into its flat
buffer, the buffers are averaged by SkipReduce, and every rank applies the same update:
the matrices' momentum, orthogonalised, and the plain gradient for the norms and the
head.

    python examples/pretrain_step.py [--ranks 4] [--skip 0] [--steps 3]
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gradient_synchronisation_gb300 as zr  # noqa: E402

D, F, VOCAB = 256, 704, 4000
# gate and up lie one behind the other: one batch of two for the update
SHAPES = {"gate": (F, D), "up": (F, D), "down": (D, F), "head": (VOCAB, D), "norm_in": (1, D), "norm_out": (1, D)}
BF = torch.bfloat16


def views(flat):
    """The weights' (or gradients') matrices as views of one flat buffer."""
    out, at = {}, 0
    for name, (r, c) in SHAPES.items():
        out[name] = flat[at:at + r * c].view(r, c)
        at += r * c
    out["gate_up"] = flat[:2 * F * D].view(2, F, D)
    return out


def size():
    return sum(r * c for r, c in SHAPES.values())


def make_weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.empty(size(), device="cuda", dtype=BF)
    for name, w in views(flat).items():
        if name.startswith("norm"):
            w.copy_(1 + 0.1 * torch.randn(w.shape, generator=g, device="cuda"))
        elif name != "gate_up":
            w.copy_(torch.randn(w.shape, generator=g, device="cuda") / w.shape[1] ** 0.5)
    return flat


def make_batches(rank, seed, rows=96, micro=2):
    """A rank's micro-batches: states, next tokens (-1: none, a prompt or padding) and
    the tokens' weights, one over those that count."""
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + rank)
    out = []
    for _ in range(micro):
        x = torch.randn(rows, D, generator=g, device="cuda").to(BF)
        target = torch.randint(0, VOCAB, (rows,), generator=g, device="cuda").int()
        target[torch.rand(rows, generator=g, device="cuda") < 0.2] = -1
        out.append(dict(x=x, target=target, weight=torch.full((rows,), 1.0 / (rows * micro), device="cuda")))
    return out


def rank_gradients(weights, grads, batches):
    """Gradients of the sum of all losses into the rank's flat buffer ``grads``; returns
    the losses' sum and the gradients of the states."""
    w, g = views(weights), views(grads)
    norm_in, norm_out = w["norm_in"][0], w["norm_out"][0]
    total, dxs = torch.zeros((), device="cuda"), []
    for n, b in enumerate(batches):
        more = dict(accumulate=n > 0)
        x = b["x"]
        y, _, r_in = zr.rms_norm(x, norm_in)
        h = zr.gated_ff(y, w["gate"], w["up"])
        z, s, r_out = zr.rms_norm(h @ w["down"].t(), norm_out, residual=x)
        loss, _, dz, _ = zr.cross_entropy_loss(z, w["head"], b["target"], weight=b["weight"], dw_vocab=g["head"], **more)
        total += loss.sum()
        ds, _ = zr.rms_norm_backward(s, norm_out, r_out, dz, dx=dz, dweight=g["norm_out"][0], **more)
        if n == 0:
            torch.mm(ds.t(), h, out=g["down"])
        else:
            g["down"].addmm_(ds.t(), h)
        dy, _, _ = zr.gated_ff_backward(y, w["gate"], w["up"], ds @ w["down"], dw_gate=g["gate"], dw_up=g["up"], **more)
        dx, _ = zr.rms_norm_backward(x, norm_in, r_in, dy, ds=ds, dx=dy, dweight=g["norm_in"][0], **more)
        dxs.append(dx)
    return total, dxs


def update(weights, grads, momentum, rate=0.02, keep=0.95):
    """Muon's update of the block's matrices, the plain gradient for the rest."""
    w, g, m = views(weights), views(grads), views(momentum)
    momentum.mul_(keep).add_(grads)
    for name in ("gate_up", "down"):
        rows, cols = w[name].shape[-2:]
        w[name].sub_(zr.orthogonalise(m[name], scale=max(1, rows / cols) ** 0.5), alpha=rate)
    for name in ("head", "norm_in", "norm_out"):
        w[name].sub_(g[name], alpha=rate)


def step(weights, grads, momenta, batches, skip=0, index=0):
    """One step of all ranks: gradients, their average, the update."""
    losses = [rank_gradients(w, g, b)[0] for w, g, b in zip(weights, grads, batches)]
    zr.skipreduce(grads, skip, mode=zr.ZR_SKIP_RANDOM, seed=1, step=index)
    for w, g, m in zip(weights, grads, momenta):
        update(w, g, m)
    return torch.stack(losses).mean()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--skip", type=int, default=0, help="Reduce-Scatter steps to skip")
    p.add_argument("--steps", type=int, default=3)
    a = p.parse_args()
    weights = [make_weights(0) for _ in range(a.ranks)]
    grads = [torch.empty_like(weights[0]) for _ in range(a.ranks)]
    momenta = [torch.zeros_like(weights[0]) for _ in range(a.ranks)]
    batches = [make_batches(r, 0) for r in range(a.ranks)]
    for i in range(a.steps):
        loss = step(weights, grads, momenta, batches, a.skip, i)
        same = all(torch.equal(weights[0], w) for w in weights[1:])
        print("step %d: loss %.4f, replicas %s" % (i, loss.item(), "equal" if same else "DIFFER"))


if __name__ == "__main__":
    main()
