"""One data-parallel training step with the library's operators.

N ranks, simulated as N rank buffers on one GPU, hold the same small model: a
gated feed-forward block, its down projection with a residual, and a head over
a vocabulary.  Each rank takes three micro-batches of its own, one for each
loss (distillation from a teacher's top logits, clipped policy loss, preference
pairs).  The block's weight gradients are written and added straight into the
rank's flat gradient buffer; the buffers are then averaged by SkipReduce, and
every rank applies the same update.

    python examples/data_parallel_step.py [--ranks 4] [--skip 0] [--steps 3]
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
SHAPES = {"gate": (F, D), "up": (F, D), "down": (D, F), "head": (VOCAB, D)}
BF = torch.bfloat16


def views(flat):
    """The weights' (or gradients') matrices as views of one flat buffer."""
    out, at = {}, 0
    for name, (r, c) in SHAPES.items():
        out[name] = flat[at:at + r * c].view(r, c)
        at += r * c
    return out


def size():
    return sum(r * c for r, c in SHAPES.values())


def make_weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.empty(size(), device="cuda", dtype=BF)
    for w in views(flat).values():
        w.copy_(torch.randn(w.shape, generator=g, device="cuda") / w.shape[1] ** 0.5)
    return flat


def make_batches(rank, seed, rows=96, k=16, pairs=4):
    """What one rank trains on: three micro-batches of token states with what
    their losses need.  Weights are one over the tokens (or pairs)."""
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + rank)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    def token(n):
        return torch.randint(0, VOCAB, (n,), generator=g, device="cuda").int()

    teacher = randn(rows, VOCAB) * 2
    top, idx = torch.topk(teacher, k)
    off = torch.arange(2 * pairs + 1, device="cuda") * (rows // (2 * pairs))
    each = torch.full((rows,), 1.0 / rows, device="cuda")
    return {
        "distill": dict(x=randn(rows, D).to(BF), idx=idx.int(), top=top,
                        lse=torch.logsumexp(teacher, 1), weight=each),
        "policy": dict(x=randn(rows, D).to(BF), action=token(rows), advantage=randn(rows),
                       ref=-8 + 0.3 * randn(rows), weight=each),
        "preference": dict(x=randn(rows, D).to(BF), target=token(rows), offsets=off,
                           ref=-8 + 0.3 * randn(rows),
                           weight=torch.full((pairs,), 1.0 / pairs, device="cuda")),
    }


def loss_and_gradient(kind, b, logits):
    """The micro-batch's loss; its gradient replaces the logits."""
    if kind == "distill":
        return zr.distill_loss(logits, b["idx"], b["top"], teacher_lse=b["lse"], weight=b["weight"],
                               dlogits=logits)[0]
    if kind == "policy":
        return zr.policy_loss(logits, b["action"], b["advantage"], ref_logp=b["ref"], kl_coef=0.05,
                              weight=b["weight"], dlogits=logits)[0]
    return zr.preference_loss(logits, b["target"], b["offsets"], b["ref"], beta=0.1,
                              weight=b["weight"], dlogits=logits)[0]


def rank_gradients(weights, grads, batches):
    """Gradients of the sum of all losses into the rank's flat buffer ``grads``;
    returns the losses' sum."""
    w, g = views(weights), views(grads)
    total = torch.zeros((), device="cuda")
    for n, (kind, b) in enumerate(batches.items()):
        x = b["x"]
        h = zr.gated_ff(x, w["gate"], w["up"], activation=zr.ZR_ACT_SILU)
        y = x + h @ w["down"].t()
        logits = y @ w["head"].t()
        total += loss_and_gradient(kind, b, logits).sum()
        dy = logits @ w["head"]
        if n == 0:
            torch.mm(logits.t(), y, out=g["head"])
            torch.mm(dy.t(), h, out=g["down"])
        else:
            g["head"].addmm_(logits.t(), y)
            g["down"].addmm_(dy.t(), h)
        zr.gated_ff_backward(x, w["gate"], w["up"], dy @ w["down"], activation=zr.ZR_ACT_SILU,
                             dw_gate=g["gate"], dw_up=g["up"], accumulate=n > 0)
    return total


def step(weights, grads, batches, skip=0, index=0, rate=0.05):
    """One step of all ranks: gradients, their average, the update."""
    losses = [rank_gradients(w, g, b) for w, g, b in zip(weights, grads, batches)]
    zr.skipreduce(grads, skip, mode=zr.ZR_SKIP_RANDOM, seed=1, step=index)
    for w, g in zip(weights, grads):
        w.sub_(g, alpha=rate)
    return torch.stack(losses).mean()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--skip", type=int, default=0, help="Reduce-Scatter steps to skip")
    p.add_argument("--steps", type=int, default=3)
    a = p.parse_args()
    weights = [make_weights(0) for _ in range(a.ranks)]
    grads = [torch.empty_like(weights[0]) for _ in range(a.ranks)]
    batches = [make_batches(r, 0) for r in range(a.ranks)]
    for i in range(a.steps):
        loss = step(weights, grads, batches, a.skip, i)
        same = all(torch.equal(weights[0], w) for w in weights[1:])
        print("step %d: loss %.4f, replicas %s" % (i, loss.item(), "equal" if same else "DIFFER"))


if __name__ == "__main__":
    main()
