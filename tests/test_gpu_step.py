"""The training step of examples/data_parallel_step.py: the averaged gradients
against automatic differentiation of the whole batch in fp64, and the replicas
staying equal."""

import math

import pytest

from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_cuda()


def reference(torch, ex, weights, batches):
    """The mean over ranks of all losses, and its gradient, in fp64."""
    flat = weights.double().requires_grad_()
    w = ex.views(flat)
    total = 0.0
    for rank in batches:
        for kind, b in rank.items():
            x = b["x"].double()
            g = x @ w["gate"].t()
            h = g * torch.sigmoid(g) * (x @ w["up"].t())
            logq = torch.log_softmax((x + h @ w["down"].t()) @ w["head"].t(), 1)
            if kind == "distill":
                p = torch.exp(b["top"].double() - b["lse"].double()[:, None])
                on = logq.gather(1, b["idx"].long())
                rest = 1 - p.sum(1)
                q_rest = 1 - torch.exp(on).sum(1)
                each = (p * (torch.log(p) - on)).sum(1) + rest * (torch.log(rest) - torch.log(q_rest))
                total = total + (each * b["weight"].double()).sum()
            elif kind == "policy":
                lp = logq.gather(1, b["action"].long()[:, None])[:, 0]
                ratio = torch.exp(lp - lp.detach())
                d = b["ref"].double() - lp
                each = 0.05 * (torch.exp(d) - d - 1) - ratio * b["advantage"].double()
                total = total + (each * b["weight"].double()).sum()
            else:
                lp = logq.gather(1, b["target"].long()[:, None])[:, 0] - b["ref"].double()
                off = b["offsets"].tolist()
                s = torch.stack([lp[i:j].sum() for i, j in zip(off, off[1:])])
                m = 0.1 * (s[0::2] - s[1::2])
                total = total - (torch.nn.functional.logsigmoid(m) * b["weight"].double()).sum()
    total = total / len(batches)
    (grad,) = torch.autograd.grad(total, flat)
    return float(total), grad


def test_averaged_gradients_match_the_whole_batch(env):
    torch, zr = env
    from examples import data_parallel_step as ex

    ranks = 3
    weights = [ex.make_weights(0) for _ in range(ranks)]
    grads = [torch.empty_like(weights[0]) for _ in range(ranks)]
    batches = [ex.make_batches(r, 1) for r in range(ranks)]
    want_loss, want = reference(torch, ex, weights[0], batches)
    losses = [ex.rank_gradients(w, g, b) for w, g, b in zip(weights, grads, batches)]
    zr.skipreduce(grads, 0)
    loss = float(torch.stack(losses).mean())
    # h, y, the logits, dlogits, dy and dh are each rounded to bf16 (2^-9), and
    # so are the gradients of each micro-batch: some ten roundings that do not
    # line up, 2^-9 sqrt(10) = 0.006 of each matrix's size; the logits' rounding
    # (2^-9 of values up to 4) moves q by 0.008.
    assert math.isfinite(loss) and abs(loss - want_loss) < 0.01 * (1 + abs(want_loss))
    for name, got in ex.views(grads[0]).items():
        ref = ex.views(want)[name]
        assert float((got.double() - ref).norm() / ref.norm()) < 0.03, name
    for g in grads[1:]:
        assert torch.equal(g, grads[0])


@pytest.mark.parametrize("skip", [0, 1])
def test_replicas_stay_equal_and_the_loss_falls(env, skip):
    torch, zr = env
    from examples import data_parallel_step as ex

    weights = [ex.make_weights(0) for _ in range(4)]
    grads = [torch.empty_like(weights[0]) for _ in range(4)]
    batches = [ex.make_batches(r, 2) for r in range(4)]
    losses = [float(ex.step(weights, grads, batches, skip, i)) for i in range(5)]
    assert all(torch.equal(weights[0], w) for w in weights[1:])
    assert losses[-1] < losses[0]


def test_refused_arguments_keep_no_memory(env):
    """A wrapper that raises gives its workspace back, whichever side refuses."""
    import ctypes

    torch, zr = env
    x, w = torch.zeros(64, 128, device="cuda").bfloat16(), torch.zeros(96, 128, device="cuda").bfloat16()
    dh, out = torch.zeros(64, 96, device="cuda").bfloat16(), torch.empty(64, 96, device="cuda").bfloat16()
    z, tok = torch.zeros(64, 50, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    off, ref = torch.tensor([0, 32, 64], device="cuda"), torch.zeros(64, device="cuda")
    odd = torch.zeros(64, 127, device="cuda").bfloat16(), torch.zeros(96, 127, device="cuda").bfloat16()
    grads = [torch.empty_like(t) for t in (x, w, w)]
    loss = [torch.empty(1, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(z)]
    calls = [
        lambda a: zr.gated_ff(odd[0], odd[1], odd[1], activation=a, out=out),
        lambda a: zr.gated_ff_backward(x, w, w, dh, activation=a, dx=grads[0], dw_gate=grads[1], dw_up=grads[2]),
        lambda a: zr.preference_loss(z, tok, off, ref, beta=a, loss=loss[0], reward=loss[1], dlogits=loss[2]),
    ]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for call in calls:
        for bad, error in (("silu", ctypes.ArgumentError), (-7, zr.ZrError)):
            with pytest.raises(error):
                call(bad)
            assert torch.cuda.memory_allocated() == before


def test_a_workspace_is_device_memory(env):
    """A workspace in host memory, or one with gaps, is refused, not written to."""
    torch, zr = env
    x, w = torch.zeros(64, 128, device="cuda").bfloat16(), torch.zeros(96, 128, device="cuda").bfloat16()
    dh = torch.zeros(64, 96, device="cuda").bfloat16()
    z, tok = torch.zeros(64, 50, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    off, ref = torch.tensor([0, 32, 64], device="cuda"), torch.zeros(64, device="cuda")
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        for call in (lambda: zr.gated_ff(x, w, w, ws=ws), lambda: zr.gated_ff_backward(x, w, w, dh, ws=ws),
                     lambda: zr.preference_loss(z, tok, off, ref, ws=ws)):
            with pytest.raises(ValueError):
                call()
