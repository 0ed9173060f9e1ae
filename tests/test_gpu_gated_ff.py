"""The gated feed-forward block and its gradients through the C ABI against the
float64 oracle.

Tolerances.  u = 2^-24: an fp32 sum of n products is off by at most (n + 8) u
times the sum of their magnitudes, the activations by 2^-20 of the size of
their arguments and results; an output rounded to bf16 by 2^-8 of itself.  In
the backward pass dg and du carry one rounding to bf16 each.
"""

import numpy as np
import pytest

from oracle import step
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -24, 2.0 ** -8
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


@pytest.fixture(scope="module")
def env():
    return require_cuda()


class Case:
    def __init__(self, torch, rows, d, f, seed=0, pad=(0, 0, 0), scale=1.0):
        rng = np.random.default_rng(seed)

        def make(r, c, s, p):
            t = torch.full((r, c + p), 5.0, dtype=torch.bfloat16, device="cuda")[:, :c]
            t.copy_(torch.from_numpy((rng.normal(size=(r, c)) * s).astype(np.float32)))
            return t

        self.x, self.dh = make(rows, d, scale, pad[0]), make(rows, f, 0.3, pad[1])
        w = make(2 * f, d, 1.0 / np.sqrt(d), pad[2])
        self.wg, self.wu = w[:f], w[f:]
        self.n = [v.double().cpu().numpy() for v in (self.x, self.wg, self.wu, self.dh)]

    def projections(self):
        x, wg, wu, _ = self.n
        c = (x.shape[1] + 8) * U
        return (x @ wg.T, x @ wu.T, c * (np.abs(x) @ np.abs(wg).T), c * (np.abs(x) @ np.abs(wu).T))

    def forward(self, act):
        x, wg, wu, _ = self.n
        want = step.gated_ff(x, wg, wu, act)
        g, u, tg, tu = self.projections()
        a, da = step.activation(g, act)
        # a' is at most 1.13 in size; second order in tg is far below
        tol = 1.2 * tg * np.abs(u) + (np.abs(a) + 1.2 * tg) * tu + 2.0 ** -20 * (np.abs(g) + np.abs(a)) * np.abs(u)
        return want, tol + BF * np.abs(want) + 1e-30

    def backward(self, act):
        x, wg, wu, dh = self.n
        dx, dwg, dwu, dg, du = step.gated_ff_backward(x, wg, wu, dh, act)
        g, u, tg, tu = self.projections()
        a, da = step.activation(g, act)
        adh = np.abs(dh)
        # |a''| is at most 1.13 as well
        tdg = adh * (1.2 * tu + np.abs(u) * (1.2 * tg + 2.0 ** -20 * (1 + np.abs(g)))) + BF * np.abs(dg)
        tdu = adh * (1.2 * tg + 2.0 ** -20 * (np.abs(g) + np.abs(a))) + BF * np.abs(du)
        f, t = wg.shape[0], x.shape[0]
        ex = tdg @ np.abs(wg) + tdu @ np.abs(wu) + (2 * f + 8) * U * (np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu))
        eg = tdg.T @ np.abs(x) + (t + 8) * U * (np.abs(dg).T @ np.abs(x))
        eu = tdu.T @ np.abs(x) + (t + 8) * U * (np.abs(du).T @ np.abs(x))
        return [(w, e * 1.1 + BF * np.abs(w) + 1e-30) for w, e in ((dx, ex), (dwg, eg), (dwu, eu))]


def check(got, want, tol, norm=None):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert off.size == 0 or off.max() <= 0, "%.3g over its tolerance" % off.max()
    if norm is not None and np.linalg.norm(want) > 0:  # roundings do not line up: far under the bound
        assert np.linalg.norm(got - want) <= norm * np.linalg.norm(want)


SHAPES = [  # rows, d, f
    (1, 1, 1), (1, 8, 16), (1, 64, 64), (2, 7, 5), (3, 100, 130), (1, 4096, 1000), (5, 72, 1048), (8, 256, 640),
    (16, 512, 96), (17, 64, 2000), (31, 1001, 333), (32, 1024, 256), (33, 40, 40), (48, 768, 1001), (64, 128, 512),
    (65, 200, 264), (100, 130, 77), (127, 64, 128), (128, 128, 128), (129, 136, 392), (200, 1000, 600),
    (256, 256, 256), (300, 333, 1111), (513, 96, 520), (1000, 64, 64), (777, 1001, 300),
    # a long k in parts of a cluster, wide tiles
    (2, 3000, 72), (150, 1500, 100), (90, 64, 3000), (1024, 520, 600),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", list(ACTS))
def test_forward(env, shape, act):
    torch, zr = env
    c = Case(torch, *shape, seed=sum(shape))
    h = zr.gated_ff(c.x, c.wg, c.wu, activation=ACTS[act])
    want, tol = c.forward(act)
    check(h, want, tol, norm=3e-3 if want.size > 64 else None)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", list(ACTS))
def test_backward(env, shape, act):
    torch, zr = env
    c = Case(torch, *shape, seed=sum(shape))
    got = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, activation=ACTS[act])
    for g, (want, tol) in zip(got, c.backward(act)):
        check(g, want, tol, norm=5e-3 if want.size > 64 else None)


@pytest.mark.parametrize("shape,act", [((1300, 2100, 2500), "silu"), ((1900, 1901, 1900), "gelu"),
                                       ((1500, 1500, 3001), "gelu_tanh")], ids=str)
def test_large(env, shape, act):
    """Products for pairs of CTAs, of several widths, with ragged ends."""
    torch, zr = env
    c = Case(torch, *shape, seed=3)
    check(zr.gated_ff(c.x, c.wg, c.wu, activation=ACTS[act]), *c.forward(act), norm=3e-3)
    got = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, activation=ACTS[act])
    for g, (want, tol) in zip(got, c.backward(act)):
        check(g, want, tol, norm=5e-3)


@pytest.mark.parametrize("rows,d,f,pad", [(5, 64, 72, (8, 3, 16)), (70, 64, 72, (8, 8, 8)), (140, 100, 60, (1, 1, 3)),
                                          (9, 24, 40, (5, 0, 0)), (150, 24, 40, (0, 0, 5)), (260, 136, 264, (24, 7, 8))])
def test_strides(env, rows, d, f, pad):
    """Rows apart from one another, also at strides that are no multiple of 16 bytes."""
    torch, zr = env
    c = Case(torch, rows, d, f, pad=pad)
    out = torch.full((rows, f + pad[1]), 9.0, dtype=torch.bfloat16, device="cuda")
    zr.gated_ff(c.x, c.wg, c.wu, out=out[:, :f])
    check(out[:, :f], *c.forward("silu"))
    assert bool((out[:, f:] == 9.0).all())
    dx = torch.full((rows, d + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((2 * f, d + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, dx=dx[:, :d], dw_gate=dw[:f, :d], dw_up=dw[f:, :d])
    for g, (want, tol) in zip((dx[:, :d], dw[:f, :d], dw[f:, :d]), c.backward("silu")):
        check(g, want, tol)
    assert bool((dx[:, d:] == 9.0).all()) and bool((dw[:, d:] == 9.0).all())


@pytest.mark.parametrize("rows,d,f", [(3, 16, 24), (200, 136, 72), (130, 33, 50)])
def test_accumulate_into_a_rank_buffer(env, rows, d, f):
    """Two micro-batches added into slices of a flat buffer, at odd offsets."""
    torch, zr = env
    c = Case(torch, rows, d, f)
    flat = torch.full((2 * f * d + 11,), 0.5, dtype=torch.bfloat16, device="cuda")
    dg, du = flat[3:3 + f * d].view(f, d), flat[3 + f * d:3 + 2 * f * d].view(f, d)
    zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, dw_gate=dg, dw_up=du)
    one = dg.clone(), du.clone()
    zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, dw_gate=dg, dw_up=du, accumulate=True)
    apart = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh)
    for got, first, own, (want, tol) in zip((dg, du), one, apart[1:], c.backward("silu")[1:]):
        assert torch.equal(first, own)
        check(got, want + first.double().cpu().numpy(), tol + 2 * BF * np.abs(want))
    assert bool((flat[:3] == 0.5).all()) and bool((flat[3 + 2 * f * d:] == 0.5).all())


def test_weight_gradients_side_by_side(env):
    """Both weight gradients as halves of the same rows."""
    torch, zr = env
    c = Case(torch, 150, 64, 96)
    want = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh)
    both = torch.full((96, 130), 9.0, dtype=torch.bfloat16, device="cuda")
    zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, dw_gate=both[:, :64], dw_up=both[:, 64:128])
    assert torch.equal(both[:, :64], want[1]) and torch.equal(both[:, 64:128], want[2])
    assert bool((both[:, 128:] == 9.0).all())


def test_parts_of_the_backward_pass(env):
    torch, zr = env
    c = Case(torch, 150, 64, 96)
    dx, dg, du = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh)
    s = torch.cuda.current_stream().cuda_stream
    need = zr.zr_gated_ff_workspace_size(150, 64, 96, 64, 64, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    only = torch.empty_like(dx)
    head = (c.x.data_ptr(), 64, c.wg.data_ptr(), c.wu.data_ptr(), 64, c.dh.data_ptr(), 96, 150, 64, 96, zr.ZR_BF16, 0, 0)
    assert zr.zr_gated_ff_backward(*head, only.data_ptr(), 64, None, None, 64, ws.data_ptr(), need, s) == zr.ZR_OK
    assert torch.equal(only, dx)
    og, ou = torch.empty_like(dg), torch.empty_like(du)
    assert zr.zr_gated_ff_backward(*head, None, 64, og.data_ptr(), ou.data_ptr(), 64, ws.data_ptr(), need, s) == zr.ZR_OK
    assert torch.equal(og, dg) and torch.equal(ou, du)


def test_no_rows(env):
    torch, zr = env
    c = Case(torch, 1, 32, 40)
    x, dh = c.x[:0], c.dh[:0]
    assert zr.gated_ff(x, c.wg, c.wu).shape == (0, 40)
    _, dg, du = zr.gated_ff_backward(x, c.wg, c.wu, dh)
    assert not dg.any() and not du.any()
    dg.fill_(3), du.fill_(4)
    zr.gated_ff_backward(x, c.wg, c.wu, dh, dw_gate=dg, dw_up=du, accumulate=True)
    assert bool((dg == 3).all()) and bool((du == 4).all())


@pytest.mark.parametrize("rows", [1, 7, 130])
@pytest.mark.parametrize("act", list(ACTS))
def test_values_that_do_not_mix(env, rows, act):
    """A NaN or infinity in one row of x stays in that row of h and dx; large
    arguments saturate the activation instead of giving NaN."""
    torch, zr = env
    c = Case(torch, rows + 1, 64, 72, scale=300.0)
    clean = zr.gated_ff(c.x, c.wg, c.wu, activation=ACTS[act])
    assert bool(torch.isfinite(clean).all())
    dclean = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, activation=ACTS[act])
    assert all(bool(torch.isfinite(v).all()) for v in dclean)
    c.x[rows, 5] = float("nan")
    h = zr.gated_ff(c.x, c.wg, c.wu, activation=ACTS[act])
    assert torch.equal(h[:rows], clean[:rows]) and bool(torch.isnan(h[rows]).all())
    dx = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, activation=ACTS[act])[0]
    assert torch.equal(dx[:rows], dclean[0][:rows]) and bool(torch.isnan(dx[rows]).all())


def test_repeats_and_streams(env):
    torch, zr = env
    c = Case(torch, 300, 264, 520)
    h = zr.gated_ff(c.x, c.wg, c.wu)
    grads = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        again = zr.gated_ff(c.x, c.wg, c.wu, stream=s)
        more = zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(again, h) and all(torch.equal(a, b) for a, b in zip(more, grads))


def test_in_a_graph(env):
    """Both calls captured in a CUDA graph and replayed on new inputs."""
    torch, zr = env
    for rows in (2, 200):
        c, d = Case(torch, rows, 128, 136, seed=1), Case(torch, rows, 128, 136, seed=2)
        h, dx = torch.empty_like(c.dh), torch.empty_like(c.x)
        dg, du = torch.empty_like(c.wg), torch.empty_like(c.wu)
        need = zr.zr_gated_ff_workspace_size(rows, 128, 136, 128, 128, 1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def both():
            zr.gated_ff(c.x, c.wg, c.wu, out=h)
            zr.gated_ff_backward(c.x, c.wg, c.wu, c.dh, dx=dx, dw_gate=dg, dw_up=du, ws=ws)

        both()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both()
        c.x.copy_(d.x), c.dh.copy_(d.dh)
        g.replay()
        torch.cuda.synchronize()
        want_h = zr.gated_ff(d.x, c.wg, c.wu)
        want = zr.gated_ff_backward(d.x, c.wg, c.wu, d.dh)
        assert torch.equal(h, want_h)
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, du), want))


def test_a_long_sum(env):
    """2^25 terms in a sum, of which few are not zero: exact, and no wait gives up."""
    torch, zr = env
    d = (1 << 25) + 8
    at = torch.tensor([0, 63, 64, (1 << 24) + 5, d - 1], device="cuda")
    x = torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, d, dtype=torch.bfloat16, device="cuda")
    x[0, at] = 1.0
    w[0, at] = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0], device="cuda").bfloat16()
    w[1, at] = 1.0
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    h = zr.gated_ff(x, w[:1], w[1:], ws=ws)
    assert zr.zr_query_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == zr.ZR_OK
    assert float(h) == 31.0 * 5  # silu(31) is 31 to 2^-40, and 155 a bf16 number
    dx, dg, du = zr.gated_ff_backward(x, w[:1], w[1:], torch.ones(1, 1, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(du, 31 * x) and torch.equal(dg, 5 * x) and torch.equal(dx, 5 * w[:1] + 31 * w[1:])


def exact_activation(np, g, act):
    """a(g) and a'(g) in 64 bits with all digits of small results."""
    import math

    if act == "gelu":
        cdf = np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in g])
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    y, dy = (g, 1.0) if act == "silu" else (k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g * g))
    s = 1 / (1 + np.exp(-y))
    return g * s, s + g * dy * s / (1 + np.exp(y))


@pytest.mark.parametrize("act", list(ACTS))
def test_activations_keep_their_digits(env, act):
    """a(g) and a'(g) down to g = -9, where gelu is 1e-18 and gelu_tanh 1e-28, to
    the rounding of the output.  x = (g, 1) and unit weights make the projections g
    and 1 without a rounding, and with dh = 1 the gradient of x is (a', a).  The
    power's argument is rounded to 2^-23 of itself, up to 70, and so is the power:
    2^-15 in all, and 2^-20 of the terms that cancel at the root of a'."""
    torch, zr = env
    g = torch.linspace(-9, 9, 2003, device="cuda").bfloat16()
    x = torch.stack([g, torch.ones_like(g)], 1)
    eye = torch.eye(2, dtype=torch.bfloat16, device="cuda")
    h = zr.gated_ff(x, eye[:1], eye[1:], activation=ACTS[act])
    dx, _, _ = zr.gated_ff_backward(x, eye[:1], eye[1:], torch.ones_like(h), activation=ACTS[act])
    n = g.double().cpu().numpy()
    a, slope = exact_activation(np, n, act)
    for got, want, cancel in ((h[:, 0], a, 0), (dx[:, 1], a, 0), (dx[:, 0], slope, 2.0 ** -20 * (np.abs(n) < 3))):
        off = np.abs(got.double().cpu().numpy() - want)
        bad = off > (BF + 2.0 ** -15) * np.abs(want) + cancel + 1e-37
        assert not bad.any(), list(zip(n[bad][:4], got.double().cpu().numpy()[bad][:4], want[bad][:4]))
