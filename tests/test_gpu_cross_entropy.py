"""Cross entropy of states over a vocabulary, and its gradients, through the C ABI
against the float64 oracle.

Tolerances.  u = 2^-24.  A logit is an fp32 sum of d products: (d + 8) u of the sum of
their magnitudes (tz).  Each power of the softmax carries its logit's error, the
rounding of its argument (3 u of up to 30) and the power's own (2^-22); a sum of them
at most 128 roundings of a half tile and one for each 32 half tiles and 8 joins.  The
gradients' powers are of distances in steps of 2^-10: off by half a step, 2^-11 ln 2 of
themselves, and 0 where they are under 2^-64.  dz is rounded to bf16 (2^-8) before the
products, which are fp32 sums again, and so are the outputs.
"""

import math

import numpy as np
import pytest

from oracle import step
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def env():
    return require_cuda()


class Case:
    def __init__(self, torch, rows, d, vocab, seed=0, pad=(0, 0), shift=0, masked=0.2, scale=1.0, weights=True):
        rng = np.random.default_rng(seed)

        def make(r, c, s, p):
            flat = torch.full((shift + r * (c + p) + 8,), 5.0, dtype=torch.bfloat16, device="cuda")
            t = flat[shift:shift + r * (c + p)].view(r, c + p)[:, :c]
            t.copy_(torch.from_numpy((rng.normal(size=(r, c)) * s).astype(np.float32)))
            return t

        self.x = make(rows, d, scale, pad[0])
        self.w = make(vocab, d, 2.0 / np.sqrt(d), pad[1])
        self.target = rng.integers(0, vocab, rows).astype(np.int32)
        self.target[rng.random(rows) < masked] = -1
        self.weight = None
        if weights:
            self.weight = rng.uniform(-0.2, 1.0, rows).astype(np.float32)
            self.weight[rng.random(rows) < masked / 2] = 0
        self.nx, self.nw = (v.double().cpu().numpy() for v in (self.x, self.w))
        self.dev = (torch.from_numpy(self.target).cuda(),
                    None if self.weight is None else torch.from_numpy(self.weight).cuda())

    def run(self, zr, **kw):
        return zr.cross_entropy_loss(self.x, self.w, self.dev[0], weight=self.dev[1], **kw)

    def want(self):
        rows, (vocab, d) = len(self.target), self.nw.shape
        loss, lse, dx, dw, dz = step.cross_entropy(self.nx, self.nw, self.target, self.weight)
        used = (self.target >= 0) & (self.target < vocab)
        k = np.where(used, 1.0 if self.weight is None else np.abs(self.weight), 0.0)
        nx = np.where(used[:, None], self.nx, 0.0)
        z = nx @ self.nw.T
        tz = (d + 8) * U * (np.abs(nx) @ np.abs(self.nw).T)
        most = tz.max(1)
        # half tiles are at least 32 wide
        rel = most + 90 * U + 2.0 ** -22 + (128 + vocab / 1024 + 16) * U
        size = np.abs(z).max(1)
        tol_lse = rel + 4 * U * (size + np.log(vocab) + 1)
        tol_loss = k * (tol_lse + most + 4 * U * (size + np.log(vocab) + 1)) + 4 * U * np.abs(loss)
        each = 2.0 ** -11 * np.log(2) + tz + most[:, None] + rel[:, None] + 2 * BF
        tdz = np.abs(dz) * each * 1.01 + k[:, None] * 2.0 ** -64
        on = np.arange(rows)[used], self.target[used]
        tdz[on] = (k * 1.01 * (tz.max(1) + most + rel))[used] + 1.01 * BF * np.abs(dz[on])
        adz = np.abs(dz)
        tol_dx = tdz @ np.abs(self.nw) + (vocab + 80) * U * (adz @ np.abs(self.nw)) + BF * 1.01 * np.abs(dx)
        tol_dw = tdz.T @ np.abs(nx) + (rows + 80) * U * (adz.T @ np.abs(nx)) + BF * 1.01 * np.abs(dw)
        return [(loss, tol_loss), (lse, np.where(k > 0, tol_lse, 0)), (dx, tol_dx + 1e-38), (dw, tol_dw + 1e-38)]


def check(got, want, tol, norm=None):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert off.size == 0 or off.max() <= 0, "%.3g over its tolerance" % off.max()
    if norm is not None and np.linalg.norm(want) > 0:  # roundings do not line up: far under the bound
        assert np.linalg.norm(got - want) <= norm * np.linalg.norm(want)


def check_all(got, case):
    for n, (g, (want, tol)) in enumerate(zip(got, case.want())):
        check(g, want, tol, norm=4e-3 if n > 1 and want.size > 500 else None)


SHAPES = [  # rows, d, vocab
    (1, 1, 1), (1, 1, 2), (2, 3, 5), (1, 8, 64), (3, 64, 65), (5, 100, 130), (16, 64, 1000), (7, 33, 1003), (1, 512, 4000),
    (64, 72, 257), (65, 256, 700), (127, 40, 128), (128, 128, 128), (130, 136, 520), (200, 1000, 333), (256, 64, 2000),
    (300, 65, 1111), (700, 24, 4097), (1000, 264, 77), (17, 2000, 90), (40, 8, 20001), (600, 512, 1500),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_loss_and_gradients(env, shape):
    torch, zr = env
    c = Case(torch, *shape, seed=sum(shape), masked=0.0 if shape[0] < 3 else 0.2)
    got = c.run(zr)
    check_all(got, c)
    loss, lse, dx, dw = c.run(zr, grad=False)
    assert dx is None and dw is None
    assert torch.equal(loss, got[0]) and torch.equal(lse, got[1])


@pytest.mark.parametrize("shape", [(1500, 520, 3000), (2100, 136, 5001)], ids=str)
def test_large(env, shape):
    torch, zr = env
    c = Case(torch, *shape, seed=5)
    check_all(c.run(zr), c)


@pytest.mark.parametrize("rows, d, vocab", [(4600, 16, 300), (9000, 24, 264)])
def test_pieces(env, rows, d, vocab):
    """More rows than a piece: dw's sums go on from one piece to the next; the last
    piece may have no rows at all once those without a target are left out."""
    torch, zr = env
    for masked in (0.05, 0.6):
        c = Case(torch, rows, d, vocab, seed=6, masked=masked)
        got = c.run(zr)
        check_all(got, c)
        dw = torch.full((vocab, d), 0.25, dtype=torch.bfloat16, device="cuda")
        c.run(zr, dw_vocab=dw, accumulate=True)
        want, tol = c.want()[3]
        check(dw, want + 0.25, tol + 2 * BF * (np.abs(want) + 0.25))


@pytest.mark.parametrize("rows, d, vocab, pad, shift", [
    (5, 64, 72, (8, 16), 0), (70, 64, 200, (3, 8), 0), (140, 100, 260, (1, 1), 1), (9, 24, 40, (5, 0), 0),
    (150, 24, 40, (0, 5), 3), (33, 7, 90, (0, 0), 5), (260, 136, 264, (24, 7), 1)])
def test_strides(env, rows, d, vocab, pad, shift):
    torch, zr = env
    c = Case(torch, rows, d, vocab, pad=pad, shift=shift)
    wide_x = torch.full((rows, d + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    flat = torch.full((vocab * (d + 5) + 3,), 9.0, dtype=torch.bfloat16, device="cuda")
    wide_w = flat[3:].view(vocab, d + 5)
    got = c.run(zr, dx=wide_x[:, :d], dw_vocab=wide_w[:, :d])
    check_all(got, c)
    assert bool((wide_x[:, d:] == 9.0).all()) and bool((wide_w[:, d:] == 9.0).all()) and bool((flat[:3] == 9.0).all())


@pytest.mark.parametrize("rows, d, vocab", [(3, 16, 24), (200, 136, 72), (130, 33, 50)])
def test_accumulate_into_a_rank_buffer(env, rows, d, vocab):
    torch, zr = env
    c = Case(torch, rows, d, vocab, masked=0.1)
    flat = torch.full((vocab * d + 11,), 0.5, dtype=torch.bfloat16, device="cuda")
    dw = flat[3:3 + vocab * d].view(vocab, d)
    c.run(zr, dw_vocab=dw)
    one = dw.clone()
    assert torch.equal(one, c.run(zr)[3])
    c.run(zr, dw_vocab=dw, accumulate=True)
    want, tol = c.want()[3]
    check(dw, want + one.double().cpu().numpy(), tol + 2 * BF * np.abs(want))
    assert bool((flat[:3] == 0.5).all()) and bool((flat[3 + vocab * d:] == 0.5).all())


def test_states_replaced_by_their_gradient(env):
    torch, zr = env
    c = Case(torch, 90, 72, 500)
    want = c.run(zr)
    x = c.x.clone()
    got = zr.cross_entropy_loss(x, c.w, c.dev[0], weight=c.dev[1], dx=x)
    assert got[2] is x and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [1, 50, 300])
def test_nothing_left(env, rows):
    """No row has a target; or there are no rows."""
    torch, zr = env
    c = Case(torch, rows, 40, 100, masked=1.1)
    c.x.fill_(float("nan"))
    for target in (c.dev[0], torch.full_like(c.dev[0], -(1 << 31))):
        loss, lse, dx, dw = zr.cross_entropy_loss(c.x, c.w, target)
        assert not loss.any() and not lse.any() and not dx.any() and not dw.any()
    dw.fill_(3)
    zr.cross_entropy_loss(c.x, c.w, c.dev[0], dw_vocab=dw, accumulate=True)
    assert bool((dw == 3).all())
    loss, lse, dx, dw = zr.cross_entropy_loss(c.x[:0], c.w, c.dev[0][:0])
    assert loss.shape == (0,) and dx.shape == (0, 40) and not dw.any()
    dw.fill_(3)
    zr.cross_entropy_loss(c.x[:0], c.w, c.dev[0][:0], dw_vocab=dw, accumulate=True)
    assert bool((dw == 3).all())


@pytest.mark.parametrize("rows, vocab", [(7, 300), (400, 1000)])
def test_rows_left_out_may_hold_anything(env, rows, vocab):
    torch, zr = env
    c = Case(torch, rows, 72, vocab, masked=0.4)
    want = [t.clone() for t in c.run(zr)]
    check_all(want, c)
    out = (c.target < 0) | (c.weight == 0)
    c.x[torch.from_numpy(out).cuda()] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(c.run(zr), want))


def test_targets_past_the_vocabulary(env):
    torch, zr = env
    c = Case(torch, 60, 64, 500, masked=0.1)
    need = zr.zr_cross_entropy_workspace_size(60, 64, 500, 64, 1, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    c.run(zr, ws=ws)
    assert zr.zr_query_status(ws.data_ptr(), s) == zr.ZR_OK
    for n, bad in ((3, 500), (41, 2 ** 31 - 1)):
        c.target[n] = bad
        c.dev[0][n] = bad
    got = c.run(zr, ws=ws)
    assert zr.zr_query_status(ws.data_ptr(), s) == zr.ZR_ERR_INVALID_ARG
    check_all(got, c)
    assert float(got[0][3]) == 0 and not got[2][41].any()


@pytest.mark.parametrize("rows", [5, 300])
def test_values_that_are_not_numbers(env, rows):
    """A NaN in a row's states is that row's loss and dx, and dw's; so is a +inf logit.
    Logits of -inf have no probability; a row of nothing else is left out."""
    torch, zr = env
    c = Case(torch, rows, 16, 600, masked=0, weights=False)
    clean = [t.clone() for t in c.run(zr)]
    c.x[1, 3] = float("nan")
    loss, lse, dx, dw = c.run(zr)
    keep = torch.arange(rows, device="cuda") != 1
    assert bool(torch.isnan(loss[1])) and bool(torch.isnan(dx[1]).all()) and bool(torch.isnan(dw).all())
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dx[keep], clean[2][keep])
    # an infinite state: logits of both signs, or one sign where the weights' column has one
    c.x[1] = 0
    c.w[:, 3] = c.w[:, 3].abs() + 0.01
    c.w[7, 3] = 0.5
    for value in (float("inf"), float("-inf")):
        c.x[:, 3] = 0
        base = [t.clone() for t in c.run(zr)]
        c.x[1, 3] = value
        loss, lse, dx, dw = c.run(zr)
        if value > 0:
            assert bool(torch.isnan(loss[1])) and bool(torch.isnan(dx[1]).all())
        else:  # every logit is -inf
            assert float(loss[1]) == 0 and not dx[1].any() and bool(torch.isfinite(dx).all())
        assert torch.equal(loss[keep], base[0][keep]) and torch.equal(dx[keep], base[2][keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_weight_that_is_not_a_number_stays_in_its_row(env, bad):
    torch, zr = env
    c = Case(torch, 40, 64, 300, masked=0)
    want = c.run(zr)
    c.dev[1][5] = bad
    loss, lse, dx, dw = c.run(zr)
    keep = torch.arange(40, device="cuda") != 5
    assert not bool(torch.isfinite(loss[5])) and not bool(torch.isfinite(dx[5]).any())
    # (the unit of dz is the largest finite weight: another one if that was row 5's)
    if float(c.dev[1][keep].abs().max()) == float(np.abs(c.weight).max()):
        assert torch.equal(loss[keep], want[0][keep]) and torch.equal(dx[keep], want[2][keep])


def test_logits_far_apart(env):
    """Logits of hundreds to the lowest that bf16 products reach: the loss is exact in
    fp32, probabilities are 0 or 1."""
    torch, zr = env
    for scale in (30.0, 3e3, 1e18):
        c = Case(torch, 40, 64, 300, scale=scale, masked=0, weights=False)
        loss, lse, dx, dw = c.run(zr)
        for g, (want, tol) in zip((loss, lse), c.want()):
            check(g, want, tol)
        assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_one_gradient_alone(env):
    torch, zr = env
    c = Case(torch, 150, 64, 700)
    _, _, dx, dw = c.run(zr)
    st = torch.cuda.current_stream().cuda_stream
    head = (c.x.data_ptr(), 64, c.w.data_ptr(), 64, 150, 64, 700, zr.ZR_BF16, c.dev[0].data_ptr(), c.dev[1].data_ptr(),
            None, None, 0)
    for want_x, want_w in ((1, 0), (0, 1)):
        need = zr.zr_cross_entropy_workspace_size(150, 64, 700, 64, want_x, want_w)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        gx, gw = torch.empty_like(dx), torch.empty_like(dw)
        assert zr.zr_cross_entropy_loss(*head, gx.data_ptr() if want_x else None, 64, gw.data_ptr() if want_w else None, 64,
                                        ws.data_ptr(), need, st) == zr.ZR_OK
        assert torch.equal(gx, dx) if want_x else torch.equal(gw, dw)


def test_gradients_against_differences(env):
    """The loss along a direction of the states and of the weights, from both sides."""
    torch, zr = env
    c = Case(torch, 64, 128, 900, masked=0.2)
    _, _, dx, dw = c.run(zr)
    x, w, dx, dw, k = (t.double().cpu() for t in (c.x, c.w, dx, dw, c.dev[1]))
    target = c.dev[0].cpu()

    def loss(x, w):
        p = torch.log_softmax(x @ w.t(), 1).gather(1, target.clamp(min=0).long()[:, None])[:, 0]
        return -(p * k)[target >= 0].sum()

    for which, g in enumerate((dx, dw)):
        along = g / g.norm()
        h = 1e-4
        d = [0, 0]
        d[which] = along * h
        slope = (loss(x + d[0], w + d[1]) - loss(x - d[0], w - d[1])) / (2 * h)
        # dz and the output are rounded to bf16: 2 x 2^-8 of the size at most
        assert abs(float(slope - g.norm())) <= 2 * BF * float(g.norm())


def test_weights_past_32_bits(env):
    """2.3e9 weights: one row that is not 0, the last; logits and gradients in closed form."""
    torch, zr = env
    rows, d, vocab = 40, 32768, 70000
    w = torch.zeros(vocab, d, dtype=torch.bfloat16, device="cuda")
    w[-1, :4] = 0.5
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:, :4] = torch.arange(rows, device="cuda")[:, None] / 4
    x[:, -1] = 1
    target = torch.full((rows,), vocab - 1, dtype=torch.int32, device="cuda")
    target[::2] = 5
    loss, lse, dx, dw = zr.cross_entropy_loss(x, w, target)
    z = torch.arange(rows, device="cuda").double() / 2
    want = torch.log(vocab - 1 + torch.exp(z))
    # half a step of log sum exp (16 at most), the power's, the sum's: 1e-5 in all
    assert float((lse - want).abs().max()) < 1e-5
    assert float((loss - (want - torch.where(target == 5, 0.0, z))).abs().max()) < 1e-5
    p = torch.exp(z - want)
    last = p - (target != 5).double()
    first = (1 - p) / (vocab - 1) - (target == 5).double()
    rest = (1 - p) / (vocab - 1)
    for got, terms in ((dx[:, 0:1], 0.5 * last[:, None]), (dw[-1, 0], last * x[:, 0].double()), (dw[-1, -1], last),
                       (dw[5, -1], first), (dw[69998, -1], rest)):
        ref, size = (terms, terms.abs()) if got.dim() else (terms.sum(), terms.abs().sum())
        # dz, the distance of a power, and the output: 2 x 2^-8 and 4e-4 of the terms' sizes
        assert bool(((got.double() - ref).abs() <= 8.3e-3 * size).all())
    assert not dx[:, 4:].any() and not dw[:, 4:-1].any()


def test_logits_past_32_bits(env):
    """A piece of 6000 x 400000 logits, all 0: dx is the mean of the weights less the
    target's, dw the difference of counts."""
    torch, zr = env
    rows, d, vocab = 6000, 1024, 400000
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(vocab, d, generator=g, device="cuda").bfloat16()
    w[:, 0] = 0
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
    target[-1] = vocab - 1
    loss, lse, dx, dw = zr.cross_entropy_loss(x, w, target)
    assert float((loss - math.log(vocab)).abs().max()) < 4e-6 and torch.equal(loss, lse)
    want = w.double().mean(0) - w[target.long()].double()
    # 1 / vocab is rounded by up to 2^-8, and so are the outputs
    tol = 2 * BF * (want.abs() + w.double().abs().mean(0)) + 1e-6
    assert bool(((dx.double() - want).abs() <= tol).all())
    count = torch.bincount(target.long(), minlength=vocab).double()
    want = rows / vocab - count
    assert bool(((dw[:, 0].double() - want).abs() <= 2 * BF * (want.abs() + rows / vocab)).all())
    assert not dw[:, 1:].any()


@pytest.mark.parametrize("rows, d, vocab", [(60, 40, 300), (300, 136, 520)])
def test_weights_of_many_sizes(env, rows, d, vocab):
    """25 decades of weights: each row's loss and dx to its own size."""
    torch, zr = env
    c = Case(torch, rows, d, vocab, seed=12)
    c.weight = (10.0 ** np.linspace(-25, 0, rows) * np.where(np.arange(rows) % 3, 1, -1)).astype(np.float32)
    c.dev = (c.dev[0], torch.from_numpy(c.weight).cuda())
    got = c.run(zr)
    for g, (want, tol) in zip(got, c.want()):
        check(g, want, tol)


@pytest.mark.parametrize("rows", [5, 300, 4600])
def test_rows_of_nothing_but_minus_infinity_leave_dw_alone(env, rows):
    """Infinite states whose every logit is -inf: the row is left out of all results, dw's
    among them."""
    torch, zr = env
    c = Case(torch, rows, 16, 600 if rows < 1000 else 130, masked=0, weights=False)
    c.w[:, 3] = c.w[:, 3].abs() + 0.01
    gone = [0, rows // 2, rows - 1]
    target = c.dev[0].clone()
    target[gone] = -1
    want = zr.cross_entropy_loss(c.x, c.w, target)
    want = [t.clone() for t in want]
    c.x[gone, 3] = float("-inf")
    got = c.run(zr)
    assert all(bool(torch.isfinite(t).all()) for t in got)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[gone] = False
    for a, b in zip(got[:3], want):
        assert torch.equal(a[keep], b[keep]) and not a[gone].any()
    # dw's terms in another order: each fp32 sum and its rounding to bf16
    c.target, c.nw = target.cpu().numpy(), c.w.double().cpu().numpy()
    c.nx[gone] = 0
    check(got[3], *c.want()[3])
    dw = torch.full_like(got[3], 0.25)
    c.run(zr, dw_vocab=dw, accumulate=True)
    assert bool(torch.isfinite(dw).all())


def test_weights_that_are_infinite(env):
    """A column of W that is -inf: a row whose state there is positive has no logit but
    -inf, and a zero dx; one whose state is 0 there is not a number."""
    torch, zr = env
    c = Case(torch, 40, 16, 300, masked=0, weights=False)
    c.w[:, 3] = float("-inf")
    c.x[:, 3] = 1
    c.x[7, 3] = 0
    loss, lse, dx, dw = c.run(zr)
    keep = torch.arange(40, device="cuda") != 7
    assert not loss[keep].any() and not dx[keep].any()
    assert bool(torch.isnan(loss[7])) and bool(torch.isnan(dx[7]).all())


def test_a_long_vocabulary(env):
    """Equal logits over 2^21 tokens, so that dx is the mean of the weights where the
    target's are 0: p = 2^-21 exactly, and what is off before the rounding to bf16 is the
    sum.  One of the tensor cores over all tokens is low by up to 1 %, a part of 2^18 terms
    by 2^-12 (cut sums have one sign; 2^-11 is allowed); the rounding keeps the order."""
    torch, zr = env
    rows, d, vocab = 4864, 1024, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    w = torch.empty(vocab, d, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.5, generator=g)
    w *= (0.5 + 1.5 * torch.rand(d, generator=g, device="cuda")).bfloat16()
    w[:, 0] = 0
    w[:512] = 0
    target = torch.randint(0, 512, (rows,), generator=g, device="cuda").int()
    loss, _, dx, dw = zr.cross_entropy_loss(x, w, target)
    assert bool((loss == math.log(2) * 21).all()) or float((loss - math.log(2) * 21).abs().max()) < 2e-6
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for lo in range(0, vocab, 1 << 18):
        want += w[lo:lo + (1 << 18)].double().sum(0)
    want /= vocab
    least, most = ((want * f).bfloat16() for f in (1 - 2.0 ** -11, 1 + 2.0 ** -14))
    assert bool((dx >= least).all()) and bool((dx <= most).all())
    count = torch.bincount(target.long(), minlength=vocab).double()
    assert bool(((dw[:, 0].double() - (rows / vocab - count)).abs() <= 2 * BF * (count + rows / vocab)).all())


@pytest.mark.parametrize("rows, masked", [(16500, 0.0), (33000, 0.1), (40000, 0.7)])
def test_pieces_without_gradients(env, rows, masked):
    """More rows than the 16384 of a piece of a loss alone, and one that the rows left out
    make empty."""
    torch, zr = env
    c = Case(torch, rows, 40, 130, seed=14, masked=masked)
    got = c.run(zr, grad=False)
    assert got[2] is None and got[3] is None
    for g, (want, tol) in zip(got[:2], c.want()):
        check(g, want, tol)


@pytest.mark.parametrize("rows, d, vocab, masked", [(4100, 24, 264, 0.0), (9000, 33, 130, 0.1), (13000, 64, 65, 0.8)])
def test_pieces_of_one_gradient(env, rows, d, vocab, masked):
    """dx alone goes in pieces of 4096 rows, dw alone in the pieces of both; each as in
    one call for all, to its bound."""
    torch, zr = env
    c = Case(torch, rows, d, vocab, seed=15, masked=masked)
    want = c.want()
    st = torch.cuda.current_stream().cuda_stream
    for dx, dw in ((1, 0), (0, 1)):
        need = zr.zr_cross_entropy_workspace_size(rows, d, vocab, d, dx, dw)
        ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")
        out = torch.full((rows if dx else vocab, d), 7.0, dtype=torch.bfloat16, device="cuda")
        loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
        assert zr.zr_cross_entropy_loss(c.x.data_ptr(), d, c.w.data_ptr(), d, rows, d, vocab, zr.ZR_BF16, c.dev[0].data_ptr(),
                                        c.dev[1].data_ptr(), loss.data_ptr(), lse.data_ptr(), 0, out.data_ptr() if dx else None,
                                        d, out.data_ptr() if dw else None, d, ws.data_ptr(), need, st) == zr.ZR_OK
        assert zr.zr_query_status(ws.data_ptr(), st) == zr.ZR_OK
        for g, (w, tol) in zip((loss, lse, out), want[:2] + [want[2 if dx else 3]]):
            check(g, w, tol)


@pytest.mark.parametrize("d, vocab", [(64, 300), (136, 5000)])
def test_targets_of_probability_near_one(env, d, vocab):
    """Rows whose target is ahead of the rest by up to 20: what its probability lacks of 1,
    1e-7 at the least here, is known to the digits of the others' logits, in the loss and in
    each row's dx."""
    torch, zr = env
    rows = 120
    c = Case(torch, rows, d, vocab, seed=21, masked=0, weights=False)
    w = c.w.float() / c.w.float().norm(dim=1, keepdim=True)
    ahead = torch.linspace(1, 26, rows, device="cuda")[:, None]
    c.w.copy_(w)
    c.x.copy_(ahead * w[c.dev[0].long()])
    c.nx, c.nw = (t.double().cpu().numpy() for t in (c.x, c.w))
    loss, lse, dx, dw = c.run(zr)
    want_loss, _, want_dx, _, dz = step.cross_entropy(c.nx, c.nw, c.target)
    on = np.arange(rows), c.target
    left = -dz[on]  # 1 - p
    assert left.min() < 1e-6 and left.min() > 1e-10
    # each probability carries its own logit's error and the target's, a power's and its sum's
    tz = 2 * (d + 8) * U * (np.abs(c.nx) @ np.abs(c.nw).T).max(1)
    rel = tz + 90 * U + 2.0 ** -22 + (128 + vocab / 1024 + 16) * U
    # (an fp32 difference of two logits is exact to half a step of their size)
    size = 4 * U * np.abs(c.nx @ c.nw.T).max(1)
    got = loss.double().cpu().numpy()
    assert (np.abs(got - want_loss) <= 1.01 * (rel + size) * np.maximum(want_loss, left) + 4 * U * want_loss).all()
    each = 2.0 ** -11 * np.log(2) + rel + size + 2 * BF
    terms = np.abs(dz) @ np.abs(c.nw)
    tol = 1.01 * each[:, None] * terms + (vocab + 80) * U * terms + BF * 1.01 * np.abs(want_dx)
    assert (np.abs(dx.double().cpu().numpy() - want_dx) <= tol + 1e-38).all()
