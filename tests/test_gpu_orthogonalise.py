"""Orthogonalised matrices through the C ABI against the float64 oracle.

Tolerances.  Two.  First, against the oracle that rounds X, A and the polynomial to
fp16 where the kernels do: what is left is bf16's rounding of the output (root mean
square 2^-8 / sqrt 3 of a value, 0.0023 at most) and roundings that fall the other way
because an fp32 sum is off by an ulp, one in thousands: 0.0026 in the 2-norm of a
thousand values or more.  (Of fewer the mean says nothing: a rounding alone may be 2^-8
= 0.0039 of its value, as 0.6972 -> 0.6953 is 0.0027, and one that falls the other way is
within the second bound, which is taken for them.)  Second, against the exact steps: a
rounding of X in step k, at most 2^-11 of X in the 2-norm of its entries, grows by the
largest divided difference of the remaining steps' polynomial over X's singular values;
so do those of A (times |b| + 2 |c| |A|, and |X|) and of the polynomial (times |X|).
Their sum bounds the error in first order.
"""

import numpy as np
import pytest

from oracle import step
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)


@pytest.fixture(scope="module")
def env():
    return require_cuda()


def half(v):
    return (np.asarray(v) * 2048).astype(np.float32).astype(np.float16).astype(np.float64) / 2048


def bound(g, coefficients):
    """The error's bound in the 2-norm of all entries, relative to the result's."""
    s = np.linalg.svd(np.asarray(g, dtype=np.float64), compute_uv=False)
    s = s / (np.linalg.norm(s) + 1e-7)
    at = [s]
    for a, b, c in coefficients:
        at.append(a * at[-1] + b * at[-1] ** 3 + c * at[-1] ** 5)

    def growth(k):
        """The largest divided difference of steps k, k + 1, ... over their arguments."""
        most = 1.0
        for (a, b, c), x in zip(coefficients[k:], at[k:]):
            grid = np.linspace(0, max(1e-9, np.abs(x).max() * 1.01), 400)
            most *= max(np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max(),
                        np.abs(a + b * grid ** 2 + c * grid ** 4).max())
        return most

    e, total = 2.0 ** -11, 0.0
    for k, (a, b, c) in enumerate(coefficients):
        x, top = at[k], np.abs(at[k]).max()
        sq, poly = x ** 2, a + b * x ** 2 + c * x ** 4
        total += e * np.linalg.norm(x) * growth(k)
        total += e * np.linalg.norm(sq) * (abs(b) + 2 * abs(c) * top ** 2) * top * growth(k + 1)
        total += e * np.linalg.norm(poly) * top * growth(k + 1)
    return total / np.linalg.norm(at[-1]) + 2.0 ** -8


def check(got, g, coefficients, eps=1e-7, scale=1.0):
    got = got.double().cpu().numpy() / scale
    assert np.isfinite(got).all()
    most = bound(g, coefficients)
    near = step.orthogonalise(g, coefficients, eps, rounded=half)
    assert np.linalg.norm(got - near) <= (2.6e-3 if got.size >= 1000 else most) * np.linalg.norm(near) + 1e-30
    want = step.orthogonalise(g, coefficients, eps)
    assert np.linalg.norm(got - want) <= most * np.linalg.norm(want) + 1e-30


SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (8, 8), (17, 40), (40, 17), (64, 64), (63, 130), (128, 128), (129, 65),
          (100, 300), (256, 704), (704, 256), (333, 333), (520, 264), (264, 1001), (1001, 264), (600, 640)]


def make(torch, shape, dt="f32", seed=0, scale=1.0):
    rng = np.random.default_rng(seed + sum(shape))
    r, c = shape[-2:]
    low = rng.normal(size=shape[:-2] + (r, 3)) @ rng.normal(size=shape[:-2] + (3, c))
    g = torch.from_numpy(((rng.normal(size=shape) + low) * scale).astype(np.float32)).cuda()
    return g.bfloat16() if dt == "bf16" else g


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_shapes(env, shape, dt):
    torch, zr = env
    g = make(torch, shape, dt, scale=1e-3)
    check(zr.orthogonalise(g), g.double().cpu().numpy(), [MUON] * 5)


@pytest.mark.parametrize("shape", [(1100, 1500), (1500, 1100), (2050, 700)], ids=str)
def test_large(env, shape):
    torch, zr = env
    g = make(torch, shape, "bf16")
    check(zr.orthogonalise(g), g.double().cpu().numpy(), [MUON] * 5)


@pytest.mark.parametrize("coefficients", [[MUON], [CUBIC] * 12, [(2.0, -1.5, 0.5)] * 6, [MUON] * 3 + [CUBIC] * 2])
def test_steps(env, coefficients):
    torch, zr = env
    for shape in ((70, 150), (150, 70)):
        g = make(torch, shape)
        got = zr.orthogonalise(g, steps=len(coefficients), coefficients=tuple(coefficients), scale=0.2)
        check(got, g.double().cpu().numpy(), coefficients, scale=0.2)
        if len(set(coefficients)) == 1:
            assert torch.equal(got, zr.orthogonalise(g, steps=len(coefficients), coefficients=coefficients[0], scale=0.2))


@pytest.mark.parametrize("count, rows, cols", [(1, 40, 70), (3, 70, 40), (16, 33, 65), (16, 65, 33), (5, 300, 136),
                                               (160, 16, 24), (700, 3, 5)])
def test_batches(env, count, rows, cols):
    """Every matrix as if it were alone, whatever its neighbours hold."""
    torch, zr = env
    g = make(torch, (count, rows, cols), "bf16")
    alone = [zr.orthogonalise(m) for m in g]
    for m, got in zip(g[:3], alone):
        check(got, m.double().cpu().numpy(), [MUON] * 5)
    out = zr.orthogonalise(g)
    # a matrix alone may be cut otherwise, its sums in another order: each rounds once
    for a, b in zip(out, alone):
        assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(b.double().norm())
    again = zr.orthogonalise(g)
    assert torch.equal(again, out)
    if count > 2:
        g[1, rows // 2, 0] = float("nan")
        g[2] = 0
        got = zr.orthogonalise(g)
        assert bool(torch.isnan(got[1]).all()) and not got[2].any()
        keep = [i for i in range(count) if i not in (1, 2)]
        assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows, cols", [(24, 40), (40, 24), (65, 33), (128, 256)])
def test_strides(env, rows, cols, dt):
    """Slices of a flat buffer at any place, rows apart, and matrices beside one another
    in the same rows."""
    torch, zr = env
    g = make(torch, (3, rows, cols), dt)
    want = zr.orthogonalise(g)
    flat = torch.zeros(3 * rows * cols + 5, dtype=g.dtype, device="cuda")
    view = flat[5:].view(3, rows, cols)
    view.copy_(g)
    assert torch.equal(zr.orthogonalise(view), want)
    wide = torch.zeros(rows, 3 * cols + 7, dtype=g.dtype, device="cuda")
    side = torch.as_strided(wide, (3, rows, cols), (cols, 3 * cols + 7, 1), 3)
    side.copy_(g)
    out = torch.full((rows, 3 * cols + 9), 9.0, dtype=torch.bfloat16, device="cuda")
    into = torch.as_strided(out, (3, rows, cols), (cols, 3 * cols + 9, 1), 4)
    assert torch.equal(zr.orthogonalise(side, out=into), want)
    assert bool((out[:, :4] == 9).all()) and bool((out[:, 4 + 3 * cols:] == 9).all())
    if dt == "bf16":
        assert torch.equal(zr.orthogonalise(view, out=view), want)
        assert bool((flat[:5] == 0).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sizes_of_values(env, dt):
    """From the smallest to the largest values of the type: the result is the same,
    unless eps counts."""
    torch, zr = env
    g = make(torch, (48, 80), dt)
    want = zr.orthogonalise(g, eps=0.0)
    for power in (-118, -90, -60, -45, -1, 30, 47, 60, 100, 120):
        moved = g * 2.0 ** power
        got = zr.orthogonalise(moved, eps=0.0)
        # (bf16 values under 2^-126 have fewer bits: entries of g under 2^-8 lose some at
        # 2^-118, and then it is another matrix)
        if torch.equal(moved.double() * 2.0 ** -power, g.double()):
            assert torch.equal(got, want), power
        else:
            check(got, moved.double().cpu().numpy(), [MUON] * 5, eps=0.0)
    # mixed sizes: what is far below the rest counts as little as it is
    mixed = g.clone()
    mixed[:, ::2] *= 2.0 ** -60
    check(zr.orthogonalise(mixed), mixed.double().cpu().numpy(), [MUON] * 5)
    check(zr.orthogonalise(g * 1e-9, eps=1e-7), (g * 1e-9).double().cpu().numpy(), [MUON] * 5, eps=1e-7)
    assert not zr.orthogonalise(torch.zeros_like(g), eps=0.0).any()
    assert not zr.orthogonalise(torch.zeros_like(g)).any()
    for bad in ("nan", "inf"):
        g[3, 5] = float(bad)
        assert bool(torch.isnan(zr.orthogonalise(g)).all())


@pytest.mark.parametrize("rows, cols", [(40, 24), (24, 40), (130, 200)])
def test_one_matrix_read_many_times(env, rows, cols):
    """A broadcast batch: its matrices are one and the same in memory."""
    torch, zr = env
    g = make(torch, (rows, cols), "bf16")
    got = zr.orthogonalise(g.expand(5, rows, cols))
    assert torch.equal(got, zr.orthogonalise(g.expand(5, rows, cols).contiguous()))
    check(got[4], g.double().cpu().numpy(), [MUON] * 5)


@pytest.mark.parametrize("shape", [(1, 300), (300, 1), (40, 70), (70, 40)], ids=str)
def test_up_to_the_range_of_the_steps(env, shape):
    """Singular values of 5.6 on entry to a step and polynomials of 31.9 still fit; what
    is past the range is not finite, and never a finite value that is wrong."""
    torch, zr = env
    g = make(torch, shape)
    if min(shape) > 1:  # one singular value, as large as X's norm, beside small ones
        g = g * 1e-4 + torch.outer(torch.ones(shape[0], device="cuda"), torch.ones(shape[1], device="cuda"))
    ng = g.double().cpu().numpy()
    for steps in ([(5.6, 0.0, 0.0), (1.0, 0.0, 0.0)], [(31.9, 0.0, 0.0)], [(2.0, 3.5, 0.0), (0.5, 0.25, 0.0)],
                  [(1.0, 0.0, 4.5), (0.25, 0.0, 0.03)], [(-5.6, 0.0, 0.0), (0.0, 1.0, 0.0)]):
        check(zr.orthogonalise(g, steps=len(steps), coefficients=tuple(steps)), ng, steps)
    if min(shape) > 1:  # (A's entries are smaller than its singular value)
        return
    for steps in ([(5.8, 0.0, 0.0), (1.0, 0.0, 0.0)], [(32.1, 0.0, 0.0)], [(33.0, 0.0, 0.0), (1.0, 0.0, 0.0)]):
        got = zr.orthogonalise(g, steps=len(steps), coefficients=tuple(steps))
        assert not bool(torch.isfinite(got).any())


@pytest.mark.parametrize("rows, cols", [(1, 1), (2, 3), (2, 8), (33, 65)])
def test_every_size_of_the_scale(env, rows, cols):
    """The result is X times the scale, rounded once, down to a scale that leaves few of
    its values normal."""
    torch, zr = env
    g = make(torch, (rows, cols))
    one = zr.orthogonalise(g).double()
    for scale in (2.0 ** -126, 1.3 * 2.0 ** -126, 1.3 * 2.0 ** -124, 1.3 * 2.0 ** -110, 1e-20, 1e20, 1.3 * 2.0 ** 120):
        want = one * scale
        # X's rounding in `one` and the result's own, which is a multiple of 2^-133
        tol = 2 * 2.0 ** -8 * want.abs() + 2.0 ** -134
        assert bool(((zr.orthogonalise(g, scale=scale).double() - want).abs() <= tol).all()), scale
    assert not zr.orthogonalise(g, scale=0.0).any()


def test_no_matrices(env):
    """An empty batch is no error, and its status word says so whatever was there."""
    torch, zr = env
    ws = torch.full((512,), 0x55, dtype=torch.uint8, device="cuda")
    out = zr.orthogonalise(torch.empty(0, 8, 16, device="cuda"), ws=ws)
    assert out.shape == (0, 8, 16)
    assert zr.zr_query_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == zr.ZR_OK
    assert bool((ws[4:] == 0x55).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("power", [0, -50, 50])
def test_a_row_of_millions_of_values(env, dt, power):
    """The norm of 2^26 + 16 values of one size, whose squares a long fp32 sum rounds the
    same way again and again.  X is 2^-13 to 6e-8 (1 / sqrt n), and so 2^-13 in fp16; a step
    of (1, 0, 0) and scales 2^-12 to either side of a bf16 half step show it to 2e-4."""
    torch, zr = env
    n = (1 << 26) + 16
    value = (1.408567 if dt == "f32" else 1.40625) * 2.0 ** power
    g = torch.full((1, n), value, dtype=torch.float32 if dt == "f32" else torch.bfloat16, device="cuda")
    for scale, want in ((1 + 2.0 ** -8 + 2.0 ** -12, 1 + 2.0 ** -7), (1 + 2.0 ** -8 - 2.0 ** -12, 1.0)):
        got = zr.orthogonalise(g, steps=1, coefficients=(1.0, 0.0, 0.0), scale=scale * 8192, eps=0.0)
        assert float(got.min()) == want == float(got.max())


@pytest.mark.parametrize("shape", [(1, (1 << 22) + 8), ((1 << 22) + 3, 5), (2, 40, (1 << 18) + 65), ((1 << 18) + 1, 130),
                                   (130, (1 << 20) + 1)], ids=str)
def test_sides_of_millions(env, shape):
    """A is a sum over the longer side, whose tensor-core sums are cut off and not rounded:
    2^18 terms or fewer to each, low by 2^-12, which is half of what its rounding to fp16
    counts in the bound.  A step of (0, 1, 0) shows A, five of them the update; both against
    the steps in fp64 on the GPU."""
    torch, zr = env
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(*shape, generator=g, device="cuda").bfloat16()
    if len(shape) == 2:
        x = x[None]
    tall = x.shape[1] > x.shape[2]
    wide = (x.transpose(1, 2) if tall else x).double()
    wide = wide / wide.flatten(1).norm(dim=1)[:, None, None]
    a = wide @ wide.transpose(1, 2)
    m, k = wide.shape[1:]
    scale = float(max(k, m) ** 0.5)
    got = zr.orthogonalise(x.view(shape), steps=1, coefficients=(0.0, 1.0, 0.0), scale=scale).double().view(x.shape)
    got = (got.transpose(1, 2) if tall else got) / scale
    want = a @ wide
    # along the result itself: A's cut sums, its rounding and X's to fp16 (which do not line up)
    along = (got * want).flatten(1).sum(1) / (want * want).flatten(1).sum(1)
    assert float((along - 1).abs().max()) <= 2.0 ** -12 + 2.0 ** -11
    del got, want
    y = wide
    for _ in range(5):
        a = y @ y.transpose(1, 2)
        p = MUON[0] * torch.eye(m, device="cuda", dtype=torch.float64) + MUON[1] * a + MUON[2] * a @ a
        y = p @ y
    got = zr.orthogonalise(x.view(shape)).double().view(x.shape)
    got = got.transpose(1, 2) if tall else got
    s = torch.linalg.eigvalsh(wide @ wide.transpose(1, 2)).clamp(min=0).sqrt()
    for n in range(len(x)):
        most = bound(torch.diag(s[n]).cpu().numpy(), [MUON] * 5)
        assert float((got[n] - y[n]).norm()) <= 1.5 * most * float(y[n].norm())
