"""The root-mean-square norm and its gradients through the C ABI against the float64
oracle.

Tolerances.  u = 2^-24.  A sum of squares is a chain of max(16, d / 1024) products in
a thread and 13 joins, each one rounding: rstd is off by half of that and 3 u, y by 2 u
more and half a step of its type.  In the backward pass hat = s rstd and dy weight
carry one rounding each, the mean the same chain; dweight's chain is a CTA's rows, the
rows a CTA has at once and the CTAs (608 at most, in eighths).
"""

import numpy as np
import pytest

from oracle import step
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SHAPES = [  # rows, d
    (1, 1), (1, 8), (3, 7), (2, 64), (5, 100), (9, 512), (4, 513), (7, 520), (1, 1001), (300, 1001), (6, 2048),
    (5, 2056), (33, 4096), (2, 4100), (700, 768), (3, 8192), (2, 9001), (2, 16384), (3, 16385), (2, 40000), (2000, 24),
    (1300, 136),
]


@pytest.fixture(scope="module")
def env():
    return require_cuda()


def dtype_of(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def matrix(torch, rng, rows, d, dt, pad=0, shift=0, scale=1.0):
    """Rows of a wider buffer that starts `shift` elements in; 7 outside."""
    flat = torch.full((shift + rows * (d + pad) + 8,), 7.0, dtype=dt, device="cuda")
    t = flat[shift:shift + rows * (d + pad)].view(rows, d + pad)[:, :d]
    t.copy_(torch.from_numpy((rng.normal(size=(rows, d)) * scale).astype(np.float32)))
    return t


def twin(torch, t):
    """The same values at the same strides and alignment (which choose the order of a sum)."""
    r, ld = t.shape[0], t.stride(0)
    flat = torch.zeros(t.storage_offset() + r * ld + 8, dtype=t.dtype, device="cuda")
    out = torch.as_strided(flat, t.shape, t.stride(), t.storage_offset())
    out.copy_(t)
    return out


def exact(t):
    return t.double().cpu().numpy()


def check(got, want, tol):
    got = exact(got)
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert off.size == 0 or off.max() <= 0, "%.3g over its tolerance" % off.max()


def chain(d):
    return (max(16, d / 1024) + 13) * U


def forward_check(y, s, rstd, weight, eps, dt):
    want, want_rstd = step.rms_norm(exact(s), exact(weight), eps)
    rel = chain(s.shape[1]) / 2 + 3 * U
    check(rstd, want_rstd, rel * want_rstd)
    check(y, want, (rel + 2 * U + HALF[dt]) * np.abs(want) + 1e-45)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["vectors", "odd"])
def test_forward(env, shape, dt, layout):
    torch, zr = env
    rng = np.random.default_rng(sum(shape))
    rows, d = shape
    pad, shift = (0, 0) if layout == "vectors" else (3, 1)
    td = dtype_of(torch, dt)
    x, res = (matrix(torch, rng, rows, d, td, pad, shift) for _ in range(2))
    w = matrix(torch, rng, 1, d, td)[0]
    y, s, rstd = zr.rms_norm(x, w, eps=1e-5)
    assert s is x
    forward_check(y, x, rstd, w, 1e-5, dt)
    out, total = (matrix(torch, rng, rows, d, td, pad, shift) for _ in range(2))
    y, s, rstd = zr.rms_norm(x, w, residual=res, out=out, sum_out=total)
    assert y is out and s is total
    assert torch.equal(s, (x.float() + res.float()).to(td))
    forward_check(y, s, rstd, w, 1e-6, dt)
    if pad and rows > 1:
        assert bool((torch.as_strided(out, (rows - 1, pad), (d + pad, 1), out.storage_offset() + d) == 7).all())
    # in place: the sum replaces the residual, y replaces x
    x2, r2 = twin(torch, x), twin(torch, res)
    zr.rms_norm(x2, w, residual=r2, out=x2, sum_out=r2)
    assert torch.equal(x2, y) and torch.equal(r2, s)


@pytest.mark.parametrize("shape", SHAPES + [(0, 64)], ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["vectors", "odd"])
def test_backward(env, shape, dt, layout):
    torch, zr = env
    rng = np.random.default_rng(sum(shape))
    rows, d = shape
    pad, shift = (0, 0) if layout == "vectors" else (5, 3)
    td = dtype_of(torch, dt)
    s, dy, ds, dx = (matrix(torch, rng, rows, d, td, pad, shift) for _ in range(4))
    w = matrix(torch, rng, 1, d, td)[0]
    rstd = zr.rms_norm(s, w)[2]
    ns, nw, ny, nd, nr = (exact(t) for t in (s, w, dy, ds, rstd))
    h = np.abs(ns * nr[:, None])
    g = np.abs(ny * nw)
    mean = (g * h).sum(1, keepdims=True) / d
    err = nr[:, None] * (4 * U * g + h * mean * (chain(d) + 6 * U))
    per_cta = rows / min(608, max(1, rows / 8)) + 8 + 608 / 8 + 8
    tol_w = (per_cta + 4) * U * (np.abs(ny) * h).sum(0)
    for branch in (None, ds):
        got = zr.rms_norm_backward(s, w, rstd, dy, ds=branch, dx=dx)
        want_x, want_w = step.rms_norm_backward(ns, nw, nr, ny, None if branch is None else nd)
        check(got[0], want_x, err + (HALF[dt] + 2 * U) * np.abs(want_x) + 1e-40)
        check(got[1], want_w, tol_w + HALF[dt] * np.abs(want_w) + 1e-40)
    # added to what is there, at an odd place of a flat buffer
    flat = torch.full((d + 9,), 0.5, dtype=td, device="cuda")
    zr.rms_norm_backward(s, w, rstd, dy, ds=ds, dx=dx, dweight=flat[3:3 + d], accumulate=True)
    check(flat[3:3 + d], want_w + 0.5, tol_w + (HALF[dt] + U) * np.abs(want_w + 0.5) + U + 1e-40)
    assert bool((flat[:3] == 0.5).all()) and bool((flat[3 + d:] == 0.5).all())
    if rows:
        # in place of each input
        for i in range(3):
            a = [twin(torch, t) for t in (s, dy, ds)]
            own = zr.rms_norm_backward(s, w, rstd, dy, ds=ds, dx=dx)[1]
            got = zr.rms_norm_backward(a[0], w, rstd, a[1], ds=a[2], dx=a[i])
            assert torch.equal(got[0], dx) and torch.equal(got[1], own)


@pytest.mark.parametrize("d", [40, 4096, 20000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sizes_of_values(env, d, dt):
    """Rows of zeros, of huge and of tiny values, and rows that are not numbers, each
    apart from the others."""
    torch, zr = env
    rng = np.random.default_rng(3)
    td = dtype_of(torch, dt)
    w = matrix(torch, rng, 1, d, td)[0]
    x = matrix(torch, rng, 6, d, td)
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4, d // 2] = float("nan")
    x[5, 1] = float("inf")
    y, _, rstd = zr.rms_norm(x, w)
    forward_check(y[:4], x[:4], rstd[:4], w, 1e-6, dt)
    assert not y[1].any()
    assert bool(torch.isnan(y[4]).all()) and bool(torch.isnan(y[5, 1])) and float(rstd[5]) == 0


def test_one_part_of_the_gradients(env):
    torch, zr = env
    rng = np.random.default_rng(4)
    s, dy = (matrix(torch, rng, 50, 200, torch.bfloat16) for _ in range(2))
    w = matrix(torch, rng, 1, 200, torch.bfloat16)[0]
    rstd = zr.rms_norm(s, w)[2]
    dx, dw = zr.rms_norm_backward(s, w, rstd, dy)
    need = zr.zr_rms_norm_workspace_size(50, 200)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    one, other = torch.empty_like(dx), torch.empty_like(dw)
    st = torch.cuda.current_stream().cuda_stream
    head = (s.data_ptr(), 200, w.data_ptr(), rstd.data_ptr(), dy.data_ptr(), 200, None, 200, 50, 200, zr.ZR_BF16, 0)
    assert zr.zr_rms_norm_backward(*head, one.data_ptr(), 200, None, None, 0, st) == zr.ZR_OK
    assert zr.zr_rms_norm_backward(*head, None, 200, other.data_ptr(), ws.data_ptr(), need, st) == zr.ZR_OK
    assert torch.equal(one, dx) and torch.equal(other, dw)


def test_rows_past_32_bits(env):
    """2.4e9 values: the last rows against a call of their own."""
    torch, zr = env
    rows, d = 600000, 4096
    s = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, _, rstd = zr.rms_norm(s, w)
    few = s[-5:].clone()
    want, _, want_rstd = zr.rms_norm(few, w)
    assert torch.equal(y[-5:], want) and torch.equal(rstd[-5:], want_rstd)
    dx, _ = zr.rms_norm_backward(s, w, rstd, y, ds=s)
    assert torch.equal(dx[-5:], zr.rms_norm_backward(few, w, want_rstd, want, ds=few)[0])


@pytest.mark.parametrize("rows, d", [(1, 2048), (5, 4096), (700, 1032), (1500, 2048)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_weight_gradient_alone_of_long_rows(env, rows, d, dt):
    torch, zr = env
    rng = np.random.default_rng(8)
    td = dtype_of(torch, dt)
    s, dy, ds = (matrix(torch, rng, rows, d, td) for _ in range(3))
    w = matrix(torch, rng, 1, d, td)[0]
    rstd = zr.rms_norm(s, w)[2]
    want = zr.rms_norm_backward(s, w, rstd, dy)[1]
    need = zr.zr_rms_norm_workspace_size(rows, d)
    ws, got = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(w)
    st = zr.zr_rms_norm_backward(s.data_ptr(), d, w.data_ptr(), rstd.data_ptr(), dy.data_ptr(), d, ds.data_ptr(), d, rows, d,
                                 zr.ZR_BF16 if dt == "bf16" else zr.ZR_F32, 0, None, d, got.data_ptr(), ws.data_ptr(), need,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == zr.ZR_OK and torch.equal(got, want)


def test_the_residual_is_the_input(env):
    """s = x + x, and many rows of one value."""
    torch, zr = env
    rng = np.random.default_rng(9)
    for rows, d in ((70, 264), (3, 5000)):
        x, w = matrix(torch, rng, rows, d, torch.bfloat16), matrix(torch, rng, 1, d, torch.bfloat16)[0]
        y, s, rstd = zr.rms_norm(x, w, residual=x)
        assert torch.equal(s, x + x)
        assert torch.equal(y, zr.rms_norm(twin(torch, s), w)[0]) and torch.equal(rstd, zr.rms_norm(s, w)[2])
    x = matrix(torch, rng, 100000, 1, torch.float32)
    y, _, rstd = zr.rms_norm(x, torch.ones(1, device="cuda"))
    forward_check(y, x, rstd, torch.ones(1), 1e-6, "f32")


@pytest.mark.parametrize("d", [1, 40, 1001, 4096, 16384, 20000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_up_to_the_largest_value(env, d, dt):
    """Rows whose sums of squares leave fp32's range by far, up to the type's largest
    finite value throughout: y is the weight, of either sign."""
    torch, zr = env
    rng = np.random.default_rng(d)
    td = dtype_of(torch, dt)
    w = matrix(torch, rng, 1, d, td)[0]
    x = matrix(torch, rng, 6, d, td)
    for n, size in enumerate((1e18, 2e19, 1e30, 1e36, 1e37)):
        x[n] *= size
    x[5] = torch.where(x[5] < 0, -1.0, 1.0) * torch.finfo(td).max
    assert bool(torch.isfinite(x).all())
    y, _, rstd = zr.rms_norm(x, w)
    # an rstd under 2^-126 is rounded to a multiple of 2^-149
    want, want_rstd = step.rms_norm(exact(x), exact(w), 1e-6)
    rel = chain(d) / 2 + 3 * U
    check(rstd, want_rstd, rel * want_rstd + 2.0 ** -150)
    check(y, want, (rel + 3 * U + HALF[dt]) * np.abs(want) + 1e-45)
    half = x * 0.5
    again, s, _ = zr.rms_norm(half, w, residual=half)
    assert torch.equal(s, x) and torch.equal(again, y)
    # eps counts there too, where it is of the squares' size
    y, _, rstd = zr.rms_norm(x[:3], w, eps=3e38)
    want, want_rstd = step.rms_norm(exact(x[:3]), exact(w), float(np.float32(3e38)))
    check(rstd, want_rstd, rel * want_rstd)
    check(y, want, (rel + 3 * U + HALF[dt]) * np.abs(want) + 1e-45)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_row_of_millions_of_values(env, dt):
    """Squares of one size: a sum of them is no worse for being long (a chain of 256, 13
    joins and the rounding of each thread's sum)."""
    torch, zr = env
    d, td = (1 << 24) + 77, dtype_of(torch, dt)
    x = torch.full((1, d), 1.1, dtype=td, device="cuda")
    w = torch.ones(d, dtype=td, device="cuda")
    y, _, rstd = zr.rms_norm(x, w)
    value = float(x[0, 0].double())
    want = 1 / np.sqrt(value * value + float(np.float32(1e-6)))
    rel = (256 + 14) * U / 2 + 3 * U
    assert abs(float(rstd[0].double()) - want) <= rel * want
    assert float((y.double() - value * want).abs().max()) <= (rel + 3 * U + HALF[dt]) * value * want
    # dy = s: the mean of dy h is the size of dy, and dx what is left of their difference
    dx, dw = zr.rms_norm_backward(x, w, rstd, x)
    r = float(rstd[0].double())
    left = r * (value - value * r * value * value * r)
    assert float((dx.double() - left).abs().max()) <= r * value * (256 + 14 + 8) * U + HALF[dt] * abs(left)
    assert float((dw.double() - value * value * r).abs().max()) <= (3 * U + HALF[dt]) * value * value * r
