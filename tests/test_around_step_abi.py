"""Argument checks of the norm, the vocabulary cross entropy and the orthogonalised
update: everything refused here is refused on the host, before anything could be
launched.  CPU only; the pointers are made up and never used."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G, H = (i << 40 for i in range(1, 9))
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def zr():
    from gradient_synchronisation_gb300 import _build

    _build.build()
    import gradient_synchronisation_gb300 as zr

    return zr


@pytest.fixture(autouse=True)
def no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")


def test_constants_match_the_header(zr):
    hdr = open(os.path.join(ROOT, "include", "zr.h")).read()
    assert int(re.search(r"#define ZR_MAX_STEPS (\d+)", hdr).group(1)) == zr.ZR_MAX_STEPS


def test_rms_norm_refusals(zr):
    def call(**k):
        a = dict(x=A, ld_x=64, r=B, ld_r=64, w=C, rows=4, d=64, dt=zr.ZR_BF16, eps=1e-6, y=D, ld_y=64, s=E, ld_s=64,
                 rstd=F)
        a.update(k)
        return zr.zr_rms_norm(*[a[n] for n in ("x", "ld_x", "r", "ld_r", "w", "rows", "d", "dt", "eps", "y", "ld_y", "s",
                                               "ld_s", "rstd")], None)

    for k in (dict(rows=-1), dict(d=0), dict(d=1 << 31), dict(rows=1 << 31), dict(dt=2), dict(eps=0.0), dict(eps=-1.0),
              dict(eps=NAN), dict(eps=INF), dict(ld_x=63), dict(ld_r=63), dict(ld_y=63), dict(ld_s=63), dict(x=0),
              dict(w=0), dict(y=0), dict(r=0), dict(s=0), dict(y=E), dict(y=E + 2), dict(y=A + 2), dict(y=A, ld_y=65),
              dict(s=B, ld_s=66), dict(s=A + 128), dict(y=C), dict(s=C + 8), dict(y=B + 6)):
        assert call(**k) == zr.ZR_ERR_INVALID_ARG, k
    for k in (dict(x=A + 1), dict(w=C + 1), dict(y=D + 1), dict(s=E + 1), dict(r=B + 1)):
        assert call(**k) == zr.ZR_ERR_ALIGNMENT, k
    assert call(rows=0, x=0, r=0, y=0, s=0) == zr.ZR_OK
    # in place, and beside one another in the same rows: let through, to the launch
    for k in (dict(y=A), dict(s=A), dict(y=B), dict(s=B), dict(y=A, s=B), dict(y=B, s=A),
              dict(y=A + 128, ld_x=128, ld_y=128)):
        assert call(**k) == zr.ZR_ERR_CUDA, k


def test_rms_norm_backward_refusals(zr):
    need = zr.zr_rms_norm_workspace_size(4, 64)
    assert need > 0 and zr.zr_rms_norm_workspace_size(0, 64) > 0
    assert zr.zr_rms_norm_workspace_size(-1, 64) == 0 == zr.zr_rms_norm_workspace_size(4, 0)

    def call(**k):
        a = dict(s=A, ld_s=64, w=B, rstd=C, dy=D, ld_dy=64, ds=E, ld_ds=64, rows=4, d=64, dt=zr.ZR_BF16, acc=0, dx=F,
                 ld_dx=64, dw=G, ws=H, n=need)
        a.update(k)
        return zr.zr_rms_norm_backward(*[a[n] for n in ("s", "ld_s", "w", "rstd", "dy", "ld_dy", "ds", "ld_ds", "rows",
                                                        "d", "dt", "acc", "dx", "ld_dx", "dw", "ws", "n")], None)

    for k in (dict(rows=-1), dict(d=0), dict(dt=7), dict(acc=2), dict(acc=-1), dict(dx=0, dw=0), dict(rstd=0), dict(s=0),
              dict(w=0), dict(dy=0), dict(ld_s=63), dict(ld_dy=63), dict(ld_ds=63), dict(ld_dx=63), dict(ws=0),
              dict(dx=A + 2), dict(dx=A, ld_dx=65), dict(dx=E + 64), dict(dw=B), dict(dw=A + 2), dict(dw=D), dict(dw=F),
              dict(dx=B)):
        assert call(**k) == zr.ZR_ERR_INVALID_ARG, k
    for k in (dict(s=A + 1), dict(dx=F + 1), dict(dw=G + 1), dict(ws=H + 8)):
        assert call(**k) == zr.ZR_ERR_ALIGNMENT, k
    assert call(n=need - 1) == zr.ZR_ERR_CAPACITY
    for k in (dict(dx=A), dict(dx=D), dict(dx=E), dict(ds=0), dict(dw=0, ws=0, n=0), dict(dx=0),
              dict(rows=0, s=0, dy=0, ds=0, dx=0, rstd=0)):
        assert call(**k) == zr.ZR_ERR_CUDA, k


def test_cross_entropy_refusals(zr):
    def need(**k):
        a = dict(rows=4, d=64, vocab=100, ld_w=64, dx=1, dw=1)
        a.update(k)
        return zr.zr_cross_entropy_workspace_size(a["rows"], a["d"], a["vocab"], a["ld_w"], a["dx"], a["dw"])

    def call(**k):
        a = dict(x=A, ld_x=64, w=B, ld_w=64, rows=4, d=64, vocab=100, dt=zr.ZR_BF16, target=C, weight=None, loss=D, lse=None,
                 acc=0, dx=E, ld_dx=64, dw=F, ld_dw=64, ws=G, n=1 << 40)
        a.update(k)
        return zr.zr_cross_entropy_loss(*[a[n] for n in ("x", "ld_x", "w", "ld_w", "rows", "d", "vocab", "dt", "target",
                                                         "weight", "loss", "lse", "acc", "dx", "ld_dx", "dw", "ld_dw", "ws",
                                                         "n")], None)

    assert need() > need(dx=0, dw=0) > 0 and need(rows=0) > 0
    for k in (dict(rows=-1), dict(d=0), dict(vocab=0), dict(ld_w=63), dict(dx=2), dict(dw=-1), dict(rows=(1 << 31) - 512)):
        assert need(**k) == 0, k
    most = (1 << 31) - 513
    for k in (dict(rows=-1), dict(d=0), dict(vocab=0), dict(vocab=1 << 31), dict(dt=3), dict(acc=2), dict(ld_x=63),
              dict(ld_w=63), dict(ld_dx=63), dict(ld_dw=63), dict(x=0), dict(w=0), dict(target=0), dict(ws=0),
              dict(loss=0, dx=0, dw=0), dict(dx=A + 2), dict(dx=A, ld_dx=65), dict(dx=B), dict(dw=B), dict(dw=B + 4),
              dict(dw=A), dict(dw=E + 8)):
        assert call(**k) == zr.ZR_ERR_INVALID_ARG, k
    assert call(dt=zr.ZR_F32) == zr.ZR_ERR_UNSUPPORTED
    for k in (dict(rows=most + 1), dict(d=most + 1, ld_x=1 << 31, ld_w=1 << 31, ld_dx=1 << 31, ld_dw=1 << 31),
              dict(vocab=most + 1)):
        assert call(**k) == zr.ZR_ERR_UNSUPPORTED, k
    for k in (dict(x=A + 1), dict(w=B + 8), dict(dx=E + 1), dict(dw=F + 1), dict(ws=G + 8), dict(ws=G + 128)):
        assert call(**k) == zr.ZR_ERR_ALIGNMENT, k
    assert call(n=need() - 1) == zr.ZR_ERR_CAPACITY
    # weights at odd strides may start anywhere; they are laid out again in the workspace
    assert need(ld_w=65) > need()
    assert call(w=B + 2, ld_w=65, n=need(ld_w=65) - 1) == zr.ZR_ERR_CAPACITY
    for k in (dict(), dict(dx=A), dict(dx=0), dict(dw=0), dict(w=B + 2, ld_w=65), dict(x=A + 2),
              dict(rows=0, x=0, target=0, dx=0)):
        assert call(**k) == zr.ZR_ERR_CUDA, k


def test_cross_entropy_workspace_has_pieces(zr):
    """Past a piece the workspace grows by the rows' states, not by their logits."""
    def need(rows, **k):
        a = dict(d=256, vocab=32000, dw=1)
        a.update(k)
        return zr.zr_cross_entropy_workspace_size(rows, a["d"], a["vocab"], a["d"], 1, a["dw"])

    logits = 2 * 32000
    assert need(4096 + 512) > (4096 + 512) * logits
    assert need(1 << 20) < need(4096 + 512) + (1 << 20) * (2 * 256 + 12) + 32000 * 256 * 4 + (1 << 26)
    assert need(1 << 20, dw=0) < need(1 << 20)


def test_orthogonalise_refusals(zr):
    need = zr.zr_orthogonalise_workspace_size(2, 32, 64)
    assert need > 0
    for k in ((-1, 32, 64), (2, 0, 64), (2, 32, 0), (2, 1 << 31, 64)):
        assert zr.zr_orthogonalise_workspace_size(*k) == 0

    def call(**k):
        a = dict(g=A, ld_g=64, step_g=2048, count=2, rows=32, cols=64, dt=zr.ZR_BF16, c=[3.4445, -4.775, 2.0315] * 5,
                 scale=1.0, eps=1e-7, out=B, ld_o=64, step_o=2048, ws=C, n=1 << 40)
        a.update(k)
        return zr.zr_orthogonalise(*[a[n] for n in ("g", "ld_g", "step_g", "count", "rows", "cols", "dt", "c", "scale",
                                                    "eps", "out", "ld_o", "step_o", "ws", "n")], None)

    one = [3.4445, -4.775, 2.0315]
    for k in (dict(dt=2), dict(count=-1), dict(rows=0), dict(cols=0), dict(c=[]), dict(c=one * 33), dict(c=[1.0, NAN, 0.0]),
              dict(c=[INF, 1.0, 0.0]), dict(scale=NAN), dict(scale=INF), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF),
              dict(ld_g=63), dict(ld_o=63), dict(g=0), dict(out=0), dict(ws=0), dict(step_g=-1), dict(step_o=-1),
              dict(step_o=2047), dict(step_o=0), dict(step_o=64, ld_o=127), dict(out=A + 2), dict(out=A, ld_o=65),
              dict(out=A, step_o=4096), dict(out=A + 4096), dict(g=B, dt=zr.ZR_F32)):
        assert call(**k) == zr.ZR_ERR_INVALID_ARG, k
    for k in (dict(g=A + 1), dict(g=A + 2, dt=zr.ZR_F32), dict(out=B + 1), dict(ws=C + 8), dict(ws=C + 128)):
        assert call(**k) == zr.ZR_ERR_ALIGNMENT, k
    assert call(n=need - 1) == zr.ZR_ERR_CAPACITY
    # sizes whose tiles or offsets would not fit are refused before a launch
    big = dict(ld_g=1 << 30, ld_o=1 << 30, step_g=1 << 50, step_o=1 << 50)
    assert call(count=1 << 26, **big) == zr.ZR_ERR_INVALID_ARG
    assert call(count=1 << 29, n=1 << 60) == zr.ZR_ERR_INVALID_ARG  # 2^41 bytes from A on: over out
    assert call(count=1 << 25, g=1 << 56, out=2 << 56, n=1 << 60) == zr.ZR_ERR_UNSUPPORTED
    assert call(count=0, g=0, out=0, ws=0) == zr.ZR_OK
    # matrices beside one another in the same rows, one read twice, in place: let through
    for k in (dict(step_g=64, ld_g=128, step_o=64, ld_o=128), dict(step_g=0), dict(out=A), dict(count=1, step_g=-5, step_o=-5),
              dict(c=one), dict(c=one * 32), dict(eps=0.0)):
        assert call(**k) == zr.ZR_ERR_CUDA, k


def test_wrappers_refuse_wrong_tensors(zr):
    import torch

    x, w, t = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: zr.rms_norm(x, w), lambda: zr.rms_norm_backward(x, w, torch.zeros(4), x),
                 lambda: zr.cross_entropy_loss(x.bfloat16(), x.bfloat16(), t), lambda: zr.orthogonalise(x)):
        with pytest.raises(ValueError):  # not on the GPU
            call()
    with pytest.raises(TypeError):
        zr.rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        zr.orthogonalise(x.half())
    with pytest.raises(ValueError):
        zr.orthogonalise(w)
    with pytest.raises(ValueError):
        zr.rms_norm(w, w)
    for c, steps in (((1.0, 2.0), 1), (((1.0, 2.0, 3.0),) * 2, 3), (((1.0, 2.0),) * 3, 3)):
        with pytest.raises(ValueError):
            zr._steps(c, steps)
    assert list(zr._steps((1.0, 2.0, 3.0), 2)) == [1, 2, 3, 1, 2, 3]
    assert list(zr._steps(((1, 2, 3), (4, 5, 6)), 2)) == [1, 2, 3, 4, 5, 6]
    assert list(zr._steps(((1, 2, 3), (4, 5, 6), (7, 8, 9)), 3)) == list(range(1, 10))


def test_orthogonalise_of_no_matrices_clears_the_status_word(zr):
    """A given workspace is written, so the call reaches the GPU that is not there."""
    args = (A, 64, 2048, 0, 32, 64, zr.ZR_BF16, [1.0, 2.0, 3.0], 1.0, 0.0, B, 64, 2048)
    assert zr.zr_orthogonalise(*args, C, 1 << 20, None) == zr.ZR_ERR_CUDA
    assert zr.zr_orthogonalise(*args, 0, 0, None) == zr.ZR_OK


def test_sizes_that_no_call_takes_have_no_workspace(zr):
    """0 bytes, not what is left of a product past 64 bits; and the calls refuse the
    sizes, whatever the workspace."""
    most = (1 << 31) - 513
    for k in ((1, most, most), (most, most, most), (1 << 26, 64, 64), (1, 1 << 30, 1 << 20)):
        assert zr.zr_orthogonalise_workspace_size(*k) == 0, k
    assert zr.zr_orthogonalise_workspace_size(1, 1 << 20, 1 << 20) > 1 << 42
    assert zr.zr_orthogonalise(A, 1 << 30, 0, 1, 1 << 20, 1 << 30, zr.ZR_BF16, [1.0, 2.0, 3.0], 1.0, 0.0, 1 << 62, 1 << 30, 0,
                               C, 1 << 20, None) == zr.ZR_ERR_UNSUPPORTED
    for k in ((most, most, most, most), (1, most, most, most), (1 << 20, 1 << 30, 1 << 20, 1 << 30),
              (1 << 30, 1 << 30, 1 << 30, (1 << 30) + 1)):
        assert zr.zr_cross_entropy_workspace_size(*k, 1, 1) == 0, k
    assert zr.zr_cross_entropy_workspace_size(1 << 20, 1 << 14, 1 << 18, 1 << 14, 1, 1) > 1 << 35
    assert zr.zr_cross_entropy_loss(A, 1 << 30, B, 1 << 30, 2, 1 << 30, 1 << 20, zr.ZR_BF16, C, None, D, None, 0, None, 0, None,
                                    0, 1 << 62, 1 << 20, None) == zr.ZR_ERR_UNSUPPORTED


def test_a_stream_is_of_the_tensors_device(zr, monkeypatch):
    """A handle says nothing of its device: it is taken for one of the tensor's, whichever
    device is the current one; a stream object of another device is refused."""
    import contextlib
    import types

    import torch

    made, current = [], []

    class Stream:
        def __init__(self, handle, device=None):
            self.handle, self.device = handle, device
            made.append(self)

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", type("ExternalStream", (Stream,), {}))
    monkeypatch.setattr(torch.cuda, "stream", use)
    x = types.SimpleNamespace(device=torch.device("cuda", 1))
    assert zr._run_on(77, lambda t, more: (t, more), x, 5) == (x, 5)
    assert made[-1] is current[-1] and made[-1].handle == 77 and made[-1].device == x.device
    own = Stream(3, torch.device("cuda", 1))
    assert zr._run_on(own, lambda t: t, x) is x and current[-1] is own
    with pytest.raises(ValueError):
        zr._run_on(Stream(3, torch.device("cuda", 0)), lambda t: t, x)


def test_sums_of_the_tensor_cores_have_a_most_of_terms(zr):
    """2^18: more rows go in pieces however wide the states are, a longer vocabulary in
    parts of dx, each with its fp32 sums in the workspace."""
    size = zr.zr_cross_entropy_workspace_size
    rows, d, vocab = 1 << 19, 1 << 18, 1000
    assert size(rows, d, vocab, d, 0, 1) < rows * (2 * d + 12) + vocab * d * 4 + 4096 * vocab * 4 + (1 << 20)
    rows, d, vocab = 4864, 1024, 1 << 21
    assert size(rows, d, vocab, d, 1, 0) - size(rows, d, vocab, d, 0, 0) >= 8 * 4096 * d * 4


def test_numbers_of_steps_that_are_refused(zr):
    """Before anything is made for them, and before 32 bits are taken of them."""
    for steps in (0, 33, 10 ** 12, (1 << 32) + 5, -1, -10 ** 12):
        with pytest.raises(zr.ZrError) as e:
            zr._steps((1.0, 2.0, 3.0), steps)
        assert e.value.status == zr.ZR_ERR_INVALID_ARG
    assert len(zr._steps((1.0, 2.0, 3.0), 32)) == 96


@pytest.mark.parametrize("d, ctas", [(200, 608), (1000, 608), (2000, 608), (3000, 456), (5000, 152), (40000, 152)])
def test_norm_workspace_holds_the_sums_of_each_kernel(zr, d, ctas):
    """A row of fp32 sums from each CTA that an SM holds at once, whichever of two kernels
    a call's alignment chooses."""
    assert zr.zr_rms_norm_workspace_size(100000, d) == ctas * d * 4
    assert zr.zr_rms_norm_workspace_size(1, d) == d * 4
