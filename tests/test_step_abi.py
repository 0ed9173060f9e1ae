"""Argument checks of the training-step calls: everything refused here is
refused on the host, before anything could be launched.  CPU only; the
pointers are made up and never used."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G = (i << 40 for i in range(1, 8))


@pytest.fixture(scope="module")
def zr():
    from gradient_synchronisation_gb300 import _build

    _build.build()
    import gradient_synchronisation_gb300 as zr

    return zr


def test_constants_match_the_header(zr):
    hdr = open(os.path.join(ROOT, "include", "zr.h")).read()
    for name in ("ZR_ACT_SILU", "ZR_ACT_GELU", "ZR_ACT_GELU_TANH"):
        assert int(re.search(name + r" = (\d+)", hdr).group(1)) == getattr(zr, name)
    assert int(re.search(r"#define ZR_MAX_TOP (\d+)", hdr).group(1)) == zr.ZR_MAX_TOP


def test_gated_ff_refusals(zr):
    def call(**k):
        a = dict(x=A, ld_x=64, wg=B, wu=C, ld_w=64, rows=4, d=64, f=32, dt=zr.ZR_BF16, act=0, h=D, ld_h=32, ws=E, n=1 << 20)
        a.update(k)
        return zr.zr_gated_ff(a["x"], a["ld_x"], a["wg"], a["wu"], a["ld_w"], a["rows"], a["d"], a["f"], a["dt"],
                              a["act"], a["h"], a["ld_h"], a["ws"], a["n"], None)

    bad = zr.ZR_ERR_INVALID_ARG
    for k in (dict(rows=-1), dict(d=0), dict(f=0), dict(d=1 << 31), dict(dt=5), dict(act=3), dict(act=-1),
              dict(ld_x=63), dict(ld_w=63), dict(ld_h=31), dict(x=0), dict(wg=0), dict(wu=0), dict(h=0),
              dict(h=A), dict(h=A + 4 * 64 * 2 - 2), dict(h=B + 2), dict(h=C + 32 * 64 * 2 - 2)):
        assert call(**k) == bad, k
    assert call(dt=zr.ZR_F32) == zr.ZR_ERR_UNSUPPORTED
    for k in (dict(x=A + 2), dict(wg=B + 8), dict(wu=C + 4), dict(h=D + 1)):
        assert call(**k) == zr.ZR_ERR_ALIGNMENT, k
    # rows at odd strides are laid out again in the workspace, from any start
    odd = dict(x=A + 2, ld_x=65)
    need = zr.zr_gated_ff_workspace_size(4, 64, 32, 65, 64, 0)
    assert need > 0 == zr.zr_gated_ff_workspace_size(4, 64, 32, 64, 64, 0)
    assert call(n=3) == zr.ZR_ERR_CAPACITY  # one is given: it holds the status word
    assert call(**odd, ws=0) == bad
    assert call(**odd, n=need - 1) == zr.ZR_ERR_CAPACITY
    assert call(**odd, ws=E + 8) == zr.ZR_ERR_ALIGNMENT
    assert call(**odd, ws=E + 128) == zr.ZR_ERR_ALIGNMENT
    assert call(rows=0, x=0, h=0) == zr.ZR_OK


def test_gated_ff_backward_refusals(zr):
    need = zr.zr_gated_ff_workspace_size(4, 64, 32, 64, 64, 1)
    assert need > 0

    def call(**k):
        a = dict(x=A, ld_x=64, wg=B, wu=C, ld_w=64, dh=D, ld_dh=32, rows=4, d=64, f=32, dt=zr.ZR_BF16, act=0, acc=0,
                 dx=E, ld_dx=64, dg=F, du=G, ld_dw=64, ws=8 << 40, n=need)
        a.update(k)
        return zr.zr_gated_ff_backward(*[a[n] for n in ("x", "ld_x", "wg", "wu", "ld_w", "dh", "ld_dh", "rows", "d",
                                                        "f", "dt", "act", "acc", "dx", "ld_dx", "dg", "du", "ld_dw",
                                                        "ws", "n")], None)

    bad = zr.ZR_ERR_INVALID_ARG
    for k in (dict(rows=-1), dict(d=0), dict(act=9), dict(acc=2), dict(ld_dh=31), dict(dh=0), dict(ld_dx=63),
              dict(ld_dw=63), dict(dg=0), dict(du=0), dict(dx=0, dg=0, du=0), dict(dx=A), dict(dx=D + 2),
              dict(dg=G + 2), dict(du=B), dict(dx=F + 64), dict(ws=0)):
        assert call(**k) == bad, k
    assert call(dt=zr.ZR_F32) == zr.ZR_ERR_UNSUPPORTED
    assert call(dg=F + 1) == zr.ZR_ERR_ALIGNMENT
    assert call(x=A + 2) == zr.ZR_ERR_ALIGNMENT
    assert call(ws=(8 << 40) + 8) == zr.ZR_ERR_ALIGNMENT
    assert call(n=need - 1) == zr.ZR_ERR_CAPACITY
    # gradients side by side in the same rows do not overlap, by one element they do
    side = dict(dg=F, ld_dw=128, dx=0, ws=0)
    assert call(**side, du=F + 63 * 2) == bad and call(**side, du=F - 65 * 2 + 4096) == bad
    assert call(**{**side, "ws": (8 << 40) + 8}, du=F + 64 * 2) == zr.ZR_ERR_ALIGNMENT  # refused for ws only
    assert zr.zr_gated_ff_workspace_size(0, 64, 32, 64, 64, 1) >= 4  # the status word, with no rows too
    assert call(rows=0, x=0, dh=0, dx=0, ws=0) == bad
    assert zr.zr_gated_ff_workspace_size(4, 64, 32, 63, 64, 1) == 0
    assert zr.zr_gated_ff_workspace_size(4, 0, 32, 64, 64, 1) == 0
    assert zr.zr_gated_ff_workspace_size(4, 64, 32, 64, 64, 2) == 0


@pytest.mark.parametrize("op", ["distill", "policy", "preference"])
def test_loss_refusals(zr, op):
    def call(**k):
        a = dict(z=A, ld=100, dt=zr.ZR_BF16, rows=4, vocab=100, tau=1.0, w=None, loss=C, dz=D, ldd=100, idx=E, top=F,
                 k=8, ld_top=8, lse=None, action=E, adv=F, old=None, ref=None, lo=0.2, hi=0.2, kl=0.0, off=F, pairs=1,
                 beta=0.1, eps=0.0, ws=G, n=zr.zr_preference_workspace_size(4))
        if op == "preference":
            a["ref"] = B
        a.update(k)
        head = (a["z"], a["ld"], a["dt"], a["rows"], a["vocab"])
        if op == "distill":
            return zr.zr_distill_loss(*head, a["idx"], a["top"], a["k"], a["ld_top"], a["lse"], a["tau"], a["w"],
                                      a["loss"], a["dz"], a["ldd"], None)
        if op == "policy":
            return zr.zr_policy_loss(*head, a["action"], a["adv"], a["old"], a["ref"], a["lo"], a["hi"], a["kl"],
                                     a["tau"], a["w"], a["loss"], None, None, a["dz"], a["ldd"], None)
        return zr.zr_preference_loss(*head, a["action"], a["off"], a["pairs"], a["ref"], a["beta"], a["eps"], a["w"],
                                     a["loss"], None, a["dz"], a["ldd"], a["ws"], a["n"], None)

    bad = zr.ZR_ERR_INVALID_ARG
    inf, nan = float("inf"), float("nan")
    cases = [dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 31) - 1, ld=1 << 31, ldd=1 << 31), dict(dt=2), dict(ld=99),
             dict(ldd=99), dict(z=0), dict(dz=A + 2), dict(dz=A, ldd=101), dict(dz=A + 798)]
    if op == "distill":
        cases += [dict(k=-1), dict(k=zr.ZR_MAX_TOP + 1, ld_top=2000), dict(ld_top=7), dict(idx=0), dict(top=0),
                  dict(loss=None, dz=None), dict(tau=0.0), dict(tau=-1.0), dict(tau=inf), dict(tau=nan), dict(tau=1e-39)]
    elif op == "policy":
        cases += [dict(action=0), dict(adv=0), dict(lo=-0.1), dict(lo=1.5), dict(lo=nan), dict(hi=-1.0), dict(hi=inf),
                  dict(kl=-1.0), dict(kl=nan), dict(kl=0.1), dict(loss=None, dz=None), dict(tau=0.0)]
    else:
        cases += [dict(action=0), dict(off=0), dict(pairs=-1), dict(ref=0), dict(beta=0.0), dict(beta=inf),
                  dict(eps=-0.1), dict(eps=1.1), dict(eps=nan), dict(loss=0), dict(ws=0)]
        assert call(ws=G + 4) == zr.ZR_ERR_ALIGNMENT
        assert call(n=100) == zr.ZR_ERR_CAPACITY
        assert zr.zr_preference_workspace_size(-1) == 0
    for k in cases:
        assert call(**k) == bad, k
    assert call(z=A + 1) == zr.ZR_ERR_ALIGNMENT
    assert call(dz=D + 1) == zr.ZR_ERR_ALIGNMENT
    if op != "preference":  # which clears its status word even then
        assert call(rows=0, z=0, dz=0, ld=100) == zr.ZR_OK


def test_wrappers_refuse_wrong_tensors(zr):
    import torch

    z = torch.zeros(2, 8)
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        zr.distill_loss(z, i, torch.zeros(2, 4))  # not on the GPU
    with pytest.raises(TypeError):
        zr.policy_loss(z.half(), i[:, 0], torch.zeros(2))
    with pytest.raises(ValueError):
        zr.gated_ff(z.bfloat16(), z.bfloat16(), z.bfloat16())
    with pytest.raises(ValueError):
        zr.preference_loss(z, i[:, 0], torch.zeros(2, dtype=torch.int64), torch.zeros(2))


def test_gated_ff_refuses_what_its_coordinates_cannot_hold(zr):
    """Tile coordinates are 32 bits: at 2 f >= 2^31 the backward pass would wrap
    to negative ones, which read as zeros.  (A workspace off its alignment: were
    the size let through, that would be refused instead, and nothing launched.)"""
    def forward(rows, d, f):
        ld = (d + 7) // 8 * 8
        return zr.zr_gated_ff(A, ld, B, C, ld, rows, d, f, zr.ZR_BF16, 0, D, f, E + 8, 1 << 60, None)

    def backward(rows, d, f):
        ld = (d + 7) // 8 * 8
        return zr.zr_gated_ff_backward(1 << 56, ld, 2 << 56, 3 << 56, ld, 4 << 56, f, rows, d, f, zr.ZR_BF16, 0, 0,
                                       5 << 56, d, 6 << 56, 7 << 56, d, (8 << 56) + 8, 1 << 62, None)

    most, half = (1 << 31) - 513, (1 << 30) - 513
    unsupported, alignment = zr.ZR_ERR_UNSUPPORTED, zr.ZR_ERR_ALIGNMENT
    assert forward(1, 8, most) == alignment and forward(1, 8, most + 1) == unsupported
    assert forward(1, most, 8) == alignment and forward(1, most + 1, 8) == unsupported
    assert forward(most, 8, 8) == alignment and forward(most + 1, 8, 8) == unsupported
    assert backward(1, 8, half) == alignment and backward(1, 8, half + 1) == unsupported
    assert backward(1, 8, 1 << 30) == unsupported and backward(1, 8, (1 << 31) - 1) == unsupported
    assert backward(1, most, 8) == alignment and backward(1, (1 << 31) - 1, 8) == unsupported
    assert backward(most, 8, 8) == alignment and backward((1 << 31) - 1, 8, 8) == unsupported


def test_matrices_past_the_address_space_are_refused(zr):
    """Offsets past 63 bits would wrap, and an output could seem to end before it
    begins.  (Each call has another fault as well, which is refused otherwise.)"""
    bad, alignment = zr.ZR_ERR_INVALID_ARG, zr.ZR_ERR_ALIGNMENT
    big = (1 << 31) - 1024

    def forward(rows, ld_x, x=A, ws=E + 8):
        return zr.zr_gated_ff(x, ld_x, B, C, 64, rows, 64, 32, zr.ZR_BF16, 0, D, 32, ws, 1 << 60, None)

    assert forward(4, 1 << 40, x=8 << 56) == alignment and forward(big, 1 << 40) == bad
    assert forward(1, 1 << 40) == alignment  # one row has no second one to step to
    assert forward(4, 64, x=(1 << 64) - 256) == bad

    def policy(rows, ld, z=A, dz=C + 1):
        return zr.zr_policy_loss(z, ld, zr.ZR_F32, rows, 100, E, F, None, None, 0.2, 0.2, 0.0, 1.0, None, D, None,
                                 None, dz, 100, None)

    assert policy(4, 1 << 30) == alignment and policy(big, 1 << 40) == bad
    assert policy(1 << 22, 1 << 40) == bad and policy(4, 100, z=(1 << 64) - 1024) == bad


def test_preference_of_more_ctas_than_a_grid_has_is_refused_first(zr):
    """(rows times parts of a row: a call of that size is refused before any kernel
    of it is launched, which here, without a GPU, would be ZR_ERR_CUDA.)"""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")

    def call(rows, vocab, dz):
        return zr.zr_preference_loss(1 << 56, vocab, zr.ZR_F32, rows, vocab, 2 << 56, 3 << 56, 1, 4 << 56, 0.1, 0.0,
                                     None, 5 << 56, None, dz, vocab, 7 << 56, 1 << 40, None)

    most = (1 << 31) - 1
    assert call(most, 40000, 6 << 56) == zr.ZR_ERR_UNSUPPORTED
    assert call(most, 40000, None) == zr.ZR_ERR_CUDA  # no gradient, no such grid
    assert call(most, 1, 6 << 56) == zr.ZR_ERR_CUDA  # one part each: it fits
