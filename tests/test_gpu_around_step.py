"""The norm, the vocabulary cross entropy and the orthogonalised update together and
among other work: a whole data-parallel step (examples/pretrain_step.py) against
automatic differentiation in fp64, and the calls on other streams, after copies and
fills, in graphs, and one right behind another many times over."""

import math
import threading

import pytest

from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_cuda()


def reference(torch, ex, weights, batches):
    """The mean over ranks of all losses, and its gradients, in fp64."""
    flat = weights.double().requires_grad_()
    w = ex.views(flat)
    xs = [[b["x"].double().requires_grad_() for b in rank] for rank in batches]

    def norm(s, weight):
        return s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * weight

    total = 0.0
    for rank, states in zip(batches, xs):
        for b, x in zip(rank, states):
            y = norm(x, w["norm_in"][0])
            g = y @ w["gate"].t()
            h = g * torch.sigmoid(g) * (y @ w["up"].t())
            z = norm(x + h @ w["down"].t(), w["norm_out"][0]) @ w["head"].t()
            used = b["target"] >= 0
            p = torch.log_softmax(z, 1).gather(1, b["target"].clamp(min=0).long()[:, None])[:, 0]
            total = total - (p * b["weight"].double())[used].sum()
    got = torch.autograd.grad(total / len(batches), [flat] + [x for s in xs for x in s])
    return float(total) / len(batches), got[0], got[1:]


def test_a_whole_step_matches_the_whole_batch(env):
    torch, zr = env
    from examples import pretrain_step as ex

    ranks = 3
    weights = [ex.make_weights(0) for _ in range(ranks)]
    grads = [torch.empty_like(weights[0]) for _ in range(ranks)]
    batches = [ex.make_batches(r, 1) for r in range(ranks)]
    want_loss, want, want_dx = reference(torch, ex, weights[0], batches)
    done = [ex.rank_gradients(w, g, b) for w, g, b in zip(weights, grads, batches)]
    zr.skipreduce(grads, 0)
    loss = float(torch.stack([d[0] for d in done]).mean())
    # y, h, s, z, dz, ds, dh, dy and each micro-batch's gradients are rounded to bf16
    # (2^-9 on average): some ten roundings that do not line up, 0.006 of each matrix
    assert math.isfinite(loss) and abs(loss - want_loss) < 0.01 * (1 + abs(want_loss))
    for name, got in ex.views(grads[0]).items():
        ref = ex.views(want)[name]
        assert float((got.double() - ref).norm() / ref.norm()) < 0.03, name
    for got, ref in zip([dx for d in done for dx in d[1]], want_dx):
        assert float((got.double() / ranks - ref).norm() / ref.norm()) < 0.03
    for g in grads[1:]:
        assert torch.equal(g, grads[0])


@pytest.mark.parametrize("skip", [0, 1])
def test_replicas_stay_equal(env, skip):
    torch, zr = env
    from examples import pretrain_step as ex

    weights = [ex.make_weights(0) for _ in range(4)]
    grads = [torch.empty_like(weights[0]) for _ in range(4)]
    momenta = [torch.zeros_like(weights[0]) for _ in range(4)]
    batches = [ex.make_batches(r, 2) for r in range(4)]
    for i in range(3):
        before = ex.views(weights[0].clone())
        assert math.isfinite(float(ex.step(weights, grads, momenta, batches, skip, i)))
        assert all(torch.equal(weights[0], w) for w in weights[1:])
        # an orthogonalised update's singular values are near 1 (0.68 to 1.21, and the
        # roundings of weights of size 0.06 to bf16)
        moved = (before["down"].double() - ex.views(weights[0])["down"].double()) / 0.02
        s = torch.linalg.svdvals(moved)
        assert 0.3 < float(s.median()) < 1.5 and float(s.max()) < 2


class Work:
    """All calls on inputs that are made from `src` by the caller."""

    def __init__(self, torch, zr, rows=300, d=256, vocab=5000):
        self.torch, self.zr = torch, zr
        g = torch.Generator(device="cuda").manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.src = [r(rows, d).to(bf), r(rows, d).to(bf), r(3, 200, 136)]
        self.x, self.res, self.g = [torch.zeros_like(t) for t in self.src]
        self.weight, self.head = (1 + 0.1 * r(d)).to(bf), (r(vocab, d) / d ** 0.5).to(bf)
        self.target = torch.randint(-1000, vocab, (rows,), generator=g, device="cuda").int()
        e = lambda *s, t=bf: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        f32 = torch.float32
        self.out = [e(rows, d), e(rows, d), e(rows, t=f32), e(rows, t=f32), e(rows, t=f32), e(rows, d), e(vocab, d), e(rows, d),
                    e(d), e(3, 200, 136)]
        need = max(zr.zr_cross_entropy_workspace_size(rows, d, vocab, d, 1, 1),
                   zr.zr_orthogonalise_workspace_size(3, 200, 136), zr.zr_rms_norm_workspace_size(rows, d))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def calls(self, ws=True):
        zr, o = self.zr, self.out
        ws = self.ws if ws else None
        y, s, rstd = zr.rms_norm(self.x, self.weight, residual=self.res, out=o[0], sum_out=o[1], rstd=o[2])
        zr.cross_entropy_loss(y, self.head, self.target, loss=o[3], lse=o[4], dx=o[5], dw_vocab=o[6], ws=ws)
        zr.rms_norm_backward(s, self.weight, rstd, o[5], ds=o[5], dx=o[7], dweight=o[8], ws=ws)
        zr.orthogonalise(self.g, out=o[9], ws=ws)

    def fill(self):
        for t, s in zip((self.x, self.res, self.g), self.src):
            t.copy_(s)

    def zero(self):
        for t in (self.x, self.res, self.g):
            t.zero_()

    def expected(self):
        self.fill()
        self.torch.cuda.synchronize()
        self.calls()
        self.torch.cuda.synchronize()
        want = [t.clone() for t in self.out]
        self.zero()
        for t in self.out:
            t.zero_()
        self.torch.cuda.synchronize()
        return want


def same(torch, got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_after_copies_and_fills_and_before_readers(env):
    torch, zr = env
    w = Work(torch, zr)
    want = w.expected()
    big = torch.empty(64 << 20, device="cuda")
    for i in range(6):
        big.normal_()  # keeps the device busy while the rest is queued
        w.fill()
        w.calls(ws=i % 2 == 0)
        got = [t.clone() for t in w.out]  # readers in the same stream
        w.zero()                          # and a writer of the inputs
        w.ws.fill_(255)                   # and of the workspace
        torch.cuda.synchronize()
        assert same(torch, got, want)


def test_after_an_event_of_another_stream(env):
    torch, zr = env
    w = Work(torch, zr)
    want = w.expected()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    big = torch.empty(64 << 20, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(a):
            big.normal_()
            w.fill()
            ready = torch.cuda.Event()
            ready.record()
        with torch.cuda.stream(b):
            b.wait_event(ready)
            w.calls()
            done = torch.cuda.Event()
            done.record()
        with torch.cuda.stream(a):
            a.wait_event(done)
            got = [t.clone() for t in w.out]
            w.zero()
        torch.cuda.synchronize()
        assert same(torch, got, want)


def test_streams_by_argument(env):
    torch, zr = env
    w = Work(torch, zr)
    want = w.expected()
    w.fill()
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        y, sm, rstd = zr.rms_norm(w.x, w.weight, residual=w.res, stream=s)
        loss, lse, dx, dw = zr.cross_entropy_loss(y, w.head, w.target, stream=s)
        dxn, dwn = zr.rms_norm_backward(sm, w.weight, rstd, dx, ds=dx, stream=s)
        u = zr.orthogonalise(w.g, stream=s)
        torch.cuda.synchronize()
        assert same(torch, [y, sm, rstd, loss, lse, dx, dw, dxn, dwn, u], want)


def test_two_streams_at_once(env):
    """Two calls of each kind beside one another, each with what it allocates itself."""
    torch, zr = env
    w = [Work(torch, zr, rows=700), Work(torch, zr, rows=300)]
    want = [v.expected() for v in w]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for v in w:
        v.fill()
    torch.cuda.synchronize()
    for _ in range(10):
        for v, s in zip(w, streams):
            with torch.cuda.stream(s):
                v.calls(ws=False)
    torch.cuda.synchronize()
    for v, t in zip(w, want):
        assert same(torch, v.out, t)


def test_in_a_graph_with_copies(env):
    torch, zr = env
    w = Work(torch, zr)
    want = w.expected()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.zero()
        w.fill()
        w.calls()
        kept = [t.clone() for t in w.out]
        w.zero()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert same(torch, kept, want)


def test_in_graphs_with_workspaces_of_their_own(env):
    """No workspace is passed: what the wrappers allocate while a graph is captured
    belongs to the graph, and two graphs replayed at once do not share it."""
    torch, zr = env
    w = Work(torch, zr, rows=130)
    want = w.expected()
    w.fill()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        v = Work(torch, zr, rows=130)
        v.fill()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            v.calls(ws=False)
        graphs.append((g, v))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s, (g, _) in zip((a, b), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, v in graphs:
            assert same(torch, v.out, want)


@pytest.mark.parametrize("rows, d, vocab", [(40, 64, 700), (300, 1001, 2501), (1200, 512, 9000), (700, 72, 3000)])
def test_calls_right_behind_one_another(env, rows, d, vocab):
    """Kernels of one call start while those of the call before drain: hundreds of calls
    without a wait, of changing sizes and inputs, have the bits of calls on their own."""
    torch, zr = env
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = (r(vocab, d) / d ** 0.5).bfloat16()
    states = [r(rows, d).bfloat16(), r(rows // 3 + 1, d).bfloat16()]
    target = [torch.randint(-vocab // 4, vocab, (len(x),), generator=g, device="cuda").int() for x in states]
    mats = [r(2, 300, 200), r(130, 400)]
    ws = torch.empty(max(zr.zr_cross_entropy_workspace_size(len(x), d, vocab, d, 1, 1) for x in states), dtype=torch.uint8,
                     device="cuda")

    def calls(k, out):
        zr.cross_entropy_loss(states[k], head, target[k], loss=out[0], lse=out[1], dx=out[2], dw_vocab=out[3], ws=ws)
        zr.orthogonalise(mats[k], out=out[4])

    def outputs(k):
        x = states[k]
        return [torch.empty(len(x), device="cuda"), torch.empty(len(x), device="cuda"), torch.empty_like(x),
                torch.empty_like(head), torch.empty(mats[k].shape, dtype=torch.bfloat16, device="cuda")]

    want = []
    for k in (0, 1):
        o = outputs(k)
        calls(k, o)
        torch.cuda.synchronize()
        want.append(o)
    got = [outputs(k) for k in (0, 1)]
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        for k in (0, 1):
            calls(k, got[k])
            if i % 10 == 9:
                for a, b in zip(got[k], want[k]):
                    bad += (a != b).sum()
    torch.cuda.synchronize()
    assert int(bad) == 0
    assert zr.zr_query_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == zr.ZR_OK


def test_refused_arguments_keep_no_memory(env):
    """A wrapper that raises gives its workspace back, whichever side refuses."""
    torch, zr = env
    x, w = torch.zeros(64, 127, device="cuda").bfloat16(), torch.zeros(96, 127, device="cuda").bfloat16()
    t, rstd = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(64, device="cuda")
    out = [torch.empty(64, device="cuda"), torch.empty(64, device="cuda"), torch.empty_like(x), torch.empty_like(w),
           torch.empty(127, device="cuda").bfloat16()]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for call in (lambda: zr.cross_entropy_loss(x, w, t, loss=out[0], lse=out[1], dx=w[:64], dw_vocab=out[3]),
                 lambda: zr.orthogonalise(x, eps=-1.0, out=out[2]),
                 lambda: zr.rms_norm_backward(x, out[4], rstd, x, dx=out[2], dweight=out[4])):
        with pytest.raises(zr.ZrError):
            call()
        assert torch.cuda.memory_allocated() == before


def test_a_workspace_is_device_memory(env):
    torch, zr = env
    x, w = torch.zeros(64, 128, device="cuda").bfloat16(), torch.zeros(128, device="cuda").bfloat16()
    t, rstd = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(64, device="cuda")
    for ws in (torch.empty(1 << 22, dtype=torch.uint8), torch.empty(1 << 22, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        for call in (lambda: zr.cross_entropy_loss(x, x, t, ws=ws), lambda: zr.orthogonalise(x, ws=ws),
                     lambda: zr.rms_norm_backward(x, w, rstd, x, ws=ws)):
            with pytest.raises(ValueError):
                call()


def test_one_workspace_is_too_small(env):
    torch, zr = env
    x = torch.zeros(64, 128, device="cuda").bfloat16()
    t = torch.zeros(64, dtype=torch.int32, device="cuda")
    small = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for call in (lambda: zr.cross_entropy_loss(x, x, t, ws=small), lambda: zr.orthogonalise(x, ws=small)):
        with pytest.raises(zr.ZrError) as e:
            call()
        assert e.value.status == zr.ZR_ERR_CAPACITY


def test_from_several_threads(env):
    """Host threads with streams and sizes of their own at once: what a thread keeps of
    its last sizes is not another's."""
    torch, zr = env
    works = [Work(torch, zr, rows=r, d=d, vocab=v) for r, d, v in ((300, 256, 5000), (40, 72, 700), (513, 1024, 2048), (7, 40, 90))]
    want = [w.expected() for w in works]
    for w in works:
        w.fill()
    torch.cuda.synchronize()
    failed = []

    def run(w, t, other):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(12):
                    w.calls(ws=i % 2 == 0)
                    zr.zr_cross_entropy_workspace_size(*other)  # other sizes in between
                torch.cuda.current_stream().synchronize()
            if not same(torch, w.out, t):
                failed.append("other bits")
        except Exception as e:  # a thread's exception would be lost
            failed.append(repr(e))

    threads = [threading.Thread(target=run, args=(w, t, (65 + i, 64, 300, 64, 1, 1)))
               for i, (w, t) in enumerate(zip(works, want))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("rows, d, vocab", [(1, 33, 70), (130, 33, 50), (65, 100, 1003), (9, 264, 4097)])
def test_what_a_workspace_holds_before(env, rows, d, vocab):
    """Bytes of 255 (NaN in every type) or 0 in the workspaces: the same bits."""
    torch, zr = env
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, dy, norm_w = r(rows, d), r(vocab, d), r(rows, d), r(d)
    target = torch.randint(-vocab // 4, vocab, (rows,), generator=g, device="cuda").int()
    batch = r(3, rows, d)
    need = max(zr.zr_cross_entropy_workspace_size(rows, d, vocab, d, 1, 1), zr.zr_orthogonalise_workspace_size(3, rows, d),
               zr.zr_rms_norm_workspace_size(rows, d))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    _, s, rstd = zr.rms_norm(x, norm_w)
    got = []
    for fill in (0, 255):
        out = []
        for call in (lambda: zr.cross_entropy_loss(x, w, target, ws=ws), lambda: zr.rms_norm_backward(s, norm_w, rstd, dy, ws=ws),
                     lambda: (zr.orthogonalise(batch, ws=ws),)):
            ws.fill_(fill)
            out += call()
        got.append(out)
    assert same(torch, *got) and all(bool(torch.isfinite(t).all()) for t in got[0])


def test_a_stream_by_its_handle(env):
    """A handle is taken for a stream of the tensors' device, and the call runs on it."""
    torch, zr = env
    x = torch.randn(70, 264, device="cuda").bfloat16()
    w = torch.ones(264, device="cuda").bfloat16()
    want = zr.rms_norm(x, w)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):  # a call on any other stream would not be captured
        got = zr.rms_norm(x, w, stream=s.cuda_stream)[0]
    got.zero_()
    g.replay()
    assert torch.equal(got, want)
