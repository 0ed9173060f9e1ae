"""The step's calls among other work: their kernels may be started before the
one ahead of them has ended, so what they read has to be complete all the same
-- after copies, fills, events of other streams, and inside graphs."""

import pytest

from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_cuda()


class Work:
    """All five calls on inputs that are made from `src` by the caller."""

    def __init__(self, torch, zr, rows=300):
        self.torch, self.zr = torch, zr
        g = torch.Generator(device="cuda").manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.src_x = r(rows, 256).bfloat16()
        self.src_z = r(rows, 20000).bfloat16()
        self.x, self.z = torch.zeros_like(self.src_x), torch.zeros_like(self.src_z)
        self.wg, self.wu = r(520, 256).bfloat16(), r(520, 256).bfloat16()
        self.dh = r(rows, 520).bfloat16()
        self.top, idx = torch.topk(r(rows, 20000), 40)
        self.idx = idx.int()
        self.tok = self.idx[:, 3].contiguous()
        self.adv = r(rows)
        self.off = torch.tensor([0, 50, 120, 200, rows], device="cuda")
        self.out = [torch.empty(rows, 520, device="cuda", dtype=torch.bfloat16), torch.empty_like(self.x),
                    torch.empty_like(self.wg), torch.empty_like(self.wu)]
        self.dz = [torch.empty_like(self.z) for _ in range(3)]
        self.loss = [torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"),
                     torch.empty(2, device="cuda")]
        self.ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")

    def calls(self):
        zr = self.zr
        zr.gated_ff(self.x, self.wg, self.wu, out=self.out[0], ws=self.ws)
        zr.gated_ff_backward(self.x, self.wg, self.wu, self.dh, dx=self.out[1], dw_gate=self.out[2],
                             dw_up=self.out[3], ws=self.ws)
        zr.distill_loss(self.z, self.idx, self.top, loss=self.loss[0], dlogits=self.dz[0])
        zr.policy_loss(self.z, self.tok, self.adv, loss=self.loss[1], dlogits=self.dz[1])
        zr.preference_loss(self.z, self.tok, self.off, self.adv, loss=self.loss[2], dlogits=self.dz[2],
                           ws=self.ws)

    def results(self):
        self.torch.cuda.synchronize()
        return [t.clone() for t in self.out + self.dz + self.loss]

    def expected(self):
        self.x.copy_(self.src_x), self.z.copy_(self.src_z)
        self.torch.cuda.synchronize()
        self.calls()
        want = self.results()
        for t in [self.x, self.z] + self.out + self.dz + self.loss:
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
    for _ in range(5):
        big.normal_()  # keeps the device busy while the rest is queued
        w.x.copy_(w.src_x), w.z.copy_(w.src_z)
        w.calls()
        got = [t.clone() for t in w.out + w.dz + w.loss]  # readers in the same stream
        w.x.zero_(), w.z.zero_()                           # and a writer of the inputs
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
            w.x.copy_(w.src_x), w.z.copy_(w.src_z)
            ready = torch.cuda.Event()
            ready.record()
        with torch.cuda.stream(b):
            b.wait_event(ready)
            w.calls()
            done = torch.cuda.Event()
            done.record()
        with torch.cuda.stream(a):
            a.wait_event(done)
            got = [t.clone() for t in w.out + w.dz + w.loss]
            w.x.zero_(), w.z.zero_()
        torch.cuda.synchronize()
        assert same(torch, got, want)


def test_in_a_graph_with_copies_and_a_second_stream(env):
    torch, zr = env
    w = Work(torch, zr)
    want = w.expected()
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w.x.zero_()
        w.x.copy_(w.src_x)
        fork = torch.cuda.Event()
        fork.record()
        with torch.cuda.stream(side):
            side.wait_event(fork)
            w.z.copy_(w.src_z)
            join = torch.cuda.Event()
            join.record()
        w.dz[0].zero_()
        s.wait_event(join)
        w.calls()
        kept = [t.clone() for t in w.out + w.dz + w.loss]
        w.x.zero_()
    for _ in range(3):
        w.z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(torch, kept, want)


def test_in_a_graph_with_workspaces_of_its_own(env):
    """No workspace is passed: what the wrappers allocate while a graph is
    captured belongs to the graph, and two graphs do not share it."""
    torch, zr = env
    w = Work(torch, zr, rows=130)
    x = torch.randn(130, 77, device="cuda").bfloat16()  # rows off 16 bytes: laid out again
    wg, wu = torch.randn(90, 77, device="cuda").bfloat16(), torch.randn(90, 77, device="cuda").bfloat16()
    dh = torch.randn(130, 90, device="cuda").bfloat16()
    w.z.copy_(w.src_z)

    def calls():
        return [zr.gated_ff(x, wg, wu), *zr.gated_ff_backward(x, wg, wu, dh),
                *zr.preference_loss(w.z, w.tok, torch.clamp(w.off, max=130), w.adv)]

    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = calls()
        graphs.append((g, out))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s, (g, _) in zip((a, b), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert same(torch, out, want)


@pytest.mark.parametrize("rows, d, f", [(8, 1024, 8192), (64, 512, 11008), (300, 128, 16384),
                                        (1500, 1024, 4096), (700, 4096, 96)])
def test_both_gradients_are_there_when_the_call_is_done(env, rows, d, f):
    """The weights' gradients are made beside the input's, and may end first or
    last: readers, the next call's kernels and writers of all inputs wait for both."""
    torch, zr = env
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 16).bfloat16()  # noqa: E731
    x, wg, wu, dh = r(rows, d), r(f, d), r(f, d), r(rows, f)
    ws = torch.empty(zr.zr_gated_ff_workspace_size(rows, d, f, d, d, 1), dtype=torch.uint8, device="cuda")
    dx, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    h = torch.empty(rows, f, dtype=torch.bfloat16, device="cuda")
    src = [t.clone() for t in (x, wg, wu, dh)]

    def call():
        zr.gated_ff_backward(x, wg, wu, dh, dx=dx, dw_gate=dg, dw_up=du, ws=ws)

    call()
    torch.cuda.synchronize()
    want = [dx.clone(), dg.clone(), du.clone()]
    zr.gated_ff(want[0], want[1], want[2], out=h)
    torch.cuda.synchronize()
    want.append(h.clone())
    for _ in range(20):
        for t in (dx, dg, du, h):
            t.fill_(float("nan"))
        call()
        zr.gated_ff(dx, dg, du, out=h)  # a kernel that may start early
        ws.fill_(255)                   # a writer of what both gradients read
        got = [t.clone() for t in (dx, dg, du, h)]
        call()
        again = [t.clone() for t in (dx, dg, du)]
        for t in (x, wg, wu, dh):
            t.zero_()
        torch.cuda.synchronize()
        for t, s in zip((x, wg, wu, dh), src):
            t.copy_(s)
        assert same(torch, got, want) and same(torch, again, want)


@pytest.mark.parametrize("rows, d, f", [(8, 1024, 8192), (130, 136, 264), (300, 128, 16384), (777, 1001, 2731),
                                        (1500, 1024, 4096), (1900, 1901, 1900)])
def test_accumulating_calls_in_a_row(env, rows, d, f):
    """Micro-batches added one after another into slices of a flat buffer: the
    weights' kernel, beside the input gradient's, reads the sums that the call
    before has just written and the activations' gradients of its own call.  The
    same bits as with nothing beside it and a synchronize after each call."""
    torch, zr = env
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 16).bfloat16()  # noqa: E731
    wg, wu = r(f, d), r(f, d)
    batches = [(r(rows, d), r(rows, f)) for _ in range(3)]
    n = zr.zr_gated_ff_workspace_size(rows, d, f, d, d, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")

    def slices():
        flat = torch.zeros(2 * f * d + 8, dtype=torch.bfloat16, device="cuda")
        return flat, flat[5:5 + f * d].view(f, d), flat[5 + f * d:5 + 2 * f * d].view(f, d)

    want, dg, du = slices()
    dxs = []
    for x, dh in batches * 4:
        s = torch.cuda.current_stream().cuda_stream
        for dxp, dgp, dup in ((dx.data_ptr(), None, None), (None, dg.data_ptr(), du.data_ptr())):
            assert zr.zr_gated_ff_backward(x.data_ptr(), d, wg.data_ptr(), wu.data_ptr(), d, dh.data_ptr(), f, rows,
                                           d, f, zr.ZR_BF16, 0, 1, dxp, d, dgp, dup, d, ws.data_ptr(), n, s) == zr.ZR_OK
            torch.cuda.synchronize()
        dxs.append(dx.clone())
    for _ in range(5):
        got, dg, du = slices()
        ws.fill_(255)
        outs = []
        for x, dh in batches * 4:
            outs.append(torch.empty_like(dx))
            zr.gated_ff_backward(x, wg, wu, dh, dx=outs[-1], dw_gate=dg, dw_up=du, accumulate=True, ws=ws)
        assert torch.equal(got, want) and same(torch, outs, dxs)
    assert zr.zr_query_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == zr.ZR_OK
