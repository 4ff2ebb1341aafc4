"""Calls on a stream that is not the current one (``stream=``) while the
current one still has work queued, and the router's and the experts' calls from
several host threads at once.  Every result is compared, bit for bit, with the
same calls made alone."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
import ep_workloads as W  # noqa: E402
from tests import moe_reference as ref  # noqa: E402
from tests.gpu_backend import dev, dev_bf16, say  # noqa: E402


class Case:
    """A layer with its router, forward and backward."""

    def __init__(self, seed, T=96, H=256, E=16, k=4, R=4, inner=128, fp8=False):
        rng = np.random.default_rng(seed)
        self.T, self.k, self.inner = T, k, inner
        self.x = dev_bf16(W.normal_bf16(rng, (T, H)))
        self.logits = dev(rng.normal(size=(T, E)).astype(np.float32))
        self.gout = dev_bf16(W.normal_bf16(rng, (T, H)))
        self.offsets = dev(np.array([0, T // 3, T], np.int32))
        self.gw = torch.empty(T, k, device="cuda")
        self.r = ep.EpRouter(T, E, k, score="sigmoid", groups=4, topk_groups=2, max_seqs=2)
        self.b = ep.EpBuffers(T, H, k, E, R, fp8=fp8)

        def weights(rows, cols):
            q = rng.integers(0, 16, size=(E, rows, cols)).astype(np.uint8)
            s = (0.5 + rng.random((E, rows, cols // 64))) * 0.2 / np.sqrt(cols)
            return dev(ref.pack_codes(q)), torch.from_numpy(s.astype(np.float32)).bfloat16().cuda()

        self.up, self.down = weights(2 * inner, H), weights(H, inner)
        # rows of the buffers that no call writes: the same in every run
        self.b.recv_x.zero_()
        self.b.recv_weights.zero_()

    def run(self, stream=None):
        b, r, kw = self.b, self.r, dict(stream=stream)
        idx, w = r.route(self.logits, **kw)
        loss = r.balance_loss(self.logits, idx, 0.1, seq_offsets=self.offsets, **kw)
        b.layout(idx, **kw)
        b.dispatch(self.x, idx, w, **kw)
        up = ep.W4Experts.pack(*self.up, swiglu=True, **kw)
        down = ep.W4Experts.pack(*self.down, **kw)
        h = b.expert_product(up, **kw)
        y = b.expert_product(down, x=h, **kw)
        b.combine(y, w, **kw)
        gw = self.gw
        gy = b.combine_backward(self.gout, w, y, grad_weights=gw, **kw)
        gx = b.dispatch_backward(gy, **kw)
        g = r.backward(self.logits, idx, gw, r.prob_grad, self.offsets, **kw)
        return [idx, w, loss, r.counts, h, y, b.out, gy, gx, gw, g]

    def check(self):
        self.b.check_status()
        self.r.check_status()


def late_writes(*tensors):
    """Queues some milliseconds of work on the current stream and behind it
    writes into blocks of these tensors' sizes, which are free again (for the
    current stream) as soon as this returns."""
    m = torch.full((4096, 4096), 2.0 ** -12, device="cuda", dtype=torch.bfloat16)
    for _ in range(40):
        m = m @ m
    blocks = [torch.empty_like(t) for t in tensors for _ in range(2)]
    for b in blocks:
        b.view(torch.uint8).fill_(0x5A)


@pytest.mark.parametrize("fp8", [False, True])
def test_results_are_not_overwritten_by_the_current_stream(fp8):
    c = Case(51, fp8=fp8)
    say(f"alone fp8={fp8}")
    want = [t.clone() for t in c.run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for n in range(3):
        say(f"beside late writes {n}")
        sizes = [t for t in want if t.numel() > 4096] + list(c.up) + list(c.down)
        late_writes(*sizes)
        got = c.run(stream=side.cuda_stream)
        torch.cuda.synchronize()
        c.check()
        for i, (a, b) in enumerate(zip(got, want)):
            rows = slice(0, c.T * c.k) if i in (4, 5, 7) else slice(None)  # rows of experts
            assert torch.equal(a[rows], b[rows]), i


def test_ranked_buffers_of_another_stream():
    """The buffers that the non-expanded path makes on its first call."""
    outs = []
    for late in (False, True):
        c = Case(52)
        side = torch.cuda.Stream()
        idx, w = c.r.route(c.logits)
        c.b.layout(idx)
        torch.cuda.synchronize()
        say(f"ranked late={late}")
        if late:
            late_writes(torch.empty(c.T * 4, 256, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(c.T * 4, 256, device="cuda"),
                        torch.empty(c.T * 4, 4, device="cuda"))
        s = side.cuda_stream
        c.b.dispatch_ranked(c.x, idx, w, stream=s)
        c.b.expand(stream=s)
        c.b.combine_ranked(c.b.recv_x, stream=s)
        torch.cuda.synchronize()
        c.check()
        outs.append((c.b.out.clone(), c.b.recv_x.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_host_threads():
    """Two threads, each with its own buffers on its own stream."""
    cases = [Case(53), Case(54, T=300, E=32, fp8=True)]
    want = [[t.clone() for t in c.run()] for c in cases]
    torch.cuda.synchronize()
    errors, got = [], [None, None]

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = cases[i].run()
            s.synchronize()
        except Exception as e:  # reported in the main thread
            errors.append(e)

    say("two threads")
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for c, g, w in zip(cases, got, want):
        c.check()
        for i, (a, b) in enumerate(zip(g, w)):
            rows = slice(0, c.T * c.k) if i in (4, 5, 7) else slice(None)
            assert torch.equal(a[rows], b[rows]), i


def test_default_stream_by_its_handle():
    """The default stream's handle, 0, and the current stream's inside a capture."""
    c = Case(55)
    want = [t.clone() for t in c.run()]
    say("default stream's handle")
    got = c.run(stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    c.check()
    for i, (a, b) in enumerate(zip(got, want)):
        rows = slice(0, c.T * c.k) if i in (4, 5, 7) else slice(None)
        assert torch.equal(a[rows], b[rows]), i
    say("capturing stream's handle")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.run(stream=torch.cuda.current_stream().cuda_stream)
    for n in range(3):
        for t in got:
            t.view(torch.uint8).fill_(n)
        g.replay()
        torch.cuda.synchronize()
        c.check()
        for i, (a, b) in enumerate(zip(got, want)):
            rows = slice(0, c.T * c.k) if i in (4, 5, 7) else slice(None)
            assert torch.equal(a[rows], b[rows]), (n, i)
        c.run()
