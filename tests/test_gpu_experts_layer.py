"""The bf16 experts and the SwiGLU checkpoint in a layer: a whole training step
through EpBuffers, captured in graphs, on other streams and from several
threads, and tensors past 2^32 values."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
import ep_workloads as W  # noqa: E402
from tests import experts_reference as ref  # noqa: E402
from tests.gpu_backend import dev, dev_bf16, host_bf16, say  # noqa: E402

U32, UBF16 = ref.U32, ref.UBF16


class Layer:
    """A layer's forward and backward: router, FP8 or bf16 dispatch, gate and up,
    SwiGLU kept in 8 bits, down, combine; then everything's gradient."""

    def __init__(self, seed, T=96, H=256, E=16, k=4, R=4, inner=200, fp8=True):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.E, self.k, self.inner, self.fp8 = T, H, E, k, inner, fp8
        self.x, self.gout = (dev_bf16(W.normal_bf16(rng, (T, H))) for _ in range(2))
        self.logits = dev(rng.normal(size=(T, E)).astype(np.float32))
        self.r = ep.EpRouter(T, E, k, score="sigmoid", scale=1.5)
        self.b = ep.EpBuffers(T, H, k, E, R, 2, fp8=fp8)
        self.up = ep.Bf16Experts(ref.to_bf16(rng.normal(size=(E, 2 * inner, H)) / 16).cuda())
        self.down = ep.Bf16Experts(ref.to_bf16(rng.normal(size=(E, H, inner)) / 14).cuda())
        self.kept = ep.SwigluCheckpoint(self.b.capacity, inner, E)
        self.sum = torch.zeros(E, 2 * inner, H, device="cuda")  # fp32 gradient of `up`
        self.gw = torch.empty(T, k, device="cuda")
        cap, bf16 = self.b.capacity, dict(dtype=torch.bfloat16, device="cuda")
        self.out = dict(gate_up=(cap, 2 * inner), h=(cap, inner), y=(cap, H), gy=(cap, H),
                        gh=(cap, inner), ggu=(cap, 2 * inner), h2=(cap, inner), gx=(cap, H))
        self.out = {n: torch.zeros(s, **bf16) for n, s in self.out.items()}
        self.out["gx0"] = torch.zeros(T, H, **bf16)
        self.out["g_down"] = torch.zeros(E, H, inner, **bf16)
        self.out["g_up"] = self.sum
        self.clear()

    def clear(self):
        """Rows of the buffers that no call writes: the same in every run."""
        for t in (self.b.recv_x, self.b.recv_weights, self.kept.codes, self.kept.scales,
                  *self.out.values()):
            t.zero_()

    def run(self, stream=None):
        b, r, kw, o = self.b, self.r, dict(stream=stream), self.out
        idx, w = r.route(self.logits, **kw)
        b.layout(idx, **kw)
        b.dispatch(self.x, idx, w, **kw)
        b.expert_product(self.up, out=o["gate_up"], **kw)
        b.swiglu_checkpoint(self.kept, o["gate_up"], out=o["h"], **kw)
        b.expert_product(self.down, x=o["h"], out=o["y"], **kw)
        b.combine(o["y"], w, **kw)
        b.combine_backward(self.gout, w, o["y"], grad_expert_out=o["gy"], grad_weights=self.gw,
                           **kw)
        b.expert_backward_rows(self.down, o["gy"], out=o["gh"], **kw)
        b.swiglu_backward(self.kept, o["gh"], out=o["ggu"], h=o["h2"], **kw)
        b.expert_backward_weights(self.down, o["gy"], x=o["h2"], out=o["g_down"], **kw)
        b.expert_backward_weights(self.up, o["ggu"], out=self.sum, add=self.sum, **kw)
        b.expert_backward_rows(self.up, o["ggu"], out=o["gx"], **kw)
        b.dispatch_backward(o["gx"], grad_x=o["gx0"], **kw)
        r.backward(self.logits, idx, self.gw, **kw)
        return self.results()

    def results(self):
        return [*self.out.values(), self.b.out, self.gw, self.r.topk_idx, self.r.grad_logits,
                self.kept.codes, self.kept.scales]

    def check(self):
        self.b.check_status()
        self.r.check_status()


def near(got, want, size, terms):
    """bf16 results of sums of that many terms."""
    err = ref.sum_error(terms, size)
    bad = np.abs(got - want) > err + (np.abs(want) + err) * UBF16 + 1e-37
    assert not bad.any(), np.max(np.abs(got - want) / (np.abs(want) + 1e-9))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 40, 700])
def test_training_step(T, fp8):
    """Every step against its 64-bit form on what the step before left."""
    c = Layer(T, T=T, fp8=fp8)
    say(f"training step T={T} fp8={fp8}")
    c.sum.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    c.check()
    b, E, I = c.b, c.E, c.inner
    off, cnt = b.expert_offsets.cpu().numpy(), b.num_tokens_per_expert.cpu().numpy()
    live = np.zeros(b.capacity, bool)
    for _, lo, hi in ref.expert_rows(off, cnt, b.capacity):
        live[lo:hi] = True
    o = {n: t.double().cpu().numpy() for n, t in c.out.items()}
    wu, wd = (e.weights.double().cpu().numpy() for e in (c.up, c.down))
    if fp8:
        xv = b.recv_x.view(torch.float8_e4m3fn).float().double().cpu().numpy() * np.repeat(
            b.recv_scales.double().cpu().numpy(), 128, axis=1)
    else:
        xv = b.recv_x.double().cpu().numpy()
    y, size = ref.product(xv, wu, off, cnt)
    near(o["gate_up"][live], y[live], size[live], c.H)
    codes, scales = ref.checkpoint(o["gate_up"][live])
    got = c.kept.codes.view(torch.float8_e4m3fn).double().cpu().numpy()
    assert np.array_equal(got[live], codes)
    assert np.array_equal(c.kept.scales.double().cpu().numpy()[live], scales)
    want = ref.silu(o["gate_up"][live][:, :I]) * o["gate_up"][live][:, I:]
    near(o["h"][live], want, np.abs(want), 8)
    y, size = ref.product(o["h"], wd, off, cnt)
    near(o["y"][live], y[live], size[live], I)
    y, size = ref.rows_grad(o["gy"], wd, off, cnt)
    near(o["gh"][live], y[live], size[live], c.H)
    kept = ref.kept(codes, scales, I)
    want, h2 = ref.swiglu_grad(kept, o["gh"][live])
    s, gate, up = ref.sigmoid(kept[:, :I]), kept[:, :I], kept[:, I:]
    size = np.concatenate([np.abs(o["gh"][live] * up * s) * (1 + np.abs(gate) * (1 - s)),
                           np.abs(o["gh"][live] * gate * s)], axis=1)
    near(o["ggu"][live], want, size, 8)
    near(o["h2"][live], h2, np.abs(h2), 8)
    y, size = ref.weights_grad(o["gy"], o["h2"], off, cnt)
    near(o["g_down"], y, size, int(cnt.max()))
    if fp8:
        xv = ref.rounded(xv.astype(np.float32))
    y, size = ref.weights_grad(o["ggu"], xv, off, cnt)
    assert np.all(np.abs(o["g_up"] - 3 - y) <= ref.sum_error(int(cnt.max()) + 1, size + 3))
    y, size = ref.rows_grad(o["ggu"], wu, off, cnt)
    near(o["gx"][live], y[live], size[live], 2 * I)


def test_one_rank_at_a_time():
    """Each rank's experts on its own rows give what all experts give at once."""
    c = Layer(5, T=50)
    say("one rank at a time")
    c.run()
    b, n = c.b, c.E // 4
    for r in range(4):
        part = slice(r * n, (r + 1) * n)
        up = ep.Bf16Experts(c.up.weights[part])
        kept = ep.SwigluCheckpoint(b.capacity, c.inner, n)
        lo, hi = int(b.expert_offsets[r * n]), int(b.expert_offsets[(r + 1) * n])
        rows = torch.zeros(b.capacity, dtype=torch.bool, device="cuda")
        rows[lo:hi] = b.row_src[lo:hi] >= 0
        gu = b.expert_product(up, rank=r)
        assert torch.equal(gu[rows], c.out["gate_up"][rows])
        h = b.swiglu_checkpoint(kept, gu, rank=r)
        assert torch.equal(h[rows], c.out["h"][rows])
        ggu, h2 = b.swiglu_backward(kept, c.out["gh"], rank=r)
        assert torch.equal(ggu[rows], c.out["ggu"][rows])
        assert torch.equal(h2[rows], c.out["h2"][rows])
        gw = b.expert_backward_weights(up, ggu, dtype=torch.float32, rank=r)
        assert torch.equal(gw, c.sum[part])
        gx = b.expert_backward_rows(up, ggu, rank=r)
        assert torch.equal(gx[rows], c.out["gx"][rows])
    with pytest.raises(ValueError):
        b.expert_backward_rows(c.up, c.out["ggu"], rank=4)


def fill(c, seed):
    g = np.random.default_rng(seed)
    c.x.copy_(dev_bf16(W.normal_bf16(g, (c.T, c.H))))
    c.gout.copy_(dev_bf16(W.normal_bf16(g, (c.T, c.H))))
    c.logits.copy_(dev(g.normal(size=(c.T, c.E)).astype(np.float32)))
    c.clear()


@pytest.mark.parametrize("fp8", [False, True])
def test_training_step_in_a_graph(fp8):
    """Two layers captured and replayed in turn on new inputs, with eager steps
    of a third between, each replay against an eager step."""
    layers, eager = [Layer(7, fp8=fp8), Layer(7, fp8=fp8)], Layer(7, fp8=fp8)
    graphs = []
    for i, c in enumerate(layers):
        fill(c, i)
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        say(f"capture {i} fp8={fp8}")
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for n in range(4):
        say(f"replay {n}")
        for i, (g, c) in enumerate(zip(graphs, layers)):
            fill(c, 10 * n + i)
            g.replay()
        for i, c in enumerate(layers):
            fill(eager, 10 * n + i)
            want = eager.run()
            torch.cuda.synchronize()
            for a, b in zip(c.results(), want):
                assert torch.equal(a, b)
            c.check()
        eager.check()


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


def test_results_are_not_overwritten_by_the_current_stream():
    """Results that the calls allocate themselves, on a side stream."""
    c = Layer(8, T=300)
    c.run()
    at = c.b.expert_offsets, c.b.num_tokens_per_expert
    o, live = c.out, np.zeros(c.b.capacity, bool)
    for _, lo, hi in ref.expert_rows(at[0].cpu().numpy(), at[1].cpu().numpy(), c.b.capacity):
        live[lo:hi] = True
    rows = dev(live)

    def calls(stream):
        kw = dict(stream=stream)
        h = c.kept.save(o["gate_up"], *at, **kw)
        ggu, h2 = c.kept.backward(o["gh"], *at, **kw)
        return [c.up.product(c.b.recv_x, c.b.recv_scales, *at, **kw)[rows], h[rows], ggu[rows],
                h2[rows], c.up.backward_rows(ggu, *at, **kw)[rows],
                c.up.backward_weights(c.b.recv_x, c.b.recv_scales, ggu, *at, **kw)]

    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for n in range(3):
        say(f"beside late writes {n}")
        late_writes(o["gate_up"], o["h"], o["gx"], want[-1])
        with torch.cuda.stream(side):  # the selections of rows run there too
            got = calls(side.cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_share_weights_and_repeats_are_bit_equal():
    a, b = Layer(9, T=500), Layer(9, T=500)
    b.up, b.down = a.up, a.down
    fill(a, 1)
    want = [t.clone() for t in a.run()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for n in range(3):
        say(f"two streams {n}")
        for c in (a, b):
            fill(c, 1)
        torch.cuda.synchronize()
        for c, s in zip((a, b), streams):
            c.run(stream=s.cuda_stream)
        torch.cuda.synchronize()
        for c in (a, b):
            for x, y in zip(c.results(), want):
                assert torch.equal(x, y)
            c.check()


def test_threads():
    """Four host threads, each with its own layer and stream."""
    layers = [Layer(20 + i, T=64) for i in range(4)]
    want = []
    for c in layers:
        fill(c, 3)
        want.append([t.clone() for t in c.run()])
    torch.cuda.synchronize()
    streams, errors = [torch.cuda.Stream() for _ in layers], []
    for c in layers:
        c.sum.zero_()
    torch.cuda.synchronize()

    def work(c, s):
        try:
            for _ in range(5):
                with torch.cuda.stream(s):
                    c.sum.zero_()
                c.run(stream=s.cuda_stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    say("threads")
    threads = [threading.Thread(target=work, args=a) for a in zip(layers, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, w in zip(layers, want):
        for x, y in zip(c.results(), w):
            assert torch.equal(x, y)


# --------------------------------------------------------------------------
# Large tensors
# --------------------------------------------------------------------------

def test_weights_past_32_bits():
    """3 experts of 30000 x 49152: the last begins past 2^31 values, and within it
    rows do, in bytes, past 2^32."""
    E, N, K = 3, 30000, 49152
    say("weights past 2^32 bytes")
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for e in range(E):
        for lo in range(0, N, 5000):
            w[e, lo:lo + 5000] = torch.randint(-2, 3, (5000, K), generator=g,
                                               device="cuda").bfloat16()
    experts = ep.Bf16Experts(w)
    for counts in ([0, 0, 5], [1, 0, 90]):  # streamed, tiled
        rows = sum(counts)
        x = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").bfloat16()
        gy = torch.randint(-2, 3, (rows, N), generator=g, device="cuda").bfloat16()
        off = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        at = off, dev(np.array(counts, np.int32))
        y, gx = experts.product(x, None, *at), experts.backward_rows(gy, *at)
        lo = counts[0]
        for n0 in (0, N - 300, 21846):  # 21846 rows of the last are past 2^31 bytes
            want = x[lo:].float() @ w[2, n0:n0 + 300].float().t()
            assert torch.equal(y[lo:, n0:n0 + 300], want.bfloat16())
        for c0 in (0, K - 264):
            want = torch.zeros(rows - lo, 264, device="cuda")
            for n0 in range(0, N, 5000):
                want += gy[lo:, n0:n0 + 5000].float() @ w[2, n0:n0 + 5000, c0:c0 + 264].float()
            assert torch.equal(gx[lo:, c0:c0 + 264], want.bfloat16())


def test_rows_past_32_bits():
    """Rows whose values begin past 2^32: 150000 of 32768, two experts of a few
    rows at the ends; their gradients and checkpoint too."""
    cap, K, N, F = 150000, 32768, 24, 16384
    say("rows past 2^32 values")
    counts, off = [3, 70], [0, cap - 70]
    x = torch.zeros(cap, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for lo, n in zip(off, counts):
        x[lo:lo + n] = torch.randint(-2, 3, (n, K), generator=g, device="cuda").bfloat16()
    w = torch.randint(-2, 3, (2, N, K), generator=g, device="cuda").bfloat16()
    gy = torch.zeros(cap, N, dtype=torch.bfloat16, device="cuda")
    gy[:3], gy[cap - 70:] = 1.0, 2.0
    at = dev(np.array(off, np.int32)), dev(np.array(counts, np.int32))
    e = ep.Bf16Experts(w)
    y = e.product(x, None, *at)
    gw = e.backward_weights(x, None, gy, *at, dtype=torch.float32)
    gx = e.backward_rows(gy, *at)
    c = ep.SwigluCheckpoint(cap, F, 2)
    h = c.save(x, *at)
    ggu, h2 = c.backward(h, *at)
    for i, (lo, n) in enumerate(zip(off, counts)):
        assert torch.equal(y[lo:lo + n], (x[lo:lo + n].float() @ w[i].float().t()).bfloat16())
        assert torch.equal(gw[i], gy[lo:lo + n].float().t() @ x[lo:lo + n].float())
        assert torch.equal(gx[lo:lo + n], (gy[lo:lo + n].float() @ w[i].float()).bfloat16())
        gate, up = x[lo:lo + n, :F].double(), x[lo:lo + n, F:].double()
        want = torch.nn.functional.silu(gate) * up
        # integers of 2 bits are kept exactly
        for got in (h, h2):
            d = (got[lo:lo + n].double() - want).abs()
            assert (d <= want.abs() * (UBF16 + 24 * U32)).all()
        want = torch.nn.functional.silu(gate) * h[lo:lo + n].double()
        d = (ggu[lo:lo + n, F:].double() - want).abs()
        assert (d <= want.abs() * (UBF16 + 24 * U32)).all()
