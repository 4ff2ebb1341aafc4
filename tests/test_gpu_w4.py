"""The experts' products with 4-bit weights on the GPU.

Where inputs are small integers and scales powers of two, every sum is exact
in fp32 and the result has to be the bf16 rounding of the exact one, bit for
bit.  Elsewhere a sum of K terms of fp32 is off by at most K half steps of the
sum of magnitudes of what the matrix instruction adds (16 + q in 0..31 for
each |q - z| of the weight), the output by a half step of bf16."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
import ep_workloads as W  # noqa: E402
from tests import moe_reference as ref  # noqa: E402
from tests.gpu_backend import dev, dev_bf16, host_bf16, say  # noqa: E402

U32, UBF16 = ref.U32, ref.UBF16


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16()


def draw(rng, E, K, N, group, zeros, swiglu, exact):
    rows = N * (2 if swiglu else 1)
    q = rng.integers(0, 16, size=(E, rows, K)).astype(np.uint8)
    if exact:
        s = 2.0 ** rng.integers(-3, 2, size=(E, rows, K // group))
    else:
        s = (0.5 + rng.random((E, rows, K // group))) * 0.2 / np.sqrt(K)
    s = bf16(s)
    z = rng.integers(0, 16, size=(E, rows, K // group)).astype(np.uint8) if zeros else None
    return q, s, z


def packed(q, s, z, swiglu):
    return ep.W4Experts.pack(dev(ref.pack_codes(q)), s.cuda(), None if z is None else dev(z),
                             swiglu=swiglu)


def draw_rows(rng, cap, K, fp8, exact):
    """(x on the device, scales on the device or None, the values in 64 bits)"""
    if exact:
        v = rng.integers(-4, 5, size=(cap, K)).astype(np.float64)
    else:
        v = rng.normal(size=(cap, K))
    if not fp8:
        t = bf16(v)
        return t.cuda(), None, t.double().numpy()
    t = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn)
    if exact:
        s = (2.0 ** rng.integers(-2, 3, size=(cap, K // 128))).astype(np.float32)
    else:
        s = (rng.random((cap, K // 128)) + 0.1).astype(np.float32)
    val = t.float().double().numpy() * np.repeat(s.astype(np.float64), 128, axis=1)
    return t.view(torch.uint8).cuda(), dev(s), val


def offsets_of(counts, gap=0):
    return np.concatenate([[0], np.cumsum(np.asarray(counts) + gap)]).astype(np.int32)


SHAPES = [  # E, K, N, group, counts
    (1, 128, 1, 128, [1]), (1, 128, 16, 128, [16]), (2, 256, 17, 128, [3, 0]),
    (3, 32, 40, 32, [0, 1, 17]), (2, 96, 33, 32, [5, 31]), (2, 192, 64, 64, [2, 40]),
    (4, 1024, 100, 64, [0, 0, 7, 1]), (5, 640, 130, 128, [33, 1, 0, 64, 2]),
    (1, 512, 200, 32, [130]), (8, 384, 96, 128, [9, 8, 7, 6, 5, 4, 3, 200]),
]


@pytest.mark.parametrize("E,K,N,group,counts", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_exact_and_rounded(E, K, N, group, counts, fp8, zeros, swiglu):
    if fp8 and K % 128:
        pytest.skip("FP8 rows come in blocks of 128")
    rng = np.random.default_rng(K + N)
    cap = int(sum(counts)) + 2 * E
    off = offsets_of(counts, gap=2)
    for exact in (True, False):
        say(f"product E={E} K={K} N={N} group={group} counts={counts} fp8={fp8} zeros={zeros} "
            f"swiglu={swiglu} exact={exact}")
        q, s, z = draw(rng, E, K, N, group, zeros, swiglu, exact)
        x, xs, xv = draw_rows(rng, cap, K, fp8, exact)
        experts = packed(q, s, z, swiglu)
        out = torch.full((cap, N), 99.0, dtype=torch.bfloat16, device="cuda")
        experts.product(x, xs, dev(off), dev(np.array(counts, np.int32)), out)
        got = out.float().cpu().numpy()
        w = ref.weights(q, s.float().numpy(), z, group)
        rows, _ = ref.product(xv, w, off, counts, swiglu)
        _, size = ref.product(xv, np.repeat(np.abs(s.double().numpy()), group, axis=2) * 32.0, off,
                              counts, swiglu)
        for r in range(cap):
            if r not in rows:
                assert (got[r] == 99.0).all(), f"row {r} is no expert's and was written"
                continue
            want = rows[r]
            if exact and not swiglu:
                assert np.array_equal(got[r], bf16(want).float().numpy()), f"row {r}"
                continue
            e = int(np.searchsorted(off, r, side="right")) - 1
            err = (0 if exact else K + 8) * U32 * size[r]
            if swiglu:
                # y = silu(a) b: silu has a slope of at most 1.1, the function and the
                # two products are off by 12 half steps
                ww = w[e] @ xv[r]
                a, b = ww[:N], ww[N:]
                sil = a / (1 + np.exp(-a))
                err = 1.1 * err[:N] * (np.abs(b) + err[N:]) + np.abs(sil) * err[N:] \
                    if not exact else 0.0
                err = err + 12 * U32 * np.abs(want)
            tol = err + (np.abs(want) + err) * UBF16 + 1e-37
            assert np.all(np.abs(got[r] - want) <= tol), (r, np.max(np.abs(got[r] - want) / tol))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K,N,counts", [(7168, 512, [4, 0, 1, 30]), (2048, 1000, [70, 129, 3, 0])])
def test_product_long_sums(fp8, K, N, counts):
    """At the sizes of a model: rounding to bf16 alone gives at most 2^-8 of the
    result's norm, and sums of random signs add next to nothing."""
    rng = np.random.default_rng(K)
    q, s, _ = draw(rng, 4, K, N, 128, False, False, False)
    cap = sum(counts)
    off = offsets_of(counts)
    x, xs, xv = draw_rows(rng, cap, K, fp8, False)
    say(f"long sums K={K} N={N} fp8={fp8}")
    out = packed(q, s, None, False).product(x, xs, dev(off), dev(np.array(counts, np.int32)))
    rows, _ = ref.product(xv, ref.weights(q, s.float().numpy(), None, 128), off, counts, False)
    want = np.stack([rows[r] for r in range(cap)])
    d = np.linalg.norm(out.float().cpu().numpy() - want, axis=1)
    assert np.all(d <= UBF16 * np.linalg.norm(want, axis=1))


def test_pack_matches_the_layout():
    """ep_w4_pack against the layout's definition, nibble by nibble."""
    rng = np.random.default_rng(1)
    for E, K, N, group, swiglu in ((2, 160, 19, 32, True), (1, 256, 16, 128, False),
                                   (3, 64, 5, 64, True)):
        q, s, z = draw(rng, E, K, N, group, True, swiglu, True)
        halves = 2 if swiglu else 1
        say(f"pack E={E} K={K} N={N} group={group}")
        p = packed(q, s, z, swiglu)
        assert np.array_equal(p.w_codes.cpu().numpy(), ref.tile_codes(q, halves))
        n16, G = -(-N // 16), K // group

        def tiles(v):
            full = np.zeros((E, halves, n16 * 16, G), v.dtype)
            full[:, :, :N] = v.reshape(E, halves, N, G)
            return full.reshape(E, halves, n16, 16, G).transpose(0, 1, 2, 4, 3)

        assert np.array_equal(host_bf16(p.w_scales), tiles(host_bf16(s)))
        assert np.array_equal(p.w_zeros.cpu().numpy(), tiles(z))


def test_every_code_and_row_value():
    """Each of the 16 codes against each power of two and each FP8 code, one
    product at a time: exact, subnormal codes included."""
    K, N = 128, 16
    q = np.broadcast_to(np.arange(16, dtype=np.uint8)[None, :, None], (1, N, K)).copy()
    s = bf16(np.ones((1, N, 1)))
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    x = np.zeros((len(codes), K), np.uint8)
    x[np.arange(len(codes)), np.arange(len(codes)) % K] = codes
    say("every FP8 code")
    out = packed(q, s, None, False).product(dev(x), torch.ones(len(codes), 1, device="cuda"),
                                            dev(np.array([0], np.int32)),
                                            dev(np.array([len(codes)], np.int32)))
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    want = bf16(v[:, None] * (np.arange(16) - 8)[None]).float().numpy()
    assert np.array_equal(out.float().cpu().numpy(), want)
    pw = np.arange(-100, 100)
    xb = np.zeros((len(pw), K), np.float32)
    xb[np.arange(len(pw)), np.arange(len(pw)) % K] = 2.0 ** pw
    say("powers of two")
    out = packed(q, s, None, False).product(bf16(xb).cuda(), None, dev(np.array([0], np.int32)),
                                            dev(np.array([len(pw)], np.int32)))
    assert np.array_equal(out.float().cpu().numpy(),
                          (2.0 ** pw)[:, None] * (np.arange(16) - 8)[None])


def test_rows_past_the_capacity_and_bad_offsets_are_left_alone():
    rng = np.random.default_rng(2)
    E, K, N = 4, 128, 32
    q, s, _ = draw(rng, E, K, N, 128, False, False, True)
    p = packed(q, s, None, False)
    x, _, xv = draw_rows(rng, 10, K, False, True)
    out = torch.full((14, N), 5.0, dtype=torch.bfloat16, device="cuda")
    off, cnt = [0, 4, -3, 2 ** 31 - 1], [3, 100, 5, 7]
    say("rows past the capacity")
    p.product(x, None, dev(np.array(off, np.int32)), dev(np.array(cnt, np.int32)), out)
    got = out.float().cpu().numpy()
    rows, _ = ref.product(xv, ref.weights(q, s.float().numpy(), None, 128), [0, 4], [3, 100],
                          False)
    assert sorted(rows) == [0, 1, 2] + list(range(4, 10))
    for r in range(14):
        if r in rows:
            assert np.array_equal(got[r], bf16(rows[r]).float().numpy())
        else:
            assert (got[r] == 5.0).all()
    say("no rows at all")
    p.product(x[:0], None, dev(np.array(off, np.int32)), dev(np.array(cnt, np.int32)), out)
    p.product(x, None, dev(np.zeros(4, np.int32)), dev(np.zeros(4, np.int32)), out)
    assert np.array_equal(out.float().cpu().numpy(), got)


def test_python_refusals():
    rng = np.random.default_rng(3)
    q, s, _ = draw(rng, 2, 128, 32, 128, False, False, True)
    p = packed(q, s, None, False)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x[:, :64]), dict(x=x.float()), dict(off=off[:1]), dict(cnt=off[:1]),
                dict(out=out[:3]), dict(out=out.float()), dict(x=x.t().contiguous().t()),
                dict(xs=torch.ones(4, 1, device="cuda")), dict(cnt=off.long()),
                dict(x=x.cpu())):
        a = dict(x=x, xs=None, off=off, cnt=off, out=out)
        a.update(bad)
        with pytest.raises(ValueError):
            p.product(a["x"], a["xs"], a["off"], a["cnt"], a["out"])


# --------------------------------------------------------------------------
# The operators together, as a layer uses them
# --------------------------------------------------------------------------

def layer_inputs(rng, T, H, E, inner):
    x = W.normal_bf16(rng, (T, H))
    centroids = (rng.normal(size=(H, E)) / np.sqrt(H)).astype(np.float32)
    q1, s1, _ = draw(rng, E, H, inner, 128, False, True, False)
    q2, s2, z2 = draw(rng, E, inner, H, 64, True, False, False)
    return x, centroids, (q1, s1), (q2, s2, z2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_layer_forward(T, fp8):
    """route -> layout -> dispatch -> gate/up with SwiGLU -> down -> combine,
    all on the device without a synchronisation, against the same in 64 bits
    from the rounded intermediate rows."""
    rng = np.random.default_rng(T)
    H, E, k, R, inner, A = 256, 16, 4, 4, 192, 4
    x, cen, (q1, s1), (q2, s2, z2) = layer_inputs(rng, T, H, E, inner)
    xd = dev_bf16(x)
    logits = xd.float() @ dev(cen)
    mask = np.ones(T, np.uint8)
    mask[T // 2:T // 2 + T // 8] = 0
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    router = ep.EpRouter(T, E, k, score="sigmoid", groups=4, topk_groups=2, group_topn=2,
                         scale=2.5)
    b = ep.EpBuffers(T, H, k, E, R, A, fp8=fp8)
    up, down = packed(q1, s1, None, True), packed(q2, s2, z2, False)
    mid = torch.zeros(b.capacity, inner, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(b.capacity, H, dtype=torch.bfloat16, device="cuda")
    say(f"layer T={T} fp8={fp8}")
    idx, w = router.route(logits, bias=dev(bias), token_mask=dev(mask))
    b.layout(idx)
    b.dispatch(xd, idx, w)
    b.expert_product(up, out=mid)
    b.expert_product(down, x=mid, out=y)
    out = b.combine(y, w).float().cpu().numpy()
    b.check_status()
    router.check_status()
    ids, ww, _ = ref.route(logits.cpu().numpy(), k, "sigmoid", bias, mask, 4, 2, 2, True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ids)
    off, cnt = b.expert_offsets.cpu().numpy(), b.num_tokens_per_expert.cpu().numpy()
    if fp8:
        xv = b.recv_x.view(torch.float8_e4m3fn).float().cpu().double().numpy() * np.repeat(
            b.recv_scales.cpu().double().numpy(), 128, axis=1)
    else:
        xv = b.recv_x.cpu().double().numpy()
    w1 = ref.weights(q1, s1.float().numpy(), None, 128)
    w2 = ref.weights(q2, s2.float().numpy(), z2, 64)
    rows, _ = ref.product(xv, w1, off, cnt, True)
    m = mid.cpu().double().numpy()
    for r, want in rows.items():
        assert np.linalg.norm(m[r] - want) <= UBF16 * np.linalg.norm(want)
    rows, _ = ref.product(m, w2, off, cnt, False)
    yy = y.cpu().double().numpy()
    for r, want in rows.items():
        assert np.linalg.norm(yy[r] - want) <= UBF16 * np.linalg.norm(want)
    slot = b.tok_slot_row.cpu().numpy()
    for t in range(T):
        want = np.zeros(H)
        big = np.zeros(H)
        for j in range(k):
            if slot[t, j] >= 0:
                want += ww[t, j] * yy[slot[t, j]]
                big += np.abs(ww[t, j] * yy[slot[t, j]])
        # gates within 60 half steps, a sum of k terms, one rounding
        assert np.all(np.abs(out[t] - want) <= UBF16 * np.abs(want) + big * (64 + k) * U32 * 2)


def test_one_rank_at_a_time():
    """Each rank's weights on its own rows give what all weights give at once."""
    rng = np.random.default_rng(11)
    T, H, E, k, R = 50, 128, 8, 3, 4
    idx = dev(W.random_routes(rng, T, E, k, 0.1))
    b = ep.EpBuffers(T, H, k, E, R, 2)
    b.layout(idx)
    b.dispatch(dev_bf16(W.normal_bf16(rng, (T, H))), idx, None)
    q, s, _ = draw(rng, E, H, 48, 128, False, False, False)
    whole = torch.zeros(b.capacity, 48, dtype=torch.bfloat16, device="cuda")
    parts = torch.zeros_like(whole)
    b.expert_product(packed(q, s, None, False), out=whole)
    for r in range(R):
        b.expert_product(packed(q[2 * r:2 * r + 2], s[2 * r:2 * r + 2], None, False), out=parts,
                         rank=r)
    assert torch.equal(whole, parts) and whole.abs().sum() > 0
    with pytest.raises(ValueError):
        b.expert_product(packed(q, s, None, False), rank=R)


def test_training_step():
    """Forward and backward of the path with the router: the gates' gradient of
    combine_backward and the balance loss reach the logits."""
    rng = np.random.default_rng(12)
    T, H, E, k, R = 60, 64, 8, 3, 2
    x, xl = W.normal_bf16(rng, (T, H)), rng.normal(size=(T, E)).astype(np.float32)
    offsets = np.array([0, 25, T], np.int32)
    router = ep.EpRouter(T, E, k, max_seqs=2)
    b = ep.EpBuffers(T, H, k, E, R)
    logits = dev(xl)
    idx, w = router.route(logits)
    loss = router.balance_loss(logits, idx, 0.1, seq_offsets=dev(offsets))
    b.layout(idx)
    b.dispatch(dev_bf16(x), idx, w)
    b.combine(b.recv_x, w)  # experts that return their rows
    gout = dev_bf16(W.normal_bf16(rng, (T, H)))
    gw = torch.empty(T, k, device="cuda")
    b.combine_backward(gout, w, b.recv_x, grad_weights=gw)
    g = router.backward(logits, idx, gw, prob_grad=router.prob_grad, seq_offsets=dev(offsets),
                        grad_loss=torch.ones(1, device="cuda"))
    b.check_status()
    router.check_status()
    ids = idx.cpu().numpy()
    want, size = ref.grad(xl, ids, gw.cpu().numpy(), "softmax", True, 1.0,
                          router.prob_grad.cpu().numpy(), offsets)
    assert np.all(np.abs(g.cpu().numpy() - want) <= size * 120 * U32)
    assert np.isclose(loss.item(), ref.balance(xl, ids, 0.1, "softmax", offsets)[0], rtol=1e-5)
    per_expert = router.counts.sum(dim=0).to(torch.int32)
    assert torch.equal(per_expert, b.num_tokens_per_expert)


def test_layer_in_a_graph():
    """The whole layer captured once and replayed on new inputs, with eager
    calls between, two graphs of two routers and buffers among them."""
    rng = np.random.default_rng(13)
    T, H, E, k, R, inner = 24, 256, 16, 4, 4, 128
    x, cen, (q1, s1), (q2, s2, z2) = layer_inputs(rng, T, H, E, inner)
    up, down = packed(q1, s1, None, True), packed(q2, s2, z2, False)
    offsets = dev(np.array([0, 10, T], np.int32))

    def build():
        st = dict(x=torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"),
                  logits=torch.zeros(T, E, device="cuda"),
                  gw=torch.zeros(T, k, device="cuda"))
        st["router"] = ep.EpRouter(T, E, k, score="sigmoid", max_seqs=2)
        st["b"] = ep.EpBuffers(T, H, k, E, R)
        st["mid"] = torch.zeros(st["b"].capacity, inner, dtype=torch.bfloat16, device="cuda")
        st["y"] = torch.zeros(st["b"].capacity, H, dtype=torch.bfloat16, device="cuda")
        return st

    def step(st):
        r, b = st["router"], st["b"]
        idx, w = r.route(st["logits"])
        r.balance_loss(st["logits"], idx, 0.1, seq_offsets=offsets)
        b.layout(idx)
        b.dispatch(st["x"], idx, w)
        b.expert_product(up, out=st["mid"])
        b.expert_product(down, x=st["mid"], out=st["y"])
        b.combine(st["y"], w)
        r.backward(st["logits"], idx, st["gw"], prob_grad=r.prob_grad, seq_offsets=offsets)

    def outputs(st):
        r, b = st["router"], st["b"]
        return [v.clone() for v in (r.topk_idx, r.topk_weights, r.loss, r.counts, r.mean_probs,
                                    r.prob_grad, b.out, r.grad_logits)]

    def fill(st, seed):
        g = np.random.default_rng(seed)
        st["x"].copy_(dev_bf16(W.normal_bf16(g, (T, H))))
        st["logits"].copy_(dev(g.normal(size=(T, E)).astype(np.float32)))
        st["gw"].copy_(dev(g.normal(size=(T, k)).astype(np.float32)))

    states = [build(), build()]
    eager = build()
    graphs = []
    for i, st in enumerate(states):
        fill(st, i)
        step(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        say(f"capture {i}")
        with torch.cuda.graph(g):
            step(st)
        graphs.append(g)
    for n in range(4):
        say(f"replay {n}")
        for i, (g, st) in enumerate(zip(graphs, states)):
            fill(st, 10 * n + i)
            g.replay()
        torch.cuda.synchronize()
        for i, st in enumerate(states):
            got = outputs(st)
            fill(eager, 10 * n + i)
            step(eager)
            torch.cuda.synchronize()
            for a, c in zip(got, outputs(eager)):
                assert torch.equal(a, c)
            st["b"].check_status()
            st["router"].check_status()


def test_two_streams_and_repeats_are_bit_equal():
    """Calls of separate buffers on two streams at once, and repeated calls."""
    rng = np.random.default_rng(14)
    E, K, N = 8, 512, 160
    q, s, _ = draw(rng, E, K, N, 128, False, True, False)
    p = packed(q, s, None, True)
    cnt = np.array([5, 0, 40, 1, 17, 16, 2, 33], np.int32)
    off = dev(offsets_of(cnt))
    x, _, _ = draw_rows(rng, int(cnt.sum()), K, False, False)
    T, G = 500, 64
    logits = dev(rng.normal(size=(T, G)).astype(np.float32))
    cnt = dev(cnt)
    first = p.product(x, None, off, cnt)
    r0 = ep.EpRouter(T, G, 6)
    r0.balance_loss(logits, r0.route(logits)[0], 1.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    routers = [ep.EpRouter(T, G, 6) for _ in streams]
    outs = [[] for _ in streams]
    for _ in range(3):
        for i, (st, r) in enumerate(zip(streams, routers)):
            with torch.cuda.stream(st):
                outs[i].append(p.product(x, None, off, cnt))
                r.balance_loss(logits, r.route(logits)[0], 1.0)
    torch.cuda.synchronize()
    for i, r in enumerate(routers):
        for o in outs[i]:
            assert torch.equal(o, first)
        assert torch.equal(r.topk_idx, r0.topk_idx) and torch.equal(r.loss, r0.loss)
        assert torch.equal(r.mean_probs, r0.mean_probs)


def test_weights_are_those_of_the_object():
    """Rewritten in place they are used, and no other tensor can take their place."""
    rng = np.random.default_rng(21)
    q = rng.integers(0, 256, size=(2, 48, 32), dtype=np.uint8)
    s = torch.ones(2, 48, 1, dtype=torch.bfloat16)
    w = ep.W4Experts.pack(dev(q), s.cuda())
    x = torch.from_numpy(rng.integers(-4, 5, size=(5, 64)).astype(np.float32)).bfloat16().cuda()
    off, cnt = dev(np.array([0, 3], np.int32)), dev(np.array([3, 2], np.int32))
    first = w.product(x, None, off, cnt).float().cpu()
    with pytest.raises(AttributeError):
        w.w_codes = w.w_codes.clone()
    w.w_scales.mul_(2)  # exact in bf16
    assert torch.equal(w.product(x, None, off, cnt).float().cpu(), 2 * first)
    with pytest.raises(ep.EpError):  # rows written over those that others still read
        w2 = ep.W4Experts.pack(dev(q[:, :, :]), s.cuda())
        buf = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
        w2.product(buf, None, off, cnt, out=buf.view(-1)[:240].view(5, 48))


def test_many_experts_of_few_rows():
    """Enough experts and columns that 17 to 32 rows are tiled, beside experts
    of fewer rows, of more and of none: exact sums."""
    E, K, N, group = 96, 64, 4200, 64
    rng = np.random.default_rng(22)
    counts = rng.integers(15, 34, size=E)
    counts[[3, 50]] = 0
    counts[[4, 60, 95]] = [1, 16, 32]
    counts[[5, 70]] = [70, 130]
    off = offsets_of(counts)
    cap = int(off[-1]) - 3  # the last expert's last rows are cut off
    assert min(cap // 16, E) * -(-(-(-N // 16)) // 8) >= 4 * 768
    q, s, _ = draw(rng, E, K, N, group, False, False, True)
    x, _, xv = draw_rows(rng, cap, K, False, True)
    say("many experts of few rows")
    out = packed(q, s, None, False).product(x, None, dev(off), dev(counts.astype(np.int32)))
    w = ref.weights(q, s.float().numpy(), None, group)
    got = out.float().cpu().numpy()
    for e in range(E):
        lo, hi = off[e], min(off[e + 1], cap)
        want = bf16(xv[lo:hi] @ w[e].T).float().numpy()
        assert np.array_equal(got[lo:hi], want), e


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_past_32_bits(fp8):
    """Experts whose rows of x lie past 2^32 values, and one whose output does.
    Sums are exact: whole steps of 2^-5, and 7168 terms of random signs of at
    most 256 (their mean square 30^2) stay far below the 2^19 that fp32 holds of
    such steps."""
    K, N = 7168, 1024
    cap = (1 << 32) // N + 200
    off = np.array([0, cap - 150, cap - 90, cap - 20], np.int32)
    cnt = np.array([3, 9, 50, 30], np.int32)  # the last is cut off
    rng = np.random.default_rng(23)
    q, s, _ = draw(rng, 4, K, N, 128, False, False, True)
    rows = np.concatenate([np.arange(o, min(o + c, cap)) for o, c in zip(off, cnt)])
    x, xs, xv = draw_rows(rng, len(rows), K, fp8, True)
    at = torch.from_numpy(rows).cuda()
    say(f"rows past 32 bits fp8={fp8}")
    big = torch.zeros((cap, K), dtype=x.dtype, device="cuda")
    big[at] = x
    scales = None
    if fp8:
        scales = torch.ones((cap, K // 128), device="cuda")
        scales[at] = xs
    out = torch.zeros((cap, N), dtype=torch.bfloat16, device="cuda")
    packed(q, s, None, False).product(big, scales, dev(off), dev(cnt), out)
    got = out[at].float().cpu().numpy()
    w = ref.weights(q, s.float().numpy(), None, 128)
    e = np.searchsorted(off, rows, side="right") - 1
    for i in range(len(rows)):
        want = w[e[i]] @ xv[i]
        assert np.array_equal(got[i], bf16(want).float().numpy()), rows[i]
    out[at] = 0
    assert not bool(out.any())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows", [7, 130])
def test_fp8_sums_keep_small_terms(group, zeros, rows):
    """In every 128 columns one code of 448, whose weights are zero (code and
    zero point equal), beside codes of n 2^-9, |n| <= 15: the result is made of
    terms 2^15 and more below the largest that is summed.  It is exact: the sums
    are of x (16 + q) / 16, whole steps of 2^-13, the large one at most
    448 x 31 / 16 = 868 and the others together 127 x 15 x 31 steps, below 2^23
    steps in all."""
    rng = np.random.default_rng(31)
    K, N = 384, 48
    v = rng.integers(-15, 16, size=(rows, K)) * 2.0 ** -9
    at = 128 * np.arange(K // 128) + rng.integers(0, 128, size=K // 128)
    v[:, at] = 448.0 * rng.choice([-1.0, 1.0], size=(rows, len(at)))
    q = rng.integers(0, 16, size=(1, N, K)).astype(np.uint8)
    z = rng.integers(0, 16, size=(1, N, K // group)).astype(np.uint8) if zeros else None
    q[:, :, at] = 8 if z is None else z[:, :, at // group]
    s = bf16(np.ones((1, N, K // group)))
    x = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(x.double().numpy(), v)
    say(f"fp8 sums group={group} zeros={zeros} rows={rows}")
    out = packed(q, s, z, False).product(x.view(torch.uint8).cuda(),
                                         torch.ones(rows, K // 128, device="cuda"),
                                         dev(np.array([0], np.int32)),
                                         dev(np.array([rows], np.int32)))
    want = v @ ref.weights(q, s.float().numpy(), z, group)[0].T
    assert np.array_equal(out.float().cpu().numpy(), bf16(want).float().numpy())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [5, 70])
def test_product_over_the_whole_range(group, zeros, fp8, rows):
    """Rows at the top and the bottom of their types and scales that bring the
    result back: finite wherever the result is.  Exact: rows are one power of
    two with any signs and each matrix has one scale, so a sum is at most
    256 x 31 steps of a power of two."""
    rng = np.random.default_rng(41)
    K, N = 256, 40
    if fp8:  # power of the codes, of the rows' scales, of the weights' scales
        cases = [(8, 119, -30), (-9, 115, 12), (8, -110, 120), (-9, -60, 100), (8, -126, 20)]
    else:
        cases = [(127, 0, -30), (127, 0, -120), (-100, 0, 120), (-126, 0, 126), (-133, 0, 100),
                 (0, 0, 110), (0, 0, -110)]
    q = rng.integers(0, 16, size=(1, N, K)).astype(np.uint8)
    z = rng.integers(0, 16, size=(1, N, K // group)).astype(np.uint8) if zeros else None
    sign = rng.choice([-1.0, 1.0], size=(rows, K))
    off, cnt = dev(np.array([0], np.int32)), dev(np.array([rows], np.int32))
    for px, ps, pw in cases:
        say(f"range group={group} zeros={zeros} fp8={fp8} rows={rows} powers={px, ps, pw}")
        v = torch.from_numpy(sign * 2.0 ** px)
        x, xs = v.to(torch.bfloat16), None
        if fp8:
            x = v.to(torch.float8_e4m3fn)
            xs = torch.full((rows, K // 128), 2.0 ** ps, device="cuda")
        assert torch.equal(x.double(), v)
        s = torch.full((1, N, K // group), 2.0 ** pw).to(torch.bfloat16)
        out = packed(q, s, z, False).product((x.view(torch.uint8) if fp8 else x).cuda(), xs, off,
                                             cnt)
        w = ref.weights(q, s.double().numpy(), z, group)[0]
        want = torch.from_numpy((sign @ w.T) * 2.0 ** (px + ps)).to(torch.bfloat16)
        assert bool(torch.isfinite(want).all())
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_weights_past_the_cache(fp8, group, zeros, swiglu):
    """Weights of more than 256 MiB, which are read past the caches: experts of
    no row, of one, of a full row tile and of two, and one that is tiled.  The
    matrices repeat after 64 rows, so that the reference stays small: exact, as
    every repetition of the columns has to be."""
    rng = np.random.default_rng(71)
    E, K, N = 12, 8192, 3200 if swiglu else 6400
    halves = 2 if swiglu else 1
    counts = [1, 0, 3, 16, 1, 0, 17, 33, 0, 2, 32, 1]
    off = offsets_of(counts)
    cap = int(off[-1])
    assert min(cap, E) * halves * -(-N // 16) * (K // 128) * 1024 > 1 << 28
    base = rng.integers(0, 16, size=(E, halves, 64, K)).astype(np.uint8)
    s = 2.0 ** rng.integers(-3, 2, size=(E, halves, 64, K // group))
    z = rng.integers(0, 16, size=(E, halves, 64, K // group)).astype(np.uint8) if zeros else None

    def whole(v, dtype):
        t = torch.from_numpy(v).cuda().to(dtype)
        return t.repeat(1, 1, N // 64, 1).reshape(E, halves * N, -1)

    codes = whole(ref.pack_codes(base), torch.uint8)
    say(f"weights past the cache fp8={fp8} group={group} zeros={zeros} swiglu={swiglu}")
    w = ep.W4Experts.pack(codes, whole(s, torch.bfloat16),
                          None if z is None else whole(z, torch.uint8), swiglu=swiglu)
    del codes
    x, xs, xv = draw_rows(rng, cap, K, fp8, True)
    out = w.product(x, xs, dev(off), dev(np.array(counts, np.int32)))
    got = out.float().cpu().numpy().reshape(cap, N // 64, 64)
    assert (got == got[:, :1]).all()
    small = ref.weights(base.reshape(E, halves * 64, K), s.reshape(E, halves * 64, -1),
                        None if z is None else z.reshape(E, halves * 64, -1), group)
    rows, _ = ref.product(xv, small, off, counts, swiglu)
    want = np.stack([rows[r] for r in range(cap)])
    if swiglu:  # silu and two products: 12 half steps, then the output's rounding
        assert np.all(np.abs(got[:, 0] - want) <= np.abs(want) * (UBF16 + 13 * U32) + 1e-37)
    else:
        assert np.array_equal(got[:, 0], bf16(want).float().numpy())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_few_rows_tiled(fp8, group, zeros, swiglu):
    """48 experts wide enough that 17 to 32 rows are tiled, beside experts that
    are streamed: exact sums, the matrices repeating after 40 rows."""
    rng = np.random.default_rng(91)
    E, K, N = 48, 256, 4200 if swiglu else 8400
    halves = 2 if swiglu else 1
    counts = [17, 32, 16, 1, 0, 24, 31, 33, 18, 15, 64, 2, 20, 0, 65, 17] * 3
    off = offsets_of(counts, gap=1)
    cap = int(off[-1]) - 1
    assert min(cap // 16, E) * -(-(halves * -(-N // 16)) // 8) >= 4 * 768
    base = rng.integers(0, 16, size=(E, halves, 40, K)).astype(np.uint8)
    s = 2.0 ** rng.integers(-3, 2, size=(E, halves, 40, K // group))
    z = rng.integers(0, 16, size=(E, halves, 40, K // group)).astype(np.uint8) if zeros else None

    def whole(v, dtype):
        t = torch.from_numpy(v).cuda().to(dtype)
        return t.repeat(1, 1, N // 40, 1).reshape(E, halves * N, -1)

    say(f"few rows tiled fp8={fp8} group={group} zeros={zeros} swiglu={swiglu}")
    w = ep.W4Experts.pack(whole(ref.pack_codes(base), torch.uint8), whole(s, torch.bfloat16),
                          None if z is None else whole(z, torch.uint8), swiglu=swiglu)
    x, xs, xv = draw_rows(rng, cap, K, fp8, True)
    out = torch.full((cap, N), 99.0, dtype=torch.bfloat16, device="cuda")
    w.product(x, xs, dev(off), dev(np.array(counts, np.int32)), out)
    got = out.float().cpu().numpy().reshape(cap, N // 40, 40)
    assert (got == got[:, :1]).all()
    small = ref.weights(base.reshape(E, halves * 40, K), s.reshape(E, halves * 40, -1),
                        None if z is None else z.reshape(E, halves * 40, -1), group)
    rows, _ = ref.product(xv, small, off, counts, swiglu)
    for r in range(cap):
        if r not in rows:
            assert (got[r] == 99.0).all(), r
        elif swiglu:
            tol = np.abs(rows[r]) * (UBF16 + 13 * U32) + 1e-37
            assert np.all(np.abs(got[r, 0] - rows[r]) <= tol), r
        else:
            assert np.array_equal(got[r, 0], bf16(rows[r]).float().numpy()), r


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_that_are_not_finite_keep_to_themselves(fp8, swiglu):
    """NaN and infinities in some rows, the last of an expert's among them: their
    outputs are not finite, all others are as they were."""
    rng = np.random.default_rng(101)
    E, K, N = 3, 256, 40
    q, s, z = draw(rng, E, K, N, 128, True, swiglu, False)
    counts = [5, 17, 70]
    off = offsets_of(counts)
    x, xs, _ = draw_rows(rng, 92, K, fp8, False)
    w = packed(q, s, z, swiglu)
    o, c = dev(off), dev(np.array(counts, np.int32))
    say(f"rows that are not finite fp8={fp8} swiglu={swiglu}")
    want = w.product(x, xs, o, c)
    rows = [0, 4, 6, 20, 21, 50, 91]
    for i, r in enumerate(rows):
        if not fp8:
            x[r, 37 * i % K] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        elif i % 2:
            x[r, 37 * i % K] = 0x7F | (0x80 if i % 4 == 1 else 0)
        else:
            xs[r, i % 2] = (float("nan"), float("inf"))[i % 4 // 2]
    got = w.product(x, xs, o, c)
    bad = torch.zeros(92, dtype=torch.bool)
    bad[rows] = True
    bad = bad.cuda()
    assert not bool(torch.isfinite(got[bad]).any())
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("zeros", [False, True])
def test_weights_with_another_storage(zeros):
    """The packed tensors' storage may be replaced between calls, also by way of
    the host; what does not fit is refused."""
    rng = np.random.default_rng(51)
    E, K, N, counts = 2, 256, 48, [3, 20]
    q, s, z = draw(rng, E, K, N, 128, zeros, False, True)
    x, _, _ = draw_rows(rng, sum(counts), K, False, True)
    at = dev(offsets_of(counts)), dev(np.array(counts, np.int32))
    w = packed(q, s, z, False)
    say(f"4-bit weights with another storage zeros={zeros}")
    want = w.product(x, None, *at)
    kept = [t for t in (w.w_codes, w.w_scales, w.w_zeros) if t is not None]
    olds = [t.data for t in kept]
    for t in kept:
        t.data = t.cpu()
    with pytest.raises(ValueError):
        w.product(x, None, *at)
    for t, old in zip(kept, olds):
        t.data = t.cuda()
        old.zero_()
    assert torch.equal(w.product(x, None, *at), want)
    for t in kept:
        was = t.data
        for other in (was[:1], was.transpose(2, 3)):
            t.data = other
            with pytest.raises(ValueError):
                w.product(x, None, *at)
        t.data = was
    assert torch.equal(w.product(x, None, *at), want)
