"""The router, its balance loss and their gradient on the GPU against the
plain 64-bit implementations of tests/moe_reference.py.

Tolerances, in half steps of fp32 (2^-24): an exponential of x - m is off by
2 (the function) and |x - m| (the argument's rounding), a score or weight made
of two of them, a sum of up to 2^10 terms in a tree (10 + 6), a quotient and
a product by  2 (2 + |x - m|) + 18;  a sum over tokens adds one per addition."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
from tests import moe_reference as ref  # noqa: E402
from tests.gpu_backend import dev, say  # noqa: E402

U32, UBF16 = ref.U32, ref.UBF16


def draw_logits(rng, T, E, bf16, spread=1.5):
    x = (rng.normal(size=(T, E)) * spread).astype(np.float32)
    t = torch.from_numpy(x)
    if bf16:
        t = t.bfloat16()
    return t.float().numpy(), t


def score_steps(x):
    """Half steps a weight or probability of each row may be off by.  Distances
    count up to 110: exp(-110) < 2e-48, so a term further off is zero within
    the absolute 1e-37 that every comparison allows (fp32 holds no more of it)."""
    fin = np.where(np.isfinite(x), x, 0.0).astype(np.float64)
    d = np.minimum(np.abs(fin - fin.max(axis=1, keepdims=True)), 110) + np.minimum(
        np.abs(fin).max(axis=1, keepdims=True), 110)
    return 2 * (2 + d.max(axis=1)) + 18


def check_route(got, x, k, **kw):
    idx, w = got[0].cpu().numpy(), got[1].cpu().numpy()
    ids, ww, bad = ref.route(x, k, **kw)
    assert np.array_equal(idx, ids)
    tol = np.abs(ww) * (score_steps(x) * U32)[:, None] + 1e-37
    assert np.all(np.abs(w - ww) <= tol), np.max(np.abs(w - ww) / tol)
    return bad


SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 8, 8), (17, 60, 4), (33, 64, 6), (16, 65, 5),
         (40, 100, 32), (64, 128, 8), (31, 200, 7), (129, 256, 8), (9, 257, 9), (12, 512, 16),
         (7, 1000, 32), (4, 1024, 10)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_sizes(T, E, k, score, bf16):
    rng = np.random.default_rng(T * 1000 + E)
    x, t = draw_logits(rng, T, E, bf16)
    for normalize, scale in ((True, 1.0), (False, 2.5)):
        say(f"route T={T} E={E} k={k} {score} bf16={bf16} normalize={normalize}")
        r = ep.EpRouter(T, E, k, score=score, normalize=normalize, scale=scale,
                        logits_dtype=t.dtype)
        got = r.route(t.cuda())
        r.check_status()
        check_route(got, x, k, score=score, normalize=normalize, scale=scale)


@pytest.mark.parametrize("E,G,tg,topn,k", [(8, 2, 1, 1, 3), (8, 8, 3, 2, 3), (60, 5, 2, 2, 6),
                                           (64, 8, 4, 1, 6), (64, 64, 9, 2, 9), (96, 3, 1, 2, 32),
                                           (128, 16, 4, 2, 8), (256, 8, 4, 1, 8),
                                           (256, 8, 4, 2, 8), (256, 64, 7, 2, 8), (320, 5, 2, 2, 8),
                                           (1024, 32, 4, 1, 12), (1024, 2, 1, 2, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_groups_and_bias(E, G, tg, topn, k, score, biased, bf16):
    T = 37
    rng = np.random.default_rng(E * 100 + G)
    x, t = draw_logits(rng, T, E, bf16)
    bias = (rng.normal(size=E) * 0.1).astype(np.float32) if biased else None
    say(f"route groups E={E} G={G} keep={tg} topn={topn} {score} bias={biased} bf16={bf16}")
    r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn,
                    logits_dtype=t.dtype)
    got = r.route(t.cuda(), bias=None if bias is None else dev(bias))
    r.check_status()
    check_route(got, x, k, score=score, bias=bias, groups=G, topk_groups=tg, group_topn=topn)


def test_route_ties_go_to_the_lowest_index():
    """Equal logits, equal keys, and keys that 32 bits cannot tell apart."""
    T, E, k = 6, 256, 8
    x = np.zeros((T, E), np.float32)
    x[1] = np.repeat(np.arange(E // 4, dtype=np.float32) % 3, 4)
    x[2, ::2] = -0.0
    x[3] = np.float32(1) + (np.arange(E) % 5).astype(np.float32) * np.float32(2 ** -23)
    x[4] = 30 + (np.arange(E) % 7).astype(np.float32) * np.float32(2 ** -19)  # sigmoid ~ 1
    x[5] = -np.finfo(np.float32).max
    for score in ("softmax", "sigmoid"):
        for bias in (None, np.zeros(E, np.float32)):
            for G, tg, topn in ((1, 1, 1), (8, 4, 2), (16, 3, 1)):
                say(f"ties {score} bias={bias is not None} G={G}")
                r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn,
                                normalize=False)
                idx, w = r.route(dev(x), bias=None if bias is None else dev(bias))
                r.check_status()
                ids, _, _ = ref.route(x, k, score, bias, groups=G, topk_groups=tg,
                                      group_topn=topn, normalize=False)
                assert np.array_equal(idx.cpu().numpy(), ids)


def test_route_close_keys():
    """Scores that 32 bits round together, in and across groups: every token is
    decided in 64 bits.  Logits a few units of the last place apart, at the
    flat end of the sigmoid and in the middle of a softmax."""
    rng = np.random.default_rng(17)
    for E, G, tg, topn, k in ((64, 1, 1, 1, 8), (64, 8, 3, 2, 6), (256, 8, 4, 2, 8),
                              (100, 5, 2, 1, 12), (512, 16, 4, 2, 7), (1024, 8, 3, 2, 32),
                              (16, 4, 2, 2, 3)):
        T = 23
        base = np.float32(4.0) + rng.integers(-6, 7, size=(T, E)).astype(np.float32) * np.float32(
            2.0 ** -20)
        x = np.where(rng.random((T, E)) < 0.3, base, rng.normal(size=(T, E))).astype(np.float32)
        bias = np.where(rng.random(E) < 0.5, 0, rng.integers(-2, 3, size=E) * 2.0 ** -23).astype(
            np.float32)
        for score in ("sigmoid", "softmax"):
            for b in (None, bias, bias + np.float32(0.25)):
                say(f"close keys E={E} G={G} {score} bias={b is not None}")
                r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn)
                got = r.route(dev(x), bias=None if b is None else dev(b))
                r.check_status()
                check_route(got, x, k, score=score, bias=b, groups=G, topk_groups=tg,
                            group_topn=topn)


def test_route_bias_of_the_lowest_value():
    """Experts and whole groups put last by a bias of the type's lowest value,
    beside logits of -inf: the sums of two such keys pass the 32-bit range, and
    those experts still come before those that cannot be selected."""
    rng = np.random.default_rng(18)
    low = np.finfo(np.float32).min
    for E, G, tg, topn, k in ((16, 4, 2, 2, 6), (16, 1, 1, 1, 8), (64, 8, 3, 2, 8),
                              (60, 5, 2, 2, 7), (256, 8, 4, 2, 8), (256, 8, 4, 1, 20),
                              (512, 1, 1, 1, 8), (1024, 8, 2, 2, 8)):
        T = 19
        x = rng.normal(size=(T, E)).astype(np.float32)
        x[rng.random((T, E)) < 0.2] = -np.inf
        x[: T // 2, : E // 2] = -np.inf
        for share in (0.5, 0.97, 1.0):
            bias = np.where(rng.random(E) < share, low, 0).astype(np.float32)
            bias[: E // max(G, 2)] = low
            for score in ("sigmoid", "softmax"):
                say(f"lowest bias E={E} G={G} topn={topn} share={share} {score}")
                r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn)
                got = r.route(dev(x), bias=dev(bias))
                r.check_status()
                check_route(got, x, k, score=score, bias=bias, groups=G, topk_groups=tg,
                            group_topn=topn)


def test_route_masked_experts_tokens_and_bad_rows():
    """-inf logits and biases, fewer selectable experts than slots, whole rows
    of -inf, the type's lowest values, masked tokens that hold NaN, and rows
    that hold NaN or +inf."""
    T, E, k = 12, 24, 4
    rng = np.random.default_rng(5)
    x, _ = draw_logits(rng, T, E, False)
    x[0] = -np.inf
    x[1, 2:] = -np.inf                       # two left
    x[2] = np.finfo(np.float32).min
    x[2, 7] = 0
    x[3] = np.finfo(np.float32).min
    x[4, ::3] = -np.inf
    x[5] = np.nan                            # masked
    x[6, 3] = np.inf                         # masked
    x[7] = -200.0                            # sigmoid scores that underflow
    x[7, 4] = -180.0
    mask = np.ones(T, np.uint8)
    mask[[5, 6, 11]] = 0
    bias = (rng.normal(size=E) * 0.1).astype(np.float32)
    bias[9] = -np.inf
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for G, tg, topn in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (12, 2, 2)):
                say(f"masks {score} bias={b is not None} G={G} topn={topn}")
                r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn)
                got = r.route(dev(x), bias=None if b is None else dev(b), token_mask=dev(mask))
                r.check_status()
                check_route(got, x, k, score=score, bias=b, mask=mask, groups=G, topk_groups=tg,
                            group_topn=topn)
    for col, v in ((0, np.nan), (23, np.inf)):
        y = x.copy()
        y[9, col] = v
        r = ep.EpRouter(T, E, k)
        idx, w = r.route(dev(y), token_mask=dev(mask))
        with pytest.raises(ep.EpError) as err:
            r.check_status()
        assert err.value.status == ep.EP_ERR_NONFINITE
        assert (idx[9] == -1).all() and (w[9] == 0).all() and (idx[8] >= 0).all()
    for v in (np.nan, np.inf):
        y = bias.copy()
        y[3] = v
        r = ep.EpRouter(T, E, k, score="sigmoid")
        idx, w = r.route(dev(x), bias=dev(y), token_mask=dev(mask))
        with pytest.raises(ep.EpError) as err:
            r.check_status()
        assert err.value.status == ep.EP_ERR_NONFINITE and (idx[8] == -1).all()


def test_route_unaligned_rows():
    """Logits that start in the middle of a 16-byte piece."""
    rng = np.random.default_rng(6)
    for E in (64, 61):
        for bf16 in (False, True):
            x, t = draw_logits(rng, 20, E, bf16)
            buf = torch.zeros(20 * E + 1, dtype=t.dtype, device="cuda")
            view = buf[1:].view(20, E)
            view.copy_(t)
            say(f"unaligned E={E} bf16={bf16}")
            r = ep.EpRouter(20, E, 5, logits_dtype=t.dtype)
            check_route(r.route(view), x, 5)
            w = rng.normal(size=(20, 5)).astype(np.float32)
            g = torch.empty(20 * E + 1, dtype=t.dtype, device="cuda")
            out = r.backward(view, r.topk_idx, dev(w), grad_logits=g[1:].view(20, E))
            check_grad(out, x, r.topk_idx.cpu().numpy(), w, bf16)


# --------------------------------------------------------------------------

def draw_route(rng, T, E, k, off=0.1):
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < off] = -1
    ids[rng.random(T) < off] = -1
    return ids


def draw_offsets(rng, T, S):
    cuts = np.sort(rng.integers(0, T + 1, size=S - 1))
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


BAL = [(1, 1, 1, 1), (1, 8, 2, 1), (7, 60, 3, 3), (64, 64, 6, 1), (65, 64, 6, 2), (63, 65, 5, 63),
       (300, 256, 8, 1), (300, 256, 8, 7), (1000, 128, 4, 90), (200, 512, 3, 2), (77, 1000, 32, 5),
       (3000, 8, 2, 4)]


@pytest.mark.parametrize("T,E,k,S", BAL)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_balance(T, E, k, S, score, bf16):
    rng = np.random.default_rng(T + E)
    x, t = draw_logits(rng, T, E, bf16)
    ids = draw_route(rng, T, E, k)
    x[(ids < 0).all(axis=1)] = 0  # the reference's padding; the kernel gets NaN there
    t = t.clone()
    t[torch.from_numpy((ids < 0).all(axis=1))] = float("nan")
    offsets = None if S == 1 else draw_offsets(rng, T, S)
    say(f"balance T={T} E={E} k={k} S={S} {score} bf16={bf16}")
    r = ep.EpRouter(T, E, k, score=score, logits_dtype=t.dtype, max_seqs=S + 1)
    loss = r.balance_loss(t.cuda(), dev(ids), 0.7,
                          seq_offsets=None if offsets is None else dev(offsets))
    r.check_status()
    l, counts, n, mean, q = ref.balance(x, ids, 0.7, score, offsets)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert np.array_equal(r.seq_tokens.cpu().numpy(), n)
    # a tile's sum of probabilities: at most 128 additions in fp32, the rest in 64 bits
    rel = (score_steps(x).max() + 128) * U32
    assert np.all(np.abs(r.mean_probs.cpu().numpy() - mean) <= rel * mean + 1e-30)
    assert np.all(np.abs(r.prob_grad.cpu().numpy() - q) <= 4 * U32 * q)
    assert abs(loss.item() - l) <= rel * l + 1e-30


def test_many_empty_sequences():
    """Thousands of sequences without a token among a few that have some."""
    T, E, k, S = 150, 8, 2, 5000
    rng = np.random.default_rng(15)
    x, t = draw_logits(rng, T, E, False)
    ids = draw_route(rng, T, E, k)
    offsets = np.zeros(S + 1, np.int32)
    offsets[1000:] = 37
    offsets[1001:] = 90
    offsets[4000:] = T
    q = rng.normal(size=(S, E)).astype(np.float32)
    say("many empty sequences")
    r = ep.EpRouter(T, E, k, max_seqs=S)
    loss = r.balance_loss(t.cuda(), dev(ids), 0.5, seq_offsets=dev(offsets))
    r.check_status()
    l, counts, n, mean, pg = ref.balance(x, ids, 0.5, "softmax", offsets)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert np.array_equal(r.seq_tokens.cpu().numpy(), n)
    rel = (score_steps(x).max() + 128) * U32
    assert abs(loss.item() - l) <= rel * l
    assert np.all(np.abs(r.prob_grad.cpu().numpy() - pg) <= 4 * U32 * pg)
    g = r.backward(t.cuda(), dev(ids), None, prob_grad=dev(q), seq_offsets=dev(offsets))
    check_grad(g, x, ids, None, False, prob_grad=q, offsets=offsets)


def test_large_batches_cross_passes_and_tiles():
    """Enough tokens that a workgroup takes several passes, tiles grow past 32
    tokens and the router's workgroups take tokens in turn: checked on a sample
    of rows, and the counts and means on all of them."""
    T, E, k, S = 70001, 64, 6, 9
    rng = np.random.default_rng(16)
    x, t = draw_logits(rng, T, E, True)
    mask = (rng.random(T) >= 0.1).astype(np.uint8)
    offsets = draw_offsets(rng, T, S)
    u = rng.normal(size=(T, k)).astype(np.float32)
    say("large batch")
    r = ep.EpRouter(T, E, k, score="sigmoid", logits_dtype=torch.bfloat16, max_seqs=S)
    xd = t.cuda()
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    idx, w = r.route(xd, bias=dev(bias), token_mask=dev(mask))
    r.balance_loss(xd, idx, 0.1, seq_offsets=dev(offsets))
    g = r.backward(xd, idx, dev(u), prob_grad=r.prob_grad, seq_offsets=dev(offsets))
    r.check_status()
    ids = idx.cpu().numpy()
    rows = np.unique(np.concatenate([np.arange(40), rng.integers(0, T, 400), np.arange(T - 40, T)]))
    want, ww, _ = ref.route(x[rows], k, "sigmoid", bias, mask[rows])
    assert np.array_equal(ids[rows], want)
    tol = ww * (score_steps(x[rows]) * U32)[:, None]
    assert np.all(np.abs(w.cpu().numpy()[rows] - ww) <= tol)
    assert np.array_equal(ids[:, 0] < 0, mask == 0)
    on = mask != 0
    p = ref.probabilities(x, "sigmoid")
    rel = (score_steps(x).max() + 128) * U32
    for s in range(S):
        lo, hi = offsets[s], offsets[s + 1]
        have = ids[lo:hi][on[lo:hi]].reshape(-1)
        assert np.array_equal(r.counts[s].cpu().numpy(), np.bincount(have, minlength=E))
        n = int(on[lo:hi].sum())
        if n:
            mean = p[lo:hi][on[lo:hi]].mean(axis=0)
            assert np.all(np.abs(r.mean_probs[s].cpu().numpy() - mean) <= rel * mean)
    pg = r.prob_grad.cpu().numpy()
    seq = np.searchsorted(offsets[1:], rows, side="right")
    for s in np.unique(seq):
        sel = rows[seq == s]
        check_grad(g[torch.from_numpy(sel).cuda()], x[sel], ids[sel], u[sel], True,
                   score="sigmoid", prob_grad=pg[s:s + 1])


def test_balance_empty_and_all_masked():
    for T in (0, 5):
        r = ep.EpRouter(T, 8, 2)
        x = torch.full((T, 8), float("nan"), device="cuda")
        ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
        say(f"balance of nothing T={T}")
        assert r.balance_loss(x, ids, 1.0).item() == 0
        r.check_status()
        assert (r.counts == 0).all() and (r.prob_grad == 0).all() and (r.mean_probs == 0).all()
        assert (r.seq_tokens == 0).all()
        g = r.backward(x, ids, torch.zeros(T, 2, device="cuda"), prob_grad=r.prob_grad)
        assert (g == 0).all() and g.shape == (T, 8)
        r.route(x, token_mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
        r.check_status()
        assert (r.topk_idx == -1).all() and (r.topk_weights == 0).all()


def test_bad_offsets_and_ids_are_reported():
    T, E, k = 130, 8, 2
    rng = np.random.default_rng(7)
    x, t = draw_logits(rng, T, E, False)
    ids = draw_route(rng, T, E, k)
    for bad in ([0, 90, 20, T], [1, 20, 90, T], [0, 20, 90, T - 1], [0, -5, 90, T],
                [0, 20, 10 ** 6, T], [0, 20, 90, 10 ** 6]):
        say(f"bad offsets {bad}")
        r = ep.EpRouter(T, E, k, max_seqs=3)
        r.balance_loss(dev(x), dev(ids), 1.0, seq_offsets=dev(np.array(bad, np.int32)))
        with pytest.raises(ep.EpError) as err:
            r.check_status()
        assert err.value.status == ep.EP_ERR_SEQS
        r.backward(dev(x), dev(ids), None, r.prob_grad,
                   seq_offsets=dev(np.array(bad, np.int32)))
        torch.cuda.synchronize()
    for v in (E, -2, 2 ** 31 - 1):
        y = ids.copy()
        y[3] = v
        y[3, 0] = 1
        say(f"bad id {v}")
        r = ep.EpRouter(T, E, k)
        r.balance_loss(dev(x), dev(y), 1.0)
        with pytest.raises(ep.EpError) as err:
            r.check_status()
        assert err.value.status == ep.EP_ERR_INVALID_ROUTE
        y[3, 1] = -1
        counts = ref.balance(x, y, 1.0)[1]
        assert np.array_equal(r.counts.cpu().numpy(), counts)
        r = ep.EpRouter(T, E, k)
        u = rng.normal(size=(T, k)).astype(np.float32)
        z = y.copy()
        z[3, 1] = v
        g = r.backward(dev(x), dev(z), dev(u))
        check_grad(g, x, y, u, False)
        with pytest.raises(ep.EpError):
            r.check_status()


# --------------------------------------------------------------------------

def check_grad(got, x, ids, u, bf16, **kw):
    want, size = ref.grad(x, ids, u, **kw)
    got = got.float().cpu().numpy()
    # each term: a score or two (score_steps each), products and differences (8), and
    # a sum over the experts (2^10 terms of a tree, 16, in each lane 16)
    tol = size * ((2 * score_steps(x) + 40) * U32)[:, None] + 1e-37
    if bf16:
        tol = tol + np.abs(want) * UBF16 * (1 + 1e-6)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


GRAD = [(1, 1, 1, 1), (1, 8, 2, 1), (3, 7, 7, 2), (17, 60, 4, 3), (33, 64, 6, 1), (16, 65, 5, 4),
        (40, 100, 32, 1), (50, 256, 8, 9), (9, 512, 20, 2), (6, 1000, 32, 2), (5, 1024, 3, 1)]


@pytest.mark.parametrize("T,E,k,S", GRAD)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
def test_backward(T, E, k, S, score, normalize, bf16):
    rng = np.random.default_rng(T + E)
    x, t = draw_logits(rng, T, E, bf16)
    ids = draw_route(rng, T, E, k)
    off = (ids < 0).all(axis=1)
    t = t.clone()
    t[torch.from_numpy(off)] = float("nan")  # padding: not read into any result
    u = rng.normal(size=(T, k)).astype(np.float32)
    nan_u = np.where(ids < 0, np.float32(np.nan), u)
    q = rng.normal(size=(S, E)).astype(np.float32)
    offsets = None if S == 1 else draw_offsets(rng, T, S)
    so = None if offsets is None else dev(offsets)
    r = ep.EpRouter(T, E, k, score=score, normalize=normalize, scale=1.5, logits_dtype=t.dtype,
                    max_seqs=S)
    kw = dict(score=score, normalize=normalize, scale=1.5)
    for name, uu, qq, gl in (("gates", nan_u, None, None), ("loss", None, q, 3.0),
                             ("both", nan_u, q, 0.25), ("loss of 1", None, q, None)):
        say(f"backward T={T} E={E} k={k} S={S} {score} normalize={normalize} bf16={bf16} {name}")
        out = torch.full((T, E), 7.0, dtype=t.dtype, device="cuda")
        g = r.backward(t.cuda(), dev(ids), None if uu is None else dev(uu),
                       prob_grad=None if qq is None else dev(qq), seq_offsets=so,
                       grad_loss=None if gl is None else torch.full((1,), gl, device="cuda"),
                       grad_logits=out)
        r.check_status()
        check_grad(g, np.where(off[:, None], 0, x), ids, None if uu is None else u, bf16,
                   prob_grad=qq, offsets=offsets, grad_loss=1.0 if gl is None else gl, **kw)


def test_backward_masked_and_extreme_logits():
    """-inf and lowest logits beside the selected ones, scores that underflow."""
    T, E, k = 6, 16, 3
    rng = np.random.default_rng(8)
    x, _ = draw_logits(rng, T, E, False)
    x[0, 3:] = -np.inf
    x[1, 4:] = np.finfo(np.float32).min
    x[2] -= 300
    x[3] += 300
    x[4, 0] = 90
    ids = np.array([[0, 1, 2], [0, 1, 3], [5, 4, 9], [1, 2, 3], [0, 7, 2], [3, -1, 1]], np.int32)
    u = rng.normal(size=(T, k)).astype(np.float32)
    q = rng.normal(size=(1, E)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            say(f"extreme {score} normalize={normalize}")
            r = ep.EpRouter(T, E, k, score=score, normalize=normalize)
            g = r.backward(dev(x), dev(ids), dev(u), prob_grad=dev(q))
            r.check_status()
            check_grad(g, x, ids, u, False, score=score, normalize=normalize, prob_grad=q)


def test_backward_against_differences():
    """The kernels' gradient against differences of the kernels' own forward:
    a step h of the logits, error h^2 / 6 of a third derivative (order 1) and
    fp32 forward values (2^-22) over h."""
    T, E, k = 4, 12, 3
    rng = np.random.default_rng(9)
    # a quarter between neighbours: no step moves an expert in or out
    x = np.array([rng.permutation(E) for _ in range(T)], np.float32) / 4 - 1.5
    u = rng.normal(size=(T, k)).astype(np.float32)
    h = 2.0 ** -6
    for score in ("softmax", "sigmoid"):
        r = ep.EpRouter(T, E, k, score=score)
        idx = r.route(dev(x))[0].cpu().numpy()
        r.balance_loss(dev(x), dev(idx), 1.0)
        g = r.backward(dev(x), dev(idx), dev(u), prob_grad=r.prob_grad).cpu().numpy()
        bias = np.zeros(E, np.float32)

        def value(z):
            # the ids stay: only their weights and the loss move
            i, w = r.route(dev(z), bias=dev(bias))
            i, w = i.cpu().numpy(), w.cpu().numpy().astype(np.float64)
            assert np.array_equal(np.sort(i), np.sort(idx))
            order = np.argsort(i, axis=1)
            back = np.argsort(np.argsort(idx, axis=1), axis=1)
            w = np.take_along_axis(np.take_along_axis(w, order, axis=1), back, axis=1)
            return (w * u).sum() + r.balance_loss(dev(z), dev(idx), 1.0).item()

        for t in range(T):
            for e in range(E):
                d = np.zeros_like(x)
                d[t, e] = h
                up, down = value(x + d), value(x - d)
                assert abs(g[t, e] - (up - down) / (2 * h)) < h * h + 16 * 2.0 ** -22 / h


def test_offsets_past_32_bits():
    """More than 2^32 logits: a block of rows again and again has the same
    selection, gates and gradient in every place, and counts that add up."""
    B, n, E, k = 4096, 4100, 256, 8
    T = B * n
    assert T * E > 1 << 32
    rng = np.random.default_rng(19)
    x, t = draw_logits(rng, B, E, True)
    u = torch.from_numpy(rng.normal(size=(B, k)).astype(np.float32)).cuda()
    say("offsets past 32 bits")
    small = ep.EpRouter(B, E, k, logits_dtype=torch.bfloat16)
    xb = t.cuda()
    ids, w = small.route(xb)
    check_route((ids, w), x, k)
    gb = small.backward(xb, ids, u)
    r = ep.EpRouter(T, E, k, logits_dtype=torch.bfloat16)
    xd = xb.repeat(n, 1)
    got_ids, got_w = r.route(xd)
    assert bool((got_ids.view(n, B, k) == ids).all())
    assert bool((got_w.view(n, B, k) == w).all())
    g = r.backward(xd, got_ids, u.repeat(n, 1))
    for i in range(0, n, 100):  # in parts: the comparison needs memory too
        assert bool((g.view(n, B, E)[i:i + 100] == gb).all()), i
    r.balance_loss(xd, got_ids, 1.0)
    r.check_status()
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).cpu().numpy()
    assert np.array_equal(r.counts[0].cpu().numpy(), counts * n)
    assert r.seq_tokens.item() == T
    mean = ref.probabilities(x, "softmax").mean(axis=0)
    rel = (score_steps(x).max() + 256) * U32
    assert np.all(np.abs(r.mean_probs[0].cpu().numpy() - mean) <= rel * mean)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_large_finite_biases(score):
    """Experts put last or first by large finite biases of either sign: the
    others' order is that of their own keys, sums of two keys that cancel
    included."""
    rng = np.random.default_rng(61)
    for E, G, tg, topn, k in ((64, 1, 1, 1, 8), (64, 1, 1, 1, 3), (64, 8, 3, 2, 6), (60, 5, 2, 2, 6),
                              (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (100, 1, 1, 1, 20),
                              (512, 16, 4, 2, 12), (1024, 8, 2, 2, 8)):
        T = 31
        x = rng.normal(size=(T, E)).astype(np.float32)
        x[::3] = np.round(x[::3] * 4) / 4  # equal keys among them
        for big in (1e4, 1e9, 3e38):
            for signs in ([-1], [1], [-1, 1]):
                bias = (rng.normal(size=E) * 0.05).astype(np.float32)
                at = rng.permutation(E)[: max(2, E // 8)]
                bias[at] = np.float32(big) * rng.choice(signs, size=len(at)).astype(np.float32)
                # neighbours in size that round apart, and pairs that add up to nearly nothing
                bias[at[: len(at) // 2]] *= np.float32(1 - 2.0 ** -20)
                say(f"large biases E={E} G={G} topn={topn} k={k} {score} big={big} signs={signs}")
                r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn)
                got = r.route(dev(x), bias=dev(bias))
                r.check_status()
                check_route(got, x, k, score=score, bias=bias, groups=G, topk_groups=tg,
                            group_topn=topn)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg,topn", [(256, 8, 4, 2), (64, 1, 1, 1)])
def test_route_with_experts_put_last_costs_no_more(score, E, G, tg, topn):
    """A large finite bias on some experts leaves the other tokens' selection to
    32 bits: at most twice the time of the call without it (64-bit keys for all
    tokens take ten times as long)."""
    T, k = 65536, 8
    rng = np.random.default_rng(62)
    x = dev(rng.normal(size=(T, E)).astype(np.float32))
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    r = ep.EpRouter(T, E, k, score=score, groups=G, topk_groups=tg, group_topn=topn)

    def best_time(b):
        b = dev(b)
        times = []
        for _ in range(5):
            start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(5):
                r.route(x, bias=b)
            stop.record()
            stop.synchronize()
            times.append(start.elapsed_time(stop) / 5)
        return min(times)

    say(f"time with experts put last E={E} G={G} {score}")
    plain = best_time(bias)
    for big in (-1e4, -1e9, float(np.finfo(np.float32).min)):
        last = bias.copy()
        last[::17] = big
        took = best_time(last)
        say(f"  plain {1e3 * plain:.1f} us, bias {big:g}: {1e3 * took:.1f} us")
        assert took <= 2 * plain
    r.check_status()


@pytest.mark.parametrize("bf16", [False, True])
def test_fast_exponential_on_the_device(bf16):
    """Softmax rows of two experts, each a sequence of its own, so that
    mean_probs is exp(x) / (1 + exp(x)): the exponential's bound of
    (1.23 |x| + 3) 2^-24, a sum, a quotient and a product, and the mean."""
    T = 4000
    v = np.linspace(0, 87, T).astype(np.float32)
    x = np.stack([np.zeros(T, np.float32), -v], axis=1)
    t = torch.from_numpy(x)
    t = t.bfloat16() if bf16 else t
    x = t.double().numpy()
    ids = dev(np.zeros((T, 1), np.int32))
    say(f"fast exponential bf16={bf16}")
    r = ep.EpRouter(T, 2, 1, logits_dtype=t.dtype, max_seqs=T)
    r.balance_loss(t.cuda(), ids, 1.0, seq_offsets=dev(np.arange(T + 1, dtype=np.int32)))
    r.check_status()
    got = r.mean_probs[:, 1].double().cpu().numpy()
    want = np.exp(x[:, 1]) / (1 + np.exp(x[:, 1]))
    assert np.all(np.abs(got / want - 1) <= (1.23 * -x[:, 1] + 3 + 6) * U32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_repeated_ids_count_as_often(score, normalize):
    """The same expert in two and more slots of a token: each slot counts, and
    its gradient adds up."""
    rng = np.random.default_rng(81)
    for T, E, k in ((21, 8, 2), (40, 64, 6), (17, 256, 8), (9, 300, 32)):
        x, t = draw_logits(rng, T, E, False)
        ids = draw_route(rng, T, E, k)
        ids[::2, 1] = ids[::2, 0]
        ids[::4] = ids[::4, :1]
        u = rng.normal(size=(T, k)).astype(np.float32)
        q = rng.normal(size=(1, E)).astype(np.float32)
        say(f"repeated ids T={T} E={E} k={k} {score} normalize={normalize}")
        r = ep.EpRouter(T, E, k, score=score, normalize=normalize)
        g = r.backward(t.cuda(), dev(ids), dev(u), prob_grad=dev(q))
        check_grad(g, x, ids, u, False, score=score, normalize=normalize, prob_grad=q)
        loss = r.balance_loss(t.cuda(), dev(ids), 0.3)
        r.check_status()
        l, counts, n, _, pg = ref.balance(x, ids, 0.3, score)
        assert np.array_equal(r.counts.cpu().numpy(), counts)
        assert np.array_equal(r.seq_tokens.cpu().numpy(), n)
        assert abs(loss.item() - l) <= (score_steps(x).max() + 128) * U32 * l
        assert np.all(np.abs(r.prob_grad.cpu().numpy() - pg) <= 4 * U32 * pg)
