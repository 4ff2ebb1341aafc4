"""The plain 64-bit implementations the GPU tests compare with: their
gradients against differences of their own forward passes, and their
selection against a search over every choice of experts."""
import itertools

import numpy as np
import pytest

from tests import moe_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_formula_against_differences(score, normalize):
    rng = np.random.default_rng(1)
    T, E, k, S = 5, 7, 3, 2
    x = rng.normal(size=(T, E))
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)], np.int32)
    ids[1, 2] = -1
    ids[3] = -1
    offsets = np.array([0, 2, T])
    u = rng.normal(size=(T, k))
    q = rng.normal(size=(S, E))
    seq = np.searchsorted(offsets[1:], np.arange(T), side="right")
    on = (ids >= 0).any(axis=1)

    def value(z):
        w = np.where(ids >= 0, ref.gates(z, ids, score, normalize, 1.7), 0.0)
        return (w * u).sum() + 0.3 * (ref.probabilities(z, score) * q[seq] * on[:, None]).sum()

    got, _ = ref.grad(x, ids, u, score, normalize, 1.7, q, offsets, 0.3)
    h = 1e-5
    for t, e in itertools.product(range(T), range(E)):
        d = np.zeros_like(x)
        d[t, e] = h
        # central differences: error h^2 / 6 of a third derivative of order 1, and
        # rounding 2^-52 / h of a value of order 1
        assert abs(got[t, e] - (value(x + d) - value(x - d)) / (2 * h)) < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_that_of_the_loss(score):
    """prob_grad, taken through the probabilities, is the derivative of the loss."""
    rng = np.random.default_rng(2)
    T, E, k = 6, 5, 2
    x = rng.normal(size=(T, E))
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)], np.int32)
    ids[2] = -1
    offsets = [0, 3, 3, T]
    _, _, _, _, q = ref.balance(x, ids, 0.5, score, offsets)
    got, _ = ref.grad(x, ids, None, score, prob_grad=q, offsets=np.array(offsets))
    h = 1e-5
    for t, e in itertools.product(range(T), range(E)):
        d = np.zeros_like(x)
        d[t, e] = h
        up, down = (ref.balance(x + s * d, ids, 0.5, score, offsets)[0] for s in (1, -1))
        assert abs(got[t, e] - (up - down) / (2 * h)) < 1e-8


def test_balanced_load_has_loss_coef():
    """Every expert with the same count and probability: f = P E = 1, loss = coef."""
    E, k = 8, 2
    x = np.zeros((E, E))
    ids = np.array([[t, (t + 1) % E] for t in range(E)], np.int32)
    loss, counts, n, mean, _ = ref.balance(x, ids, 0.25)
    assert np.isclose(loss, 0.25) and (counts == 2).all() and n[0] == E


def test_route_is_the_best_choice():
    """The selected set has the largest sum of keys of all sets that lie in
    topk_groups groups which are the best ones."""
    rng = np.random.default_rng(3)
    E, k, G, tg = 8, 3, 4, 2
    for t in range(20):
        x = rng.normal(size=(1, E)).astype(np.float32)
        bias = rng.normal(size=E).astype(np.float32) * 0.1
        ids, w, _ = ref.route(x, k, "sigmoid", bias, groups=G, topk_groups=tg, group_topn=2)
        key = 1 / (1 + np.exp(-x[0].astype(np.float64))) + bias
        gk = key.reshape(G, 2).sum(axis=1)
        best_groups = max(itertools.combinations(range(G), tg), key=lambda c: gk[list(c)].sum())
        inside = [e for e in range(E) if e // 2 in best_groups]
        best = max(itertools.combinations(inside, k), key=lambda c: key[list(c)].sum())
        assert set(ids[0]) == set(best)
        assert np.all(np.diff(key[ids[0]]) <= 0) and np.isclose(w.sum(), 1.0)


def test_tiles_hold_every_code_once():
    """The tiled layout is a permutation of the codes (and zero padding)."""
    rng = np.random.default_rng(4)
    q = rng.integers(0, 16, size=(2, 2 * 19, 160)).astype(np.uint8)
    t = ref.tile_codes(q, 2)
    assert t.shape == (2, 2, 2, 2, 1024)
    nib = np.stack([t & 15, t >> 4]).reshape(-1)
    assert np.array_equal(np.bincount(nib, minlength=16)[1:],
                          np.bincount(q.reshape(-1), minlength=16)[1:])
    assert ref.pack_codes(q).shape == (2, 38, 80)


def test_bound_of_the_fast_exponential():
    """exp(x) as the router's kernels take it, exp2 of the fp32 product with the
    fp32 constant: even an exact exp2 stays within the stated bound less the 2
    that are left for the hardware's."""
    import os
    import re

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "combine_get_dispatch_amd", "csrc", "ep_router.hip")
    text = open(path).read()
    const = np.float32(float.fromhex(re.search(r"exp2f\(v \* (0x1\.[0-9a-f]+p\+0)f\)", text).group(1)))
    per, plus = re.search(r"exp2 of x log2\(e\), off by\s*//\s*\(([\d.]*) ?\|x\| \+ (\d)\) 2\^-24",
                          text).groups()
    x = -np.random.default_rng(5).uniform(0, 87, 4_000_000).astype(np.float32)
    got = np.exp2((x * const).astype(np.longdouble))
    off = np.abs(got / np.exp(x.astype(np.longdouble)) - 1).astype(np.float64) * 2.0 ** 24
    assert np.all(off <= float(per or 1) * np.abs(x) + int(plus) - 2 + 1e-3)
