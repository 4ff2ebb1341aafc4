"""The 8-bit SwiGLU checkpoint and its gradient on the GPU.  Codes and scales
are exact; h and the gradients are fp32 expressions of a few operations and an
exponential, rounded once to bf16."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
from tests import experts_reference as ref  # noqa: E402
from tests.gpu_backend import dev, say  # noqa: E402

U32, UBF16 = ref.U32, ref.UBF16


def layout_of(counts, gap):
    off = np.concatenate([[0], np.cumsum(np.asarray(counts) + gap)]).astype(np.int32)
    return off, int(off[-1])


def live_rows(off, counts, cap):
    live = np.zeros(cap, bool)
    for _, lo, hi in ref.expert_rows(off, counts, cap):
        live[lo:hi] = True
    return live


def decoded(t):
    return t.view(torch.float8_e4m3fn).double().cpu().numpy()


def close(got, want, size=None):
    """12 half steps of fp32 of the expression's size, one of bf16."""
    err = 12 * U32 * (np.abs(want) if size is None else size)
    return np.abs(got - want) <= err + (np.abs(want) + err) * UBF16 + 1e-37


SHAPES = [(1, [1]), (2, [0, 3]), (16, [5, 0, 1]), (127, [2, 3]), (128, [4, 1]), (129, [1, 0, 9]),
          (200, [7, 30]), (256, [3] * 40), (1001, [9, 2]), (1408, [1, 0, 70]), (2048, [300, 5])]


@pytest.mark.parametrize("F,counts", SHAPES)
def test_save_and_backward(F, counts):
    rng = np.random.default_rng(F)
    off, cap = layout_of(counts, 2)
    live = live_rows(off, counts, cap)
    v = ref.rounded(rng.normal(size=(cap, 2 * F)) * np.exp(rng.normal(size=(cap, 1)) * 2))
    v[live.argmax()] = 0.0  # a row of zeros
    gh = ref.rounded(rng.normal(size=(cap, F)))
    gate_up, grad = v.copy(), gh.copy()
    gate_up[~live], grad[~live] = np.nan, np.nan
    c = ep.SwigluCheckpoint(cap, F, len(counts))
    c.codes.fill_(0x55)
    c.scales.fill_(7.0)
    h = torch.full((cap, F), 99.0, dtype=torch.bfloat16, device="cuda")
    at = dev(off), dev(np.array(counts, np.int32))
    say(f"save F={F} counts={counts}")
    assert c.save(ref.to_bf16(gate_up).cuda(), *at, out=h) is h
    codes, scales = ref.checkpoint(v[live])
    assert np.array_equal(decoded(c.codes)[live], codes)
    assert np.array_equal(c.scales.double().cpu().numpy()[live], scales)
    assert (c.codes.cpu().numpy()[~live] == 0x55).all()
    assert (c.scales.cpu().numpy()[~live] == 7.0).all()
    got = h.double().cpu().numpy()
    assert (got[~live] == 99.0).all()
    assert np.all(close(got[live], ref.silu(v[live, :F]) * v[live, F:]))

    say(f"backward F={F} counts={counts}")
    g, h2 = torch.full((cap, 2 * F), 99.0, dtype=torch.bfloat16, device="cuda"), torch.full_like(
        h, 99.0)
    c.backward(ref.to_bf16(grad).cuda(), *at, out=g, h=h2)
    kept = ref.kept(codes, scales, F)
    want, wh = ref.swiglu_grad(kept, gh[live])
    s, gate, up = ref.sigmoid(kept[:, :F]), kept[:, :F], kept[:, F:]
    size = np.concatenate([np.abs(gh[live] * up * s) * (1 + np.abs(gate) * (1 - s)),
                           np.abs(gh[live] * gate * s)], axis=1)
    g, h2 = g.double().cpu().numpy(), h2.double().cpu().numpy()
    assert (g[~live] == 99.0).all() and (h2[~live] == 99.0).all()
    assert np.all(close(g[live], want, size))
    assert np.all(close(h2[live], wh))
    say("without h")
    g3 = torch.full((cap, 2 * F), 99.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_swiglu_checkpoint_backward(len(counts), F, c.codes, c.scales,
                                     ref.to_bf16(grad).cuda(), *at, g3, None)
    assert np.array_equal(g3.double().cpu().numpy(), g)


@pytest.mark.parametrize("F", [64, 128, 136, 75])
def test_every_scale_and_border(F):
    """Blocks whose largest value is at and beside 448 times a power of two, over
    the type's whole range."""
    most = []
    for e in list(range(-133, -95, 3)) + [-20, -1, 0, 1, 30, 118]:
        for m in (1.0, 1.7421875, 1.75, 1.7578125, 1.984375):
            most.append(m * 2.0 ** e)
    most = ref.rounded(np.array([0.0] + most))
    rng = np.random.default_rng(F)
    v = np.zeros((len(most), 2 * F))
    v[:] = ref.rounded(most[:, None] * rng.uniform(-1, 1, size=v.shape))
    v[np.arange(len(most)), rng.integers(0, F, len(most))] = most
    v[np.arange(len(most)), F + rng.integers(0, F, len(most))] = -most
    at = dev(np.array([0], np.int32)), dev(np.array([len(most)], np.int32))
    c = ep.SwigluCheckpoint(len(most), F, 1)
    say(f"borders F={F}")
    c.save(ref.to_bf16(v).cuda(), *at)
    codes, scales = ref.checkpoint(v)
    assert np.array_equal(c.scales.double().cpu().numpy(), scales)
    assert np.array_equal(decoded(c.codes), codes)


@pytest.mark.parametrize("F", [128, 75])
def test_values_that_are_not_finite(F):
    """NaN codes in their places, and no part in the others' scale."""
    rng = np.random.default_rng(1)
    v = ref.rounded(rng.normal(size=(6, 2 * F)))
    v[1, 3], v[2, F], v[3, 2 * F - 1], v[4, :F] = np.inf, np.nan, -np.inf, np.nan
    at = dev(np.array([0], np.int32)), dev(np.array([6], np.int32))
    c = ep.SwigluCheckpoint(6, F, 1)
    say("values that are not finite")
    h = c.save(ref.to_bf16(v).cuda(), *at).double().cpu().numpy()
    codes, scales = ref.checkpoint(v)
    assert np.array_equal(decoded(c.codes), codes, equal_nan=True)
    assert np.array_equal(c.scales.double().cpu().numpy(), scales)
    bad = ~(np.isfinite(v[:, :F]) & np.isfinite(v[:, F:]))
    assert np.array_equal(np.isfinite(h), ~bad)
    gh = ref.rounded(rng.normal(size=(6, F)))
    g, h2 = c.backward(ref.to_bf16(gh).cuda(), *at)
    assert np.array_equal(np.isfinite(h2.float().cpu().numpy()), ~bad)
    ok = np.isfinite(g.float().cpu().numpy())
    assert np.array_equal(ok[:, :F], ~bad) and np.array_equal(ok[:, F:], np.isfinite(v[:, :F]))


def test_large_gates():
    """Gates of any size: no infinity times zero."""
    gates = [0.0, 1.0, -1.0, 87.0, -87.0, -88.5, -95.0, 200.0, -200.0, 1e30, -1e30, 2.0 ** 126,
             -2.0 ** 126]
    v = np.zeros((len(gates), 256))
    v[:, :128] = ref.rounded(np.array(gates))[:, None]
    v[:, 128:] = ref.rounded(np.array([1e-3, 3.0, -2.0, 1e3] * 32))
    gh = ref.rounded(np.array([1.0, -1e3, 1e-3, 7.0] * 32))[None].repeat(len(gates), axis=0)
    at = dev(np.array([0], np.int32)), dev(np.array([len(gates)], np.int32))
    c = ep.SwigluCheckpoint(len(gates), 128, 1)
    say("large gates")
    h = c.save(ref.to_bf16(v).cuda(), *at).double().cpu().numpy()
    want = ref.silu(v[:, :128]) * v[:, 128:]
    big = np.abs(want) < 3e38
    assert np.all(close(h, want)[big]) and not np.isnan(h).any()
    g, h2 = c.backward(ref.to_bf16(gh).cuda(), *at)
    kept = ref.kept(*ref.checkpoint(v), 128)
    want, wh = ref.swiglu_grad(kept, gh)
    s, gate, up = ref.sigmoid(kept[:, :128]), kept[:, :128], kept[:, 128:]
    size = np.concatenate([np.abs(gh * up * s) * (1 + np.abs(gate) * (1 - s)),
                           np.abs(gh * gate * s)], axis=1)
    for got, w, z in ((g, want, size), (h2, wh, np.abs(wh))):
        got = got.double().cpu().numpy()
        assert not np.isnan(got).any()
        inside = np.abs(w) < 3e38
        assert np.all(close(got, w, z)[inside])


def test_checkpoint_as_fp8_rows():
    """The checkpoint's codes and scales are FP8 rows of a product, which sees
    exactly the kept values."""
    rng = np.random.default_rng(2)
    F, N, rows = 128, 48, 20
    v = ref.rounded(rng.normal(size=(rows, 2 * F)))
    w = rng.integers(-4, 5, size=(1, N, 2 * F)).astype(np.float64)
    at = dev(np.array([0], np.int32)), dev(np.array([rows], np.int32))
    c = ep.SwigluCheckpoint(rows, F, 1)
    c.save(ref.to_bf16(v).cuda(), *at)
    say("a checkpoint as rows")
    got = ep.Bf16Experts(ref.to_bf16(w).cuda()).product(c.codes, c.scales, *at)
    kept = ref.kept(*ref.checkpoint(v), F)
    assert np.array_equal(ref.rounded(kept), kept)
    y, size = ref.product(kept, w, [0], [rows])
    err = ref.sum_error(2 * F, size)
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= err + (np.abs(y) + err) * UBF16)


def test_rows_past_the_capacity():
    rng = np.random.default_rng(3)
    F, cap = 40, 9
    off, cnt = np.array([2, 5, -1, 9], np.int32), np.array([2, 100, 4, 3], np.int32)
    v = ref.rounded(rng.normal(size=(cap, 2 * F)))
    c = ep.SwigluCheckpoint(cap, F, 4)
    c.codes.fill_(0x33)
    c.scales.fill_(5.0)
    h = torch.full((cap + 3, F), 99.0, dtype=torch.bfloat16, device="cuda")
    say("rows past the capacity")
    c.save(ref.to_bf16(v).cuda(), dev(off), dev(cnt), out=h)
    live = live_rows(off, cnt, cap)
    assert live.sum() == 6
    assert (c.codes.cpu().numpy()[~live] == 0x33).all()
    assert np.array_equal(decoded(c.codes)[live], ref.checkpoint(v)[0][live])
    got = h.double().cpu().numpy()
    assert (got[:cap][~live] == 99.0).all() and (got[cap:] == 99.0).all()
    assert (got[:cap][live] != 99.0).all()


@pytest.mark.parametrize("F", [40, 136])
def test_a_row_is_the_same_beside_any_other(F):
    """Large gates take another form of the exponential: for their own values alone."""
    rng = np.random.default_rng(F)
    n = 64
    v = ref.rounded(rng.normal(size=(n, 2 * F)) * 9)
    beside = v.copy()
    beside[::2] = ref.rounded(rng.normal(size=(n // 2, 2 * F)) * 400)
    grad = ref.to_bf16(ref.rounded(rng.normal(size=(n, F)))).cuda()
    at = dev(np.array([0], np.int32)), dev(np.array([n], np.int32))
    got = []
    for rows in (v, beside):
        c = ep.SwigluCheckpoint(n, F, 1)
        h = c.save(ref.to_bf16(rows).cuda(), *at)
        got.append([t[1::2] for t in (h, c.codes, c.scales, *c.backward(grad, *at))])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_checkpoint_moved_away_and_back():
    """Codes and scales kept in host memory between save and backward, and other
    tensors in their old places."""
    rng = np.random.default_rng(4)
    n, F = 32, 200
    v = ref.to_bf16(ref.rounded(rng.normal(size=(n, 2 * F)))).cuda()
    grad = ref.to_bf16(ref.rounded(rng.normal(size=(n, F)))).cuda()
    at = dev(np.array([0], np.int32)), dev(np.array([n], np.int32))
    c = ep.SwigluCheckpoint(n, F, 1)
    say("a checkpoint moved away and back")
    c.save(v, *at)
    want = c.backward(grad, *at)
    olds = c.codes.data, c.scales.data
    for t in (c.codes, c.scales):
        t.data = t.cpu()
    olds[0].fill_(0x7F)
    olds[1].fill_(float("nan"))
    for call in (lambda: c.backward(grad, *at), lambda: c.save(v, *at)):
        with pytest.raises(ValueError):
            call()
    for t in (c.codes, c.scales):
        t.data = t.cuda()
    for a, b in zip(c.backward(grad, *at), want):
        assert torch.equal(a, b)
    for t in olds:
        t.zero_()
    c.save(v, *at)
    assert not olds[0].any() and not olds[1].any()
