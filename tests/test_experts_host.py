"""Refusals of the bf16 experts' products, their gradients and the SwiGLU
checkpoint: each call below is rejected before anything touches a device, so
these run without one; and the plain forms the GPU tests compare with, against
differences."""
import ctypes

import numpy as np
import pytest
import torch

import combine_get_dispatch_amd as ep
from tests import experts_reference as ref


def _fake(n, by=0):
    return ctypes.c_void_p(0x1000000 * n + by)  # never dereferenced: rejected first


def _experts(E=2, K=256, N=32):
    return ep.ep_experts_t(E, K, N)


def _product(x=_experts(), dtype=0, rows=_fake(1), scales=None, w=_fake(2), swiglu=0, off=_fake(3),
             cnt=_fake(4), cap=8, out=_fake(5)):
    return ep.lib().ep_expert_product(ctypes.byref(x), dtype, rows, scales, w, swiglu, off, cnt,
                                      cap, out, None)


def _rows(x=_experts(), grad=_fake(1), w=_fake(2), off=_fake(3), cnt=_fake(4), cap=8,
          out=_fake(5)):
    return ep.lib().ep_expert_product_backward_rows(ctypes.byref(x), grad, w, off, cnt, cap, out,
                                                    None)


def _weights(x=_experts(), dtype=0, rows=_fake(1), scales=None, grad=_fake(2), off=_fake(3),
             cnt=_fake(4), cap=8, gtype=2, add=None, out=_fake(5)):
    return ep.lib().ep_expert_product_backward_weights(
        ctypes.byref(x), dtype, rows, scales, grad, off, cnt, cap, gtype, add, out, None)


@pytest.mark.parametrize("bad", [dict(E=0), dict(E=1025), dict(K=0), dict(K=1 << 20), dict(N=0),
                                 dict(N=1 << 20), dict(N=-8), dict(K=-8)], ids=str)
def test_bad_experts_rejected(bad):
    for call in (_product, _rows, _weights):
        assert call(x=_experts(**bad)) == ep.EP_ERR_INVALID_ARG and ep.lib().ep_last_error()


@pytest.mark.parametrize("call", [_product, _rows, _weights])
def test_what_the_calls_share(call):
    for kw in (dict(off=None), dict(cnt=None), dict(cap=-1), dict(cap=(1 << 31) - 1),
               dict(x=_experts(E=1024), cap=1 << 28), dict(out=None)):
        assert call(**kw) == ep.EP_ERR_INVALID_ARG, kw


def test_product_rejections():
    for kw in (dict(dtype=2), dict(dtype=3), dict(dtype=1), dict(rows=None), dict(w=None),
               dict(rows=_fake(1, 8)), dict(w=_fake(2, 8)), dict(out=_fake(5, 1)),
               dict(dtype=1, scales=_fake(6, 2)), dict(x=_experts(N=33), swiglu=1),
               dict(x=_experts(K=192), dtype=1, scales=_fake(6)),
               dict(out=_fake(1)), dict(out=_fake(1, 8 * 256 * 2 - 2)),
               dict(out=_fake(1, -(8 * 32 * 2 - 2))), dict(out=_fake(2, 2 * 32 * 256 * 2 - 2)),
               dict(dtype=1, scales=_fake(6), out=_fake(6, 8 * 2 * 4 - 2))):
        assert _product(**kw) == ep.EP_ERR_INVALID_ARG, kw
    assert _product(cap=0, rows=None, out=None) == ep.EP_OK
    assert ep.lib().ep_expert_product(None, 0, _fake(1), None, _fake(2), 0, _fake(3), _fake(4), 8,
                                      _fake(5), None) == ep.EP_ERR_INVALID_ARG


def test_rows_gradient_rejections():
    for kw in (dict(grad=None), dict(w=None), dict(grad=_fake(1, 8)), dict(w=_fake(2, 4)),
               dict(out=_fake(5, 1)), dict(out=_fake(1, 8 * 32 * 2 - 2)),
               dict(out=_fake(2, 2 * 32 * 256 * 2 - 2))):
        assert _rows(**kw) == ep.EP_ERR_INVALID_ARG, kw
    assert _rows(cap=0, grad=None, out=None) == ep.EP_OK


def test_weights_gradient_rejections():
    for kw in (dict(dtype=2), dict(dtype=1), dict(rows=None), dict(grad=None), dict(gtype=1),
               dict(gtype=3), dict(rows=_fake(1, 8)), dict(grad=_fake(2, 2)),
               dict(out=_fake(5, 8)), dict(add=_fake(6, 4)),
               dict(x=_experts(K=192), dtype=1, scales=_fake(6)),
               dict(out=_fake(1)), dict(out=_fake(2)), dict(add=_fake(5, 16)),
               dict(add=_fake(5, 2 * 32 * 256 * 4 - 16)),
               dict(dtype=1, scales=_fake(5, 64)), dict(cap=0, out=None)):
        assert _weights(**kw) == ep.EP_ERR_INVALID_ARG, kw


def _save(E=2, F=200, gate_up=_fake(1), off=_fake(2), cnt=_fake(3), cap=8, h=_fake(4),
          codes=_fake(5), scales=_fake(6)):
    return ep.lib().ep_swiglu_checkpoint(E, F, gate_up, off, cnt, cap, h, codes, scales, None)


def _use(E=2, F=200, codes=_fake(1), scales=_fake(2), grad=_fake(3), off=_fake(4), cnt=_fake(5),
         cap=8, out=_fake(6), h=_fake(7)):
    return ep.lib().ep_swiglu_checkpoint_backward(E, F, codes, scales, grad, off, cnt, cap, out, h,
                                                  None)


def test_checkpoint_rejections():
    for call in (_save, _use):
        for kw in (dict(E=0), dict(E=1025), dict(F=0), dict(F=1 << 20), dict(off=None),
                   dict(cnt=None), dict(cap=-1), dict(cap=(1 << 31) - 1),
                   dict(E=1024, cap=1 << 28), dict(codes=None), dict(scales=None),
                   dict(scales=_fake(9, 2)), dict(codes=_fake(9, 8)), dict(h=_fake(9, 2))):
            assert call(**kw) == ep.EP_ERR_INVALID_ARG, (call.__name__, kw)
    for kw in (dict(gate_up=None), dict(h=None), dict(gate_up=_fake(1, 4)), dict(h=_fake(1)),
               dict(codes=_fake(1, 8 * 200 * 4 - 16)), dict(scales=_fake(4, 8 * 200 * 2 - 4)),
               dict(codes=_fake(4))):
        assert _save(**kw) == ep.EP_ERR_INVALID_ARG, kw
    for kw in (dict(grad=None), dict(out=None), dict(grad=_fake(3, 2)), dict(out=_fake(6, 8)),
               dict(h=_fake(3)), dict(h=_fake(6, 8 * 200 * 4 - 16)), dict(out=_fake(1)),
               dict(out=_fake(3)), dict(h=_fake(2))):
        assert _use(**kw) == ep.EP_ERR_INVALID_ARG, kw
    none = dict(codes=None, scales=None, h=None)
    assert _save(cap=0, gate_up=None, **none) == ep.EP_OK
    assert _use(cap=0, grad=None, out=None, **none) == ep.EP_OK


def test_python_checks():
    w = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    x, g = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.bfloat16)
    at = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (w.float(), w[0], w[0, 0], w[:, :, :64], w.transpose(1, 2)):
        with pytest.raises(ValueError):
            ep.Bf16Experts(bad)
    e = ep.Bf16Experts(w)
    with pytest.raises(ValueError):  # host tensors
        e.product(x, None, *at)
    with pytest.raises(ValueError):
        e.backward_rows(g, *at)
    with pytest.raises(ValueError):
        e.backward_weights(x, None, g, *at)
    with pytest.raises(ValueError):  # other widths, other row counts
        e.product(g, None, *at)
    with pytest.raises(ValueError):
        e.backward_rows(x, *at)
    with pytest.raises(ValueError):
        e.backward_weights(x[:3], None, g, *at)
    with pytest.raises(ValueError):
        e.backward_weights(x, None, g, *at, dtype=torch.float16)
    c = ep.SwigluCheckpoint(4, 16, 2, device="cpu")
    assert c.codes.shape == (4, 32) and c.scales.shape == (4, 2)
    assert ep.SwigluCheckpoint(4, 129, 2, device="cpu").scales.shape == (4, 4)
    with pytest.raises(ValueError):
        c.save(g, *at)
    with pytest.raises(ValueError):  # more rows than are kept
        c.save(torch.zeros(5, 32, dtype=torch.bfloat16), *at)
    with pytest.raises(ValueError):
        c.backward(g, *at)


@pytest.mark.parametrize("stream", [None, 7])
def test_results_come_from_the_calls_stream(monkeypatch, stream):
    from combine_get_dispatch_amd import moe

    seen = []
    for name in ("_expert_product", "_backward_rows", "_save", "_use"):
        monkeypatch.setattr(moe, name, lambda *a: seen.append(a[-1]))
    monkeypatch.setattr(moe, "ep_expert_product_backward_weights",
                        lambda *a, **k: seen.append(k["stream"]))

    def empty(s, *size, **kw):
        seen.append(s)
        return torch.empty(*size, **kw)

    monkeypatch.setattr(moe, "_empty", empty)
    x, g = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.bfloat16)
    e = ep.Bf16Experts(torch.zeros(2, 32, 128, dtype=torch.bfloat16))
    assert e.product(x, None, None, None, stream=stream).shape == (4, 32)
    half = ep.Bf16Experts(e.weights, swiglu=True)
    assert half.product(x, None, None, None, stream=stream).shape == (4, 16)
    assert e.backward_rows(g, None, None, stream=stream).shape == (4, 128)
    gw = e.backward_weights(x, None, g, None, None, stream=stream)
    assert gw.shape == (2, 32, 128) and gw.dtype == torch.bfloat16
    gw = e.backward_weights(x, None, g, None, None, add=gw.float(), stream=stream)
    assert gw.dtype == torch.float32
    assert e.backward_weights(x, None, g, None, None, out=gw, stream=stream) is gw
    c = ep.SwigluCheckpoint(4, 16, 2, device="cpu")
    assert c.save(g, None, None, stream=stream).shape == (4, 16)
    a, b = c.backward(g[:, :16], None, None, stream=stream)
    assert a.shape == (4, 32) and b.shape == (4, 16)
    assert set(seen) == {stream} and len(seen) == 7 + 8 + 1


def test_e4m3_form_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = np.unique(codes[np.isfinite(codes)])
    assert np.array_equal(ref.e4m3(codes), codes)
    v = np.concatenate([(codes[1:] + codes[:-1]) / 2, np.linspace(-448, 448, 4001),
                        2.0 ** np.arange(-14, 8)])  # ties, values, powers of two
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(v.astype(np.float32).astype(np.float64)), want)


def test_plain_gradients_against_differences():
    rng = np.random.default_rng(3)
    off, cnt = [0, 3, 5], [3, 0, 4]
    x, w = rng.normal(size=(9, 5)), rng.normal(size=(3, 4, 5))
    g = rng.normal(size=(9, 4))

    def total(x, w):
        return np.nansum(ref.product(x, w, off, cnt)[0] * g)

    step = 1e-6
    gx, gw = ref.rows_grad(g, w, off, cnt)[0], ref.weights_grad(g, x, off, cnt)[0]
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = step
        want = (total(x + d, w) - total(x - d, w)) / (2 * step)
        assert abs(want - (0 if np.isnan(gx[i]) else gx[i])) < 1e-7
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = step
        assert abs((total(x, w + d) - total(x, w - d)) / (2 * step) - gw[i]) < 1e-7
    v, gh = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    gv, h = ref.swiglu_grad(v, gh)
    assert np.allclose(h, ref.silu(v[:, :4]) * v[:, 4:])
    for i in np.ndindex(v.shape):
        d = np.zeros_like(v)
        d[i] = step
        a, b = (np.sum(ref.swiglu_grad(v + t, gh)[1] * gh) for t in (d, -d))
        assert abs((a - b) / (2 * step) - gv[i]) < 1e-7


@pytest.mark.parametrize("N,K", [(64, 64), (32, 128)])
def test_weights_are_looked_at_at_each_call(N, K):
    """A tensor's storage, shape, strides and type may be replaced with the
    address unchanged."""
    def other(change):
        t = torch.zeros(2, N, K, dtype=torch.bfloat16)
        e, at = ep.Bf16Experts(t), t.data_ptr()
        t.data = change(t)
        assert t.data_ptr() == at
        return e

    for change in (lambda t: t.transpose(1, 2), lambda t: t[:1], lambda t: t[:, :N // 2],
                   lambda t: t[:, :, :K // 2], lambda t: t[:, ::2], lambda t: t.view(2, K, N)
                   if N != K else t.view(4, N // 2, K), lambda t: t.view(torch.float16),
                   lambda t: t.view(torch.int16)):
        with pytest.raises(ValueError, match="^w "):
            other(change)._where()
    t = torch.zeros(2, N, K, dtype=torch.bfloat16)
    e = ep.Bf16Experts(t)
    t.data = torch.zeros_like(t)
    assert e._where() == (-1, t.data_ptr())


def test_checkpoint_is_looked_at_at_each_call():
    """Its tensors' storage may be replaced; what does not fit is refused."""
    c = ep.SwigluCheckpoint(4, 200, 2, device="cpu")
    for t, name in ((c.codes, "codes"), (c.scales, "scales")):
        was = t.data
        t.data = torch.ones_like(was)  # moved: the calls take it where it is
        assert c._where() == (-1, 4, c.codes.data_ptr(), c.scales.data_ptr())
        for other in (was[:3], was.t().contiguous().t(), was.view(torch.int8), was[:, :1]):
            t.data = other
            with pytest.raises(ValueError, match=f"^{name} "):
                c._where()
        t.data = was
    assert c._where() == (-1, 4, c.codes.data_ptr(), c.scales.data_ptr())


def test_weights_whose_storage_was_freed():
    """Views of a flat tensor whose storage is given back between steps."""
    from combine_get_dispatch_amd import moe

    flat = torch.zeros(4, 32, 128, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 1, 2, 1, 1024, dtype=torch.uint8), torch.zeros(
        4, 1, 2, 1, 16, dtype=torch.bfloat16)
    experts = [ep.Bf16Experts(flat), ep.Bf16Experts(flat[2:])]
    packed = moe._packed(codes[2:], scales[2:], None)
    calls = [e._where for e in experts] + [lambda: moe._packed_at(packed)]
    for call in calls:
        call()
    for t in (flat, codes, scales):
        for n in (0, 16):
            size = t.untyped_storage().nbytes()
            t.untyped_storage().resize_(n)
            for call in calls[:2] if t is flat else calls[2:]:
                with pytest.raises(ValueError, match="storage"):
                    call()
            t.untyped_storage().resize_(size)
            for call in calls:
                call()
