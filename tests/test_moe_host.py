"""Refusals of the router's and the experts' products' entry points: each
call below is rejected before anything touches a device, so these run
without one."""
import ctypes

import pytest
import torch

import combine_get_dispatch_amd as ep


def _fake(n):
    return ctypes.c_void_p(0x100000 * n)  # never dereferenced: rejected first


def _router(T=16, E=8, k=2, score=0, G=1, tg=1, topn=1, norm=1, scale=1.0):
    return ep.ep_router_t(T, E, k, score, G, tg, topn, norm, scale)


def _route(r, dtype=ep.EP_DTYPE_F32, logits=_fake(1), idx=_fake(2), w=_fake(3), status=_fake(4)):
    return ep.lib().ep_route(ctypes.byref(r), dtype, logits, None, None, idx, w, status, None)


BAD_ROUTERS = [
    dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(score=2),
    dict(score=-1), dict(G=0), dict(G=3), dict(E=130, G=65), dict(G=2, tg=3), dict(G=2, tg=0),
    dict(G=8, tg=1, k=2), dict(topn=0), dict(topn=3), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(T=(1 << 31) - 1, E=1024),
]


@pytest.mark.parametrize("bad", BAD_ROUTERS, ids=str)
def test_bad_router_rejected(bad):
    r = _router(**bad)
    assert _route(r) == ep.EP_ERR_INVALID_ARG and ep.lib().ep_last_error()
    with pytest.raises(ep.EpError):
        ep.ep_balance_workspace_bytes(r, 1)
    st = ep.lib().ep_route_backward(ctypes.byref(r), ep.EP_DTYPE_F32, _fake(1), _fake(2), None,
                                    None, None, 1, None, _fake(3), _fake(4), None)
    assert st == ep.EP_ERR_INVALID_ARG


def test_route_rejections():
    r = _router()
    assert ep.lib().ep_route(None, 2, _fake(1), None, None, _fake(2), _fake(3), _fake(4),
                             None) == ep.EP_ERR_INVALID_ARG
    assert _route(r, dtype=ep.EP_DTYPE_FP8_E4M3) == ep.EP_ERR_INVALID_ARG
    assert _route(r, logits=None) == ep.EP_ERR_INVALID_ARG
    assert _route(r, logits=ctypes.c_void_p(0x100002)) == ep.EP_ERR_INVALID_ARG
    for kw in (dict(idx=None), dict(w=None), dict(status=None)):
        assert _route(r, **kw) == ep.EP_ERR_INVALID_ARG
    assert _route(_router(T=0), logits=None, idx=None, w=None, status=None) == ep.EP_OK


def _balance(r, S=1, seqs=None, coef=1.0, ws=_fake(5), wsb=1 << 20, outs=None, dtype=2,
             idx=_fake(2)):
    outs = [_fake(6 + i) for i in range(6)] if outs is None else outs
    return ep.lib().ep_balance_loss(ctypes.byref(r), dtype, _fake(1), idx, seqs, S, coef, ws, wsb,
                                    *outs, None)


def test_balance_rejections():
    r = _router()
    assert _balance(r, S=0) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, S=2) == ep.EP_ERR_INVALID_ARG          # several sequences, no offsets
    assert _balance(r, S=1 << 24, seqs=_fake(3)) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, coef=float("nan")) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, wsb=16) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, ws=ctypes.c_void_p(0x100010)) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, ws=None) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, dtype=1) == ep.EP_ERR_INVALID_ARG
    assert _balance(r, idx=None) == ep.EP_ERR_INVALID_ARG
    for i in range(6):
        outs = [_fake(6 + j) for j in range(6)]
        outs[i] = None
        assert _balance(r, outs=outs) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_balance_workspace_bytes(_router(T=0), 1) > 0


def test_backward_rejections():
    r = _router()

    def call(dtype=2, logits=_fake(1), idx=_fake(2), q=None, seqs=None, S=1, out=_fake(3),
             status=_fake(4)):
        return ep.lib().ep_route_backward(ctypes.byref(r), dtype, logits, idx, None, q, seqs, S,
                                          None, out, status, None)

    for kw in (dict(dtype=1), dict(logits=None), dict(idx=None), dict(out=None),
               dict(status=None), dict(q=_fake(5), S=2), dict(q=_fake(5), S=0),
               dict(out=ctypes.c_void_p(0x100002))):
        assert call(**kw) == ep.EP_ERR_INVALID_ARG


def _w4(E=2, K=256, N=32, group=128, swiglu=0):
    return ep.ep_w4_t(E, K, N, group, swiglu)


@pytest.mark.parametrize("bad", [dict(E=0), dict(E=1025), dict(K=0), dict(K=-128), dict(K=192),
                                 dict(K=1 << 24), dict(N=0), dict(N=1 << 20), dict(group=16),
                                 dict(group=256), dict(K=48, group=32)], ids=str)
def test_bad_w4_rejected(bad):
    w = _w4(**bad)
    with pytest.raises(ep.EpError):
        ep.ep_w4_packed_sizes(w)
    L = ep.lib()
    assert L.ep_w4_pack(ctypes.byref(w), _fake(1), _fake(2), None, _fake(3), _fake(4), None,
                        None) == ep.EP_ERR_INVALID_ARG
    assert L.ep_expert_product_w4(ctypes.byref(w), 0, _fake(1), None, _fake(2), _fake(3), None,
                                  _fake(4), _fake(5), 8, _fake(6), None) == ep.EP_ERR_INVALID_ARG


def test_packed_sizes():
    assert ep.ep_w4_packed_sizes(_w4()) == (2 * 2 * 2 * 1024, 2 * 2 * 2 * 16)
    assert ep.ep_w4_packed_sizes(_w4(E=3, K=96, N=17, group=32, swiglu=1)) == (
        3 * 2 * 2 * 1024, 3 * 2 * 2 * 3 * 16)


def test_product_rejections():
    w = _w4()
    L = ep.lib()

    def call(w=w, dtype=0, x=_fake(1), xs=None, codes=_fake(2), scales=_fake(3), off=_fake(4),
             cnt=_fake(5), cap=8, out=_fake(6)):
        return L.ep_expert_product_w4(ctypes.byref(w), dtype, x, xs, codes, scales, None, off, cnt,
                                      cap, out, None)

    for kw in (dict(dtype=2), dict(dtype=1), dict(x=None), dict(codes=None), dict(scales=None),
               dict(off=None), dict(cnt=None), dict(cap=-1), dict(cap=(1 << 31) - 1),
               dict(out=None), dict(x=ctypes.c_void_p(0x100008)),
               dict(out=_fake(1)), dict(out=ctypes.c_void_p(0x100000 + 8 * 256 * 2 - 2)),
               dict(x=ctypes.c_void_p(0x600000 + 8 * 32 * 2 - 16)),
               dict(w=_w4(E=1024), cap=1 << 28),
               dict(codes=ctypes.c_void_p(0x100008)),
               dict(w=_w4(K=96, group=32), dtype=1, xs=_fake(7))):
        assert call(**kw) == ep.EP_ERR_INVALID_ARG, kw
    assert call(cap=0, x=None, out=None) == ep.EP_OK
    assert L.ep_w4_pack(ctypes.byref(w), _fake(1), _fake(2), _fake(3), _fake(4), _fake(5), None,
                        None) == ep.EP_ERR_INVALID_ARG
    assert L.ep_w4_pack(ctypes.byref(w), _fake(1), None, None, _fake(4), _fake(5), None,
                        None) == ep.EP_ERR_INVALID_ARG


def test_python_checks():
    with pytest.raises(ValueError):
        ep.EpRouter(4, 8, 2, score="tanh", device="cpu")
    with pytest.raises(ep.EpError):
        ep.EpRouter(4, 8, 9, device="cpu")
    r = ep.EpRouter(4, 8, 2, max_seqs=2, device="cpu")
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):  # host tensors
        r.route(x)
    with pytest.raises(ValueError):
        r.route(x.bfloat16())
    with pytest.raises(ValueError):
        r.balance_loss(x, r.topk_idx, 1.0, seq_offsets=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        r.balance_loss(x, r.topk_idx, 1.0, seq_offsets=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):  # two rows of scales for three of codes
        ep.W4Experts.pack(torch.zeros(1, 3, 16, dtype=torch.uint8),
                          torch.zeros(1, 3, 1, dtype=torch.bfloat16), swiglu=True)
    with pytest.raises(ep.EpError):  # groups of 16
        ep.W4Experts.pack(torch.zeros(1, 4, 16, dtype=torch.uint8),
                          torch.zeros(1, 4, 2, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ep.W4Experts(torch.zeros(1, 3, 1, 1, 1024, dtype=torch.uint8), torch.zeros(1), None, 16,
                     128, 128)


def test_status_names():
    assert ep.lib().ep_status_string(ep.EP_ERR_SEQS) != b"unknown status"
    assert ep.lib().ep_status_string(ep.EP_ERR_SEQS + 1) == b"unknown status"


def test_packed_weights_are_looked_at_at_each_call(monkeypatch):
    """Their tensors' storage may be replaced; what does not fit is refused."""
    from combine_get_dispatch_amd import moe

    monkeypatch.setattr(moe, "_device", lambda t, name: t.get_device())  # host tensors here
    E, K, N = 2, 256, 32
    for zeros in (False, True):
        codes = torch.zeros(E, 1, 2, 2, 1024, dtype=torch.uint8)
        scales = torch.zeros(E, 1, 2, 2, 16, dtype=torch.bfloat16)
        z = torch.zeros(E, 1, 2, 2, 16, dtype=torch.uint8) if zeros else None
        w = ep.W4Experts(codes, scales, z, N, K, 128)

        def at():
            return -1, [t if t is None else t.data_ptr() for t in (codes, scales, z)]

        assert moe._packed_at(w._weights) == at()
        for t, name in ((codes, "w_codes"), (scales, "w_scales"), (z, "w_zeros")):
            if t is None:
                continue
            was = t.data
            t.data = torch.ones_like(was)  # moved: the calls take it where it is
            assert moe._packed_at(w._weights) == at()
            for other in (was[:1], was.transpose(2, 3), was.view(torch.int8)):
                t.data = other
                with pytest.raises(ValueError, match=f"^{name} "):
                    moe._packed_at(w._weights)
            t.data = was
        assert moe._packed_at(w._weights) == at()
