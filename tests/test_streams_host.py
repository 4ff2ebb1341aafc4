"""Tensors that a call allocates come from the memory of the stream the call
runs on: a block of another stream's may still be read or written by work
queued there.  Shown without a device: torch's allocation and stream switch are
replaced by recorders, the library's calls by nothing."""
import contextlib
import types

import pytest
import torch

import combine_get_dispatch_amd as ep
from combine_get_dispatch_amd import moe


@pytest.fixture
def allocations(monkeypatch):
    """The stream of each allocation, in order (None: the current one)."""
    active, seen = [None], []
    empty = torch.empty

    class External:
        def __init__(self, handle, device=None):
            self.handle = handle

    @contextlib.contextmanager
    def switched(stream):
        active.append(stream.handle)
        yield
        active.pop()

    def recorded(*size, **kw):
        seen.append(active[-1])
        return empty(*size, **kw)

    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", switched)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch, "empty_like", lambda t, dtype=None: recorded(
        t.shape, dtype=dtype or t.dtype, device=t.device))
    return seen


def _experts():
    w = object.__new__(ep.W4Experts)
    w.cfg, w._ref, w._weights = ep.ep_w4_t(2, 128, 32, 128, 0), None, None
    return w


@pytest.mark.parametrize("stream", [None, 7])
def test_product_and_pack(monkeypatch, allocations, stream):
    for name in ("_product", "ep_w4_pack"):
        monkeypatch.setattr(moe, name, lambda *a, **k: None)
    monkeypatch.setattr(ep.W4Experts, "__init__", lambda self, *a: None)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    assert _experts().product(x, None, None, None, stream=stream).shape == (4, 32)
    ep.W4Experts.pack(torch.zeros(2, 32, 64, dtype=torch.uint8),
                      torch.zeros(2, 32, 1, dtype=torch.bfloat16),
                      torch.zeros(2, 32, 1, dtype=torch.uint8), stream=stream)
    assert allocations == [stream] * 4
    allocations.clear()
    out = torch.zeros(4, 32, dtype=torch.bfloat16)
    assert _experts().product(x, None, None, None, out=out, stream=stream) is out
    assert allocations == []


@pytest.mark.parametrize("stream", [None, 7])
def test_buffers(monkeypatch, allocations, stream):
    for name in ("ep_dispatch_backward", "ep_combine_backward", "ep_dispatch_ranked",
                 "ep_combine_ranked"):
        monkeypatch.setattr(ep, name, lambda *a, **k: None)
    b = object.__new__(ep.EpBuffers)
    b.__dict__.update(
        cfg=ep._cfg(4, 128, 2, 8, 2, 1), capacity=8, handle=None, fp8=True, expert_offsets=None,
        num_tokens_per_expert=None, recv_x=torch.zeros(8, 128, dtype=torch.uint8), status=None,
        recv_scales=None, workspace=None, tok_slot_row=None,
        out=torch.zeros(4, 128, dtype=torch.bfloat16))
    b.dispatch_backward(None, stream=stream)
    b.combine_backward(b.out, None, None, stream=stream)
    experts = types.SimpleNamespace(product=lambda *a, **k: k["stream"])
    assert b.expert_product(experts, stream=stream) is stream
    assert allocations == [stream] * 2
    b.dispatch_ranked(None, None, None, stream=stream)
    b.combine_ranked(None, stream=stream)
    assert len(allocations) > 8 and set(allocations) == {stream}
