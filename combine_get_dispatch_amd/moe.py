"""Python binding of include/ep_moe.h: the router in front of the dispatch /
combine path, and behind it the experts' products with 4-bit or bf16 weights,
the latter's gradients, and the 8-bit checkpoint of the SwiGLU between them.

The functions carry the C names and take preallocated torch tensors on the
current device; ``EpRouter``, ``W4Experts``, ``Bf16Experts`` and
``SwigluCheckpoint`` keep the buffers, the workspace and the weights of one
configuration.  The package exports all of them.
"""
from __future__ import annotations

import ctypes

from . import (EP_DTYPE_BF16, EP_DTYPE_F32, EP_DTYPE_FP8_E4M3, _check, _empty, _ptr, _stream,
               lib)

EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": EP_SCORE_SOFTMAX, "sigmoid": EP_SCORE_SIGMOID}


class ep_router_t(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_topk", ctypes.c_int32), ("score", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_topn", ctypes.c_int32), ("normalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class ep_w4_t(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32), ("group", ctypes.c_int32),
                ("swiglu", ctypes.c_int32)]


class ep_experts_t(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32)]


def register(L):
    """Argument types of this header's functions (called once, by lib())."""
    P, S, i32, i64, f32 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                           ctypes.c_float)
    router, w4 = ctypes.POINTER(ep_router_t), ctypes.POINTER(ep_w4_t)
    experts = ctypes.POINTER(ep_experts_t)
    types = {
        "ep_route": [router, ctypes.c_int, P, P, P, P, P, P, P],
        "ep_balance_workspace_bytes": [router, i32, ctypes.POINTER(S)],
        "ep_balance_loss": [router, ctypes.c_int, P, P, P, i32, f32, P, S, P, P, P, P, P, P, P],
        "ep_route_backward": [router, ctypes.c_int, P, P, P, P, P, i32, P, P, P, P],
        "ep_w4_packed_sizes": [w4, ctypes.POINTER(i64), ctypes.POINTER(i64)],
        "ep_w4_pack": [w4, P, P, P, P, P, P, P],
        "ep_expert_product_w4": [w4, ctypes.c_int, P, P, P, P, P, P, P, i64, P, P],
        "ep_expert_product": [experts, ctypes.c_int, P, P, P, i32, P, P, i64, P, P],
        "ep_expert_product_backward_rows": [experts, P, P, P, P, i64, P, P],
        "ep_expert_product_backward_weights": [experts, ctypes.c_int, P, P, P, P, P, i64,
                                               ctypes.c_int, P, P, P],
        "ep_swiglu_checkpoint": [i32, i32, P, P, P, i64, P, P, P, P],
        "ep_swiglu_checkpoint_backward": [i32, i32, P, P, P, P, P, i64, P, P, P],
    }
    for name, args in types.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int


def _device(t, name):
    """The current device, where the library launches: its tensors live there."""
    import torch

    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a device tensor")
    if d != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return d


def _at(t, dev, dtype, shape, name):
    """Device pointer of a contiguous tensor of this type and shape (None: any)
    on device dev; None passes NULL."""
    if t is None:
        return None
    if (t.dtype is dtype and (shape is None or t.shape == shape) and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    _ptr(t, dtype, shape, name)  # says what is wrong
    raise ValueError(f"{name} is on {t.device}, not on the current device")


def _logits_dtype(t):
    import torch

    if t.dtype == torch.float32:
        return EP_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return EP_DTYPE_BF16
    raise ValueError(f"logits must be float32 or bfloat16, not {t.dtype}")


def _num_seqs(seq_offsets):
    if seq_offsets is None:
        return 1
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets must be int32 [num_seqs + 1] with at least one sequence")
    return seq_offsets.numel() - 1


def ep_route(router: ep_router_t, logits, bias, token_mask, topk_idx, topk_weights, status,
             stream=None):
    import torch

    T, E, k = router.num_tokens, router.num_experts, router.num_topk
    d = _device(logits, "logits")
    st = lib().ep_route(
        ctypes.byref(router), _logits_dtype(logits),
        _at(logits, d, logits.dtype, (T, E), "logits"),
        _at(bias, d, torch.float32, (E,), "bias"),
        _at(token_mask, d, torch.uint8, (T,), "token_mask"),
        _at(topk_idx, d, torch.int32, (T, k), "topk_idx"),
        _at(topk_weights, d, torch.float32, (T, k), "topk_weights"),
        _at(status, d, torch.int32, (1,), "status"), _stream(stream))
    _check(st, "ep_route")


def ep_balance_workspace_bytes(router: ep_router_t, num_seqs: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().ep_balance_workspace_bytes(ctypes.byref(router), int(num_seqs),
                                            ctypes.byref(n)), "ep_balance_workspace_bytes")
    return n.value


def ep_balance_loss(router: ep_router_t, logits, topk_idx, seq_offsets, coef, workspace, counts,
                    seq_tokens, mean_probs, prob_grad, loss, status, stream=None):
    import torch

    T, E, k, S = router.num_tokens, router.num_experts, router.num_topk, _num_seqs(seq_offsets)
    i32, f32, d = torch.int32, torch.float32, _device(logits, "logits")
    st = lib().ep_balance_loss(
        ctypes.byref(router), _logits_dtype(logits),
        _at(logits, d, logits.dtype, (T, E), "logits"),
        _at(topk_idx, d, i32, (T, k), "topk_idx"),
        _at(seq_offsets, d, i32, None, "seq_offsets"), S, float(coef),
        _at(workspace, d, torch.uint8, None, "workspace"), workspace.numel(),
        _at(counts, d, i32, (S, E), "counts"), _at(seq_tokens, d, i32, (S,), "seq_tokens"),
        _at(mean_probs, d, f32, (S, E), "mean_probs"),
        _at(prob_grad, d, f32, (S, E), "prob_grad"), _at(loss, d, f32, (1,), "loss"),
        _at(status, d, i32, (1,), "status"), _stream(stream))
    _check(st, "ep_balance_loss")


def ep_route_backward(router: ep_router_t, logits, topk_idx, grad_weights, prob_grad, seq_offsets,
                      grad_loss, grad_logits, status, stream=None):
    import torch

    T, E, k = router.num_tokens, router.num_experts, router.num_topk
    S = _num_seqs(seq_offsets) if prob_grad is not None else 1
    i32, f32, d = torch.int32, torch.float32, _device(logits, "logits")
    st = lib().ep_route_backward(
        ctypes.byref(router), _logits_dtype(logits),
        _at(logits, d, logits.dtype, (T, E), "logits"),
        _at(topk_idx, d, i32, (T, k), "topk_idx"),
        _at(grad_weights, d, f32, (T, k), "grad_weights"),
        _at(prob_grad, d, f32, (S, E), "prob_grad"),
        _at(seq_offsets, d, i32, None, "seq_offsets"), S,
        _at(grad_loss, d, f32, (1,), "grad_loss"),
        _at(grad_logits, d, logits.dtype, (T, E), "grad_logits"),
        _at(status, d, i32, (1,), "status"), _stream(stream))
    _check(st, "ep_route_backward")


def ep_w4_packed_sizes(w4: ep_w4_t):
    """Bytes of the packed codes, and values of the packed scales (and zeros)."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ep_w4_packed_sizes(ctypes.byref(w4), ctypes.byref(a), ctypes.byref(b)),
           "ep_w4_packed_sizes")
    return a.value, b.value


def ep_w4_pack(w4: ep_w4_t, codes, scales, zeros, w_codes, w_scales, w_zeros, stream=None):
    import torch

    rows = (2 if w4.swiglu else 1) * w4.out_features
    groups = (w4.num_experts, rows, w4.in_features // w4.group)
    nb, ns = ep_w4_packed_sizes(w4)
    _sized(w_codes, nb, "w_codes")
    _sized(w_scales, ns, "w_scales")
    _sized(w_zeros, ns, "w_zeros")
    d = _device(codes, "codes")
    st = lib().ep_w4_pack(
        ctypes.byref(w4),
        _at(codes, d, torch.uint8, (w4.num_experts, rows, w4.in_features // 2), "codes"),
        _at(scales, d, torch.bfloat16, groups, "scales"),
        _at(zeros, d, torch.uint8, groups, "zeros"),
        _at(w_codes, d, torch.uint8, None, "w_codes"),
        _at(w_scales, d, torch.bfloat16, None, "w_scales"),
        _at(w_zeros, d, torch.uint8, None, "w_zeros"), _stream(stream))
    _check(st, "ep_w4_pack")


def _sized(t, n, name):
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} values, expected {n}")


def ep_expert_product_w4(w4: ep_w4_t, x, x_scales, w_codes, w_scales, w_zeros, expert_offsets,
                         num_tokens_per_expert, out, stream=None):
    """x: bf16 [capacity, K], or uint8 E4M3 codes with x_scales.  expert_offsets
    may have one entry more than there are experts, as the layout's has."""
    nb, ns = ep_w4_packed_sizes(w4)
    _sized(w_codes, nb, "w_codes")
    _sized(w_scales, ns, "w_scales")
    _sized(w_zeros, ns, "w_zeros")
    _product(w4, ctypes.byref(w4), x, x_scales, _packed(w_codes, w_scales, w_zeros),
             expert_offsets, num_tokens_per_expert, out, stream)


def _packed(w_codes, w_scales, w_zeros):
    """What _weights_kept_at takes for each of the packed tensors, or None."""
    import torch

    return [None if t is None else (t, dtype, t.shape, name) for t, dtype, name in
            ((w_codes, torch.uint8, "w_codes"), (w_scales, torch.bfloat16, "w_scales"),
             (w_zeros, torch.uint8, "w_zeros"))]


def _packed_at(packed):
    """Their device, and the pointers, at this call."""
    dev, codes = _weights_kept_at(*packed[0])
    pointers = [codes]
    for p in packed[1:]:
        d, at = (dev, None) if p is None else _weights_kept_at(*p)
        if d != dev:
            raise ValueError(f"{p[3]} is on {p[0].device}, w_codes on {packed[0][0].device}")
        pointers.append(at)
    return dev, pointers


def _product(w4, ref, x, x_scales, weights, expert_offsets, num_tokens_per_expert, out, stream):
    import torch

    K, N, E = w4.in_features, w4.out_features, w4.num_experts
    fp8 = x_scales is not None
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected (rows, {K})")
    cap = x.shape[0]
    if out.dim() != 2 or out.shape[1] != N or out.shape[0] < cap:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected (>= {cap}, {N})")
    if expert_offsets.dim() != 1 or expert_offsets.shape[0] not in (E, E + 1):
        raise ValueError(f"expert_offsets has shape {tuple(expert_offsets.shape)}, "
                         f"expected ({E},) or ({E + 1},)")
    d = _device(x, "x")
    at, pointers = _packed_at(weights)
    if d != at:
        raise ValueError("the weights are not on the current device")
    st = lib().ep_expert_product_w4(
        ref, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _at(x, d, torch.uint8 if fp8 else torch.bfloat16, None, "x"),
        _at(x_scales, d, torch.float32, (cap, K // 128), "x_scales"), *pointers,
        _at(expert_offsets, d, torch.int32, None, "expert_offsets"),
        _at(num_tokens_per_expert, d, torch.int32, (E,), "num_tokens_per_expert"), cap,
        _at(out, d, torch.bfloat16, None, "out"), _stream(stream))
    _check(st, "ep_expert_product_w4")


def _expert_rows(t, cols, name):
    """Rows of a tensor [capacity, cols]."""
    s = t.shape
    if len(s) != 2 or s[1] != cols:
        raise ValueError(f"{name} has shape {tuple(s)}, expected (rows, {cols})")
    return s[0]


def _rows_at(t, dev, dtype, rows, cols, name):
    """Device pointer of a contiguous tensor of at least these rows; None passes NULL."""
    if t is None:
        return None
    s = t.shape
    if len(s) != 2 or s[1] != cols or s[0] < rows:
        raise ValueError(f"{name} has shape {tuple(s)}, expected (>= {rows}, {cols})")
    return _at(t, dev, dtype, s, name)


def _expert_at(expert_offsets, num_tokens_per_expert, E, d):
    """Pointers of the layout's arrays; expert_offsets may have one entry more
    than there are experts, as the layout's has."""
    import torch

    if expert_offsets.dim() != 1 or expert_offsets.shape[0] not in (E, E + 1):
        raise ValueError(f"expert_offsets has shape {tuple(expert_offsets.shape)}, "
                         f"expected ({E},) or ({E + 1},)")
    return (_at(expert_offsets, d, torch.int32, None, "expert_offsets"),
            _at(num_tokens_per_expert, d, torch.int32, (E,), "num_tokens_per_expert"))


def _x_at(x, x_scales, K, d):
    """Type and pointers of bf16 rows, or of E4M3 codes and their scales."""
    import torch

    if x_scales is None:
        return EP_DTYPE_BF16, _at(x, d, torch.bfloat16, None, "x"), None
    return (EP_DTYPE_FP8_E4M3, _at(x, d, torch.uint8, None, "x"),
            _at(x_scales, d, torch.float32, (x.shape[0], K // 128), "x_scales"))


def _weight_shape(experts):
    return experts.num_experts, experts.out_features, experts.in_features


def _weights_at(w, experts):
    """Their device, and the pointer."""
    import torch

    d = _device(w, "w")
    return d, _at(w, d, torch.bfloat16, _weight_shape(experts), "w")


def _kept_at(t, dtype, shape, name):
    """Device and pointer of a contiguous tensor of this type and shape.  For
    tensors that an object holds from call to call: their storage, shape, strides
    and type may have been replaced (by ``.data``), the address left as it was."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} with strides {t.stride()}, "
                         f"expected contiguous {dtype} {tuple(shape)}")
    return t.get_device(), t.data_ptr()


def _weights_kept_at(t, dtype, shape, name):
    """The same of weights, which may be a part of a larger tensor whose storage
    is given back for a while: a part of none still has an address."""
    if t.untyped_storage().nbytes() < (t.storage_offset() + t.numel()) * t.itemsize:
        raise ValueError(f"{name} reaches past the end of its storage")
    return _kept_at(t, dtype, shape, name)


def _here(t, name, other, what):
    """The device of a call whose weights or checkpoint are on `other`."""
    d = _device(t, name)
    if d != other:
        raise ValueError(f"{what} not on the current device")
    return d


def ep_expert_product(experts: ep_experts_t, x, x_scales, w, swiglu, expert_offsets,
                      num_tokens_per_expert, out, stream=None):
    """x: bf16 [capacity, K], or uint8 E4M3 codes with x_scales."""
    _device(x, "x")
    _expert_product(experts, ctypes.byref(experts), x, x_scales, _weights_at(w, experts),
                    1 if swiglu else 0, expert_offsets, num_tokens_per_expert, out, stream)


def _expert_product(experts, ref, x, x_scales, w, swiglu, expert_offsets, num_tokens_per_expert,
                    out, stream):
    import torch

    K, N = experts.in_features, experts.out_features
    cap = _expert_rows(x, K, "x")
    d = _here(x, "x", w[0], "the weights are")
    st = lib().ep_expert_product(
        ref, *_x_at(x, x_scales, K, d), w[1], swiglu,
        *_expert_at(expert_offsets, num_tokens_per_expert, experts.num_experts, d), cap,
        _rows_at(out, d, torch.bfloat16, cap, N // 2 if swiglu else N, "out"), _stream(stream))
    if st:
        _check(st, "ep_expert_product")


def ep_expert_product_backward_rows(experts: ep_experts_t, grad_out, w, expert_offsets,
                                    num_tokens_per_expert, grad_x, stream=None):
    _device(grad_out, "grad_out")
    _backward_rows(experts, ctypes.byref(experts), grad_out, _weights_at(w, experts),
                   expert_offsets, num_tokens_per_expert, grad_x, stream)


def _backward_rows(experts, ref, grad_out, w, expert_offsets, num_tokens_per_expert, grad_x,
                   stream):
    import torch

    N = experts.out_features
    cap = _expert_rows(grad_out, N, "grad_out")
    d = _here(grad_out, "grad_out", w[0], "the weights are")
    st = lib().ep_expert_product_backward_rows(
        ref, _at(grad_out, d, torch.bfloat16, None, "grad_out"), w[1],
        *_expert_at(expert_offsets, num_tokens_per_expert, experts.num_experts, d), cap,
        _rows_at(grad_x, d, torch.bfloat16, cap, experts.in_features, "grad_x"), _stream(stream))
    if st:
        _check(st, "ep_expert_product_backward_rows")


def ep_expert_product_backward_weights(experts: ep_experts_t, x, x_scales, grad_out,
                                       expert_offsets, num_tokens_per_expert, add, grad_w,
                                       stream=None):
    """grad_w: bf16 or fp32 [experts, N, K], written whole; add: the same type
    and shape (grad_w itself to add to it), or None."""
    import torch

    K, N = experts.in_features, experts.out_features
    cap = _expert_rows(grad_out, N, "grad_out")
    if _expert_rows(x, K, "x") != cap:
        raise ValueError(f"x has {x.shape[0]} rows, grad_out {cap}")
    dtype = grad_w.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"grad_w must be float32 or bfloat16, not {dtype}")
    d, shape = _device(grad_out, "grad_out"), _weight_shape(experts)
    st = lib().ep_expert_product_backward_weights(
        ctypes.byref(experts), *_x_at(x, x_scales, K, d),
        _at(grad_out, d, torch.bfloat16, None, "grad_out"),
        *_expert_at(expert_offsets, num_tokens_per_expert, experts.num_experts, d), cap,
        EP_DTYPE_F32 if dtype is torch.float32 else EP_DTYPE_BF16,
        _at(add, d, dtype, shape, "add"), _at(grad_w, d, dtype, shape, "grad_w"),
        _stream(stream))
    if st:
        _check(st, "ep_expert_product_backward_weights")


def _checkpoint_shape(cap, features):
    return cap, 2 * -(-features // 128)


def _checkpoint_at(codes, scales, features):
    """Their device, rows and pointers."""
    import torch

    rows = _expert_rows(codes, 2 * features, "codes")
    if scales.shape[0] < rows:
        rows = scales.shape[0]
    d = _device(codes, "codes")
    return (d, rows, _at(codes, d, torch.uint8, None, "codes"),
            _rows_at(scales, d, torch.float32, 0, _checkpoint_shape(0, features)[1], "scales"))


def ep_swiglu_checkpoint(num_experts, features, gate_up, expert_offsets, num_tokens_per_expert, h,
                         codes, scales, stream=None):
    _device(gate_up, "gate_up")
    _save(num_experts, features, gate_up, expert_offsets, num_tokens_per_expert, h,
          _checkpoint_at(codes, scales, features), stream)


def _save(num_experts, features, gate_up, expert_offsets, num_tokens_per_expert, h, kept, stream):
    import torch

    cap = _expert_rows(gate_up, 2 * features, "gate_up")
    if kept[1] < cap:
        raise ValueError(f"gate_up has {cap} rows, the checkpoint {kept[1]}")
    d = _here(gate_up, "gate_up", kept[0], "the checkpoint is")
    st = lib().ep_swiglu_checkpoint(
        num_experts, features, _at(gate_up, d, torch.bfloat16, None, "gate_up"),
        *_expert_at(expert_offsets, num_tokens_per_expert, num_experts, d), cap,
        _rows_at(h, d, torch.bfloat16, cap, features, "h"), kept[2], kept[3], _stream(stream))
    if st:
        _check(st, "ep_swiglu_checkpoint")


def ep_swiglu_checkpoint_backward(num_experts, features, codes, scales, grad_h, expert_offsets,
                                  num_tokens_per_expert, grad_gate_up, h, stream=None):
    _device(grad_h, "grad_h")
    _use(num_experts, features, _checkpoint_at(codes, scales, features), grad_h, expert_offsets,
         num_tokens_per_expert, grad_gate_up, h, stream)


def _use(num_experts, features, kept, grad_h, expert_offsets, num_tokens_per_expert, grad_gate_up,
         h, stream):
    import torch

    cap = _expert_rows(grad_h, features, "grad_h")
    if kept[1] < cap:
        raise ValueError(f"grad_h has {cap} rows, the checkpoint {kept[1]}")
    d = _here(grad_h, "grad_h", kept[0], "the checkpoint is")
    st = lib().ep_swiglu_checkpoint_backward(
        num_experts, features, kept[2], kept[3],
        _at(grad_h, d, torch.bfloat16, None, "grad_h"),
        *_expert_at(expert_offsets, num_tokens_per_expert, num_experts, d), cap,
        _rows_at(grad_gate_up, d, torch.bfloat16, cap, 2 * features, "grad_gate_up"),
        _rows_at(h, d, torch.bfloat16, cap, features, "h"), _stream(stream))
    if st:
        _check(st, "ep_swiglu_checkpoint_backward")


class EpRouter:
    """The router of one configuration: selection, balance loss and their
    gradient, with the outputs and the workspace allocated once.  Results are
    views of these buffers: the next call of the same method overwrites them.
    One call at a time may use them (as the workspace of EpBuffers).  They are
    made on the current stream: another stream waits for it before its first
    call."""

    def __init__(self, num_tokens, num_experts, num_topk, score="softmax", groups=1,
                 topk_groups=1, group_topn=1, normalize=True, scale=1.0, logits_dtype=None,
                 max_seqs=1, device="cuda"):
        import torch

        if score not in _SCORES:
            raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
        self.cfg = ep_router_t(num_tokens, num_experts, num_topk, _SCORES[score], groups,
                               topk_groups, group_topn, 1 if normalize else 0, float(scale))
        self.logits_dtype = torch.float32 if logits_dtype is None else logits_dtype
        self.max_seqs = int(max_seqs)
        dev = torch.device(device)
        T, E, k, S = num_tokens, num_experts, num_topk, self.max_seqs
        i32, f32 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.float32, device=dev)
        ws = ep_balance_workspace_bytes(self.cfg, S)  # checks the configuration too
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, **i32)
        self.topk_idx = torch.empty((T, k), **i32)
        self.topk_weights = torch.empty((T, k), **f32)
        self.loss = torch.empty(1, **f32)
        self.grad_logits = torch.empty((T, E), dtype=self.logits_dtype, device=dev)
        self._counts, self._seq_tokens = torch.empty((S, E), **i32), torch.empty(S, **i32)
        self._mean_probs = torch.empty((S, E), **f32)
        self._prob_grad = torch.empty((S, E), **f32)
        self._views(S)

    def _views(self, S):
        if S > self.max_seqs:
            raise ValueError(f"{S} sequences, but the buffers hold max_seqs = {self.max_seqs}")
        self.counts, self.seq_tokens = self._counts[:S], self._seq_tokens[:S]
        self.mean_probs, self.prob_grad = self._mean_probs[:S], self._prob_grad[:S]

    def _typed(self, logits):
        if logits.dtype != self.logits_dtype:
            raise ValueError(f"logits has dtype {logits.dtype}, expected {self.logits_dtype}")

    def route(self, logits, bias=None, token_mask=None, stream=None):
        """Expert ids [T, k] (-1: none) and gates [T, k] of the k best experts."""
        self._typed(logits)
        ep_route(self.cfg, logits, bias, token_mask, self.topk_idx, self.topk_weights,
                 self.status, stream=stream)
        return self.topk_idx, self.topk_weights

    def balance_loss(self, logits, topk_idx, coef, seq_offsets=None, stream=None):
        """The loss [1]; fills counts, seq_tokens, mean_probs and prob_grad."""
        self._typed(logits)
        S = _num_seqs(seq_offsets)
        if S != self.counts.shape[0]:
            self._views(S)
        ep_balance_loss(self.cfg, logits, topk_idx, seq_offsets, coef, self.workspace,
                        self.counts, self.seq_tokens, self.mean_probs, self.prob_grad, self.loss,
                        self.status, stream=stream)
        return self.loss

    def backward(self, logits, topk_idx, grad_weights, prob_grad=None, seq_offsets=None,
                 grad_loss=None, grad_logits=None, stream=None):
        """Gradient for the logits of the gates (grad_weights, or None) and of
        the balance loss (prob_grad of its forward, times grad_loss)."""
        self._typed(logits)
        out = self.grad_logits if grad_logits is None else grad_logits
        ep_route_backward(self.cfg, logits, topk_idx, grad_weights, prob_grad, seq_offsets,
                          grad_loss, out, self.status, stream=stream)
        return out

    def check_status(self, stream=None):
        from . import ep_read_status

        ep_read_status(self.status, stream=stream)


class W4Experts:
    """Packed 4-bit weights of a set of experts (W4Experts.pack lays out
    row-major ones) and their product.  They are read in place at each call, and
    may be rewritten in place or moved (by ``.data``); other tensors are another
    W4Experts."""

    def __init__(self, w_codes, w_scales, w_zeros, out_features, in_features, group):
        if w_codes.dim() < 2:
            raise ValueError("w_codes must be [experts, halves, ...]")
        E, halves = w_codes.shape[:2]
        if halves not in (1, 2):
            raise ValueError(f"w_codes has {halves} matrices per expert, expected 1 or 2")
        self.cfg = ep_w4_t(E, in_features, out_features, group, 1 if halves == 2 else 0)
        nb, ns = ep_w4_packed_sizes(self.cfg)
        _sized(w_codes, nb, "w_codes")
        _sized(w_scales, ns, "w_scales")
        _sized(w_zeros, ns, "w_zeros")
        self._tensors = w_codes, w_scales, w_zeros
        self._ref = ctypes.byref(self.cfg)
        self._weights = _packed(w_codes, w_scales, w_zeros)
        _device(w_codes, "w_codes")
        _packed_at(self._weights)

    @property
    def w_codes(self):
        return self._tensors[0]

    @property
    def w_scales(self):
        return self._tensors[1]

    @property
    def w_zeros(self):
        return self._tensors[2]

    @classmethod
    def pack(cls, codes, scales, zeros=None, swiglu=False, stream=None):
        """codes uint8 [experts, rows, K / 2] (column 2 i in the low half of
        byte i), scales bf16 and zeros uint8 [experts, rows, K / group]; with
        swiglu the rows are the gate's, then the up projection's."""
        import torch

        if codes.dim() != 3 or scales.dim() != 3 or scales.shape[2] < 1:
            raise ValueError("codes and scales must be [experts, rows, columns]")
        E, rows, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
        halves = 2 if swiglu else 1
        if rows % halves or K % scales.shape[2]:
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} "
                             "do not make whole matrices and groups")
        N, group = rows // halves, K // scales.shape[2]
        cfg = ep_w4_t(E, K, N, group, 1 if swiglu else 0)
        ep_w4_packed_sizes(cfg)
        n16, k128, dev = -(-N // 16), -(-K // 128), codes.device
        w_codes = _empty(stream, (E, halves, n16, k128, 1024), dtype=torch.uint8, device=dev)
        groups = (E, halves, n16, K // group, 16)
        w_scales = _empty(stream, groups, dtype=torch.bfloat16, device=dev)
        w_zeros = (_empty(stream, groups, dtype=torch.uint8, device=dev)
                   if zeros is not None else None)
        ep_w4_pack(cfg, codes, scales, zeros, w_codes, w_scales, w_zeros, stream=stream)
        return cls(w_codes, w_scales, w_zeros, N, K, group)

    def product(self, x, x_scales, expert_offsets, num_tokens_per_expert, out=None, stream=None):
        """bf16 [rows, out_features]: each expert's rows times its weights.
        Rows that are no expert's are left as they are.  Without ``out`` the
        result belongs to the stream the call runs on."""
        import torch

        if out is None:
            out = _empty(stream, (x.shape[0], self.cfg.out_features), dtype=torch.bfloat16,
                         device=x.device)
        _product(self.cfg, self._ref, x, x_scales, self._weights, expert_offsets,
                 num_tokens_per_expert, out, stream)
        return out


class Bf16Experts:
    """bf16 weights [experts, out_features, in_features] of a set of experts,
    their product and its gradients.  With swiglu the rows of a weight matrix
    are the gate's, then the up projection's, and ``product`` gives
    silu(gate) * up; the gradients are those of the plain product (gate and
    up), which an object without swiglu on the same weights gives.  The
    weights are read in place at each call, and may be rewritten in place or
    moved (by ``.data``) in their shape and type; other tensors are another
    Bf16Experts."""

    def __init__(self, weights, swiglu=False):
        import torch

        if weights.dim() != 3 or weights.dtype != torch.bfloat16:
            raise ValueError("weights must be bf16 [experts, out_features, in_features]")
        if not weights.is_contiguous():
            raise ValueError("weights must be contiguous")
        self._weights, self.swiglu = weights, bool(swiglu)
        E, N, K = weights.shape
        self.cfg = ep_experts_t(E, K, N)
        self._ref = ctypes.byref(self.cfg)
        self._given = weights, weights.dtype, weights.shape, "w"

    @property
    def weights(self):
        return self._weights

    def _where(self):
        """Device and pointer at this call."""
        return _weights_kept_at(*self._given)

    def product(self, x, x_scales, expert_offsets, num_tokens_per_expert, out=None, stream=None):
        """bf16 [rows, out_features] (half of them with swiglu): each expert's
        rows times its weights.  Rows that are no expert's are left as they
        are.  Without ``out`` the result belongs to the stream the call runs on
        (so for the other methods)."""
        import torch

        if out is None:
            N = self.cfg.out_features // (2 if self.swiglu else 1)
            out = _empty(stream, (x.shape[0], N), dtype=torch.bfloat16, device=x.device)
        _expert_product(self.cfg, self._ref, x, x_scales, self._where(), 1 if self.swiglu else 0,
                        expert_offsets, num_tokens_per_expert, out, stream)
        return out

    def backward_rows(self, grad_out, expert_offsets, num_tokens_per_expert, out=None,
                      stream=None):
        """bf16 [rows, in_features]: the plain product's gradient for its rows."""
        import torch

        if out is None:
            out = _empty(stream, (grad_out.shape[0], self.cfg.in_features), dtype=torch.bfloat16,
                         device=grad_out.device)
        _backward_rows(self.cfg, self._ref, grad_out, self._where(), expert_offsets,
                       num_tokens_per_expert, out, stream)
        return out

    def backward_weights(self, x, x_scales, grad_out, expert_offsets, num_tokens_per_expert,
                         out=None, add=None, dtype=None, stream=None):
        """The plain product's gradient for the weights, in their shape: bf16,
        or fp32 by ``dtype`` or ``out``, plus ``add`` (which may be ``out``)."""
        import torch

        if out is None:
            dtype = dtype or (torch.bfloat16 if add is None else add.dtype)
            out = _empty(stream, tuple(self._weights.shape), dtype=dtype,
                         device=grad_out.device)
        ep_expert_product_backward_weights(self.cfg, x, x_scales, grad_out, expert_offsets,
                                           num_tokens_per_expert, add, out, stream=stream)
        return out


class SwigluCheckpoint:
    """The 8-bit checkpoint of a layer's gate and up rows: codes
    [capacity, 2 features], scales [capacity, 2 ceil(features / 128)].  They
    are allocated once, on the current stream (another stream waits for it
    before its first call), and the next ``save`` overwrites them.  Between the
    calls they may be elsewhere (``codes.data = codes.cpu()``, and back)."""

    def __init__(self, capacity, features, num_experts, device="cuda"):
        import torch

        dev = torch.device(device)
        self.capacity, self.features = int(capacity), int(features)
        self.num_experts = int(num_experts)
        self._codes = torch.empty((self.capacity, 2 * self.features), dtype=torch.uint8,
                                  device=dev)
        self._scales = torch.empty(_checkpoint_shape(self.capacity, self.features),
                                   dtype=torch.float32, device=dev)
        self._given = [(t, t.dtype, t.shape, name)
                       for t, name in ((self._codes, "codes"), (self._scales, "scales"))]

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    def _where(self):
        """Device, rows and pointers at this call."""
        d, codes = _kept_at(*self._given[0])
        other, scales = _kept_at(*self._given[1])
        if other != d:
            raise ValueError(f"scales is on {self._scales.device}, codes on {self._codes.device}")
        return d, self.capacity, codes, scales

    def save(self, gate_up, expert_offsets, num_tokens_per_expert, out=None, stream=None):
        """bf16 [rows, features]: silu(gate) * up; keeps gate and up."""
        import torch

        if out is None:
            out = _empty(stream, (gate_up.shape[0], self.features), dtype=torch.bfloat16,
                         device=gate_up.device)
        _save(self.num_experts, self.features, gate_up, expert_offsets, num_tokens_per_expert, out,
              self._where(), stream)
        return out

    def backward(self, grad_h, expert_offsets, num_tokens_per_expert, out=None, h=None,
                 stream=None):
        """(bf16 [rows, 2 features], bf16 [rows, features]): the gradient for
        gate and up, and silu(gate) * up of the kept values."""
        import torch

        rows, kw = grad_h.shape[0], dict(dtype=torch.bfloat16, device=grad_h.device)
        if out is None:
            out = _empty(stream, (rows, 2 * self.features), **kw)
        if h is None:
            h = _empty(stream, (rows, self.features), **kw)
        _use(self.num_experts, self.features, self._where(), grad_h, expert_offsets,
             num_tokens_per_expert, out, h, stream)
        return out, h
