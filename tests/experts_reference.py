"""Plain 64-bit forms of the experts' bf16 products, their gradients, and the
8-bit checkpoint of the SwiGLU between them (include/ep_moe.h)."""
import numpy as np
import torch

UBF16, U32 = 2.0 ** -8, 2.0 ** -24  # half a step, relative to the value


def to_bf16(a):
    """numpy -> bf16 tensor, nearest even (from 64 bits through 32)."""
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16()


def rounded(a):
    return to_bf16(a).double().numpy()


def expert_rows(offsets, counts, cap):
    """[(expert, first row, last row + 1)] inside the buffers."""
    out = []
    for e, n in enumerate(counts):
        lo = int(offsets[e])
        hi = min(lo + int(n), cap)
        if lo >= 0 and hi > lo:
            out.append((e, lo, hi))
    return out


def silu(y):
    with np.errstate(over="ignore"):
        return y / (1 + np.exp(-y))


def product(x, w, offsets, counts):
    """(y, sums of magnitudes), NaN in rows that are no expert's."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    size = np.full_like(y, np.nan)
    for e, lo, hi in expert_rows(offsets, counts, x.shape[0]):
        y[lo:hi] = x[lo:hi] @ w[e].T
        size[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    return y, size


def rows_grad(g, w, offsets, counts):
    return product(g, np.swapaxes(w, 1, 2), offsets, counts)


def weights_grad(g, x, offsets, counts):
    E = len(counts)
    y = np.zeros((E, g.shape[1], x.shape[1]))
    size = np.zeros_like(y)
    for e, lo, hi in expert_rows(offsets, counts, x.shape[0]):
        y[e] = g[lo:hi].T @ x[lo:hi]
        size[e] = np.abs(g[lo:hi]).T @ np.abs(x[lo:hi])
    return y, size


def sum_error(terms, size):
    """A sum of that many terms in fp32: each step off by half a step of a
    partial sum, which is at most the sum of magnitudes; a few more for the
    order inside a matrix instruction."""
    return (terms + 8) * U32 * size


def e4m3(v):
    """Nearest even E4M3 number of finite values within 448, as values."""
    a = np.abs(v)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.round(v / step) * step  # np.round: half to even


def checkpoint(gate_up):
    """[rows, 2 F] values (finite or not) -> (codes' values, scales
    [rows, 2 blocks]) by the definition."""
    rows, F = gate_up.shape[0], gate_up.shape[1] // 2
    blocks = -(-F // 128)
    codes, scales = np.empty_like(gate_up), np.empty((rows, 2 * blocks))
    for r in range(rows):
        for half in range(2):
            for b in range(blocks):
                lo, hi = half * F + b * 128, half * F + min(F, b * 128 + 128)
                v = gate_up[r, lo:hi]
                ok = np.isfinite(v)
                most = np.max(np.abs(v[ok]), initial=0.0)
                e = -100
                while most > 448 * 2.0 ** e:
                    e += 1
                scales[r, half * blocks + b] = 2.0 ** e
                codes[r, lo:hi] = np.where(ok, e4m3(np.where(ok, v, 0.0) / 2.0 ** e), np.nan)
    return codes, scales


def kept(codes, scales, F):
    """What codes [rows, 2 F] and scales stand for."""
    at = np.arange(F) // 128
    blocks = scales.shape[1] // 2
    return codes * np.concatenate([scales[:, at], scales[:, blocks + at]], axis=1)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def swiglu_grad(gate_up, grad):
    F = grad.shape[1]
    g, u = gate_up[:, :F], gate_up[:, F:]
    s = sigmoid(g)
    return np.concatenate([grad * u * s * (1 + g * (1 - s)), grad * g * s], axis=1), g * s * u
