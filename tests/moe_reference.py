"""Plain implementations in 64 bits of the router, its balance loss, their
gradient and the experts' 4-bit products, straight from their definitions and
apart from the library.  numpy only."""
import numpy as np

U32 = 2.0 ** -24  # half a step of fp32, relative
UBF16 = 2.0 ** -8


def scores(x, score):
    """log of the scores, in 64 bits; -inf stays."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if score == "softmax":
            m = x.max(axis=-1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            return x - m - np.log(np.exp(x - m).sum(axis=-1, keepdims=True))
        return np.where(x > 0, 0.0, x) - np.log1p(np.exp(-np.abs(x)))


def route(x, k, score="softmax", bias=None, mask=None, groups=1, topk_groups=1, group_topn=1,
          normalize=True, scale=1.0):
    """(ids, weights, bad): bad[t] where a logit or key is NaN or +inf."""
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    bad = np.zeros(T, bool)
    by_logit = bias is None and (groups == 1 or group_topn == 1)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        row = x[t].astype(np.float64)
        if np.isnan(row).any() or (row == np.inf).any():
            bad[t] = True
            continue
        if np.all(row == -np.inf):
            continue
        ls = scores(row, score)
        key = row.copy() if by_logit else np.exp(ls) + (0 if bias is None else
                                                        bias.astype(np.float64))
        key[row == -np.inf] = -np.inf
        if np.isnan(key).any() or (key == np.inf).any():
            bad[t] = True
            continue
        if groups > 1:
            per = E // groups
            gk = np.full(groups, -np.inf)
            for g in range(groups):
                best = np.sort(key[g * per:(g + 1) * per])[::-1][:group_topn]
                best = best[best > -np.inf]
                if len(best):
                    gk[g] = best.sum()
            keep = np.argsort(-gk, kind="stable")[:topk_groups]
            allowed = np.zeros(E, bool)
            for g in keep:
                allowed[g * per:(g + 1) * per] = True
            key = np.where(allowed, key, -np.inf)
        order = [e for e in np.argsort(-key, kind="stable")[:k] if key[e] > -np.inf]
        ids[t, :len(order)] = order
        s = ls[order]
        if normalize and len(order):
            s = s - s.max()
            s = s - np.log(np.exp(s).sum())
        w[t, :len(order)] = scale * np.exp(s)
    return ids, w, bad


def probabilities(x, score):
    ls = scores(x, score)
    m = ls.max(axis=1, keepdims=True)
    e = np.exp(ls - np.where(np.isfinite(m), m, 0.0))
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def balance(x, ids, coef, score="softmax", offsets=None):
    """loss, counts, tokens, mean probabilities, gradient for them."""
    T, E = x.shape
    k = ids.shape[1]
    offsets = [0, T] if offsets is None else list(offsets)
    S = len(offsets) - 1
    on = (ids >= 0).any(axis=1)
    p = np.zeros((T, E))
    if on.any():
        p[on] = probabilities(x[on], score)
    counts, n, mean = np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros((S, E))
    for s in range(S):
        lo, hi = offsets[s], offsets[s + 1]
        for e in ids[lo:hi].reshape(-1):
            if e >= 0:
                counts[s, e] += 1
        n[s] = on[lo:hi].sum()
        if n[s]:
            mean[s] = p[lo:hi].sum(axis=0) / n[s]
    live = max(1, int((n > 0).sum()))
    f = E * counts / (k * np.maximum(n, 1)[:, None])
    loss = coef / live * (f * mean).sum()
    return loss, counts, n, mean, coef / live * f / np.maximum(n, 1)[:, None]


def gates(x, ids, score, normalize, scale):
    """Weights of given ids (a function of the logits, for differences)."""
    ls = scores(x, score)
    s = np.where(ids >= 0, np.take_along_axis(ls, np.maximum(ids, 0), axis=1), -np.inf)
    if normalize:
        m = s.max(axis=1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        tot = np.exp(s - m).sum(axis=1, keepdims=True)
        return scale * np.exp(s - m) / np.where(tot > 0, tot, 1.0)
    return scale * np.exp(s)


def grad(x, ids, u, score="softmax", normalize=True, scale=1.0, prob_grad=None, offsets=None,
         grad_loss=1.0):
    """(gradient, size): size bounds the terms each element is the sum of."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        slots = np.flatnonzero(ids[t] >= 0)
        if not len(slots):
            continue
        e = ids[t, slots]
        s = np.exp(scores(x[t], score))
        one_minus = 1.0 if score == "softmax" else np.exp(scores(-x[t], "sigmoid"))
        if u is not None:
            v = u[t, slots].astype(np.float64)
            if normalize:
                w = gates(x[t:t + 1], ids[t:t + 1], score, True, 1.0)[0, slots]
                d, b = w * (v - (w * v).sum()), w * (np.abs(v) + (w * np.abs(v)).sum())
                if score == "sigmoid":
                    d, b = d * one_minus[e], b * one_minus[e]
                np.add.at(out[t], e, scale * d)
                np.add.at(size[t], e, abs(scale) * b)
            elif score == "softmax":
                np.add.at(out[t], e, scale * s[e] * v)
                np.add.at(size[t], e, abs(scale) * s[e] * np.abs(v))
                out[t] -= scale * s * (s[e] * v).sum()
                size[t] += abs(scale) * s * (s[e] * np.abs(v)).sum()
            else:
                np.add.at(out[t], e, scale * s[e] * one_minus[e] * v)
                np.add.at(size[t], e, abs(scale) * s[e] * one_minus[e] * np.abs(v))
        if prob_grad is not None:
            seq = 0 if offsets is None else int(np.searchsorted(offsets[1:], t, side="right"))
            q = prob_grad[seq].astype(np.float64)
            p = probabilities(x[t:t + 1], score)[0]
            d = grad_loss * p * (q - (q * p).sum())
            b = abs(grad_loss) * p * (np.abs(q) + (np.abs(q) * p).sum())
            if score == "sigmoid":
                d, b = d * one_minus, b * one_minus
            out[t] += d
            size[t] += b
    return out, size


# --------------------------------------------------------------------------
# 4-bit weights
# --------------------------------------------------------------------------

def pack_codes(q):
    """[..., K] codes 0..15 -> [..., K / 2] bytes, column 2 i in the low half."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def tile_codes(q, halves):
    """The packed codes of q [E, halves * N, K] by the layout's definition, one
    nibble at a time."""
    E, HN, K = q.shape
    N = HN // halves
    n16, k128 = -(-N // 16), -(-K // 128)
    out = np.zeros((E, halves, n16, k128, 64, 4), np.uint32)
    q = q.reshape(E, halves, N, K)
    for n in range(N):
        for c in range(K):
            lane = n % 16 + 16 * (c % 32 // 8)
            word, i = c % 128 // 32, c % 8
            shift = 4 * (i // 2) + (16 if i % 2 else 0)
            out[:, :, n // 16, c // 128, lane, word] |= q[:, :, n, c].astype(np.uint32) << shift
    return np.ascontiguousarray(out).view(np.uint8).reshape(E, halves, n16, k128, 1024)


def weights(q, scales, zeros, group):
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=2)
    return (q.astype(np.float64) - z) * np.repeat(scales.astype(np.float64), group, axis=2)


def product(x, w, offsets, counts, swiglu):
    """{row: fp64 outputs} of the experts' rows, and the sums of magnitudes."""
    cap = x.shape[0]
    rows, size = {}, {}
    for e in range(len(counts)):
        for r in range(offsets[e], min(offsets[e] + counts[e], cap)):
            y = w[e] @ x[r]
            b = np.abs(w[e]) @ np.abs(x[r])
            if swiglu:
                n = len(y) // 2
                with np.errstate(over="ignore"):
                    sig = 1 / (1 + np.exp(-y[:n]))
                rows[r], size[r] = y[:n] * sig * y[n:], b
            else:
                rows[r], size[r] = y, b
    return rows, size
