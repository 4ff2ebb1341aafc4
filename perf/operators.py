"""The router, its balance loss, their gradient, and the experts' products with
4-bit weights, as measured: cases, inputs, plain forms and exact results.

Four operators, named by a case's "op":

route     logits -> expert ids and gates of the k best experts of each token
balance   logits and expert ids -> load-balance loss, counts per expert, the
          mean probabilities, and the loss's gradient for them
grad      gradient of the gates and of the balance loss for the logits
product   expert-major rows (bf16, or FP8 with a scale per 128 values) times
          the experts' 4-bit weights (one scale per group, optional zero
          points), plain or with a SwiGLU epilogue
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _route(name, T, E, k, **kw):
    c = dict(op="route", tokens=T, experts=E, topk=k, dtype="fp32", score="softmax", bias=False,
             groups=1, topk_groups=1, group_topn=1, normalize=True, scale=1.0, masked=0.0)
    return _named(name, c, kw)


def _balance(name, T, E, k, **kw):
    c = dict(op="balance", tokens=T, experts=E, topk=k, dtype="fp32", score="softmax", seqs=1,
             masked=0.0)
    return _named(name, c, kw)


def _grad(name, T, E, k, **kw):
    c = dict(op="grad", tokens=T, experts=E, topk=k, dtype="fp32", score="softmax", normalize=True,
             scale=1.0, seqs=1, balance=True, masked=0.0)
    return _named(name, c, kw)


def _product(name, rows, experts, K, N, **kw):
    c = dict(op="product", rows=rows, experts=experts, hit=experts, in_features=K, out_features=N,
             group=128, x="bf16", zeros=False, swiglu=False)
    return _named(name, c, kw)


def _named(name, c, kw):
    c.update(kw)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one token of a decode step, sigmoid scores with a selection bias and group limits
        _route("route_token", 1, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4,
               group_topn=2, scale=2.5),
        # a prefill batch with the group limits of the Large workload
        _route("route_prefill", 4096, 256, 8, groups=8, topk_groups=4),
        # a long training batch, bf16 logits, with padded tokens
        _route("route_train_bf16", 131072, 64, 6, dtype="bf16", normalize=False, masked=0.05),
        # a long batch with bias and groups
        _route("route_train_bias", 65536, 256, 8, score="sigmoid", bias=True, groups=8,
               topk_groups=4, group_topn=2, scale=2.5),
        # a batch as one sequence, at the Skewed workload's experts
        _balance("balance_batch", 8192, 64, 6),
        # a packed batch: many sequences of uneven lengths, padded tokens
        _balance("balance_packed", 65536, 256, 8, dtype="bf16", score="sigmoid", seqs=37,
                 masked=0.05),
        # a small training step with an odd number of experts
        _grad("grad_small_odd", 333, 60, 4, normalize=False, seqs=3),
        # a long training step
        _grad("grad_train", 65536, 256, 8, score="sigmoid", scale=2.5, seqs=16, masked=0.02),
        # one decoded token: its 8 experts of 64, gate and up projections
        _product("product_token", 8, 64, 4096, 1024, hit=8, swiglu=True),
        # one rank's share of the Decode workload: FP8 rows, gate and up projections
        _product("product_decode_fp8", 128, 32, 7168, 2048, x="fp8", swiglu=True),
        # odd sizes: group 64, zero points, a ragged output width, experts without rows
        _product("product_odd", 75, 16, 1472, 1001, hit=11, group=64, zeros=True),
        # one rank's share of the Prefill workload: down projection
        _product("product_prefill", 4096, 32, 2048, 7168),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _router_size(rng):
    """Tokens, experts, k: at most as many logits as the largest listed cases."""
    E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384, 512, rng.randint(2, 300)])
    T = _log(rng, 1, min(131072, 65536 * 256 // E))
    k = rng.randint(1, min(8, E))
    return T, E, k


def draw(rng):
    op = rng.choice(["route", "balance", "grad", "product"])
    if op == "route":
        T, E, k = _router_size(rng)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        tg = rng.randint(max(1, -(-k * groups // E)), groups)
        topn = rng.choice([1, 2])
        return _route(None, T, E, k, dtype=rng.choice(["fp32", "bf16"]),
                      score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                      groups=groups, topk_groups=tg, group_topn=topn,
                      normalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                      masked=rng.choice([0.0, 0.1]))
    if op == "balance":
        T, E, k = _router_size(rng)
        return _balance(None, T, E, k, dtype=rng.choice(["fp32", "bf16"]),
                        score=rng.choice(["softmax", "sigmoid"]),
                        seqs=_log(rng, 1, max(1, min(64, T))), masked=rng.choice([0.0, 0.1]))
    if op == "grad":
        T, E, k = _router_size(rng)
        return _grad(None, T, E, max(k, min(2, E)), dtype=rng.choice(["fp32", "bf16"]),
                     score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), seqs=_log(rng, 1, max(1, min(64, T))),
                     balance=rng.random() < 0.7, masked=rng.choice([0.0, 0.1]))
    fp8 = rng.random() < 0.5
    group = rng.choice([32, 64, 128])
    K = 128 * _log(rng, 2, 56) if fp8 else group * _log(rng, -(-256 // group), 7168 // group)
    swiglu = rng.random() < 0.5
    N = _log(rng, 64, 2048 if swiglu else 4096)
    experts = rng.choice([4, 8, 16, 24, 32])
    most = max(8, min(4096, 4096 * 2048 * 7168 // (K * N * (2 if swiglu else 1))))
    rows = _log(rng, 1, most)
    return _product(None, rows, experts, K, N, hit=rng.randint(1, experts), group=group,
                    x="fp8" if fp8 else "bf16", zeros=rng.random() < 0.4, swiglu=swiglu)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _dt(name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def _logits(case, g):
    T, E = case["tokens"], case["experts"]
    # hidden . expert centroid: a popularity per expert and a token's own part
    return (_randn(g, T, E) * 1.4 + 0.5 * _randn(g, 1, E)).to(_dt(case["dtype"]))


def _mask(case, g):
    if not case["masked"]:
        return None
    return (torch.rand(case["tokens"], generator=g, device=DEV) >= case["masked"]).to(torch.uint8)


def _seq_offsets(T, S, g):
    """Uneven sequence lengths that add up to T (some may be empty)."""
    if S == 1:
        return None
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV).sort().values
    ends = torch.tensor([T], device=DEV)
    return torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)


def _some_route(case, logits, mask):
    """Expert ids of a plain top-k of the logits, -1 in the rows of padded tokens."""
    idx = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices
    idx = idx[:, :case["topk"]].to(torch.int32)
    if mask is not None:
        idx = torch.where(mask[:, None] != 0, idx, -1)
    return idx.contiguous()


def _counts(rows, experts, hit, seed):
    """Rows per expert: `hit` experts share them unevenly, the others have none."""
    import random

    r = random.Random(seed)
    c = [0] * experts
    chosen = r.sample(range(experts), min(hit, experts, rows))
    for e in chosen:
        c[e] = 1
    for _ in range(rows - len(chosen)):
        c[chosen[r.randrange(len(chosen))]] += 1
    return c


def _tiles(codes, scales, zeros, halves):
    """The tiled form of row-major weights: `halves` matrices of N rows each
    (gate and up of a SwiGLU), rows padded to 16 and columns to 128.  A tile is
    16 rows x 128 columns: 64 lanes x 4 words, lane l and word w hold row
    l % 16, columns 32 w + 8 (l / 16) + 0..7, column 2p in bits 4p.. and
    column 2p + 1 in bits 16 + 4p.. of the word."""
    E, HN, K2 = codes.shape
    N, K = HN // halves, 2 * K2
    q = torch.stack([codes & 15, codes >> 4], dim=-1).view(E, halves, N, K)
    N16, K128 = -(-N // 16), -(-K // 128)
    full = torch.zeros(E, halves, N16 * 16, K128 * 128, dtype=torch.uint8, device=codes.device)
    full[:, :, :N, :K] = q
    # e, half, row tile, row, column tile, word, lane group, pair, parity
    t = full.view(E, halves, N16, 16, K128, 4, 4, 4, 2)
    # nibble order of a word, lowest first: pairs' even columns, then their odd ones
    t = t.permute(0, 1, 2, 4, 6, 3, 5, 8, 7).reshape(E, halves, N16, K128, 64, 16, 2)
    w = (t[..., 0] | (t[..., 1] << 4)).contiguous()

    def by_tile(v):
        if v is None:
            return None
        G = v.shape[-1]
        p = torch.zeros(E, halves, N16 * 16, G, dtype=v.dtype, device=v.device)
        p[:, :, :N] = v.view(E, halves, N, G)
        return p.view(E, halves, N16, 16, G).transpose(3, 4).contiguous()

    return w, by_tile(scales), by_tile(zeros)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    if case["op"] == "product":
        E, K, N, G = case["experts"], case["in_features"], case["out_features"], case["group"]
        halves = 2 if case["swiglu"] else 1
        counts = _counts(case["rows"], E, case["hit"], seed)
        rows = case["rows"]
        s["max_rows"] = max(counts)
        c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        s["counts"] = c
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV),
                                  torch.cumsum(c, 0).to(torch.int32)])
        s["codes"] = torch.randint(0, 256, (E, halves * N, K // 2), generator=g, device=DEV,
                                   dtype=torch.uint8)
        u = torch.rand(E, halves * N, K // G, generator=g, device=DEV)
        s["scales"] = ((0.5 + u) * (0.2 / math.sqrt(K))).to(torch.bfloat16)
        s["zeros"] = (torch.randint(5, 12, (E, halves * N, K // G), generator=g, device=DEV,
                                    dtype=torch.uint8) if case["zeros"] else None)
        s["w_codes"], s["w_scales"], s["w_zeros"] = _tiles(s["codes"], s["scales"], s["zeros"],
                                                           halves)
        x = _randn(g, rows, K)
        if case["x"] == "fp8":
            # one scale per row and 128 values, as FP8 dispatch leaves them
            b = x.view(rows, K // 128, 128)
            sc = b.abs().amax(dim=2) / 448.0
            s["x"] = (b / sc[:, :, None]).reshape(rows, K).to(torch.float8_e4m3fn).view(torch.uint8)
            s["x_scales"] = sc.contiguous()
        else:
            s["x"], s["x_scales"] = x.to(torch.bfloat16), None
        return s
    s["logits"] = _logits(case, g)
    mask = _mask(case, g)
    if case["op"] == "route":
        s["mask"] = mask
        s["bias"] = _randn(g, case["experts"]) * 0.05 if case["bias"] else None
        return s
    s["idx"] = _some_route(case, s["logits"], mask)
    s["seq_offsets"] = _seq_offsets(case["tokens"], case["seqs"], g)
    if case["op"] == "balance":
        return s
    T, E, k, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
    s["grad_weights"] = _randn(g, T, k) * 1e-2
    # what the loss's forward hands to the backward: its gradient for the probabilities
    f = torch.rand(S, E, generator=g, device=DEV) * 2
    s["prob_grad"] = f * (1e-2 / T) if case["balance"] else None
    s["grad_loss"] = torch.full((1,), 1024.0, device=DEV) if case["balance"] else None
    return s


# --------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, 64 where 32 lose what matters
# --------------------------------------------------------------------------

def _softmax(x):
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _scores(x, score):
    return _softmax(x) if score == "softmax" else _sigmoid(x)


def _plain_route(s):
    c = s["case"]
    E, k, G = c["experts"], c["topk"], c["groups"]
    T = c["tokens"]
    # the order of the experts is decided in 64 bits: neighbours may be closer than 32 hold
    x = s["logits"].double()
    key = _scores(x, c["score"])
    if s["bias"] is not None:
        key = key + s["bias"].double()
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        group = best[:, :, :min(c["group_topn"], E // G)].sum(dim=2)
        order = torch.sort(group, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order[:, :c["topk_groups"]], True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = _scores(s["logits"].float(), c["score"]).gather(1, idx)
    if c["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * c["scale"]
    idx = idx.to(torch.int32)
    if s["mask"] is not None:
        on = s["mask"][:, None] != 0
        idx, w = torch.where(on, idx, -1), torch.where(on, w, 0.0)
    return idx, w


def _probs(x, score):
    p = _scores(x, score)
    return p if score == "softmax" else p / p.sum(dim=1, keepdim=True)


def _token_seq(s, T):
    """Sequence of each token."""
    if s["seq_offsets"] is None:
        return torch.zeros(T, dtype=torch.int64, device=s["idx"].device)
    t = torch.arange(T, device=s["idx"].device)
    return torch.searchsorted(s["seq_offsets"][1:].long(), t, right=True)


def _by_sequence(v, member):
    """Sums of the rows of v over each sequence, in 64 bits (long sums): the
    product with the [sequences, tokens] table of ones and zeros."""
    return torch.matmul(member, v.double())


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["topk"]
    idx = s["idx"].long()
    on = (idx >= 0).any(dim=1)
    p = _probs(s["logits"].float(), c["score"]) * on[:, None]
    hot = torch.zeros(T, E + 1, dtype=torch.int64, device=idx.device)
    hot.scatter_add_(1, torch.where(idx < 0, E, idx), torch.ones_like(idx))
    at = torch.arange(c["seqs"], device=idx.device)
    member = (at[:, None] == _token_seq(s, T)).double()
    counts = _by_sequence(hot[:, :E], member)
    tokens = _by_sequence(on[:, None], member)[:, 0]
    sums = _by_sequence(p, member)
    n = tokens.clamp(min=1)[:, None]
    mean = sums / n
    f = counts * (E / k) / n
    seqs = (tokens > 0).sum().clamp(min=1)
    grad = f / n * (COEF / seqs)
    loss = (f * mean).sum().reshape(1) * (COEF / seqs)
    return (loss.float(), counts.to(torch.int32), tokens.to(torch.int32), mean.float(),
            grad.float())


def _plain_grad(s):
    c = s["case"]
    T = c["tokens"]
    x = s["logits"].float()
    idx = s["idx"].long()
    valid = idx >= 0
    at = idx.clamp(min=0)
    sc = _scores(x, c["score"])
    u = torch.where(valid, s["grad_weights"], 0.0)
    w = torch.where(valid, sc.gather(1, at), 0.0)
    if c["normalize"]:
        p = w / w.sum(dim=1, keepdim=True).clamp(min=1e-30)
        d = c["scale"] * p * (u - (u * p).sum(dim=1, keepdim=True))  # d(log score)
        if c["score"] == "sigmoid":
            d = d * (1 - w)
        gl = torch.zeros_like(x).scatter_add_(1, at, torch.where(valid, d, 0.0))
    elif c["score"] == "softmax":
        gl = torch.zeros_like(x).scatter_add_(1, at, c["scale"] * w * u)
        gl = gl - sc * (c["scale"] * (w * u).sum(dim=1, keepdim=True))
    else:
        gl = torch.zeros_like(x).scatter_add_(1, at, c["scale"] * w * (1 - w) * u)
    if s["prob_grad"] is not None:
        p = _probs(x, c["score"])
        q = s["prob_grad"][_token_seq(s, T)]
        d = s["grad_loss"] * p * (q - (q * p).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - sc)
        gl = gl + torch.where(valid.any(dim=1, keepdim=True), d, 0.0)
    return gl.to(s["logits"].dtype)


def _weights(s, dtype):
    c = s["case"]
    E, K, G = c["experts"], c["in_features"], c["group"]
    rows = s["codes"].shape[1]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1).view(E, rows, K // G, G)
    z = 8 if s["zeros"] is None else s["zeros"][..., None]
    q = q.to(torch.int8) - (z if isinstance(z, int) else z.to(torch.int8))
    return (q.to(dtype) * s["scales"][..., None].to(dtype)).view(E, rows, K)


def _rows(s, dtype):
    if s["x_scales"] is None:
        return s["x"].to(dtype)
    r, K = s["x"].shape
    x = s["x"].view(torch.float8_e4m3fn).to(torch.float32).to(dtype).view(r, K // 128, 128)
    return (x * s["x_scales"][:, :, None].to(dtype)).view(r, K)


def _plain_product(s):
    c = s["case"]
    E, K, N = c["experts"], c["in_features"], c["out_features"]
    R, M = c["rows"], s["max_rows"]
    # rows of each expert side by side, padded to the longest
    pos = torch.arange(R, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), pos, right=True)
    r = pos - s["offsets"].long()[e]
    x = torch.zeros(E, M, K, device=DEV)
    x[e, r] = _rows(s, torch.float32)
    w = _weights(s, torch.float32)
    y = torch.matmul(w, x.transpose(1, 2).contiguous())[e, :, r]
    if c["swiglu"]:
        y = y[:, :N] * _sigmoid(y[:, :N]) * y[:, N:]
    return y.to(torch.bfloat16)


COEF = 0.01


def run(s):
    c = s["case"]
    if not own:
        return {"route": _plain_route, "balance": _plain_balance, "grad": _plain_grad,
                "product": _plain_product}[c["op"]](s)
    import combine_get_dispatch_amd as ep

    if c["op"] == "product":
        if "experts" not in s:  # made once: the weights' handle and the output rows
            s["experts"] = ep.W4Experts(s["w_codes"], s["w_scales"], s["w_zeros"],
                                        c["out_features"], c["in_features"], c["group"])
            s["out"] = torch.empty(c["rows"], c["out_features"], dtype=torch.bfloat16, device=DEV)
        return s["experts"].product(s["x"], s["x_scales"], s["offsets"], s["counts"], s["out"])
    if "router" not in s:  # made once: the router's buffers
        s["router"] = ep.EpRouter(
            c["tokens"], c["experts"], c["topk"], score=c["score"], groups=c.get("groups", 1),
            topk_groups=c.get("topk_groups", 1), group_topn=c.get("group_topn", 1),
            normalize=c.get("normalize", True), scale=c.get("scale", 1.0),
            logits_dtype=s["logits"].dtype, max_seqs=c.get("seqs", 1))
    r = s["router"]
    if c["op"] == "route":
        return r.route(s["logits"], bias=s["bias"], token_mask=s["mask"])
    if c["op"] == "balance":
        loss = r.balance_loss(s["logits"], s["idx"], COEF, seq_offsets=s["seq_offsets"])
        return loss, r.counts, r.seq_tokens, r.mean_probs, r.prob_grad
    return r.backward(s["logits"], s["idx"], s["grad_weights"], prob_grad=s["prob_grad"],
                      seq_offsets=s["seq_offsets"], grad_loss=s["grad_loss"])


# --------------------------------------------------------------------------
# Exact results, from the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_log_scores(x, score):
    if score == "softmax":
        return x - torch.logsumexp(x, dim=1, keepdim=True)
    return torch.where(x > 0, 0.0, x) - torch.log1p(torch.exp(-x.abs()))


def _exact_route(s):
    c = s["case"]
    T, E, k, G = c["tokens"], c["experts"], c["topk"], c["groups"]
    ls = _exact_log_scores(s["logits"].double(), c["score"])
    key = torch.exp(ls) + (0 if s["bias"] is None else s["bias"].double())
    if G > 1:
        top = key.view(T, G, -1).topk(min(c["group_topn"], E // G), dim=2).values.sum(dim=2)
        # a group is kept if fewer than topk_groups stand before it
        a, b = top[:, :, None], top[:, None, :]
        low = torch.ones(G, G, device=DEV).tril(-1).bool()
        before = ((b > a) | ((b == a) & low)).sum(dim=2)
        out = (before >= c["topk_groups"])[:, torch.arange(E, device=DEV) // (E // G)]
        key = torch.where(out, -math.inf, key)
    left = key.clone()
    ids = []
    for _ in range(k):  # the best left, the first of equals
        best = left.amax(dim=1, keepdim=True)
        i = (left == best).to(torch.uint8).argmax(dim=1)
        ids.append(i)
        left.scatter_(1, i[:, None], -math.inf)
    idx = torch.stack(ids, dim=1)
    w = ls.gather(1, idx)
    w = torch.exp(w - torch.logsumexp(w, dim=1, keepdim=True)) if c["normalize"] else torch.exp(w)
    w = w * c["scale"]
    idx = idx.to(torch.int32)
    if s["mask"] is not None:
        off = (s["mask"] == 0)[:, None]
        idx, w = idx.masked_fill(off, -1), w.masked_fill(off, 0.0)
    return idx, w


def _exact_probs(x, score):
    ls = _exact_log_scores(x, score)
    return torch.exp(ls - torch.logsumexp(ls, dim=1, keepdim=True))


def _bounds(s, T):
    return [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()


def _exact_balance(s):
    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["topk"]
    p = _exact_probs(s["logits"].double(), c["score"])
    at = _bounds(s, T)
    counts, tokens, means = [], [], []
    for lo, hi in zip(at, at[1:]):
        i = s["idx"][lo:hi]
        on = (i >= 0).any(dim=1)
        counts.append(torch.bincount(i[i >= 0].long(), minlength=E))
        n = int(on.sum())
        tokens.append(n)
        means.append(p[lo:hi][on].sum(dim=0) / max(n, 1))
    live = max(1, sum(n > 0 for n in tokens))
    n = torch.tensor(tokens, device=DEV)
    counts, mean = torch.stack(counts), torch.stack(means)
    f = E * counts.double() / (k * n.clamp(min=1)[:, None])
    loss = COEF / live * (f * mean).sum().reshape(1)
    return (loss, counts.to(torch.int32), n.to(torch.int32), mean,
            COEF / live * f / n.clamp(min=1)[:, None])


def _exact_grad(s):
    # the derivative of sum(u w) + g sum(q p) by torch's own differentiation in 64 bits
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    valid = s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    with torch.enable_grad():
        ls = _exact_log_scores(x, c["score"])
        sel = ls.gather(1, at)
        if c["normalize"]:
            sel = sel - torch.logsumexp(sel, dim=1, keepdim=True)
        w = c["scale"] * torch.exp(sel)
        total = (torch.where(valid, w, 0.0) * s["grad_weights"].double()).sum()
        if s["prob_grad"] is not None:
            q = s["prob_grad"].double()[_token_seq(s, c["tokens"])]
            p = torch.exp(ls - torch.logsumexp(ls, dim=1, keepdim=True))
            total = total + s["grad_loss"].double() * (q * p * valid.any(dim=1, keepdim=True)).sum()
        total.sum().backward()
    return x.grad


def _exact_product(s):
    c = s["case"]
    E, K, N = c["experts"], c["in_features"], c["out_features"]
    x = s["x"].double() if s["x_scales"] is None else (
        s["x"].view(torch.float8_e4m3fn).double() * s["x_scales"].double().repeat_interleave(128, 1))
    out = torch.empty(c["rows"], N, dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    for e in range(E):
        if at[e] == at[e + 1]:
            continue
        codes = s["codes"][e]
        q = torch.empty(codes.shape[0], K, dtype=torch.float64, device=DEV)
        q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        z = 8.0 if s["zeros"] is None else s["zeros"][e].double().repeat_interleave(c["group"], 1)
        w = (q - z) * s["scales"][e].double().repeat_interleave(c["group"], 1)
        y = x[at[e]:at[e + 1]] @ w.T
        if c["swiglu"]:
            a, b = y[:, :N], y[:, N:]
            y = a / (1 + torch.exp(-a)) * b
        out[at[e]:at[e + 1]] = y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "balance": _exact_balance, "grad": _exact_grad,
            "product": _exact_product}[case["op"]](s)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "product":
        K, N, G = case["in_features"], case["out_features"], case["group"]
        n = N * (2 if case["swiglu"] else 1)
        hit = min(case["hit"], case["experts"], case["rows"])
        weights = hit * (n * K // 2 + n * (K // G) * (3 if case["zeros"] else 2))
        row = K + 4 * (K // 128) if case["x"] == "fp8" else 2 * K
        return dict(bytes=weights + case["rows"] * (row + 2 * N), flops=2.0 * case["rows"] * n * K)
    T, E, k = case["tokens"], case["experts"], case["topk"]
    logits = T * E * (4 if case["dtype"] == "fp32" else 2)
    S = case.get("seqs", 1)
    if case["op"] == "route":
        # a score, its comparison with the best so far
        return dict(bytes=logits + T * (1 if case["masked"] else 0) + 4 * E + 8 * T * k,
                    flops=10.0 * T * E)
    if case["op"] == "balance":
        return dict(bytes=logits + 4 * T * k + 4 * (S + 1) + S * (12 * E + 4) + 4,
                    flops=10.0 * T * E)
    return dict(bytes=2 * logits + 8 * T * k + 4 * S * E, flops=10.0 * T * E)
