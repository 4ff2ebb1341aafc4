"""The experts' products with bf16 weights, their gradients, and the 8-bit
checkpoint of the activation between them, as measured: cases, inputs, plain
forms and exact results.

Five operators, named by a case's "op":

product       expert-major rows (bf16, or FP8 with a scale per 128 values)
              times the experts' bf16 weights, plain or with a SwiGLU epilogue
rows_grad     gradient of the product for its rows
weights_grad  gradient of the product for the weights, in bf16 or fp32, alone
              or added to what earlier batches left
save          SwiGLU of gate and up rows, and their checkpoint: E4M3 with a
              power-of-two scale per 128 values
use           from the checkpoint and the gradient of the SwiGLU rows: the
              gradient of gate and up, and the SwiGLU rows again
"""
import math
import random

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _product(name, rows, experts, K, N, **kw):
    c = dict(op="product", rows=rows, experts=experts, hit=experts, in_features=K, out_features=N,
             x="bf16", swiglu=False)
    return _named(name, c, kw)


def _rows_grad(name, rows, experts, K, N, **kw):
    c = dict(op="rows_grad", rows=rows, experts=experts, hit=experts, in_features=K,
             out_features=N)
    return _named(name, c, kw)


def _weights_grad(name, rows, experts, K, N, **kw):
    c = dict(op="weights_grad", rows=rows, experts=experts, hit=experts, in_features=K,
             out_features=N, x="bf16", grad="bf16", add=False)
    return _named(name, c, kw)


def _checkpoint(op, name, rows, experts, inner, **kw):
    c = dict(op=op, rows=rows, experts=experts, hit=experts, inner=inner)
    return _named(name, c, kw)


def _named(name, c, kw):
    c.update(kw)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one decoded token: its 8 experts of 64, gate and up projections
        _product("product_token", 8, 64, 4096, 2048, hit=8, swiglu=True),
        # one rank's share of the Decode workload: FP8 rows, gate and up projections
        _product("product_decode_fp8", 128, 32, 7168, 4096, x="fp8", swiglu=True),
        # one rank's share of the Prefill workload: FP8 rows, gate and up projections
        _product("product_prefill_fp8", 4096, 32, 7168, 4096, x="fp8", swiglu=True),
        # a rank's rows of a training step (8 ranks of 4096 tokens): down projection
        _product("product_train", 32768, 32, 2048, 7168),
        # a small batch with odd sizes and experts without rows
        _rows_grad("rows_grad_odd", 333, 16, 1480, 1001, hit=11),
        # the training step's gradient through the gate and up projections
        _rows_grad("rows_grad_train", 32768, 32, 7168, 4096),
        # gradient accumulation over small batches: fp32, an expert without rows
        _weights_grad("weights_grad_accumulate", 4096, 8, 2048, 7168, hit=7, grad="fp32",
                      add=True),
        # the training step's gate and up projections, x as FP8 dispatch left it
        _weights_grad("weights_grad_train_fp8", 32768, 32, 7168, 4096, x="fp8"),
        # a few rows of an odd width
        _checkpoint("save", "save_small_odd", 85, 16, 1001, hit=9),
        # the training step's activation
        _checkpoint("save", "save_train", 32768, 32, 2048),
        _checkpoint("use", "use_small_odd", 85, 16, 1001, hit=9),
        _checkpoint("use", "use_train", 32768, 32, 2048),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_WEIGHTS = 32 * 7168 * 4096   # of the listed cases
MOST_PRODUCTS = 32768 * 7168 * 4096


def _size(rng, fp8):
    """Rows, experts, K, N: at most the largest listed cases' weights and products."""
    experts = rng.choice([1, 2, 4, 8, 16, 24, 32, 64])
    if fp8:
        K = 128 * _log(rng, 1, 56)
    else:
        K = _log(rng, 64, 7168)
        if rng.random() < 0.7:
            K = (K + 7) // 8 * 8
    N = _log(rng, 64, min(7168, MOST_WEIGHTS // (experts * K)))
    if rng.random() < 0.7:
        N = N // 8 * 8
    rows = _log(rng, 1, max(8, min(32768, MOST_PRODUCTS // (K * N))))
    return rows, experts, K, N


def draw(rng):
    op = rng.choice(["product", "product", "rows_grad", "weights_grad", "save", "use"])
    fp8 = rng.random() < 0.5
    if op == "product":
        rows, experts, K, N = _size(rng, fp8)
        return _product(None, rows, experts, K, N // 2 * 2, hit=rng.randint(1, experts),
                        x="fp8" if fp8 else "bf16", swiglu=rng.random() < 0.5)
    if op == "rows_grad":
        rows, experts, K, N = _size(rng, False)
        return _rows_grad(None, rows, experts, K, N, hit=rng.randint(1, experts))
    if op == "weights_grad":
        rows, experts, K, N = _size(rng, fp8)
        # FP8 rows come with bf16 gradients, of about their own precision
        grad = "bf16" if fp8 else rng.choice(["bf16", "fp32"])
        return _weights_grad(None, rows, experts, K, N, hit=rng.randint(1, experts),
                             x="fp8" if fp8 else "bf16", grad=grad, add=rng.random() < 0.5)
    experts = rng.choice([1, 4, 8, 16, 32, 64, 256])
    inner = _log(rng, 32, 4096)
    if rng.random() < 0.6:
        inner = (inner + 7) // 8 * 8
    return _checkpoint(op, None, _log(rng, 1, min(32768, 32768 * 2048 // inner)), experts, inner,
                       hit=rng.randint(1, experts))


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


def _counts(rows, experts, hit, seed):
    """Rows per expert: `hit` experts of uneven popularity, the others have none."""
    r = random.Random(seed)
    c = [0] * experts
    chosen = r.sample(range(experts), min(hit, experts, rows))
    for e in chosen:
        c[e] = 1
    pull = [math.exp(0.3 * r.gauss(0, 1)) for _ in chosen]
    for e in r.choices(chosen, pull, k=rows - len(chosen)):
        c[e] += 1
    return c


def _weights(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = _randn(g, N, K) / math.sqrt(K)
    return w


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    R, E = case["rows"], case["experts"]
    counts = _counts(R, E, case["hit"], seed)
    s["max_rows"] = max(counts)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    s["counts"] = c
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV),
                              torch.cumsum(c, 0).to(torch.int32)])
    if case["op"] in ("save", "use"):
        N = case["inner"]
        # gate and up of a layer: their sizes differ from row to row
        size = torch.exp(0.5 * _randn(g, R, 1))
        s["gate_up"] = (_randn(g, R, 2 * N) * size).to(torch.bfloat16)
        if case["op"] == "use":
            s["codes"], s["scales"] = _encode(s["gate_up"], N)
            s["grad"] = (_randn(g, R, N) * 1e-3).to(torch.bfloat16)
        return s
    K, N = case["in_features"], case["out_features"]
    if case["op"] in ("product", "weights_grad"):
        x = _randn(g, R, K)
        if case["x"] == "fp8":
            # one scale per row and 128 values, as FP8 dispatch leaves them
            b = x.view(R, K // 128, 128)
            sc = b.abs().amax(dim=2) / 448.0
            s["x"] = (b / sc[:, :, None]).reshape(R, K).to(torch.float8_e4m3fn).view(torch.uint8)
            s["x_scales"] = sc.contiguous()
        else:
            s["x"], s["x_scales"] = x.to(torch.bfloat16), None
    if case["op"] in ("product", "rows_grad"):
        s["w"] = _weights(g, E, N, K)
    if case["op"] in ("rows_grad", "weights_grad"):
        s["grad"] = (_randn(g, R, N) * 1e-3).to(torch.bfloat16)
    if case["op"] == "weights_grad":
        s["add"] = None
        if case["add"]:
            s["add"] = (_randn(g, E, N, K) * 1e-3 * math.sqrt(R / E)).to(_dt(case["grad"]))
    return s


# --------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, rounded once at the end
# --------------------------------------------------------------------------

def _rows(s):
    if s["x_scales"] is None:
        return s["x"].float()
    R, K = s["x"].shape
    x = s["x"].view(torch.float8_e4m3fn).float().view(R, K // 128, 128)
    return (x * s["x_scales"][:, :, None]).view(R, K)


def _places(s):
    """Expert of each row, and its place there."""
    pos = torch.arange(s["case"]["rows"], device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), pos, right=True)
    return e, pos - s["offsets"].long()[e]


def _by_expert(s, v):
    """Rows of each expert side by side, padded with zeros to the longest."""
    e, r = _places(s)
    p = torch.zeros(s["case"]["experts"], s["max_rows"], v.shape[1], device=DEV)
    p[e, r] = v
    return p


def _plain_product(s):
    y = torch.bmm(_by_expert(s, _rows(s)), s["w"].float().transpose(1, 2).contiguous())
    e, r = _places(s)
    y = y[e, r]
    if s["case"]["swiglu"]:
        N = s["case"]["out_features"] // 2
        y = y[:, :N] / (1 + torch.exp(-y[:, :N])) * y[:, N:]
    return y.to(torch.bfloat16)


def _plain_rows_grad(s):
    y = torch.bmm(_by_expert(s, s["grad"].float()), s["w"].float())
    e, r = _places(s)
    return y[e, r].to(torch.bfloat16)


def _plain_weights_grad(s):
    g = _by_expert(s, s["grad"].float()).transpose(1, 2).contiguous()
    y = torch.bmm(g, _by_expert(s, _rows(s)))
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(_dt(s["case"]["grad"]))


def _blocks(v, N):
    """Gate and up rows in blocks of 128 values, padded with zeros: [rows, 2, blocks, 128]."""
    R, G = v.shape[0], -(-N // 128)
    p = torch.zeros(R, 2, G * 128, dtype=v.dtype, device=v.device)
    p[:, :, :N] = v.view(R, 2, N)
    return p.view(R, 2, G, 128)


def _encode(gate_up, N):
    """E4M3 codes [rows, 2 N] and scales [rows, 2 ceil(N / 128)]: the smallest
    power of two, from 2^-100 on, with which the block's values stay within 448."""
    R = gate_up.shape[0]
    b = _blocks(gate_up.float(), N)
    m, e = torch.frexp(b.abs().amax(dim=3))
    e = torch.where(m > 0.875, e - 8, e - 9)   # 448 = 0.875 * 2^9
    e = torch.where(m == 0, -100, e).clamp(min=-100)
    scale = torch.ldexp(torch.ones_like(m), e)
    codes = (b / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return (codes.view(R, 2, -1)[:, :, :N].reshape(R, 2 * N).contiguous(),
            scale.view(R, -1).contiguous())


def _decode(codes, scales, N):
    b = _blocks(codes.view(torch.float8_e4m3fn).float(), N)
    R, _, G, _ = b.shape
    return (b * scales.view(R, 2, G, 1)).view(R, 2, G * 128)[:, :, :N]


def _plain_save(s):
    N = s["case"]["inner"]
    x = s["gate_up"].float()
    g, u = x[:, :N], x[:, N:]
    codes, scales = _encode(s["gate_up"], N)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16), codes.view(torch.float8_e4m3fn), scales


def _plain_use(s):
    v = _decode(s["codes"], s["scales"], s["case"]["inner"])
    g, u, d = v[:, 0], v[:, 1], s["grad"].float()
    sg = 1 / (1 + torch.exp(-g))
    grad = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], dim=1)
    return grad.to(torch.bfloat16), (g * sg * u).to(torch.bfloat16)


def run(s):
    c = s["case"]
    if not own:
        return {"product": _plain_product, "rows_grad": _plain_rows_grad,
                "weights_grad": _plain_weights_grad, "save": _plain_save,
                "use": _plain_use}[c["op"]](s)
    import combine_get_dispatch_amd as ep

    R, E = c["rows"], c["experts"]
    if "out" not in s:  # made once: the weights' handle or the checkpoint, and the outputs
        bf16 = dict(dtype=torch.bfloat16, device=DEV)
        if c["op"] == "product":
            s["experts"] = ep.Bf16Experts(s["w"], swiglu=c["swiglu"])
            s["out"] = torch.empty(R, c["out_features"] // (2 if c["swiglu"] else 1), **bf16)
        elif c["op"] == "rows_grad":
            s["experts"] = ep.Bf16Experts(s["w"])
            s["out"] = torch.empty(R, c["in_features"], **bf16)
        elif c["op"] == "weights_grad":
            s["cfg"] = ep.ep_experts_t(E, c["in_features"], c["out_features"])
            s["out"] = torch.empty(E, c["out_features"], c["in_features"], dtype=_dt(c["grad"]),
                                   device=DEV)
        else:
            s["checkpoint"] = ep.SwigluCheckpoint(R, c["inner"], E)
            s["out"] = torch.empty(R, c["inner"], **bf16)
            if c["op"] == "use":
                s["checkpoint"].codes.copy_(s["codes"])
                s["checkpoint"].scales.copy_(s["scales"])
                s["grad_gate_up"] = torch.empty(R, 2 * c["inner"], **bf16)
    at = s["offsets"], s["counts"]
    if c["op"] == "product":
        return s["experts"].product(s["x"], s["x_scales"], *at, out=s["out"])
    if c["op"] == "rows_grad":
        return s["experts"].backward_rows(s["grad"], *at, out=s["out"])
    if c["op"] == "weights_grad":
        ep.ep_expert_product_backward_weights(s["cfg"], s["x"], s["x_scales"], s["grad"], *at,
                                              s["add"], s["out"])
        return s["out"]
    if c["op"] == "save":
        k = s["checkpoint"]
        return k.save(s["gate_up"], *at, out=s["out"]), k.codes.view(torch.float8_e4m3fn), k.scales
    return s["checkpoint"].backward(s["grad"], *at, out=s["grad_gate_up"], h=s["out"])


# --------------------------------------------------------------------------
# Exact results, from the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_rows(s, lo, hi):
    if s["x_scales"] is None:
        return s["x"][lo:hi].double()
    return (s["x"][lo:hi].view(torch.float8_e4m3fn).double()
            * s["x_scales"][lo:hi].double().repeat_interleave(128, 1))


def _each_expert(s):
    at = s["offsets"].tolist()
    return [(e, at[e], at[e + 1]) for e in range(s["case"]["experts"])]


def _exact_product(s):
    c = s["case"]
    N = c["out_features"]
    out = torch.empty(c["rows"], N, dtype=torch.float64, device=DEV)
    for e, lo, hi in _each_expert(s):
        out[lo:hi] = _exact_rows(s, lo, hi) @ s["w"][e].double().T
    if not c["swiglu"]:
        return out
    gate, up = out[:, :N // 2], out[:, N // 2:]
    return gate * torch.sigmoid(gate) * up


def _exact_rows_grad(s):
    out = torch.empty(s["case"]["rows"], s["case"]["in_features"], dtype=torch.float64, device=DEV)
    for e, lo, hi in _each_expert(s):
        out[lo:hi] = s["grad"][lo:hi].double() @ s["w"][e].double()
    return out


def _exact_weights_grad(s):
    c = s["case"]
    out = torch.zeros(c["experts"], c["out_features"], c["in_features"], dtype=torch.float64,
                      device=DEV)
    if s["add"] is not None:
        out += s["add"]
    for e, lo, hi in _each_expert(s):
        out[e] += s["grad"][lo:hi].double().T @ _exact_rows(s, lo, hi)
    return out


def _exact_save(s):
    N = s["case"]["inner"]
    codes, scales = [], []
    x = s["gate_up"].double()
    for half in (x[:, :N], x[:, N:]):
        for lo in range(0, N, 128):
            v = half[:, lo:lo + 128]
            e = torch.ceil(torch.log2(v.abs().amax(dim=1, keepdim=True) / 448))
            # log2 decides up to a rounding: the border itself by the inequality
            e = torch.where(v.abs().amax(dim=1, keepdim=True) > 448 * torch.exp2(e), e + 1, e)
            e = torch.where(v.abs().amax(dim=1, keepdim=True) <= 448 * torch.exp2(e - 1), e - 1, e)
            scale = torch.exp2(e.clamp(min=-100))
            v = v / scale
            # a step is 2^-3 of the value's power of two, 2^-9 from the smallest normal one down
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            codes.append(torch.round(v / step) * step)
            scales.append(scale)
    gate, up = x[:, :N], x[:, N:]
    return gate * torch.sigmoid(gate) * up, torch.cat(codes, dim=1), torch.cat(scales, dim=1)


def _exact_use(s):
    # the gradient by torch's own differentiation in 64 bits
    N = s["case"]["inner"]
    at = torch.arange(N, device=DEV) // 128
    sc = s["scales"].double().view(s["case"]["rows"], 2, -1)[:, :, at].reshape(-1, 2 * N)
    x = (s["codes"].view(torch.float8_e4m3fn).double() * sc).requires_grad_(True)
    with torch.enable_grad():
        h = torch.nn.functional.silu(x[:, :N]) * x[:, N:]
        h.backward(s["grad"].double())
    return x.grad, h.detach()


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "rows_grad": _exact_rows_grad,
            "weights_grad": _exact_weights_grad, "save": _exact_save,
            "use": _exact_use}[case["op"]](s)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    R = case["rows"]
    if case["op"] in ("save", "use"):
        N = case["inner"]
        kept = 2 * N + 8 * -(-N // 128)  # codes and scales of a row
        # save: gate and up, h;  use: the gradient of h, that of gate and up, h
        return dict(bytes=R * (kept + 4 * N + 2 * N + (2 * N if case["op"] == "use" else 0)),
                    flops=20.0 * R * N)
    K, N = case["in_features"], case["out_features"]
    hit = min(case["hit"], case["experts"], R)
    row = K + 4 * (K // 128) if case.get("x") == "fp8" else 2 * K
    flops = 2.0 * R * N * K
    if case["op"] == "product":
        out = N // 2 if case["swiglu"] else N
        return dict(bytes=2 * hit * N * K + R * (row + 2 * out), flops=flops)
    if case["op"] == "rows_grad":
        return dict(bytes=2 * hit * N * K + 2 * R * (N + K), flops=flops)
    size = (4 if case["grad"] == "fp32" else 2) * (2 if case["add"] else 1)
    return dict(bytes=R * (row + 2 * N) + case["experts"] * N * K * size, flops=flops)
