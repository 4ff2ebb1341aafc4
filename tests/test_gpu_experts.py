"""The experts' products with bf16 weights and their gradients on the GPU.

Where inputs are small integers (and scales powers of two) every sum is exact
in fp32, and the result has to be the rounding of the exact one, bit for bit.
Elsewhere a sum of L terms of fp32 is off by at most L + 8 half steps of the
sum of magnitudes, the output by a half step of its type.  FP8 rows enter the
product unrounded (a sum of 128 codes is scaled, one more half step), and the
weights' gradient as bf16(code * scale): that is what the reference multiplies.

Rows that are no expert's, and weights of experts without rows, are NaN: they
may enter no result."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_amd as ep  # noqa: E402
from tests import experts_reference as ref  # noqa: E402
from tests.gpu_backend import dev, say  # noqa: E402

U32, UBF16 = ref.U32, ref.UBF16


def layout_of(counts, gap):
    """Offsets with `gap` rows behind each expert, and the rows in all."""
    off = np.concatenate([[0], np.cumsum(np.asarray(counts) + gap)]).astype(np.int32)
    return off, int(off[-1])


def only_experts(v, off, counts):
    """NaN in the rows that are no expert's."""
    out = np.full_like(v, np.nan)
    for _, lo, hi in ref.expert_rows(off, counts, v.shape[0]):
        out[lo:hi] = v[lo:hi]
    return out


def draw_rows(rng, cap, K, exact):
    return rng.integers(-4, 5, size=(cap, K)).astype(np.float64) if exact else ref.rounded(
        rng.normal(size=(cap, K)))


def draw_fp8(rng, cap, K, exact, round_to_bf16):
    """(codes, scales on the device, the values that enter the product)"""
    v = draw_rows(rng, cap, K, exact)
    t = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn)
    if exact:
        s = 2.0 ** rng.integers(-2, 3, size=(cap, K // 128))
    else:
        s = (rng.random((cap, K // 128)) + 0.1).astype(np.float32).astype(np.float64)
    val = t.float().double().numpy() * np.repeat(s, 128, axis=1)
    if round_to_bf16:  # a product of 4 and 24 bits, rounded to 24, then to 8
        val = ref.rounded(val.astype(np.float32))
    return t.view(torch.uint8).cuda(), dev(s.astype(np.float32)), val


def draw_x(rng, cap, K, fp8, exact, off, counts, round_to_bf16=False):
    if fp8:
        x, xs, xv = draw_fp8(rng, cap, K, exact, round_to_bf16)
        dead = torch.from_numpy(np.isnan(only_experts(xv, off, counts)[:, 0])).cuda()
        x[dead] = 0x7F
        xs[dead] = float("nan")
        return x, xs, xv
    xv = draw_rows(rng, cap, K, exact)
    return ref.to_bf16(only_experts(xv, off, counts)).cuda(), None, xv


def draw_w(rng, counts, N, K, exact):
    E = len(counts)
    w = rng.integers(-4, 5, size=(E, N, K)).astype(np.float64) if exact else ref.rounded(
        rng.normal(size=(E, N, K)) / np.sqrt(K))
    t = w.copy()
    t[np.asarray(counts) == 0] = np.nan
    return ref.to_bf16(t).cuda(), w


def check_rows(got, want, size, terms, exact):
    """bf16 rows; NaN in `want`: not an expert's, still 99."""
    got = got.double().cpu().numpy()
    dead = np.isnan(want)
    assert (got[dead] == 99.0).all(), "a row that is no expert's was written"
    if exact:
        w = ref.rounded(np.where(dead, 99.0, want))
        bad = got != w
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], w[bad][:4])
        return
    err = ref.sum_error(terms, size)
    tol = err + (np.abs(want) + err) * UBF16 + 1e-37
    d = np.abs(got - want)
    assert np.all(d[~dead] <= tol[~dead]), np.max((d / tol)[~dead])


def many(seed, experts, *large):
    """Experts enough for the large tiles: a few rows each, and some of many."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 4, experts)
    c[rng.choice(experts, len(large), replace=False)] = large
    return [int(n) for n in c]


SHAPES = [  # K, N, counts
    (128, 80, many(1, 180, 513, 64, 65)), (264, 272, many(2, 190, 300, 129)),
    (384, 48, many(3, 200, 255, 192, 128)), (64, 48, many(5, 1024, 300)), (72, 536, many(4, 170, 257, 700)),
    (1, 1, [1]), (8, 8, [1]), (33, 18, [3, 0]), (128, 40, [0, 1, 17]), (256, 130, [65, 1, 0, 64]),
    (1024, 100, [0, 7]), (640, 264, [33, 1, 0, 129, 2]), (384, 96, [9, 8, 7, 6, 5, 4, 3, 200]),
    (512, 520, [300]), (136, 1002, [257, 31]), (384, 512, [130, 256, 0, 511]), (72, 64, [16] * 9),
    (1920, 256, [2, 4, 1, 15, 16, 17]), (512, 128, [3, 0, 5]), (2176, 80, [1, 0, 0, 14]),
    (896, 34, [16]), (640, 96, [0, 40, 9]), (136, 66, [2, 30, 1]), (2048, 24, [100, 31, 32, 33]), (904, 776, [64, 128, 192]),
]


def name(v):
    """of a test's counts"""
    return f"{len(v)}x{max(v)}" if isinstance(v, list) and len(v) > 12 else None


@pytest.mark.parametrize("K,N,counts", SHAPES, ids=name)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product(K, N, counts, fp8, swiglu):
    if fp8 and K % 128:
        pytest.skip("FP8 rows come in blocks of 128")
    if swiglu and N % 2:
        pytest.skip("gate and up are halves")
    rng = np.random.default_rng(K + N)
    off, cap = layout_of(counts, 2)
    for exact in (True, False):
        say(f"product K={K} N={N} counts={counts[:9]} fp8={fp8} swiglu={swiglu} exact={exact}")
        x, xs, xv = draw_x(rng, cap, K, fp8, exact, off, counts)
        wt, w = draw_w(rng, counts, N, K, exact)
        out = torch.full((cap, N // 2 if swiglu else N), 99.0, dtype=torch.bfloat16, device="cuda")
        got = ep.Bf16Experts(wt, swiglu=swiglu).product(x, xs, dev(off),
                                                        dev(np.array(counts, np.int32)), out=out)
        assert got is out
        y, size = ref.product(xv, w, off, counts)
        if not swiglu:
            check_rows(out, y, size, K, exact)
            continue
        # h = silu(a) b: silu has a slope of at most 1.1, the function and the
        # products are off by 12 half steps
        h = N // 2
        a, b, err = y[:, :h], y[:, h:], 0.0 * size if exact else ref.sum_error(K, size)
        want = ref.silu(a) * b
        e = (1.1 * err[:, :h] * (np.abs(b) + err[:, h:]) + np.abs(ref.silu(a)) * err[:, h:]
             + 12 * U32 * np.abs(want))
        g = out.double().cpu().numpy()
        dead = np.isnan(want)
        assert (g[dead] == 99.0).all()
        tol = e + (np.abs(want) + e) * UBF16 + 1e-37
        assert np.all(np.abs(g - want)[~dead] <= tol[~dead])


@pytest.mark.parametrize("K,N,counts", SHAPES + [(40, 33, [5, 70]), (1001, 131, [3, 129])],
                         ids=name)
def test_rows_gradient(K, N, counts):
    rng = np.random.default_rng(K + N + 1)
    off, cap = layout_of(counts, 1)
    for exact in (True, False):
        say(f"rows' gradient K={K} N={N} counts={counts[:9]} exact={exact}")
        gv = draw_rows(rng, cap, N, exact)
        g = ref.to_bf16(only_experts(gv, off, counts)).cuda()
        wt, w = draw_w(rng, counts, N, K, exact)
        out = torch.full((cap, K), 99.0, dtype=torch.bfloat16, device="cuda")
        ep.Bf16Experts(wt).backward_rows(g, dev(off), dev(np.array(counts, np.int32)), out=out)
        check_rows(out, *ref.rows_grad(gv, w, off, counts), N, exact)


@pytest.mark.parametrize("K,N,counts", SHAPES + [(40, 33, [5, 70]), (1001, 131, [3, 129])],
                         ids=name)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("add", ["none", "apart", "in place"])
def test_weights_gradient(K, N, counts, fp8, dtype, add):
    if fp8 and K % 128:
        pytest.skip("FP8 rows come in blocks of 128")
    rng = np.random.default_rng(K + N + 2)
    off, cap = layout_of(counts, 3)
    E = len(counts)
    for exact in (True, False):
        say(f"weights' gradient K={K} N={N} counts={counts[:9]} fp8={fp8} {dtype} add={add} "
            f"exact={exact}")
        gv = draw_rows(rng, cap, N, exact)
        g = ref.to_bf16(only_experts(gv, off, counts)).cuda()
        x, xs, xv = draw_x(rng, cap, K, fp8, exact, off, counts, round_to_bf16=True)
        want, size = ref.weights_grad(gv, xv, off, counts)
        out = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
        before = None
        if add != "none":
            av = (rng.integers(-64, 65, size=(E, N, K)).astype(np.float64) if exact
                  else ref.rounded(rng.normal(size=(E, N, K))))
            before = torch.from_numpy(av.astype(np.float32)).to(dtype).cuda()
            want, size = want + av, size + np.abs(av)
            if add == "in place":
                out = before
        e = ep.Bf16Experts(torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda"))
        e.backward_weights(x, xs, g, dev(off), dev(np.array(counts, np.int32)), out=out,
                           add=before)
        got = out.double().cpu().numpy()
        if exact:
            if dtype == torch.bfloat16:
                want = ref.rounded(want)
            assert np.array_equal(got, want), np.argwhere(got != want)[:4]
            continue
        err = ref.sum_error(max(counts) + 1, size)
        if dtype == torch.bfloat16:
            err = err + (np.abs(want) + err) * UBF16
        d = np.abs(got - want)
        assert np.all(d <= err + 1e-37), np.max(d / (err + 1e-37))


def test_fp8_rows_are_rounded_once():
    """The weights' gradient against the unrounded rows: 2^-8 of each value at
    most, and the sum's own rounding."""
    rng = np.random.default_rng(5)
    K, N, counts = 512, 96, [40, 3]
    off, cap = layout_of(counts, 0)
    x, xs, raw = draw_fp8(rng, cap, K, False, False)
    gv = draw_rows(rng, cap, N, False)
    say("rounding of FP8 rows")
    e = ep.Bf16Experts(torch.zeros(2, N, K, dtype=torch.bfloat16, device="cuda"))
    got = e.backward_weights(x, xs, ref.to_bf16(gv).cuda(), dev(off),
                             dev(np.array(counts, np.int32)), dtype=torch.float32)
    y, size = ref.weights_grad(gv, raw, off, counts)
    err = size * UBF16 + ref.sum_error(40, size * (1 + UBF16))
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= err)


@pytest.mark.parametrize("K,N", [(128, 64), (75, 33)])
def test_rows_past_the_capacity_and_bad_offsets_are_left_alone(K, N):
    rng = np.random.default_rng(6)
    E, cap = 4, 10
    off, cnt = np.array([0, 4, -3, 2 ** 31 - 1], np.int32), np.array([3, 100, 5, 7], np.int32)
    xv, w = draw_rows(rng, cap, K, True), rng.integers(-4, 5, size=(E, N, K)).astype(np.float64)
    gv = draw_rows(rng, cap, N, True)
    e = ep.Bf16Experts(ref.to_bf16(w).cuda())
    x, g = ref.to_bf16(xv).cuda(), ref.to_bf16(gv).cuda()
    for name, call, rows, width, form in (("product", lambda o, c, out: e.product(
            x, None, o, c, out=out), xv, N, ref.product), ("rows' gradient",
            lambda o, c, out: e.backward_rows(g, o, c, out=out), gv, K, ref.rows_grad)):
        say(f"{name}: rows past the capacity")
        out = torch.full((cap + 4, width), 99.0, dtype=torch.bfloat16, device="cuda")
        call(dev(off), dev(cnt), out)
        want = np.full((cap + 4, width), 99.0)
        y = form(rows, w, off, cnt)[0]
        want[:cap] = np.where(np.isnan(y), 99.0, ref.rounded(np.nan_to_num(y)))
        assert np.array_equal(out.double().cpu().numpy(), want)
        say(f"{name}: no rows")
        call(dev(off), dev(np.zeros(4, np.int32)), out)
        call(dev(off), dev(np.full(4, -7, np.int32)), out)
        assert np.array_equal(out.double().cpu().numpy(), want)
    say("weights' gradient: rows past the capacity, experts without rows")
    gw = e.backward_weights(x, None, g, dev(off), dev(cnt), dtype=torch.float32)
    assert np.array_equal(gw.double().cpu().numpy(), ref.weights_grad(gv, xv, off, cnt)[0])
    say("weights' gradient: no rows at all, no capacity")
    for rows in (cap, 0):
        gw.fill_(float("nan"))
        e.backward_weights(x[:rows], None, g[:rows], dev(off), dev(np.zeros(4, np.int32)), out=gw)
        assert not gw.any()
        add = torch.randn_like(gw)
        e.backward_weights(x[:rows], None, g[:rows], dev(off), dev(np.zeros(4, np.int32)), out=gw,
                           add=add)
        assert torch.equal(gw, add)


@pytest.mark.parametrize("K,N", [(256, 128), (75, 33)])
def test_rows_that_are_not_finite_stay_by_themselves(K, N):
    rng = np.random.default_rng(7)
    counts = [70, 20]
    off, cap = layout_of(counts, 0)
    at, cnt = dev(off), dev(np.array(counts, np.int32))
    wt, _ = draw_w(rng, counts, N, K, False)
    e = ep.Bf16Experts(wt)
    for width, call in ((K, lambda v: e.product(v, None, at, cnt)),
                        (N, lambda v: e.backward_rows(v, at, cnt))):
        v = ref.to_bf16(draw_rows(rng, cap, width, False)).cuda()
        say(f"rows that are not finite, width {width}")
        clean = call(v)
        dirty = v.clone()
        dirty[3, width - 1], dirty[64, 0], dirty[89, 1] = float("inf"), float("nan"), -float("inf")
        got = call(dirty)
        bad = torch.zeros(cap, dtype=torch.bool, device="cuda")
        bad[[3, 64, 89]] = True
        assert torch.equal(got[~bad], clean[~bad])
        assert not torch.isfinite(got[bad]).any()


@pytest.mark.parametrize("swiglu", [False, True])
def test_results_between_16_byte_boundaries(swiglu):
    """Results may begin anywhere: by tiles, few rows and gradients."""
    rng = np.random.default_rng(8)
    K, N = 128, 80
    for counts in ([3], [40, 100], many(4, 180, 200)):
        off, cap = layout_of(counts, 0)
        at = dev(off), dev(np.array(counts, np.int32))
        wt, _ = draw_w(rng, counts, N, K, False)
        wt = wt.nan_to_num()
        x = ref.to_bf16(draw_rows(rng, cap, K, False)).cuda()
        e = ep.Bf16Experts(wt, swiglu=swiglu)
        say(f"results between 16-byte boundaries, {len(counts)} experts")
        want = e.product(x, None, *at)
        for by in (1, 3, 4):
            flat = torch.full((want.numel() + 8,), 99.0, dtype=torch.bfloat16, device="cuda")
            out = flat[by:by + want.numel()].view(want.shape)
            assert torch.equal(e.product(x, None, *at, out=out), want)
            assert (flat[:by] == 99.0).all() and (flat[by + want.numel():] == 99.0).all()
        g = ref.to_bf16(draw_rows(rng, cap, N, False)).cuda()
        want = e.backward_rows(g, *at)
        flat = torch.full((want.numel() + 8,), 99.0, dtype=torch.bfloat16, device="cuda")
        out = flat[1:1 + want.numel()].view(want.shape)
        # another order of the same sums
        d = (e.backward_rows(g, *at, out=out).double() - want.double()).abs()
        size = 2 * ref.sum_error(N, 6 * 4 * N ** 0.5) + want.double().abs() * 2 * UBF16
        assert (d <= size).all() and flat[0] == 99.0 and (flat[1 + want.numel():] == 99.0).all()


def test_large_and_small_values():
    """Rows and weights of any size: sums in fp32's range are finite."""
    K, N = 256, 64
    for scale in (1e-30, 1e30):
        say(f"rows of {scale}")
        x = torch.full((70, K), scale, dtype=torch.bfloat16, device="cuda")
        w = torch.full((1, N, K), 1 / scale, dtype=torch.bfloat16, device="cuda")
        at = dev(np.array([0], np.int32)), dev(np.array([70], np.int32))
        want = ref.rounded(K * float(x[0, 0]) * float(w[0, 0, 0]))
        got = ep.Bf16Experts(w).product(x, None, *at)
        assert np.array_equal(got.double().cpu().numpy(), np.full((70, N), want))


# Row tiles of an expert go through the columns in bands of eight: more than
# eight tiles of 256 rows and of 128 (few tiles in all), a last band of one and
# of more, and beside them experts of one tile and of none.
BANDS = [(128, 520, many(8, 180, 2500, 2049)), (256, 264, [1100, 3, 0, 40]),
         (384, 776, [2, 2304, 0, 1, 1025] + [1, 0, 257] * 30), (128, 40, [0, 1030, 2200])]


@pytest.mark.parametrize("K,N,counts", BANDS, ids=name)
@pytest.mark.parametrize("fp8", [False, True])
def test_product_over_bands_of_row_tiles(K, N, counts, fp8):
    rng = np.random.default_rng(N + len(counts))
    off, cap = layout_of(counts, 1)
    say(f"bands K={K} N={N} counts={counts[:5]} fp8={fp8}")
    x, xs, xv = draw_x(rng, cap, K, fp8, True, off, counts)
    wt, w = draw_w(rng, counts, N, K, True)
    at = dev(off), dev(np.array(counts, np.int32))
    out = torch.full((cap, N), 99.0, dtype=torch.bfloat16, device="cuda")
    ep.Bf16Experts(wt).product(x, xs, *at, out=out)
    y, size = ref.product(xv, w, off, counts)
    check_rows(out, y, size, K, True)
    if fp8:
        return
    say("rows' gradient")  # of the product turned over: the same sums
    out.fill_(99.0)
    ep.Bf16Experts(wt.transpose(1, 2).contiguous()).backward_rows(x, *at, out=out)
    check_rows(out, y, size, K, True)


# rows of the weights: 19, 10 and 9 tiles of 128 or 256, by few tiles in all, some, many
@pytest.mark.parametrize("K,N,counts", [(384, 2312, [70, 3]), (640, 2312, [5, 0, 64, 1, 130, 9]),
                                        (264, 2056, [1, 2, 70, 0] * 16)], ids=name)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("add", [False, True])
def test_weights_gradient_over_bands_of_row_tiles(K, N, counts, fp8, dtype, add):
    if fp8 and K % 128:
        pytest.skip("FP8 rows come in blocks of 128")
    rng = np.random.default_rng(K + N)
    off, cap = layout_of(counts, 2)
    E = len(counts)
    say(f"bands of the weights' gradient K={K} N={N} counts={counts[:6]} fp8={fp8} {dtype} "
        f"add={add}")
    gv = draw_rows(rng, cap, N, True)
    g = ref.to_bf16(only_experts(gv, off, counts)).cuda()
    x, xs, xv = draw_x(rng, cap, K, fp8, True, off, counts, round_to_bf16=True)
    want = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e, lo, hi in ref.expert_rows(off, counts, cap):
        want[e] = torch.from_numpy(gv[lo:hi].T @ xv[lo:hi]).cuda()
    out = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
    if add:
        out = torch.randint(-64, 65, (E, N, K), device="cuda").to(dtype)
        want += out.double()
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    ep.Bf16Experts(w).backward_weights(x, xs, g, dev(off), dev(np.array(counts, np.int32)),
                                       out=out, add=out if add else None)
    assert torch.equal(out, want.float().to(dtype))


@pytest.mark.parametrize("counts", [[5], [70], [3, 70] * 90], ids=["few", "tiles", "many"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_over_the_whole_range(counts, fp8, swiglu):
    """Rows, scales and weights at the top and the bottom of their types, that
    bring the result back: finite wherever the result is.  Exact: a row is one
    power of two, times 1.5 by its scales, with any signs, and a matrix another
    one times -3 .. 3, so a sum is at most 256 x 9 steps of a power of two."""
    rng = np.random.default_rng(42)
    K, N = 256, 40
    if fp8:  # power of the codes, of the rows' scales, of the weights
        cases = [(8, -30, 118), (8, 119, -30), (-9, 115, 12), (8, -110, 120), (-9, -60, 120),
                 (8, -126, 20), (0, 127, -120), (-9, 127, -126), (8, -10, -110), (8, 118, -126)]
    else:
        cases = [(127, 0, -30), (127, 0, -120), (-100, 0, 120), (-126, 0, 120), (0, 0, 110),
                 (0, 0, -110)]
    off, cap = layout_of(counts, 0)
    at = dev(off), dev(np.array(counts, np.int32))
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], size=(cap, K))).cuda()
    small = torch.from_numpy(rng.integers(-3, 4, size=(len(counts), N, K)).astype(float)).cuda()
    sums = torch.cat([sign[lo:hi] @ small[e].T for e, lo, hi in ref.expert_rows(off, counts, cap)])
    for px, ps, pw in cases:
        say(f"range counts={counts[:2]} fp8={fp8} swiglu={swiglu} powers={px, ps, pw}")
        v = sign * 2.0 ** px
        x, xs, by = v.bfloat16(), None, 1.0
        if fp8:
            x, by = v.to(torch.float8_e4m3fn), 1.5
            xs = torch.full((cap, K // 128), by * 2.0 ** ps, device="cuda")
        assert torch.equal(x.double(), v)
        w = (small * 2.0 ** pw).bfloat16()
        assert torch.equal(w.double(), small * 2.0 ** pw)
        y = sums * by * 2.0 ** (px + ps + pw)
        got = ep.Bf16Experts(w, swiglu=swiglu).product(x.view(torch.uint8) if fp8 else x, xs, *at)
        if not swiglu:
            want = y.float().bfloat16()
            assert torch.isfinite(want).all() and torch.equal(got, want)
            continue
        # 12 half steps, as in test_product, and a step of fp32's smallest numbers
        # in the exponential; a result past fp32's range is infinite and one below
        # its normal numbers may lose bits
        g, u = y[:, :N // 2], y[:, N // 2:]
        want = g / (1 + torch.exp(-g)) * u
        inside = want.abs() < 2.0 ** 127
        err = want.abs() * 12 * U32 + (g * u).abs() * 2.0 ** -149
        tol = err + (want.abs() + err) * UBF16 + 2.0 ** -125
        assert ((got.double() - want).abs() <= tol)[inside].all()
        assert not torch.isnan(got).any()


@pytest.mark.parametrize("counts", [[5], [70], [3, 70, 129] * 60], ids=["few", "tiles", "many"])
def test_fp8_rows_beside_rows_of_other_scales(counts):
    """Any scale beside any other, on both sides of those that the kernels treat
    another way; and scales that are not finite stay by themselves.  Exact: small
    integers times one power of two per row."""
    rng = np.random.default_rng(43)
    K, N = 256, 72
    off, cap = layout_of(counts, 0)
    at = dev(off), dev(np.array(counts, np.int32))
    x, _, xv = draw_fp8(rng, cap, K, True, False)
    v = x.view(torch.float8_e4m3fn).double()
    w, wv = draw_w(rng, counts, N, K, True)
    scales = 2.0 ** rng.choice([-126, -100, -30, -2, 0, 1, 31, 32, 33, 60, 100], size=cap)
    say(f"scales beside others, counts={counts[:3]}")

    def product(s):
        xs = torch.from_numpy(np.repeat(s[:, None], K // 128, axis=1)).float().cuda()
        return ep.Bf16Experts(w).product(x, xs, *at)

    sums = torch.cat([v[lo:hi] @ torch.from_numpy(wv[e].T).cuda()
                      for e, lo, hi in ref.expert_rows(off, counts, cap)])
    want = (sums * torch.from_numpy(scales).cuda()[:, None]).float().bfloat16()
    assert torch.equal(product(scales), want)
    bad = rng.random(cap) < 0.2
    bad[0] = True
    dirty = np.where(bad, rng.choice([np.inf, -np.inf, np.nan], size=cap), scales)
    got = product(dirty)
    assert torch.equal(got[torch.from_numpy(~bad).cuda()], want[torch.from_numpy(~bad).cuda()])
    assert not torch.isfinite(got[torch.from_numpy(bad).cuda()]).any()


@pytest.mark.parametrize("K,N,counts", [(384, 272, many(6, 260, 300, 65)), (264, 528, many(7, 175, 129))],
                         ids=name)
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_gradient_of_many_tiles(K, N, counts, fp8):
    """More than a thousand tiles, several of each expert, shared by the steps they take."""
    if fp8 and K % 128:
        pytest.skip("FP8 rows come in blocks of 128")
    rng = np.random.default_rng(K)
    off, cap = layout_of(counts, 1)
    say(f"weights' gradient of many tiles K={K} N={N} fp8={fp8}")
    x, xs, xv = draw_x(rng, cap, K, fp8, True, off, counts, True)
    dyv = draw_rows(rng, cap, N, True)
    dy = ref.to_bf16(only_experts(dyv, off, counts)).cuda()
    w = torch.zeros(len(counts), N, K, dtype=torch.bfloat16, device="cuda")
    got = ep.Bf16Experts(w).backward_weights(x, xs, dy, dev(off), dev(np.array(counts, np.int32)),
                                             dtype=torch.float32).cpu().numpy()
    for e, lo, hi in ref.expert_rows(off, counts, cap):
        assert np.array_equal(got[e], dyv[lo:hi].T @ xv[lo:hi]), e


@pytest.mark.parametrize("K,fp8", [(64, False), (72, False), (128, False), (192, False), (128, True),
                                   (256, True), (384, True)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_short_sums_of_many_full_tiles(K, fp8, swiglu):
    """A stage or a few per tile, several tiles one after the other: a tile's
    stores are on their way while the next ones' rows and columns come."""
    rng = np.random.default_rng(K)
    N = 1040
    counts = [int(n) for n in rng.choice([128, 256, 65, 300], size=180)]
    off, cap = layout_of(counts, 0)
    say(f"short sums K={K} fp8={fp8} swiglu={swiglu}")
    x, xs, xv = draw_x(rng, cap, K, fp8, True, off, counts)
    w = torch.randint(-4, 5, (len(counts), N, K), device="cuda").to(torch.bfloat16)
    n = dev(np.array(counts, np.int32))
    y = ep.Bf16Experts(w).product(x, xs, dev(off), n)
    xd = torch.from_numpy(xv).cuda()
    sums = torch.empty(cap, N, dtype=torch.float64, device="cuda")
    for e, lo, hi in ref.expert_rows(off, counts, cap):
        sums[lo:hi] = xd[lo:hi] @ w[e].double().T
    assert torch.equal(y, sums.float().bfloat16())
    if swiglu:
        # sums are exact: an exponential, a division and two products, then bf16
        h = ep.Bf16Experts(w, swiglu=True).product(x, xs, dev(off), n).double()
        g, u = sums[:, :N // 2], sums[:, N // 2:]
        want = g / (1 + torch.exp(-g)) * u
        tol = want.abs() * (12 * U32 + UBF16 * (1 + 12 * U32)) + 1e-37
        assert ((h - want).abs() <= tol).all()
    elif not fp8:  # the rows' gradient of the product turned over
        dx = ep.Bf16Experts(w.transpose(1, 2).contiguous()).backward_rows(x, dev(off), n)
        assert torch.equal(dx, y)


# (experts, K, N, the rows of each hit expert): all have more than 256 MiB of weights
PAST_CACHE = [(40, 2048, 2048, [3] * 40), (40, 2048, 2040, [70] + [0, 20] * 19 + [129]),
              (20, 4096, 2064, [1] * 16 + [0] * 4), (33, 2176, 2048, [0] + [17] * 32)]


@pytest.mark.parametrize("E,K,N,counts", PAST_CACHE, ids=["3", "uneven", "one", "17"])
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_past_the_cache(E, K, N, counts, fp8):
    """Small integers: sums are exact, so every form of the kernel has to give
    the same bits, with SwiGLU too, as calls over a few experts at a time."""
    rng = np.random.default_rng(E + K)
    off, cap = layout_of(counts, 1)
    say(f"weights past the cache E={E} K={K} N={N} fp8={fp8}")
    x, xs, xv = draw_x(rng, cap, K, fp8, True, off, counts)
    w = torch.randint(-4, 5, (E, N, K), device="cuda").to(torch.bfloat16)
    dyv = draw_rows(rng, cap, N, True)
    dy = ref.to_bf16(only_experts(dyv, off, counts)).cuda()
    n = np.array(counts, np.int32)

    def run(swiglu, from_expert, to_expert):
        part = ep.Bf16Experts(w[from_expert:to_expert], swiglu=swiglu)
        o = dev(off[from_expert:to_expert + 1])
        k = dev(n[from_expert:to_expert])
        out = torch.full((cap, N // 2 if swiglu else N), 99.0, dtype=torch.bfloat16, device="cuda")
        part.product(x, xs, o, k, out=out)
        dx = torch.full((cap, K), 99.0, dtype=torch.bfloat16, device="cuda")
        part.backward_rows(dy, o, k, out=dx)
        return out, dx

    y, dx = run(False, 0, E)
    h, _ = run(True, 0, E)
    y_want = torch.full_like(y, 99.0)
    dx_want = torch.full_like(dx, 99.0)
    xd, dyd = torch.from_numpy(xv).cuda(), torch.from_numpy(dyv).cuda()
    for e, lo, hi in ref.expert_rows(off, counts, cap):
        y_want[lo:hi] = (xd[lo:hi] @ w[e].double().T).float().bfloat16()
        dx_want[lo:hi] = (dyd[lo:hi] @ w[e].double()).float().bfloat16()
    assert torch.equal(y, y_want) and torch.equal(dx, dx_want)
    for e in range(0, E, 7):
        to = min(E, e + 7)
        lo, hi = int(off[e]), int(off[to])
        h_part, dx_part = run(True, e, to)
        assert torch.equal(h[lo:hi], h_part[lo:hi]) and torch.equal(dx[lo:hi], dx_part[lo:hi])


def test_weights_with_another_storage():
    """A tensor's storage may be replaced between calls; what does not fit is refused."""
    t = torch.zeros(2, 32, 128, dtype=torch.bfloat16, device="cuda")
    e = ep.Bf16Experts(t)
    x = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(4, 32, dtype=torch.bfloat16, device="cuda")
    off, n = dev(np.array([0, 2, 4], np.int32)), dev(np.array([2, 2], np.int32))
    assert (e.product(x, None, off, n) == 0).all()
    t.data = torch.ones_like(t)
    assert (e.product(x, None, off, n) == 128).all()
    assert (e.backward_rows(g, off, n) == 32).all()
    t.data = torch.ones(2, 16, 128, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: e.product(x, None, off, n), lambda: e.backward_rows(g, off, n)):
        with pytest.raises(ValueError):
            call()


def test_weights_changed_at_the_same_address():
    """What the calls would read another way than the tensor now says is refused."""
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    off, n = dev(np.array([0, 2, 4], np.int32)), dev(np.array([2, 2], np.int32))
    for change in (lambda t: t.transpose(1, 2), lambda t: t[:1], lambda t: t[:, :32],
                   lambda t: t.view(torch.float16)):
        t = torch.ones(2, 64, 64, dtype=torch.bfloat16, device="cuda")
        e, at = ep.Bf16Experts(t), t.data_ptr()
        assert (e.product(x, None, off, n) == 64).all()
        t.data = change(t)
        assert t.data_ptr() == at
        for call in (lambda: e.product(x, None, off, n), lambda: e.backward_rows(x, off, n)):
            with pytest.raises(ValueError):
                call()
    t.data = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    assert (e.product(x, None, off, n) == 0).all()
    t.data = t.cpu()
    with pytest.raises(ValueError):
        e.product(x, None, off, n)


def test_python_refusals():
    e = ep.Bf16Experts(torch.zeros(2, 32, 128, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, gx, gw = g.clone(), x.clone(), torch.zeros(2, 32, 128, device="cuda")
    for bad in (dict(x=x[:, :64]), dict(x=x.float()), dict(off=off[:1]), dict(cnt=off[:1]),
                dict(out=out[:3]), dict(out=out.float()), dict(x=x.t().contiguous().t()),
                dict(xs=torch.ones(4, 1, device="cuda")), dict(cnt=off.long()), dict(x=x.cpu()),
                dict(out=out.t().contiguous().t())):
        a = dict(dict(x=x, xs=None, off=off, cnt=off, out=out), **bad)
        with pytest.raises(ValueError):
            e.product(a["x"], a["xs"], a["off"], a["cnt"], out=a["out"])
    for bad in (dict(g=g[:, :16]), dict(g=g.float()), dict(out=gx[:3]), dict(out=gx.half()),
                dict(off=off.long()), dict(g=g.cpu())):
        a = dict(dict(g=g, off=off, out=gx), **bad)
        with pytest.raises(ValueError):
            e.backward_rows(a["g"], a["off"], off, out=a["out"])
    for bad in (dict(g=g[:3]), dict(x=x.float()), dict(out=gw[:1]), dict(out=gw.half()),
                dict(add=gw.bfloat16()), dict(add=gw[:, :31]), dict(xs=torch.ones(4, device="cuda"))):
        a = dict(dict(g=g, x=x, xs=None, out=gw, add=None), **bad)
        with pytest.raises(ValueError):
            e.backward_weights(a["x"], a["xs"], a["g"], off, off, out=a["out"], add=a["add"])
    with pytest.raises(ep.EpError):  # rows that begin between 16-byte boundaries
        e.product(torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 128),
                  None, off, off)
    with pytest.raises(ep.EpError):  # a result over its input
        ep.Bf16Experts(torch.zeros(2, 128, 128, dtype=torch.bfloat16, device="cuda")).product(
            x, None, off, off, out=x)
