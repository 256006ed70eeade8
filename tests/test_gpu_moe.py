"""GPU parity of the operators around the packed-MXFP4 products: epilogues,
products grouped by expert, the router and the weighted sum.

Products are compared bit for bit on operands whose every partial sum fp32
holds exactly.  Activations, weights and weighted sums are compared within
the half steps (2^-24 relative for fp32, 2^-8 for bf16) of the operations
that they take, as derived beside each check."""
import itertools

import numpy as np
import pytest
import torch

from oracle import moe_ref as moe
from oracle import mxfp4_ref as mx
from synthetic_inputs import to_bf16_values

pytestmark = pytest.mark.gpu
F32, F64 = np.float32, np.float64
U24, U8 = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ar():
    import post_weight_quantization_autoround_amd as mod
    assert torch.cuda.is_available()
    return mod


def _dev(a, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if bf16 else t


def _np(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


TABLE = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def _operand(rng, k, *lead):
    """Packed operand [*lead, k] on the GPU and its fp64 values there.  Values are multiples of 2^-2 of magnitude at most
    12: products of two such are multiples of 2^-4 of at most 144, and K < 2^24 / (16 * 144) = 7281 of them sum
    exactly in fp32 in any order, with 100 units to spare for K <= 7200: a bias and a residual of at most 512 each, in
    multiples of 2^-4, and their sum too where K <= 6000."""
    assert k <= 6000
    packed = rng.integers(0, 256, (*lead, k // 2), np.uint8)
    packed[packed % 16 == 8] &= 0xF0
    packed[packed // 16 == 8] &= 0x0F
    packed, scale = _dev(packed), _dev(rng.integers(126, 129, (*lead, k // 32)).astype(np.uint8))
    v = _dev(TABLE)[torch.stack((packed & 15, packed >> 4), -1).reshape(*lead, k).int()]
    return packed, scale, v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=-1)


def _exact(rng, *shape):
    """fp64 values that bf16 holds, multiples of 2^-4 of magnitude at most 8."""
    return _dev(rng.integers(-128, 129, shape) / 16.0)


# Every kernel and tile that the dense products choose from, as their own tests have it: few rows, 32 to 256 rows a tile, K
# that ends inside a stage and of several turns of the rings, on and off dword boundaries of the scale rows.
SHAPES = [(1, 1, 32), (1, 16, 64), (2, 33, 96), (15, 17, 128), (12, 900, 736), (13, 900, 736), (16, 256, 2048),
          (17, 129, 288), (17, 9000, 1504), (20, 1500, 2016), (20, 20000, 1056), (33, 3000, 4128), (40, 5000, 288),
          (65, 48, 1120), (130, 4200, 416), (130, 4200, 1024), (130, 9000, 288), (257, 511, 544), (300, 9000, 640),
          (300, 17000, 288), (520, 17000, 288), (520, 17000, 768), (600, 9000, 352), (1100, 8000, 1088),
          (2000, 8300, 160), (2000, 8300, 512)]
SHAPES += [(512, 11008, 512), (600, 9000, 640), (513, 8196, 256)]      # packed X in the tile kernel's 128x256


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_exact(ar, m, n, k):
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    x16 = X.bfloat16()
    P = X @ W.t()
    bias, res = _exact(rng, n), _exact(rng, m, n)
    for i, (b, r, out, act) in enumerate([("f32", "bf16", "f32", "none"), ("bf16", "f32", "bf16", "relu"),
                                          (None, "bf16", "bf16", "none"), ("bf16", None, "f32", "relu"),
                                          (None, None, "bf16", "none")]):
        want = P if b is None else P + bias
        want = want.clamp(min=0) if act == "relu" else want
        want = (want if r is None else want + res).float().to(DT[out])
        more = dict(bias=None if b is None else bias.to(DT[b]), residual=None if r is None else res.to(DT[r]), act=act,
                    out_dtype=DT[out])
        print(f"a16 {m}x{n}x{k} {i}", flush=True)
        assert torch.equal(ar.mxfp4_linear(x16, wp, ws, **more), want), i
        print(f"a4 {m}x{n}x{k} {i}", flush=True)
        assert torch.equal(ar.mxfp4_linear_a4(xp, xs, wp, ws, **more), want), i
    if m * n < 1 << 22:      # without an epilogue: the plain product, bit for bit
        assert torch.equal(ar.mxfp4_linear(x16, wp, ws), ar.mxfp4_gemm(x16, wp, ws))
        assert torch.equal(ar.mxfp4_linear_a4(xp, xs, wp, ws), ar.mxfp4_gemm_a4(xp, xs, wp, ws))


@pytest.mark.parametrize("m,n", [(1, 40), (3, 101), (16, 4097), (40, 5000), (300, 1003), (300, 9000), (520, 17000)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_strides_and_in_place(ar, m, n, out):
    k = 288
    rng = np.random.default_rng(m + n)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    bias, res = _exact(rng, n), _exact(rng, m, n)
    want = (X @ W.t() + bias + res).float().to(DT[out])
    calls = [lambda **kw: ar.mxfp4_linear(X.bfloat16(), wp, ws, bias=bias.bfloat16(), out_dtype=DT[out], **kw),
             lambda **kw: ar.mxfp4_linear_a4(xp, xs, wp, ws, bias=bias.float(), out_dtype=DT[out], **kw)]
    for call, (left, pad), rdt in itertools.product(calls, [(0, 0), (4, 4), (1, 2), (8, 3)], ["f32", "bf16"]):
        # rows of Y and of the residual inside wider buffers, which stay as they are around them
        rbuf = torch.full((m, left + n + pad), 3.0, dtype=DT[rdt], device="cuda")
        rbuf[:, left:left + n] = res.to(DT[rdt])
        buf = torch.full((m + 2, left + n + pad), 7.0, dtype=DT[out], device="cuda")
        print(f"{m}x{n} {out} {left} {pad} {rdt}", flush=True)
        call(residual=rbuf[:, left:left + n], out=buf[1:-1, left:left + n])
        assert torch.equal(buf[1:-1, left:left + n], want)
        buf[1:-1, left:left + n] = 7.0
        assert (buf == 7).all()
    for call, left in itertools.product(calls, [0, 1]):      # onto the residual itself
        buf = torch.full((m, left + n), 5.0, dtype=DT[out], device="cuda")
        view = buf[:, left:]
        view.copy_(res)
        assert call(residual=view, out=view) is view
        assert torch.equal(view, want) and (buf[:, :left] == 5).all()


# with the test above every kernel of both forms, the larger ones with columns in fours and not
STRIDED = [(20, 17001, 96), (130, 4201, 384), (300, 4203, 384), (600, 9000, 384), (600, 9001, 512), (520, 17000, 384),
           (520, 17001, 512), (2000, 8300, 160), (2000, 8301, 160)]


@pytest.mark.parametrize("m,n,k", STRIDED)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_strides_and_in_place_over_the_tiles(ar, m, n, k, out):
    rng = np.random.default_rng(m + n + k)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    bias, res = _exact(rng, n), _exact(rng, m, n)
    want = (X @ W.t() + bias + res).float().to(DT[out])
    calls = [lambda **kw: ar.mxfp4_linear(X.bfloat16(), wp, ws, bias=bias.bfloat16(), out_dtype=DT[out], **kw),
             lambda **kw: ar.mxfp4_linear_a4(xp, xs, wp, ws, bias=bias.float(), out_dtype=DT[out], **kw)]
    for call, (left, pad), rdt in itertools.product(calls, [(0, 0), (4, 4), (1, 2)], ["f32", "bf16"]):
        rbuf = torch.full((m, left + n + pad), 3.0, dtype=DT[rdt], device="cuda")
        rbuf[:, left:left + n] = res.to(DT[rdt])
        buf = torch.full((m + 2, left + n + pad), 7.0, dtype=DT[out], device="cuda")
        print(f"{m}x{n}x{k} {out} {left} {pad} {rdt}", flush=True)
        call(residual=rbuf[:, left:left + n], out=buf[1:-1, left:left + n])
        assert torch.equal(buf[1:-1, left:left + n], want)
        buf[1:-1, left:left + n] = 7.0
        assert (buf == 7).all()
    for call, left in itertools.product(calls, [0, 1]):      # onto the residual itself
        buf = torch.full((m + 2, left + n), 5.0, dtype=DT[out], device="cuda")
        view = buf[1:-1, left:]
        view.copy_(res)
        assert call(residual=view, out=view) is view
        assert torch.equal(view, want)
        view[:] = 5
        assert (buf == 5).all()


ACTS = ["relu", "silu", "gelu", "gelu_tanh"]


def _act_bound(v, act, out):
    """Half steps that act(v) may be off by, relative to it, v carrying one rounding of its own (2^-24 |v|).

    silu, gelu_tanh: v s1 s2 with s = h, h = exp(-|u| / 2) from an argument with a relative error of c 2^-24 (c = 3 for
    silu: v's, the product's and expf's own 2 half steps stand apart; 12 for gelu_tanh's u, a product of v, its square, two
    constants and a sum that do not cancel), which moves h by |u| / 2 of it, twice: |u| c, plus 2 for v itself, 2 * 4 for
    the two expf's, 8 for the sum, quotient and products.  relu: v's own.
    gelu: v / 2 erfc(z), z = -v / sqrt 2 carrying 4 half steps, which erfc multiplies by at most 2 z^2 + 2 = v^2 + 2 (its
    logarithmic derivative for z > 0): 4 (v^2 + 2), plus 2 for v and 2 * 16 for erfcf and the products.
    For bf16 the hardware's exponential: its argument's error counts the same, 2^-16 is added in all."""
    a = np.abs(v)
    if act == "relu":
        steps = 2.0 + 0 * a
    elif act == "gelu":
        steps = 34 + 4 * (a * a + 2)
    else:
        u = a if act == "silu" else 1.5957691216 * a * (1 + 0.044715 * a * a)
        steps = 18 + (3 if act == "silu" else 12) * np.minimum(u, 210)
    return steps * U24 + (2.0 ** -16 + U8 if out == "bf16" else 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 2048, 32), (40, 2048, 64), (300, 9000, 160), (520, 17000, 256)])
def test_activations(ar, act, m, n, k):
    rng = np.random.default_rng(m)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    xs[:], X = xs - 2, X / 4
    some = np.unique(np.concatenate([np.arange(4), rng.integers(0, m, 4)]) % m)     # rows that are compared
    bias = np.concatenate([np.linspace(-30, 8, n - 40), np.linspace(-110, 110, 20), 10.0 ** np.arange(-38, 2, 2)]).astype(F32)
    if m == 1:
        X[:], xs[:] = 0, 0
        xp[:] = 0                                # act(bias) itself
        bias = np.concatenate([bias[:1024], -np.geomspace(1e-30, 105, 1024).astype(F32)])
    P = (X[some] @ W.t()).cpu().numpy()
    v = (P.astype(F32) + bias).astype(F64)       # the fp32 sum, rounded as the kernel rounds it
    want = moe.activate(v, act)
    for out in ("f32", "bf16"):
        tol = np.abs(want) * _act_bound(v, act, out) + (2.0 ** -133 if out == "bf16" else 2.0 ** -148)   # subnormal steps
        for a4 in (False, True):
            print(f"{act} {m}x{n}x{k} {out} a4 {a4}", flush=True)
            more = dict(bias=_dev(bias), act=act, out_dtype=DT[out])
            Y = ar.mxfp4_linear_a4(xp, xs, wp, ws, **more) if a4 else ar.mxfp4_linear(X.bfloat16(), wp, ws, **more)
            err = np.abs(_np(Y[some]).astype(F64) - want)
            assert (err <= tol).all(), (err / tol).max()


def _act_bias(n):
    return np.concatenate([np.linspace(-30, 8, n - 40), np.linspace(-110, 110, 20), 10.0 ** np.arange(-38, 2, 2)]).astype(F32)


def _check_act(got, v, act, out):
    """act(v) within what test_activations allows; v as the kernel rounds it."""
    want = moe.activate(v, act)
    tol = np.abs(want) * _act_bound(v, act, out) + (2.0 ** -133 if out == "bf16" else 2.0 ** -148)
    err = np.abs(_np(got).astype(F64) - want)
    assert (err <= tol).all(), (err / tol).max()


ACT_SHAPES = [(16, 9000, 160), (20, 17000, 96), (130, 4200, 160), (300, 4200, 160), (600, 9000, 384), (2000, 8300, 160)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", ACT_SHAPES)      # with the test above every kernel of both forms
def test_activations_over_the_tiles(ar, act, m, n, k):
    rng = np.random.default_rng(m)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    xs[:], X = xs - 2, X / 4
    some = np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, 4)]))
    bias = _act_bias(n)
    v = ((X[some] @ W.t()).cpu().numpy().astype(F32) + bias).astype(F64)
    for out, a4 in itertools.product(("f32", "bf16"), (False, True)):
        print(f"{act} {m}x{n}x{k} {out} a4 {a4}", flush=True)
        more = dict(bias=_dev(bias), act=act, out_dtype=DT[out])
        Y = ar.mxfp4_linear_a4(xp, xs, wp, ws, **more) if a4 else ar.mxfp4_linear(X.bfloat16(), wp, ws, **more)
        _check_act(Y[some], v, act, out)


@pytest.mark.parametrize("act", ["none"] + ACTS)
@pytest.mark.parametrize("m", [1, 40, 300])
def test_activations_of_nonfinite_values(ar, act, m):
    n, k = 96, 64
    rng = np.random.default_rng(0)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, m)
    bias = np.zeros(n, F32)
    bias[:6] = [np.inf, -np.inf, np.nan, 3e38, -3e38, -0.0]
    v = (X @ W.t()).cpu().numpy() + bias
    res = np.zeros((m, n), F32)
    res[:, 7], res[:, 8] = np.nan, -np.inf
    want = (moe.activate(v, act) + res).astype(F32)
    for Y in (ar.mxfp4_linear(X.bfloat16(), wp, ws, bias=_dev(bias), act=act, residual=_dev(res)),
              ar.mxfp4_linear_a4(xp, xs, wp, ws, bias=_dev(bias), act=act, residual=_dev(res))):
        got = _np(Y)
        cols = [0, 1, 2, 3, 4, 7, 8]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(got[:, cols][~np.isnan(want[:, cols])], want[:, cols][~np.isnan(want[:, cols])])


def test_linear_past_32_bit_offsets(ar):
    # Y and the residual of 4.5 G elements (9 GB of bf16): rows past element 2^32 against the first ones
    m, n, k = 140_000, 32_000, 32
    rng = np.random.default_rng(9)
    wp, ws, W = _operand(rng, k, n)
    xp, xs, X = _operand(rng, k, 1000)
    res = _exact(rng, 1000, n)
    want = ((X @ W.t()).clamp(min=0) + res).float().bfloat16()
    xpd, xsd = xp.repeat(m // 1000, 1), xs.repeat(m // 1000, 1)
    Y = res.bfloat16().repeat(m // 1000, 1)
    ar.mxfp4_linear_a4(xpd, xsd, wp, ws, act="relu", residual=Y, out_dtype=torch.bfloat16, out=Y)
    for first in (0, 67_000, 134_000, m - 1000):
        assert torch.equal(Y[first:first + 1000], want), first
    Y = res.bfloat16().repeat(m // 1000, 1)
    ar.mxfp4_linear(X.bfloat16().repeat(m // 1000, 1), wp, ws, act="relu", residual=Y, out_dtype=torch.bfloat16, out=Y)
    for first in (0, 67_000, 134_000, m - 1000):
        assert torch.equal(Y[first:first + 1000], want), first


# ----------------------------------------------------------------- grouped
def _grouped_want(X, W, offsets, rows, bias, act, m):
    """fp64 on the GPU; NaN where nothing is written."""
    y = torch.full((m, W.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    zero = torch.cat((X, torch.zeros_like(X[:1])))
    for e in range(W.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            r = torch.arange(lo, hi) if rows is None else torch.from_numpy(rows[lo:hi].astype(np.int64))
            r[(r < 0) | (r >= X.shape[0])] = X.shape[0]
            y[lo:hi] = zero[r.cuda()] @ W[e].t() + (0 if bias is None else bias[e])
    return y.clamp(min=0) if act == "relu" else y


# sizes of the groups: empty ones (the first, the last, several in a row), single rows, one with everything, sizes on and
# off the tiles' rows; (leading rows of no expert, trailing ones)
GROUPS = [([1], 0, 0), ([0, 1, 0], 0, 0), ([3, 0, 0, 5, 1, 0], 0, 2), ([0, 0, 33, 64, 1, 31, 32, 0], 2, 3),
          ([130, 0, 7, 257], 0, 1), ([0, 300, 0], 1, 0), ([1] * 70, 0, 0), ([0, 2] * 100 + [90], 3, 1),
          ([0] * 999 + [4] + [0] * 24, 0, 0), ([600, 20, 512, 513], 0, 0)]


@pytest.mark.parametrize("sizes,lead,trail", GROUPS)
@pytest.mark.parametrize("n,k", [(33, 96), (300, 288), (1030, 1184)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_exact(ar, sizes, lead, trail, n, k, gather):
    rng = np.random.default_rng(len(sizes) + sum(sizes) + n + k)
    E = len(sizes)
    if E * n * k > 3e8:
        n = 130
    offsets = (lead + np.concatenate([[0], np.cumsum(sizes)])).astype(np.int32)
    m = int(offsets[-1]) + trail
    R = max(1, m // 3) if gather else m
    rows = rng.integers(0, R, m).astype(np.int32) if gather else None
    if gather and m > 4:
        rows[::5] = rng.choice([-1, R, -2 ** 31, 2 ** 31 - 1], len(rows[::5]))     # rows of zeros
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, R)
    bias = _exact(rng, E, n)
    o, r = _dev(offsets), None if rows is None else _dev(rows)
    for b, act, out in [(None, "none", "f32"), ("f32", "relu", "bf16"), ("bf16", "none", "f32")]:
        want = _grouped_want(X, W, offsets, rows, None if b is None else bias, act, m).float().to(DT[out])
        more = dict(rows=r, bias=None if b is None else bias.to(DT[b]), act=act, out_dtype=DT[out])
        for a4 in (False, True):
            print(f"{E} experts {m}x{n}x{k} gather {gather} {b} {act} {out} a4 {a4}", flush=True)
            buf = torch.full((m + 2, n), 7.0, dtype=DT[out], device="cuda")
            Y = buf[1:-1]
            if a4:
                ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, o, out=Y, **more)
            else:
                ar.mxfp4_grouped_gemm(X.bfloat16(), wp, ws, o, out=Y, **more)
            assert torch.equal(torch.where(want.isnan(), torch.full_like(want, 7.0), want), Y)
            assert (buf[0] == 7).all() and (buf[-1] == 7).all()


# mean rows an expert and widths that lead to each of the tiles, with skewed groups
TILED = [(5, 8, 4100, 512), (40, 8, 9000, 288), (70, 16, 4200, 1504), (130, 8, 9000, 288), (300, 8, 4200, 2016),
         (300, 6, 9000, 416), (600, 5, 4200, 1184), (1100, 4, 4200, 2304), (1100, 4, 9000, 288), (200, 64, 520, 640),
         (24, 128, 520, 2400), (2, 200, 520, 1888), (700, 8, 2100, 384), (260, 16, 2048, 128), (200, 64, 4200, 288),
         (200, 64, 4200, 384), (300, 40, 8300, 1184), (70, 64, 4200, 1184), (100, 40, 9000, 288), (70, 16, 4200, 1536),
         (33, 40, 1030, 256), (3, 300, 520, 416), (60, 700, 130, 160)]


@pytest.mark.parametrize("mean,E,n,k", TILED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_exact_over_the_tiles(ar, mean, E, n, k, gather):
    rng = np.random.default_rng(mean + E + n + k)
    sizes = rng.multinomial(mean * E, rng.dirichlet(np.full(E, 2.0)))
    sizes[E // 2] = 0
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    m = int(offsets[-1]) + 3
    R = max(1, m // 4) if gather else m
    rows = rng.integers(0, R, m).astype(np.int32) if gather else None
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, R)
    bias = _exact(rng, E, n)
    o, r = _dev(offsets), None if rows is None else _dev(rows)
    real = _grouped_want(X, W, offsets, rows, bias, "none", m)[:-3]
    for out in ("f32", "bf16"):
        want = real.float().to(DT[out])
        more = dict(rows=r, bias=bias.float(), out_dtype=DT[out])
        print(f"a16 {mean} rows x {E} x {n} x {k} gather {gather} {out}", flush=True)
        assert torch.equal(ar.mxfp4_grouped_gemm(X.bfloat16(), wp, ws, o, **more)[:-3], want)
        print(f"a4 {mean} rows x {E} x {n} x {k} gather {gather} {out}", flush=True)
        assert torch.equal(ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, o, **more)[:-3], want)


# packed X in the tile kernels (K a multiple of 128) of 64, 128 and 256 rows, and both forms in the ring's gathered loads
@pytest.mark.parametrize("mean,E,n,k", [(8, 200, 520, 512), (100, 40, 4100, 640), (300, 16, 4200, 1024), (70, 64, 2048, 416)])
@pytest.mark.parametrize("real_rows", [0, 1, 100])
def test_grouped_rows_that_do_not_exist(ar, mean, E, n, k, real_rows):
    rng = np.random.default_rng(mean + E + n + k + real_rows)
    m = mean * E
    offsets = np.concatenate([[0], np.cumsum(rng.multinomial(m, rng.dirichlet(np.full(E, 2.0))))]).astype(np.int32)
    rows = rng.integers(-2, real_rows + 2, m).astype(np.int32)
    rows[::7] = rng.choice([-1, real_rows, -2 ** 31, 2 ** 31 - 1], len(rows[::7]))
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, 100)
    xp, xs, X = xp[:real_rows], xs[:real_rows], X[:real_rows]
    bias = _exact(rng, E, n)
    zero = torch.cat((X, torch.zeros((1, k), dtype=X.dtype, device="cuda")))
    r = torch.from_numpy(rows.astype(np.int64))
    r[(r < 0) | (r >= real_rows)] = real_rows
    want = torch.empty((m, n), dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[lo:hi] = zero[r[lo:hi].cuda()] @ W[e].t() + bias[e]
    more = dict(rows=_dev(rows), bias=bias.float())
    for a4 in (True, False):
        print(f"{mean} rows x {E} x {n} x {k} of {real_rows} rows a4 {a4}", flush=True)
        Y = ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, _dev(offsets), **more) if a4 else \
            ar.mxfp4_grouped_gemm(X.bfloat16(), wp, ws, _dev(offsets), **more)
        assert torch.equal(Y, want.float())



# every kernel of both forms
ACT_TILED = [(16, 8, 520, 288), (70, 16, 4200, 160), (300, 6, 9000, 416), (1100, 4, 9000, 288), (2, 200, 520, 160),
             (200, 64, 520, 256), (24, 128, 520, 256), (260, 16, 2048, 256), (200, 64, 4200, 288), (70, 64, 4200, 160),
             (100, 40, 520, 256), (40, 64, 1030, 160)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("mean,E,n,k", ACT_TILED)
def test_grouped_activations_over_the_tiles(ar, act, mean, E, n, k):
    rng = np.random.default_rng(mean + E)
    sizes = rng.multinomial(mean * E, rng.dirichlet(np.full(E, 2.0)))
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    m, R = mean * E, max(1, mean * E // 4)
    rows = rng.integers(0, R, m).astype(np.int32)
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, R)
    xs[:], X = xs - 2, X / 4
    bias = np.stack([np.roll(_act_bias(n), 7 * e) for e in range(E)])
    some = np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, 4)]))
    expert = np.searchsorted(offsets, some, side="right") - 1
    P = np.stack([(W[e] @ X[rows[p]]).cpu().numpy() for p, e in zip(some, expert)])
    v = (P.astype(F32) + bias[expert]).astype(F64)
    for out, a4 in itertools.product(("f32", "bf16"), (False, True)):
        print(f"{act} {mean} rows x {E} x {n} x {k} {out} a4 {a4}", flush=True)
        more = dict(rows=_dev(rows), bias=_dev(bias), act=act, out_dtype=DT[out])
        Y = ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, _dev(offsets), **more) if a4 else \
            ar.mxfp4_grouped_gemm(X.bfloat16(), wp, ws, _dev(offsets), **more)
        _check_act(Y[some], v, act, out)


@pytest.mark.parametrize("mean,E,n,k", [(3, 6, 140, 96), (70, 4, 300, 416), (300, 4, 520, 288), (600, 4, 1030, 512)])
def test_grouped_keeps_experts_apart(ar, mean, E, n, k):
    # every second expert's weight and every second token are NaN throughout; the others are untouched by them
    rng = np.random.default_rng(mean)
    sizes = rng.multinomial(mean * E, np.full(E, 1 / E))
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    m = int(offsets[-1])
    rows = rng.integers(0, m, m).astype(np.int32)
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, m)
    for r in (rows, None):
        want = _grouped_want(X, W, offsets, r, None, "none", m).float()
        clean = np.repeat(np.arange(E) % 2 == 0, sizes) & ((np.arange(m) if r is None else r) % 2 == 0)
        ws2, xs2, x2 = ws.clone(), xs.clone(), X.bfloat16()
        ws2[1::2] = 255
        xs2[1::2] = 255
        x2[1::2] = float("nan")
        rr = None if r is None else _dev(r)
        for Y in (ar.mxfp4_grouped_gemm(x2, wp, ws2, _dev(offsets), rows=rr),
                  ar.mxfp4_grouped_gemm_a4(xp, xs2, wp, ws2, _dev(offsets), rows=rr)):
            assert torch.equal(Y[_dev(clean)], want[_dev(clean)])
            assert Y[_dev(~clean)].isnan().all()


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_scales_at_any_address(ar, off, gather):
    rng = np.random.default_rng(off)
    for mean, E, n, k in [(3, 5, 77, 96), (150, 4, 520, 352), (400, 4, 520, 512)]:
        sizes = rng.multinomial(mean * E, np.full(E, 1 / E))
        o = _dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))
        m = int(o[-1])
        wp, ws, W = _operand(rng, k, E, n)
        xp, xs, X = _operand(rng, k, m)
        rows = _dev(rng.integers(0, m, m).astype(np.int32)) if gather else None

        def moved(a):
            buf = torch.full((a.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
            out = buf[off:off + a.numel()].view(a.shape)
            out.copy_(a)
            assert out.data_ptr() % 4 == off
            return out

        want = ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, o, rows=rows)
        assert torch.equal(ar.mxfp4_grouped_gemm_a4(xp, moved(xs), wp, moved(ws), o, rows=rows), want)
        assert torch.equal(ar.mxfp4_grouped_gemm(X.bfloat16(), wp, moved(ws), o, rows=rows), want)


@pytest.mark.parametrize("borders", [[-5, 3, 2, 50, 7], [9, 9, 0, 0, 4], [2 ** 31 - 1, -2 ** 31, 5, 5, 2 ** 31 - 1],
                                     [0, 1000, 0, 1000, 0], [40, 30, 20, 10, 0]])
@pytest.mark.parametrize("m,n,k", [(10, 40, 96), (700, 1030, 288), (700, 1030, 256)])
def test_grouped_cuts_borders_that_do_not_ascend(ar, borders, m, n, k):
    # rows of experts whose borders are in order come out, whatever the others' are; nothing around Y is written
    rng = np.random.default_rng(m)
    wp, ws, W = _operand(rng, k, 4, n)
    xp, xs, X = _operand(rng, k, m)
    o = _dev(np.array(borders, np.int64).astype(np.int32))
    cut = np.clip(np.array(borders, np.int64), 0, m)
    spans = [(max(lo, 0), max(lo, hi)) for lo, hi in zip(cut[:-1], cut[1:])]
    owners = np.zeros(m, int)
    for lo, hi in spans:
        owners[lo:hi] += 1
    for a4 in (False, True):
        buf = torch.full((m + 2, n), 7.0, device="cuda")
        print(f"{borders} {m}x{n}x{k} a4 {a4}", flush=True)
        if a4:
            ar.mxfp4_grouped_gemm_a4(xp, xs, wp, ws, o, out=buf[1:-1])
        else:
            ar.mxfp4_grouped_gemm(X.bfloat16(), wp, ws, o, out=buf[1:-1])
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        assert (buf[1:-1][_dev(owners == 0)] == 7).all()
        if sum(hi - lo for lo, hi in spans) <= m:      # no more tiles than borders in order can need
            for e, (lo, hi) in enumerate(spans):
                alone = _dev((owners == 1) & (np.arange(m) >= lo) & (np.arange(m) < hi))
                assert torch.equal(buf[1:-1][alone], (X[alone] @ W[e].t()).float())


def test_grouped_past_32_bit_offsets(ar):
    # Y of 4.6 G elements, X and the weights of more than 2^32 bytes: the last expert's last rows among others
    E, n, k, per = 5, 4096, 2048, 225_000
    rng = np.random.default_rng(10)
    wp, ws, W = _operand(rng, k, E, n)
    xp, xs, X = _operand(rng, k, 1000)
    o = _dev((np.arange(E + 1) * per).astype(np.int32))
    x16 = X.bfloat16().repeat(E * per // 1000, 1)
    Y = ar.mxfp4_grouped_gemm(x16, wp, ws, o, out_dtype=torch.bfloat16)
    for e in (0, 2, E - 1):
        want = (X @ W[e].t()).float().bfloat16()
        for first in (e * per, (e + 1) * per - 1000):
            assert torch.equal(Y[first:first + 1000], want), (e, first)
    del Y, x16
    Y = ar.mxfp4_grouped_gemm_a4(xp.repeat(E * per // 1000, 1), xs.repeat(E * per // 1000, 1), wp, ws, o,
                                 out_dtype=torch.bfloat16)
    for e in (0, 2, E - 1):
        want = (X @ W[e].t()).float().bfloat16()
        for first in (e * per, (e + 1) * per - 1000):
            assert torch.equal(Y[first:first + 1000], want), (e, first)
    del Y
    # weights of 2^32 packed bytes and more
    E, n, k = 300, 16384, 2048
    packed = wp[0].repeat(E, 4, 1)
    scale = ws[0].repeat(E, 4, 1)
    last = rng.integers(0, 256, (n, k // 2), np.uint8) & 0x77
    packed[-1] = _dev(last)
    W = _dev(TABLE)[torch.stack((packed[-1] & 15, packed[-1] >> 4), -1).reshape(n, k).int()]
    W = W * torch.exp2(scale[-1].double() - 127).repeat_interleave(32, dim=1)
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[-1] = 50
    want = (X[:50] @ W.t()).float()
    assert torch.equal(ar.mxfp4_grouped_gemm(X[:50].bfloat16(), packed, scale, o), want)
    assert torch.equal(ar.mxfp4_grouped_gemm_a4(xp[:50], xs[:50], packed, scale, o), want)


# ------------------------------------------------------------------- route
def _check_route(ar, x, k, dtype="f32", bias=None, **kw):
    t = _dev(x.astype(F32), dtype == "bf16")
    want = moe.route(_np(t), k, bias=None if bias is None else bias.astype(F32), **kw)
    got = ar.moe_route(t, k, bias=None if bias is None else _dev(bias.astype(F32)), **kw)
    for name, g in zip(("expert", "weight", "offsets", "token", "pos"), got):
        if name == "weight":      # 64 bits (with a margin of 2^-40 for the exponentials), rounded once
            w = want["weight"]
            np.testing.assert_array_equal(np.isnan(_np(g)), np.isnan(w))
            ok = ~np.isnan(w)
            assert (np.abs(_np(g).astype(F64) - w)[ok] <= (U24 + 2.0 ** -40) * np.abs(w[ok]) + 2.0 ** -149).all()
        else:
            np.testing.assert_array_equal(_np(g), want[name], err_msg=name)


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 6), (2, 3, 3), (5, 8, 2), (7, 65, 8), (16, 128, 8), (33, 200, 64),
                                   (64, 256, 8), (100, 300, 4), (300, 60, 4), (17, 512, 1), (40, 513, 10), (9, 1024, 64),
                                   (1030, 16, 2), (4200, 32, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(ar, t, e, k, score):
    rng = np.random.default_rng(t + e + k)
    x = 1.5 * rng.standard_normal((t, e))
    for dtype, normalize, bias in [("f32", True, None), ("bf16", False, None), ("f32", False, 0.1 * rng.standard_normal(e)),
                                   ("bf16", True, 0.1 * rng.standard_normal(e))]:     # bf16 logits tie often
        _check_route(ar, x, k, dtype, bias, score=score, normalize=normalize, weight_scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_ties_and_nonfinite(ar, score, normalize, biased):
    rng = np.random.default_rng(3)
    t, e, k = 60, 70, 5
    low, inf = np.finfo(F32).min, np.inf
    x = rng.standard_normal((t, e))
    x[0] = 0.25                                            # all tied
    x[1] = -inf                                            # nothing left
    x[2], x[2, 69] = -inf, 1.0                             # one left
    x[3], x[3, [3, 68]] = -inf, [-2.0, -2.0]               # two, tied
    x[4] = low                                             # a mask of the type's lowest value leaves nothing
    x[5], x[5, 9:12] = low, [1.0, 2.0, 1.0]
    x[6, 40] = np.nan
    x[7, [5, 60]] = np.nan
    x[8, 33] = inf
    x[9, [33, 34]] = inf
    x[10], x[10, 1] = -inf, np.nan
    x[11], x[11, 7] = -inf, inf
    x[12, ::2] = -0.0
    x[12, 1::2] = 0.0
    x[13] = 1000.0 * x[13]
    x[14] = -800.0 - np.abs(x[14])                         # sigmoids that 64 bits hold as 0 or barely
    x[20:30, ::3] = -inf
    x[30:40] = np.round(2 * x[30:40]) / 2                  # many ties
    x[40:, 20:] = -inf                                     # experts without rows
    bias = None
    if biased:
        bias = np.round(8 * rng.standard_normal(e)) / 8
        bias[[2, 50]] = -inf
        bias[4] = inf
    _check_route(ar, x, k, "f32", bias, score=score, normalize=normalize)
    _check_route(ar, x[:12, :6], 6, "f32", None if bias is None else bias[:6], score=score, normalize=normalize)
    x[:, :] = -inf                                         # no token goes anywhere
    _check_route(ar, x, k, "bf16", bias, score=score, normalize=normalize)


def test_route_of_no_tokens_and_of_many(ar):
    expert, weight, offsets, token, pos = ar.moe_route(torch.empty(0, 40, device="cuda"), 4)
    assert expert.shape == weight.shape == pos.shape == (0, 4) and token.shape == (0,)
    assert offsets.shape == (41,) and int(offsets.abs().sum()) == 0
    # 2^20 tokens: the order against a stable sort
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1 << 20, 37, generator=gen, device="cuda")
    x[::7] = -float("inf")
    expert, weight, offsets, token, pos = ar.moe_route(x, 3)
    assert torch.equal(expert[1::7], torch.sort(x[1::7], dim=-1, descending=True, stable=True)[1][:, :3].int())
    assert (expert[::7] == -1).all() and (weight[::7] == 0).all() and (pos[::7] == -1).all()
    flat = torch.where(expert < 0, 37, expert).reshape(-1)
    group, slot = torch.sort(flat, stable=True)
    real = int((group < 37).sum())
    assert torch.equal(offsets, torch.searchsorted(group, torch.arange(38, device="cuda")).int())
    assert torch.equal(token[:real], (slot[:real] // 3).int()) and (token[real:] == -1).all()
    assert torch.equal(pos.reshape(-1)[slot[:real]], torch.arange(real, device="cuda", dtype=torch.int32))


# more than 2^14 slots: the experts in 1 to 16 wavefronts, 1 to 16 segments of which share the chunks, evenly and not; chunks
# of 1024 slots and of 2048
@pytest.mark.parametrize("t,e,k", [(5501, 40, 3), (2801, 65, 6), (4200, 100, 5), (6203, 128, 3), (2600, 200, 7), (5001, 256, 8),
                                   (10007, 256, 8), (2301, 300, 8), (3001, 512, 7), (20003, 512, 4), (2200, 513, 8),
                                   (1400, 1024, 13), (140_007, 256, 4)])
def test_route_order_of_many_slots(ar, t, e, k):
    gen = torch.Generator(device="cuda").manual_seed(t + e)
    x = torch.randn(t, e, generator=gen, device="cuda") + 1.5 * torch.randn(e, generator=gen, device="cuda")
    x[3::11] = -float("inf")                               # tokens of no expert, and some of fewer than k
    x[5::17, 2:] = -float("inf")
    x[:, e // 2] = -float("inf")                           # an expert without rows
    expert, weight, offsets, token, pos = ar.moe_route(x, k)
    key, index = torch.sort(x, dim=-1, descending=True, stable=True)
    want = torch.where(key[:, :k] > -float("inf"), index[:, :k], -1).int()
    assert torch.equal(expert, want) and (weight[want < 0] == 0).all()
    flat = torch.where(want < 0, e, want).reshape(-1)
    group, slot = torch.sort(flat, stable=True)
    real = int((group < e).sum())
    assert real < t * k and torch.equal(offsets, torch.searchsorted(group, torch.arange(e + 1, device="cuda").int()).int())
    assert torch.equal(token[:real], (slot[:real] // k).int()) and (token[real:] == -1).all()
    assert torch.equal(pos.reshape(-1)[slot[:real]], torch.arange(real, device="cuda", dtype=torch.int32))
    assert (pos[want < 0] == -1).all()


@pytest.mark.parametrize("t,e,k", [(2801, 65, 6), (2100, 200, 8), (2301, 256, 8), (2801, 400, 6)])
def test_route_of_many_slots_by_biased_scores(ar, t, e, k):
    rng = np.random.default_rng(t + e)
    x = 1.5 * rng.standard_normal((t, e))
    x[2::9] = -np.inf
    _check_route(ar, x, k, "f32", 0.1 * rng.standard_normal(e), score="sigmoid", weight_scale=2.5)


def test_route_at_its_limits(ar):
    t, e, k = 1 << 18, 1024, 64                          # 2^24 slots, the most experts and choices
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, e, generator=gen, device="cuda").bfloat16()      # (ties in every token)
    expert, weight, offsets, token, pos = ar.moe_route(x, k, score="sigmoid", normalize=False)
    first = 0
    for part in x.split(1 << 16):
        want = torch.sort(part, dim=-1, descending=True, stable=True)
        n = part.shape[0]
        assert torch.equal(expert[first:first + n], want[1][:, :k].int())
        # rounded once from 64 bits, where the exponential may be off by an ulp: half a step of the 24 bits
        s = torch.sigmoid(want[0][:, :k].double())
        assert ((weight[first:first + n].double() - s).abs() <= s * (2.0 ** -24 + 2.0 ** -50)).all()
        first += n
    group, slot = torch.sort(expert.reshape(-1), stable=True)
    assert torch.equal(offsets, torch.searchsorted(group, torch.arange(e + 1, dtype=torch.int32, device="cuda")).int())
    assert torch.equal(token, (slot // k).int())
    assert torch.equal(pos.reshape(-1)[slot], torch.arange(t * k, device="cuda", dtype=torch.int32))


# ----------------------------------------------------------------- combine
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 8, 4096), (3, 2, 33), (16, 6, 2052), (5, 64, 130), (7, 9, 4100),
                                   (300, 8, 520), (2000, 3, 1024)])
@pytest.mark.parametrize("z", ["f32", "bf16"])
def test_combine(ar, t, k, n, z):
    rng = np.random.default_rng(t + k + n)
    p = t * k + 3
    Z = to_bf16_values(rng.standard_normal((p, n)).astype(F32))
    pos = rng.integers(0, p, (t, k)).astype(np.int32)         # some rows twice, some not at all
    w = rng.standard_normal((t, k)).astype(F32)
    pos[rng.random((t, k)) < 0.2] = -1
    if t > 2:
        pos[1] = -1
        pos[2, 0], pos[0, k - 1] = p, 2 ** 31 - 1             # behind the last row: nothing
    w[pos < 0] = np.nan                                       # not read into the sum
    res = to_bf16_values(rng.standard_normal((t, n)).astype(F32))
    for r, out in [(None, "f32"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), (None, "bf16")]:
        ref, mag = moe.combine(Z, pos, w, None if r is None else res)
        # k products and k sums (the first onto 0) and the residual's, each a half step of at most the sum of magnitudes
        tol = (2 * k + 1) * U24 * mag
        more = dict(out_dtype=DT[out])
        got = ar.moe_combine(_dev(Z, z == "bf16"), _dev(pos), _dev(w), None if r is None else _dev(res, r == "bf16"), **more)
        err = np.abs(_np(got).astype(F64) - ref)
        assert (err <= tol + (U8 * (np.abs(ref) + tol) if out == "bf16" else 0)).all()
        if r == out:      # onto the residual itself, at an odd address of a wider buffer too
            for lead in (0, 1):
                buf = torch.full((lead + t * n + 1,), 9.0, dtype=DT[out], device="cuda")
                y = buf[lead:lead + t * n].view(t, n)
                y.copy_(_dev(res))
                assert ar.moe_combine(_dev(Z, z == "bf16"), _dev(pos), _dev(w), residual=y, out=y, **more) is y
                assert torch.equal(y, got) and buf[-1] == 9 and (buf[:lead] == 9).all()


def test_combine_carries_nan_and_infinity(ar):
    Z = torch.ones(4, 8, device="cuda")
    Z[1, 2], Z[2, 3] = float("nan"), float("inf")
    pos = torch.tensor([[0, 1], [0, 2], [0, -1], [3, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 0.0], [1.0, -1.0], [1.0, 1.0], [float("nan"), 1.0]], device="cuda")
    y = ar.moe_combine(Z, pos, w)
    assert y[0, 2].isnan() and y[0].isnan().sum() == 1          # 0 * NaN
    assert y[1, 3] == -float("inf") and (y[2] == 1).all() and y[3].isnan().all()
    assert (ar.moe_combine(Z[:0], pos, w) == 0).all()


@pytest.mark.parametrize("n", [32_000, 32_001])           # in pieces of four columns and of one
def test_combine_past_32_bit_offsets(ar, n):
    t, k = 140_000, 2
    Z = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    rows = [0, 67_108, 134_218, t - 1]
    part = _exact(np.random.default_rng(4), len(rows), n)
    Z[rows] = part.bfloat16()
    pos = torch.stack((torch.arange(t - 1, -1, -1), torch.full((t,), -1)), 1).int().cuda()
    w = torch.full((t, k), 2.0, device="cuda")
    y = ar.moe_combine(Z, pos, w, out_dtype=torch.bfloat16)
    for i, r in enumerate(rows):
        assert torch.equal(y[t - 1 - r], (2 * part[i]).bfloat16())
    assert int(y.count_nonzero()) == 0 + sum(int(part[i].count_nonzero()) for i in range(len(rows)))


# ------------------------------------------------- together, as they are used
def _layer(rng, E, H, F):
    gu, down = (0.05 * rng.standard_normal((E, 2 * F, H)), 0.05 * rng.standard_normal((E, H, F)))
    import post_weight_quantization_autoround_amd as ar

    def packed(w):
        p, s = ar.pack_mxfp4(_dev(w.astype(F32).reshape(-1, w.shape[-1])))
        return p.view(E, w.shape[1], -1), s.view(E, w.shape[1], -1)

    router = ar.pack_mxfp4(_dev((0.1 * rng.standard_normal((E, H))).astype(F32)))
    return dict(gate_up=packed(gu), down=packed(down), router=router, bias=_dev(0.1 * rng.standard_normal((E, H)).astype(F32)))


def _moe(ar, s, x, delta, k, mask):
    """A mixture-of-experts MLP on packed weights: norm with residual, router, gate and up of each token's experts, SwiGLU,
    down, weighted sum onto the residual stream."""
    hp, hs, r = ar.rmsnorm_mxfp4(x, delta=delta)
    logits = ar.mxfp4_linear_a4(hp, hs, *s["router"])
    logits = torch.where(mask[:, None], logits, -float("inf"))           # padding goes to no expert
    expert, weight, offsets, token, pos = ar.moe_route(logits, k)
    gu = x.new_zeros((token.shape[0], s["gate_up"][0].shape[1]))         # (rows behind the last are not written)
    ar.mxfp4_grouped_gemm_a4(hp, hs, *s["gate_up"], offsets, rows=token, out_dtype=torch.bfloat16, out=gu)
    f = gu.shape[1] // 2
    ap, as_ = ar.swiglu_mxfp4(gu[:, :f], gu[:, f:])
    z = ar.mxfp4_grouped_gemm_a4(ap, as_, *s["down"], offsets, bias=s["bias"], out_dtype=torch.bfloat16)
    y = ar.moe_combine(z, pos, weight, residual=r, out_dtype=torch.bfloat16)
    return dict(hp=hp, hs=hs, r=r, logits=logits, expert=expert, weight=weight, offsets=offsets, token=token, pos=pos, gu=gu,
                ap=ap, as_=as_, z=z, y=y)


@pytest.mark.parametrize("t", [1, 16, 300])
def test_moe_of_packed_operators(ar, t):
    E, H, F, k = 12, 256, 352, 3
    rng = np.random.default_rng(t)
    s = _layer(rng, E, H, F)
    x = _dev(rng.standard_normal((t, H)).astype(F32), True)
    d = _dev(rng.standard_normal((t, H)).astype(F32))
    mask = torch.ones(t, dtype=torch.bool, device="cuda")
    mask[1::5] = False
    o = {n: (v if n in ("hp", "hs", "ap", "as_") else _np(v)) for n, v in _moe(ar, s, x, d, k, mask).items()}
    want = moe.route(o["logits"], k)
    for name in ("expert", "offsets", "token", "pos"):
        np.testing.assert_array_equal(o[name], want[name])
    assert (o["expert"][~mask.cpu().numpy()] == -1).all()
    # each stage from what the one before it gave; sums of H or F products within as many half steps
    vals = lambda p, sc: mx.values(p.reshape(-1, p.shape[-1]).cpu().numpy(), sc.reshape(-1, sc.shape[-1]).cpu().numpy())  # noqa: E731
    n = int(o["offsets"][-1])
    for X, (wp, ws), bias, got, K in [(vals(o["hp"], o["hs"]), s["gate_up"], None, o["gu"], H),
                                      (vals(o["ap"], o["as_"]), s["down"], _np(s["bias"]), o["z"], F)]:
        W = vals(wp, ws).reshape(E, wp.shape[1], K)
        rows = o["token"] if bias is None else None
        ref, written = moe.grouped(X, W, o["offsets"], rows, bias)
        mag, _ = moe.grouped(np.abs(X), np.abs(W), o["offsets"], rows, None if bias is None else np.abs(bias))
        assert written[:n].all() and not written[n:].any()
        ref, mag, got = ref[:n], mag[:n], got[:n]
        tol = (K + 1) * U24 * mag
        assert (np.abs(got - ref) <= tol + U8 * (np.abs(ref) + tol)).all()
    ref, mag = moe.combine(o["z"][:n], o["pos"], o["weight"], o["r"])
    tol = (2 * k + 1) * U24 * mag
    assert (np.abs(o["y"] - ref) <= tol + U8 * (np.abs(ref) + tol)).all()


@pytest.mark.parametrize("t", [1, 16, 200])
def test_captured_graph_and_other_streams(ar, t):
    # the layer captured once and replayed with new inputs in place, so that other experts are chosen (one replay has no
    # rows at all), eager work between the replays; then two streams at once
    E, H, F, k = 12, 256, 352, 3
    rng = np.random.default_rng(50 + t)
    s = _layer(rng, E, H, F)
    x = _dev(rng.standard_normal((t, H)).astype(F32), True)
    d = _dev(rng.standard_normal((t, H)).astype(F32))
    mask = torch.ones(t, dtype=torch.bool, device="cuda")

    def run():
        o = _moe(ar, s, x, d, k, mask)
        z = ar.mxfp4_grouped_gemm(o["r"], *s["gate_up"], o["offsets"], rows=o["token"], act="silu", out=gu32.zero_())
        lin = ar.mxfp4_linear(o["r"], s["down"][0][0][:, :H // 2].contiguous(), s["down"][1][0][:, :H // 32].contiguous(),
                              bias=s["bias"][0], act="gelu", residual=o["r"])
        return {n: v for n, v in o.items() if n != "z"} | dict(z16=z, lin=lin)

    gu32 = torch.empty(t * k, 2 * F, device="cuda")
    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    torch.cuda.synchronize()
    for rep in range(5):
        x.copy_(_dev(rng.standard_normal((t, H)).astype(F32), True))
        d.mul_(-0.7)
        mask.copy_(torch.from_numpy(rng.random(t) < (0.0 if rep == 2 else 0.8)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        first = {n: v.clone() for n, v in got.items()}
        want = run()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(first[n], want[n]), (rep, n)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(_moe(ar, s, x, d, k, mask))
    torch.cuda.synchronize()
    for o in outs:
        for n in o:
            if n != "z":      # rows of z behind the last are not written
                assert torch.equal(o[n], want[n]), n
    del graph


def test_captured_route_of_many_slots(ar):
    # the form that keeps its counts in pos meanwhile, captured; replays with other scores, each against an eager call
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, b = torch.empty(7000, 48, device="cuda"), torch.zeros(48, device="cuda")
    ar.moe_route(x.zero_(), 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ar.moe_route(x, 3, score="sigmoid", bias=b)
    for rep in range(4):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        b.copy_(0.2 * torch.randn(48, generator=gen, device="cuda"))
        if rep == 2:
            x[:6990] = -float("inf")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        first = [g.clone() for g in got]
        for g, w in zip(first, ar.moe_route(x, 3, score="sigmoid", bias=b)):
            assert torch.equal(g, w), rep
        assert int(first[2][-1]) == (30 if rep == 2 else 21000)
    del graph


def test_binding_refusals(ar):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    p, s = ar.pack_mxfp4(x)
    g, gs = p.expand(2, 4, 32).contiguous(), s.expand(2, 4, 2).contiguous()
    o = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    lg = torch.zeros(4, 8, device="cuda")
    i4 = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    f4 = torch.zeros((4, 2), device="cuda")
    for call, err in [
        (lambda: ar.mxfp4_linear(x, p, s, bias=torch.zeros(5, device="cuda")), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, bias=torch.zeros(4, device="cuda", dtype=torch.half)), TypeError),
        (lambda: ar.mxfp4_linear(x, p, s, act="tanh"), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, residual=torch.zeros(4, 5, device="cuda")), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, residual=torch.zeros(4, 4, device="cuda").t()), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, out=torch.zeros(4, 4, device="cuda").t()), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, out=torch.zeros(4, 4, device="cuda", dtype=torch.bfloat16)), TypeError),
        (lambda: ar.mxfp4_linear(x[:, :32].contiguous(), p, s), ValueError),
        (lambda: ar.mxfp4_linear(x, p, s, residual=torch.zeros(1, 4, device="cuda").expand(4, 4)), ar.ARError),
        (lambda: ar.mxfp4_linear_a4(p, s[:2], p, s), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, p, s, o), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs, o[:2].contiguous()), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs, o.long()), TypeError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs, o, rows=i4), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs, o, rows=i4[:, 0]), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs[:1], o), ValueError),
        (lambda: ar.mxfp4_grouped_gemm(x, g, gs, o, bias=torch.zeros(4, device="cuda")), ValueError),
        (lambda: ar.mxfp4_grouped_gemm_a4(p, s[:2], g, gs, o), ValueError),
        (lambda: ar.mxfp4_grouped_gemm_a4(p, s, g, gs, o, act=None), ValueError),
        (lambda: ar.moe_route(lg, 0), ar.ARError),
        (lambda: ar.moe_route(lg, -1), ar.ARError),
        (lambda: ar.moe_route(lg, 9), ar.ARError),
        (lambda: ar.moe_route(lg, 2 ** 32 + 2), ar.ARError),   # 2 in 32 bits
        (lambda: ar.moe_route(lg, 2 - 2 ** 32), ar.ARError),
        (lambda: ar.moe_route(lg, 2, score="max"), ValueError),
        (lambda: ar.moe_route(lg, 2, bias=torch.zeros(4, device="cuda")), ValueError),
        (lambda: ar.moe_route(lg.half(), 2), TypeError),
        (lambda: ar.moe_combine(lg, i4, f4[:2]), ValueError),
        (lambda: ar.moe_combine(lg, i4.long(), f4), TypeError),
        (lambda: ar.moe_combine(lg, i4, f4, residual=torch.zeros(4, 7, device="cuda")), ValueError),
        (lambda: ar.moe_combine(lg, i4, f4, out=lg), ar.ARError),
    ]:
        with pytest.raises(err):
            call()
    e = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    ep, es = ar.pack_mxfp4(e)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ar.mxfp4_linear(e, p, s).shape == (0, 4) and ar.mxfp4_linear_a4(ep, es, p, s, bias=f4[0].repeat(2)).shape == (0, 4)
    assert ar.mxfp4_grouped_gemm(e, g, gs, none).shape == (0, 4)
    assert ar.mxfp4_grouped_gemm_a4(ep, es, g, gs, none, rows=none[:0]).shape == (0, 4)
    assert ar.moe_combine(lg, i4[:0], f4[:0]).shape == (0, 8)
    # rows of X that do not exist, all of them
    y = ar.mxfp4_grouped_gemm(e, g, gs, o, rows=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (y == 0).all()
