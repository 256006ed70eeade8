"""GPU parity of the packed-MXFP4 operators against the 64-bit oracle.

Codes and scale bytes are compared bit for bit.  Products are compared in two
ways: on operands whose every partial sum fp32 holds exactly, bit for bit;
and on general operands within K half-steps of fp32 of sum |x w| (each of at
most K additions rounds once; the products are exact), plus half a step of
the output type."""
import numpy as np
import pytest
import torch

from oracle import mxfp4_ref as mx
from synthetic_inputs import make_weight, to_bf16_values

pytestmark = pytest.mark.gpu
F32 = np.float32
U24 = 2.0 ** -24          # half a step of fp32, relative
U8 = 2.0 ** -8            # half a step of bf16, relative


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


def _same_packed(got, codes, scale, what=""):
    packed, sc = (t.cpu().numpy() for t in got[:2])
    np.testing.assert_array_equal(sc, scale, err_msg=what)
    np.testing.assert_array_equal(mx.unpack(packed), codes, err_msg=what)


def _hard_weight(rng, n, k):
    """A weight with blocks of zeros, ties, NaN, infinities and magnitudes from the smallest to the largest."""
    W = make_weight(rng, n, k)
    W[0] = 0.0
    if n > 1:
        W[1] = np.resize(F32([10, 0.5, -1.5, -0.1, 7, 5, -3.5, 2.5, -0.0, 0.25, 1.25, 1.75, 8, 12, -12]), k)
    if n > 3:
        W[2] *= F32(2.0 ** -126)
        W[3] *= F32(2.0 ** 120)
    if n > 6:
        W[4, 5], W[5, k - 1], W[6, 0] = np.nan, np.inf, -np.inf
    if n > 8:
        W[7], W[8] = F32(1e-45), F32(3.4e38)
    return W


# ------------------------------------------------------------ pack, unpack
@pytest.mark.parametrize("n,k", [(1, 32), (3, 96), (17, 64), (64, 2080), (5, 11008)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("clip", [False, True])
def test_pack_and_unpack(ar, n, k, bf16, clip):
    rng = np.random.default_rng(n + k)
    W = _hard_weight(rng, max(n, 9), k)[-n:] if n < 9 else _hard_weight(rng, n, k)
    W = to_bf16_values(W) if bf16 else W
    alpha = rng.uniform(0.5, 1.0, (n, k // 32)).astype(F32) if clip else None
    if clip and n > 16:
        alpha[16, 0], alpha[15, 0] = 0.0, np.nan
    codes, scale = mx.quantize(W, alpha)
    got = ar.pack_mxfp4(_dev(W, bf16), alpha=None if alpha is None else _dev(alpha))
    _same_packed(got, codes, scale)
    with np.errstate(over="ignore"):
        want = mx.values(mx.pack(codes), scale).astype(F32)
    for dt in (torch.float32, torch.bfloat16):
        v = _np(ar.unpack_mxfp4(*got, out_dtype=dt))
        np.testing.assert_array_equal(v, want)      # every value is exact in either type


def test_unpack_every_code_and_scale(ar):
    packed = np.resize(np.arange(256, dtype=np.uint8), (256, 256))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    with np.errstate(over="ignore"):
        want = mx.values(packed, scale).astype(F32)     # 2^126 * 4 and above: infinite in fp32
    for dt in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(_np(ar.unpack_mxfp4(_dev(packed), _dev(scale), out_dtype=dt)), want)


@pytest.mark.parametrize("clip", [False, True])
def test_pack_equals_the_tensor_level_quantizer(ar, clip):
    rng = np.random.default_rng(5)
    W = _dev(make_weight(rng, 128, 1024), bf16=True)
    alpha = _dev(rng.uniform(0.5, 1.0, (128, 32)).astype(F32)) if clip else None
    q = ar.qdq_rtn(W, bits=4, group_size=32, alpha=alpha, fmt=ar.AR_FMT_MXFP4)
    packed, scale = ar.pack_mxfp4(W, alpha=alpha)
    codes = torch.stack((packed & 15, packed >> 4), -1).reshape(128, 1024)
    assert torch.equal(codes, q["codes"]) and torch.equal(scale, q["zero"])
    assert torch.equal(ar.unpack_mxfp4(packed, scale), q["w_hat"])


def test_pack_past_32_bit_offsets(ar):
    n, k = 270_000, 16_384                    # 4.4 Gi elements, 8.8 GB of bf16
    W = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(6)
    rows = [0, 131_071, 131_072, 262_143, 262_144, n - 1]
    part = to_bf16_values(make_weight(rng, len(rows), k))
    W[rows] = _dev(part, bf16=True)
    packed, scale = ar.pack_mxfp4(W)
    codes, sc = mx.quantize(part)
    _same_packed((packed[rows], scale[rows]), codes, sc)
    assert int(packed.count_nonzero()) == int(packed[rows].count_nonzero())
    back = ar.unpack_mxfp4(packed, scale, out_dtype=torch.bfloat16)
    np.testing.assert_array_equal(_np(back[rows]), mx.values(mx.pack(codes), sc).astype(F32))


# --------------------------------------------------------------- RMS norm
@pytest.mark.parametrize("m,h", [(1, 32), (1, 4096), (3, 96), (5, 2080), (2, 8192), (3, 11008), (2, 20000), (1, 32768)])
@pytest.mark.parametrize("delta", ["none", "bf16", "f32"])
def test_rmsnorm(ar, m, h, delta):
    h = h // 32 * 32
    rng = np.random.default_rng(m + h)
    x = to_bf16_values((rng.standard_normal((m, h)) * rng.uniform(0.1, 30, (m, 1))).astype(F32))
    x[:, :2] *= 64
    d = None if delta == "none" else rng.standard_normal((m, h)).astype(F32)
    d = to_bf16_values(d) if delta == "bf16" else d
    w = (1 + 0.2 * rng.standard_normal(h)).astype(F32) if h % 64 == 0 else None
    c = 0.3
    r = mx.residual(x, d, c)
    codes, scale = mx.quantize(mx.rmsnorm(r, w, 1e-5))
    got = ar.rmsnorm_mxfp4(_dev(x, True), weight=None if w is None else _dev(w), eps=1e-5,
                           delta=None if d is None else _dev(d, delta == "bf16"), delta_scale=c)
    _same_packed(got, codes, scale)
    if d is None:
        assert got[2] is None
    else:
        np.testing.assert_array_equal(_np(got[2]), to_bf16_values(r))


def test_rmsnorm_hard_rows(ar):
    # rows of zeros (also with eps = 0: 0 / 0), of one value whose norm is 1 (exact ties with the weight),
    # with NaN, an infinity, with magnitudes that under- and overflow in fp32
    h = 128
    x = np.zeros((9, h), F32)
    x[1] = 3.0
    x[2] = np.resize(F32([1.0, -1.0]), h)
    x[3], x[3, 7] = 1.0, np.nan
    x[4], x[4, 40] = 1.0, np.inf
    x[5] = 2.0 ** -130
    x[6], x[6, 64] = 2.0 ** -120, 2.0 ** 100
    x[7] = 2.0 ** 127
    x[8, :32] = 1.0
    w = np.resize(F32([2.5, 0.25, 5, -0.75, 1, 3.5, 0, 1e30, 1e-30]), h)
    x = to_bf16_values(x)
    for eps in (0.0, 1e-5):
        for ww in (None, w):
            codes, scale = mx.quantize(mx.rmsnorm(x, ww, eps))
            got = ar.rmsnorm_mxfp4(_dev(x, True), weight=None if ww is None else _dev(ww), eps=eps)
            _same_packed(got, codes, scale, f"eps {eps} weight {ww is not None}")


def test_rmsnorm_weights_past_the_fp32_range(ar):
    # an element of 2^100 (its normalized value, sqrt(96), is near no border) brings r / rms of the others below fp32's
    # normal range, and weights bring them back: a block of them, and single ones beside ordinary elements
    rng = np.random.default_rng(12)
    m, h = 64, 96
    x = rng.choice([-1.0, 1.0], (m, h)) * rng.uniform(1, 2, (m, h))
    w = np.ones(h)
    x[:, 0], x[:, 1:32] = 2.0 ** 100, 0
    x[:, 32:64] *= 2.0 ** rng.integers(-54, -45, (m, 1))
    w[32:64] = rng.uniform(3e29, 1e30, 32)
    x[:, 70:90:5] *= 2.0 ** -60
    w[70:90:5] = 2.0 ** 120 * rng.uniform(1, 2, 4)
    x[0, 32:64] = 1.71875 * 2.0 ** -50
    x = to_bf16_values(x.astype(F32))
    w = w.astype(F32)
    codes, scale = mx.quantize(mx.rmsnorm(x, w, 1e-5))
    _same_packed(ar.rmsnorm_mxfp4(_dev(x, True), weight=_dev(w), eps=1e-5), codes, scale)


# ----------------------------------------------------------------- SwiGLU
@pytest.mark.parametrize("m,f,joined", [(1, 32, False), (1, 11008, True), (7, 96, True), (33, 2080, False),
                                        (130, 1024, True)])
def test_swiglu(ar, m, f, joined):
    rng = np.random.default_rng(m * f)
    g = to_bf16_values((rng.standard_normal((m, f)) * 4).astype(F32))
    u = to_bf16_values(rng.standard_normal((m, f)).astype(F32))
    if joined:
        both = _dev(np.concatenate([g, u], axis=1), True)
        gate, up = both[:, :f], both[:, f:]
    else:
        gate, up = _dev(g, True), _dev(u, True)
    codes, scale = mx.quantize(mx.swiglu(g, u))
    _same_packed(ar.swiglu_mxfp4(gate, up), codes, scale)


def test_swiglu_hard_values(ar):
    # every finite bf16 gate with factors that give ties, tiny and huge products; NaN and infinities
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    g = bits.view(F32).reshape(-1, 32)
    g = np.where(np.isfinite(g), g, F32(0.5)).astype(F32)
    for factor in (1.0, 2.5, 2.0 ** -130, 2.0 ** 100, 0.0):
        u = np.full_like(g, to_bf16_values(F32([factor]))[0])
        codes, scale = mx.quantize(mx.swiglu(g, u))
        _same_packed(ar.swiglu_mxfp4(_dev(g, True), _dev(u, True)), codes, scale, f"factor {factor}")
    g = np.ones((6, 64), F32)
    u = np.ones((6, 64), F32)
    g[0, 3], g[1, 4], g[2, 5], u[3, 6], u[4, 40] = np.nan, np.inf, -np.inf, np.nan, -np.inf
    g[5], u[5, 3] = -100.0, np.inf
    codes, scale = mx.quantize(mx.swiglu(g, u))
    _same_packed(ar.swiglu_mxfp4(_dev(g, True), _dev(u, True)), codes, scale, "nonfinite")


def test_swiglu_factors_past_the_fp32_range(ar):
    # blocks that mix ordinary elements with ones whose sigmoid or g sigmoid(g) leaves fp32's normal range (gates around
    # -88 and far below, subnormal gates) and whose factor brings the product back among the others
    g = np.zeros((4, 32), F32)
    u = np.zeros((4, 32), F32)
    g[0, :2], u[0, :2] = (1, -90), (1, 1e38)
    g[1], u[1] = 1, 1
    g[1, 7], u[1, 7] = -90, 2.0 ** 125
    g[2], u[2] = 1.3 * 2.0 ** -20, 1.3 * 2.0 ** -20
    g[2, 3], u[2, 3] = 1.71875 * 2.0 ** -131, 1.40625 * 2.0 ** 89
    g[3], u[3] = 1, 1
    g[3, 9], u[3, 9] = -88, -1.25 * 2.0 ** 122
    rng = np.random.default_rng(11)
    m, f = 64, 512
    gr = rng.standard_normal((m, f)) * 4
    ur = rng.standard_normal((m, f)) * 2.0 ** rng.integers(-40, 20, (m, f // 32)).repeat(32, axis=1)
    deep = rng.random((m, f)) < 0.05
    tiny = rng.random((m, f)) < 0.5
    far = np.where(tiny, np.sign(gr) * 2.0 ** rng.uniform(-133, -100, (m, f)), rng.uniform(-130, -80, (m, f)))
    gr = np.where(deep, far, gr)
    ur = np.where(deep, np.sign(ur) * 2.0 ** rng.uniform(60, 127.9, (m, f)), ur)
    for i, (gate, up) in enumerate([(g[j:j + 1], u[j:j + 1]) for j in range(4)] + [(gr, ur)]):
        gate, up = to_bf16_values(gate.astype(F32)), to_bf16_values(up.astype(F32))
        codes, scale = mx.quantize(mx.swiglu(gate, up))
        _same_packed(ar.swiglu_mxfp4(_dev(gate, True), _dev(up, True)), codes, scale, f"set {i}")


# --------------------------------------------------------------- products
SHAPES = [(1, 1, 32), (1, 16, 64), (1, 4096, 4096), (2, 33, 96), (3, 100, 160), (15, 17, 128), (16, 256, 2048),
          (17, 129, 288), (31, 64, 512), (32, 1000, 2080), (33, 96, 4096), (64, 130, 256), (65, 48, 1120),
          (100, 300, 736), (130, 520, 1056), (256, 256, 512), (257, 511, 544), (300, 1030, 416), (513, 260, 2304),
          (700, 40, 64), (1, 30000, 96), (40, 24, 32768)]


def _exact_operand(rng, rows, k):
    """Packed operand whose values are multiples of 2^-2 of magnitude at most 12: with one like it, products are
    multiples of 2^-4 of at most 144, and K < 2^24 / (16 * 144) = 7281 of them sum exactly in fp32 in any order.  Larger
    K have the scale 2^-1 alone: products of at most 9, K < 2^24 / (16 * 9) = 116508."""
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    codes[codes == 8] = 0
    if k > 7000:
        return mx.pack(codes), np.full((rows, k // 32), 126, np.uint8)
    return mx.pack(codes), rng.integers(126, 129, (rows, k // 32)).astype(np.uint8)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products_exact(ar, m, n, k):
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, m, k)
    X, W = mx.values(xp, xs), mx.values(wp, ws)
    ref = (X @ W.T).astype(F32)
    x16 = _dev(X.astype(F32), True)
    for dt in (torch.float32, torch.bfloat16):
        want = ref if dt == torch.float32 else to_bf16_values(ref)
        print(f"a16 {m}x{n}x{k} {dt}", flush=True)
        np.testing.assert_array_equal(_np(ar.mxfp4_gemm(x16, _dev(wp), _dev(ws), out_dtype=dt)), want)
        print(f"a4 {m}x{n}x{k} {dt}", flush=True)
        np.testing.assert_array_equal(_np(ar.mxfp4_gemm_a4(_dev(xp), _dev(xs), _dev(wp), _dev(ws), out_dtype=dt)), want)


# Every tile the products choose from (the choice goes by how many tiles there are), with K that ends inside a stage and
# K that does not, rows of scales on and off dword boundaries.
TILED = [(17, 9000, 96), (17, 20000, 1056), (40, 5000, 288), (130, 4200, 416), (130, 4200, 1024), (130, 9000, 288),
         (300, 9000, 160), (300, 9000, 640), (300, 17000, 288), (300, 17000, 384), (520, 17000, 288), (520, 17000, 768),
         (520, 17000, 128), (600, 9000, 352), (1100, 8000, 96), (1100, 8000, 1088), (2000, 8300, 160), (2000, 8300, 512),
         (12, 900, 736), (13, 900, 736), (17, 1000, 32), (20, 1500, 5088), (33, 3000, 8224), (5, 8000, 1376)]


@pytest.mark.parametrize("m,n,k", TILED)
def test_products_exact_over_the_tiles(ar, m, n, k):
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    wp, ws = (_dev(t) for t in _exact_operand(rng, n, k))
    xp, xs = (_dev(t) for t in _exact_operand(rng, m, k))
    X, W = (_dev(mx.values(*(t.cpu().numpy() for t in p))) for p in ((xp, xs), (wp, ws)))
    want = (X @ W.t()).float()                        # fp64 products and sums of these operands are exact
    for dt in (torch.float32, torch.bfloat16):
        print(f"a16 {m}x{n}x{k} {dt}", flush=True)
        assert torch.equal(ar.mxfp4_gemm(X.bfloat16(), wp, ws, out_dtype=dt), want.to(dt))
        print(f"a4 {m}x{n}x{k} {dt}", flush=True)
        assert torch.equal(ar.mxfp4_gemm_a4(xp, xs, wp, ws, out_dtype=dt), want.to(dt))


# Every tile again with K of several turns of its ring and a rest, and of whole turns in two tile columns at least (which
# start at a turn of their own, also where the last stage ends early); the two tile kernels of packed operands with
# more than one group of scales, K an odd and an even multiple of 128.
TURNS = [(20, 1500, 2016), (20, 1500, 2400), (20, 1500, 4608), (20, 1500, 3616), (17, 9000, 1504), (17, 9000, 1888),
         (17, 9000, 2400), (20, 20000, 2016), (20, 20000, 2400), (130, 4200, 1504), (130, 4200, 1888), (130, 4200, 2400),
         (130, 9000, 1504), (130, 9000, 1888), (130, 9000, 2400), (300, 9000, 2016), (300, 9000, 2400),
         (300, 17000, 2304), (300, 17000, 2432), (520, 17000, 2304), (520, 17000, 2432), (520, 17000, 992),
         (520, 17000, 1184), (2000, 8300, 1152), (2000, 8300, 1184)]


@pytest.mark.parametrize("m,n,k", TURNS)
def test_products_exact_over_turns_of_the_ring(ar, m, n, k):
    # operands as _exact_operand's, K < 7281; fp64 products and sums of them are exact
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    table = _dev(mx.values(np.arange(16, dtype=np.uint8)[None], np.full((1, 1), 127, np.uint8)))[0, 0::2]

    def operand(rows):
        packed = rng.integers(0, 256, (rows, k // 2), np.uint8)
        packed[packed % 16 == 8] &= 0xF0
        packed[packed // 16 == 8] &= 0x0F
        packed, scale = _dev(packed), _dev(rng.integers(126, 129, (rows, k // 32)).astype(np.uint8))
        v = table[torch.stack((packed & 15, packed >> 4), -1).reshape(rows, k).int()]
        return packed, scale, v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=1)

    wp, ws, W = operand(n)
    xp, xs, X = operand(m)
    want = (X @ W.t()).float()
    for dt in (torch.float32, torch.bfloat16):
        print(f"a16 {m}x{n}x{k} {dt}", flush=True)
        assert torch.equal(ar.mxfp4_gemm(X.bfloat16(), wp, ws, out_dtype=dt), want.to(dt))
        print(f"a4 {m}x{n}x{k} {dt}", flush=True)
        assert torch.equal(ar.mxfp4_gemm_a4(xp, xs, wp, ws, out_dtype=dt), want.to(dt))


@pytest.mark.parametrize("m,n,k", [(3, 40, 32), (16, 300, 288), (40, 5000, 160), (130, 4200, 288), (300, 9000, 96),
                                   (300, 17000, 288), (520, 17000, 352), (1100, 8000, 96), (2000, 8300, 160)])
def test_products_keep_rows_apart(ar, m, n, k):
    # every second row of X and of W is NaN throughout: the others, whose last stage ends where such a row begins,
    # are untouched
    rng = np.random.default_rng(m + n + k)
    wp, ws = (_dev(t) for t in _exact_operand(rng, n, k))
    xp, xs = (_dev(t) for t in _exact_operand(rng, m, k))
    X, W = (_dev(mx.values(*(t.cpu().numpy() for t in p))) for p in ((xp, xs), (wp, ws)))
    want = (X @ W.t()).float()[::2, ::2]
    ws[1::2] = 255
    xs[1::2] = 255
    x16 = X.bfloat16()
    x16[1::2] = float("nan")
    for Y in (ar.mxfp4_gemm(x16, wp, ws), ar.mxfp4_gemm_a4(xp, xs, wp, ws)):
        assert torch.equal(Y[::2, ::2], want)
        assert Y[1::2].isnan().all() and Y[:, 1::2].isnan().all()


@pytest.mark.parametrize("m,n,k", [(2, 64, 256), (40, 5000, 256), (300, 17000, 256), (520, 17000, 512)])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_scales_at_any_address(ar, m, n, k, off):
    rng = np.random.default_rng(off)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, m, k)

    def moved(a):
        buf = torch.full((a.size + 8,), 255, dtype=torch.uint8, device="cuda")
        out = buf[off:off + a.size].view(a.shape)
        out.copy_(_dev(a))
        assert out.data_ptr() % 4 == off
        return out

    args = (_dev(wp), _dev(ws))
    want = ar.mxfp4_gemm_a4(_dev(xp), _dev(xs), *args)
    assert torch.equal(ar.mxfp4_gemm_a4(_dev(xp), moved(xs), args[0], moved(ws)), want)
    x16 = ar.unpack_mxfp4(_dev(xp), moved(xs), out_dtype=torch.bfloat16)
    assert torch.equal(ar.mxfp4_gemm(x16, args[0], moved(ws)), want)


@pytest.mark.parametrize("m,n,k", [(1, 520, 4096), (16, 300, 11008), (40, 257, 2080), (130, 512, 4096),
                                   (520, 300, 1056)])
def test_products_general(ar, m, n, k):
    rng = np.random.default_rng(m + n + k)
    W = make_weight(rng, n, k)
    W[:, :32] *= F32(2.0 ** 20)
    X = to_bf16_values(rng.standard_normal((m, k)).astype(F32))
    X[0] *= F32(2.0 ** -30)
    wp, ws = ar.pack_mxfp4(_dev(W))
    xp, xs = ar.pack_mxfp4(_dev(X, True))
    Wv = mx.values(wp.cpu().numpy(), ws.cpu().numpy())
    for Xv, call in ((X, lambda dt: ar.mxfp4_gemm(_dev(X, True), wp, ws, out_dtype=dt)),
                     (mx.values(xp.cpu().numpy(), xs.cpu().numpy()),
                      lambda dt: ar.mxfp4_gemm_a4(xp, xs, wp, ws, out_dtype=dt))):
        ref, mag = mx.product(Xv, Wv)
        tol = k * U24 * mag
        err = np.abs(_np(call(torch.float32)).astype(np.float64) - ref)
        assert (err <= tol).all(), (err / mag).max()
        err = np.abs(_np(call(torch.bfloat16)).astype(np.float64) - ref)
        assert (err <= tol + U8 * (np.abs(ref) + tol)).all()


@pytest.mark.parametrize("m", [1, 20, 300])
def test_products_of_subnormal_values(ar, m):
    # X below bf16's smallest normal number times a weight of 2^120, and a weight of 2^-127 and 2^-128 (scale byte 0)
    # times an X of 2^120: products around 2^-8, exact sums
    n, k = 70, 320
    rng = np.random.default_rng(m)
    codes = rng.integers(0, 3, (n, k)).astype(np.uint8)                     # 0, 0.5, 1
    ints = rng.integers(-7, 8, (m, k)).astype(F32)
    for byte, unit in ((247, 2.0 ** -130), (0, 2.0 ** 120)):
        wp, ws = mx.pack(codes), np.full((n, k // 32), byte, np.uint8)
        X = (ints.astype(np.float64) * unit).astype(F32)
        ref = (X.astype(np.float64) @ mx.values(wp, ws).T).astype(F32)
        assert np.abs(ref).max() > 2.0 ** -12
        np.testing.assert_array_equal(_np(ar.mxfp4_gemm(_dev(X, True), _dev(wp), _dev(ws))), ref)


def test_rmsnorm_of_more_rows_than_a_launch_holds(ar):
    m, h = (1 << 25) + 1000, 32                       # 64 threads a row: 2^31 threads and some
    x = torch.zeros((m, h), dtype=torch.bfloat16, device="cuda")
    rows = [0, (1 << 25) - 1, 1 << 25, m - 1]
    rng = np.random.default_rng(3)
    part = to_bf16_values(rng.standard_normal((len(rows), h)).astype(F32))
    x[rows] = _dev(part, True)
    d = torch.zeros((m, h), dtype=torch.bfloat16, device="cuda")
    d[rows] = _dev(part, True)
    packed, scale, r = ar.rmsnorm_mxfp4(x, delta=d, delta_scale=0.5)
    rr = mx.residual(part, part, 0.5)
    codes, sc = mx.quantize(mx.rmsnorm(rr, None, 1e-5))
    _same_packed((packed[rows], scale[rows]), codes, sc)
    np.testing.assert_array_equal(_np(r[rows]), to_bf16_values(rr))
    assert int(packed.count_nonzero()) == int(packed[rows].count_nonzero())


@pytest.mark.parametrize("m", [1, 16, 40, 130, 600])
def test_products_write_their_output_only(ar, m):
    n, k = 261, 160
    rng = np.random.default_rng(m)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, m, k)
    X, W = mx.values(xp, xs), mx.values(wp, ws)
    ref = (X @ W.T).astype(F32)
    for a4 in (False, True):
        buf = torch.full((m + 2, n), 7.0, device="cuda")
        out = buf[1:m + 1]
        if a4:
            ar.mxfp4_gemm_a4(_dev(xp), _dev(xs), _dev(wp), _dev(ws), out=out)
        else:
            ar.mxfp4_gemm(_dev(X.astype(F32), True), _dev(wp), _dev(ws), out=out)
        got = _np(buf)
        np.testing.assert_array_equal(got[1:-1], ref)
        assert (got[0] == 7).all() and (got[-1] == 7).all()


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_products_carry_nan_and_infinity(ar, m):
    # a NaN block of the weight spoils its output column, a NaN or infinite activation its row, and nothing else
    n, k = 140, 320
    rng = np.random.default_rng(m)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, m, k)
    X = mx.values(xp, xs)
    W = mx.values(wp, ws)
    ref = (X @ W.T).astype(F32)
    ws2, xs2, X2 = ws.copy(), xs.copy(), X.copy()
    ws2[77, 9] = 255
    xs2[m - 1, 3] = 255
    X2[m - 1, 100] = np.nan
    ref2 = ref.copy()
    ref2[m - 1] = np.nan
    ref2[:, 77] = np.nan
    for dt in (torch.float32, torch.bfloat16):
        want = ref2 if dt == torch.float32 else to_bf16_values(ref2)
        np.testing.assert_array_equal(
            _np(ar.mxfp4_gemm(_dev(X2.astype(F32), True), _dev(wp), _dev(ws2), out_dtype=dt)), want)
        np.testing.assert_array_equal(
            _np(ar.mxfp4_gemm_a4(_dev(xp), _dev(xs2), _dev(wp), _dev(ws2), out_dtype=dt)), want)


@pytest.mark.parametrize("m,n,k", [(3, 140, 352), (12, 140, 2080), (16, 140, 320), (40, 5000, 288), (300, 140, 352),
                                   (300, 9000, 160), (520, 9000, 416)])
def test_products_carry_infinite_activations(ar, m, n, k):
    # +inf and -inf in X times a weight of either sign is an infinity, times a code 0 NaN, both signs in a row meet in
    # NaN; other rows stay as they are
    rng = np.random.default_rng(m + n)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, m, k)
    X, W = mx.values(xp, xs), mx.values(wp, ws)
    X[0, k - 1], X[m - 1, 0], X[1, 40], X[1, k - 2] = np.inf, -np.inf, np.inf, -np.inf
    want = np.where(np.isfinite(X), X, 0.0) @ W.T
    with np.errstate(invalid="ignore"):
        for i in (0, 1, m - 1):
            want[i] = (X[i] * W).sum(axis=1)
    assert np.isposinf(want).any() and np.isneginf(want).any() and np.isnan(want[[0, m - 1]]).any()
    x16, W = _dev(X.astype(F32), True), (_dev(wp), _dev(ws))
    for dt in (torch.float32, torch.bfloat16):
        ref = want.astype(F32) if dt == torch.float32 else to_bf16_values(want.astype(F32))
        np.testing.assert_array_equal(_np(ar.mxfp4_gemm(x16, *W, out_dtype=dt)), ref)


@pytest.mark.parametrize("m", [3, 300])
def test_products_of_the_longest_rows(ar, m):
    # the largest K; X is zero except for 500 columns spread over it, the first and the last block among them
    n, k = 40, (1 << 23) - 32
    rng = np.random.default_rng(m)
    cols = np.unique(np.concatenate([np.arange(32), k - 32 + np.arange(32), rng.integers(0, k, 436)]))
    wp, ws = _dev(rng.integers(0, 256, (n, k // 2), np.uint8)), torch.full((n, k // 32), 126, dtype=torch.uint8, device="cuda")
    W = mx.unpack(wp[:, cols // 2].cpu().numpy())[:, cols % 2 + 2 * np.arange(len(cols))]
    W = mx.values(mx.pack(np.pad(W, ((0, 0), (0, -len(cols) % 32)))), np.full((n, -(-len(cols) // 32)), 126, np.uint8))
    codes = rng.integers(1, 8, (m, len(cols)))                       # 0.5 .. 6
    X = np.array([0.5, 1, 1.5, 2, 3, 4, 6])[codes - 1]
    want = (X @ W[:, :len(cols)].T).astype(F32)                      # multiples of 2^-3 of at most 500 * 18: exact
    at = torch.from_numpy(cols).cuda()
    x = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    x[:, at] = _dev(codes.astype(np.uint8))
    xp = x[:, 0::2] | (x[:, 1::2] << 4)
    del x
    xs = torch.full((m, k // 32), 127, dtype=torch.uint8, device="cuda")
    x16 = ar.unpack_mxfp4(xp, xs, out_dtype=torch.bfloat16)
    np.testing.assert_array_equal(_np(x16[:, at]), X)
    np.testing.assert_array_equal(_np(ar.mxfp4_gemm(x16, wp, ws)), want)
    np.testing.assert_array_equal(_np(ar.mxfp4_gemm_a4(xp, xs, wp, ws)), want)


def test_products_past_32_bit_offsets(ar):
    # Y of 4.5 G elements (18 GB of fp32): rows past element 2^32 against the first ones
    m, n, k = 140_000, 32_000, 32
    rng = np.random.default_rng(9)
    wp, ws = _exact_operand(rng, n, k)
    xp, xs = _exact_operand(rng, 1000, k)
    ref = (mx.values(xp, xs) @ mx.values(wp, ws).T).astype(F32)
    xpd, xsd = _dev(xp).repeat(m // 1000, 1), _dev(xs).repeat(m // 1000, 1)
    want = _dev(ref)
    for a4 in (False, True):
        if a4:
            Y = ar.mxfp4_gemm_a4(xpd, xsd, _dev(wp), _dev(ws))
        else:
            Y = ar.mxfp4_gemm(ar.unpack_mxfp4(xpd, xsd, out_dtype=torch.bfloat16), _dev(wp), _dev(ws))
        for first in (0, 67_000, 134_000, m - 1000):
            assert torch.equal(Y[first:first + 1000], want), first
        del Y


# ------------------------------------------------- together, as they are used
def _mlp(ar, s, x, delta):
    """The MLP of a decoder block on packed weights and activations: norm with residual, gate and up as one product,
    SwiGLU, down projection."""
    hp, hs, r = ar.rmsnorm_mxfp4(x, weight=s["norm"], delta=delta)
    gu = ar.mxfp4_gemm_a4(hp, hs, *s["gate_up"], out_dtype=torch.bfloat16)
    f = gu.shape[1] // 2
    ap, as_ = ar.swiglu_mxfp4(gu[:, :f], gu[:, f:])
    return ar.mxfp4_gemm_a4(ap, as_, *s["down"]), r, gu, (hp, hs), (ap, as_)


@pytest.mark.parametrize("m", [1, 37, 300])
def test_mlp_of_packed_operators(ar, m):
    H, F = 256, 704
    rng = np.random.default_rng(m)
    gu_w, down_w = make_weight(rng, 2 * F, H), make_weight(rng, H, F)
    norm = (1 + 0.1 * rng.standard_normal(H)).astype(F32)
    s = dict(norm=_dev(norm), gate_up=ar.pack_mxfp4(_dev(gu_w, True)), down=ar.pack_mxfp4(_dev(down_w, True)))
    x = to_bf16_values(rng.standard_normal((m, H)).astype(F32))
    d = rng.standard_normal((m, H)).astype(F32)
    y, r, gu, hq, aq = _mlp(ar, s, _dev(x, True), _dev(d))
    rr = mx.residual(x, d, 1.0)
    np.testing.assert_array_equal(_np(r), to_bf16_values(rr))
    codes, scale = mx.quantize(mx.rmsnorm(rr, norm, 1e-5))
    _same_packed(hq, codes, scale)
    W1 = mx.values(*(t.cpu().numpy() for t in s["gate_up"]))
    ref, mag = mx.product(mx.values(mx.pack(codes), scale), W1)
    tol = H * U24 * mag
    assert (np.abs(_np(gu) - ref) <= tol + U8 * (np.abs(ref) + tol)).all()
    g = _np(gu)                                              # from here on the GPU's own bf16 product
    codes, scale = mx.quantize(mx.swiglu(g[:, :F], g[:, F:]))
    _same_packed(aq, codes, scale)
    ref, mag = mx.product(mx.values(mx.pack(codes), scale), mx.values(*(t.cpu().numpy() for t in s["down"])))
    assert (np.abs(_np(y) - ref) <= F * U24 * mag).all()


@pytest.mark.parametrize("m", [1, 16, 130])
def test_captured_graph_and_other_streams(ar, m):
    # the chain captured once and replayed with new inputs in place, eager work between the replays; then two
    # streams at once
    H, F = 256, 704
    rng = np.random.default_rng(100 + m)
    s = dict(norm=_dev(np.ones(H, F32)), gate_up=ar.pack_mxfp4(_dev(make_weight(rng, 2 * F, H))),
             down=ar.pack_mxfp4(_dev(make_weight(rng, H, F))))
    x = _dev(rng.standard_normal((m, H)).astype(F32), True)
    d = _dev(rng.standard_normal((m, H)).astype(F32))

    def both():
        y, r = _mlp(ar, s, x, d)[:2]
        return y, r, ar.mxfp4_gemm(r, *s["gate_up"]), ar.unpack_mxfp4(*s["down"])

    both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both()
    torch.cuda.synchronize()
    for rep in range(4):
        x.copy_(_dev(rng.standard_normal((m, H)).astype(F32), True))
        d.mul_(-0.7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(both())
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert torch.equal(a, b)
    del graph


def test_out_over_an_operand_is_refused(ar):
    x = torch.ones((64, 64), dtype=torch.bfloat16, device="cuda")
    p, s = ar.pack_mxfp4(x)
    with pytest.raises(ar.ARError, match="overlaps"):
        ar.mxfp4_gemm(x, p, s, out_dtype=torch.bfloat16, out=x)
    both = torch.empty((3, 64, 64), dtype=torch.bfloat16, device="cuda")   # neighbours in one allocation are no overlap
    both[1] = 1
    ar.mxfp4_gemm(both[1], p, s, out_dtype=torch.bfloat16, out=both[0])
    ar.mxfp4_gemm(both[1], p, s, out_dtype=torch.bfloat16, out=both[2])
    assert (both[0] == 64).all() and (both[2] == 64).all() and (both[1] == 1).all()


def test_binding_refusals(ar):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    p, s = ar.pack_mxfp4(x)
    for call, err in [
        (lambda: ar.pack_mxfp4(x[:, :48].contiguous()), ValueError),
        (lambda: ar.pack_mxfp4(x.half()), TypeError),
        (lambda: ar.pack_mxfp4(x.t()), ValueError),
        (lambda: ar.pack_mxfp4(x[0]), ValueError),
        (lambda: ar.pack_mxfp4(x, alpha=torch.ones(4, 3, device="cuda")), ValueError),
        (lambda: ar.unpack_mxfp4(p, s[:, :1].contiguous()), ValueError),
        (lambda: ar.unpack_mxfp4(p, s, out_dtype=torch.float16), TypeError),
        (lambda: ar.rmsnorm_mxfp4(x, weight=torch.ones(32, device="cuda")), ValueError),
        (lambda: ar.rmsnorm_mxfp4(x, delta=x[:2]), ValueError),
        (lambda: ar.swiglu_mxfp4(x, x[:, :32]), ValueError),
        (lambda: ar.swiglu_mxfp4(x.t(), x.t()), ValueError),
        (lambda: ar.swiglu_mxfp4(x[:, 4:36], x[:, 4:36]), ar.ARError),      # not 16-byte aligned
        (lambda: ar.mxfp4_gemm(x[:, :32].contiguous(), p, s), ValueError),
        (lambda: ar.mxfp4_gemm(x, p, s, out=torch.empty(4, 5, device="cuda")), ValueError),
        (lambda: ar.mxfp4_gemm(x, p, s, out_dtype=torch.bfloat16, out=torch.empty(4, 4, device="cuda")), TypeError),
        (lambda: ar.mxfp4_gemm_a4(p, s, p[:, :16].contiguous(), s), ValueError),
        (lambda: ar.mxfp4_gemm_a4(p, s[:2], p, s), ValueError),
    ]:
        with pytest.raises(err):
            call()
    e = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    ep, es = ar.pack_mxfp4(e)
    assert ep.shape == (0, 32) and es.shape == (0, 2)
    assert ar.unpack_mxfp4(ep, es).shape == (0, 64)
    assert ar.mxfp4_gemm(e, p, s).shape == (0, 4) and ar.mxfp4_gemm_a4(ep, es, p, s).shape == (0, 4)
    assert ar.swiglu_mxfp4(e, e)[0].shape == (0, 32) and ar.rmsnorm_mxfp4(e)[0].shape == (0, 32)
