"""Refusals of the epilogue and grouped MXFP4 products, the router and the
weighted sum: checked on the host before any HIP call, so these run without a
GPU."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_autoround_amd", "libautoround.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libautoround.so not built")


@pytest.fixture(scope="module")
def ar():
    import post_weight_quantization_autoround_amd as mod
    return mod


def _at(byte):
    return ctypes.c_void_p(byte)      # never dereferenced: checks fail first


ORDER = {      # every argument in order, well apart; sizes: M = 4 rows, K = 64, N = 8, E = 3
    "ar_mxfp4_linear": dict(X=0x10000, M=4, K=64, packed=0x20000, scale=0x30000, N=8, bias=0x40000, bt=0, act=0,
                            residual=0x50000, rt=0, ldr=8, Y=0x60000, yt=0, ldy=8, stream=None),
    "ar_mxfp4_linear_a4": dict(xp=0x10000, xs=0x18000, M=4, K=64, packed=0x20000, scale=0x30000, N=8, bias=0x40000, bt=0,
                               act=0, residual=0x50000, rt=0, ldr=8, Y=0x60000, yt=0, ldy=8, stream=None),
    "ar_mxfp4_grouped_gemm": dict(X=0x10000, R=4, K=64, rows=0x18000, packed=0x20000, scale=0x30000, E=3, N=8,
                                  offsets=0x38000, bias=0x40000, bt=0, act=0, Y=0x60000, yt=0, M=4, stream=None),
    "ar_mxfp4_grouped_gemm_a4": dict(xp=0x10000, xs=0x14000, R=4, K=64, rows=0x18000, packed=0x20000, scale=0x30000, E=3,
                                     N=8, offsets=0x38000, bias=0x40000, bt=0, act=0, Y=0x60000, yt=0, M=4, stream=None),
    "ar_moe_route": dict(logits=0x10000, lt=0, T=4, E=8, k=2, score=0, bias=0x20000, normalize=1, c=1.0, expert=0x30000,
                         weight=0x40000, offsets=0x50000, token=0x60000, pos=0x70000, stream=None),
    "ar_moe_combine": dict(Z=0x10000, zt=0, P=8, N=16, pos=0x20000, weight=0x30000, T=4, k=2, residual=0x40000, rt=0,
                           Y=0x50000, yt=0, stream=None),
}
POINTERS = {"X", "xp", "xs", "packed", "scale", "bias", "residual", "Y", "rows", "offsets", "logits", "expert", "weight",
            "token", "pos", "Z"}


def _call(ar, name, **kw):
    args = dict(ORDER[name])
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(ar.lib, name)(*[_at(v) if a in POINTERS and v is not None else v for a, v in args.items()])


INVALID, UNSUPPORTED = 1, 2
LIN = [(dict(packed=None), INVALID), (dict(scale=None), INVALID), (dict(Y=None), INVALID), (dict(M=-1), INVALID),
       (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=48), INVALID), (dict(yt=2), INVALID), (dict(bt=3), INVALID),
       (dict(rt=-1), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(ldy=7), INVALID),
       (dict(ldr=7), INVALID), (dict(packed=0x20004), UNSUPPORTED), (dict(Y=0x60002), UNSUPPORTED),
       (dict(Y=0x60001, yt=1), UNSUPPORTED), (dict(bias=0x40002), UNSUPPORTED), (dict(bias=0x40001, bt=1), UNSUPPORTED),
       (dict(residual=0x50002), UNSUPPORTED), (dict(residual=0x50001, rt=1), UNSUPPORTED), (dict(K=1 << 23), UNSUPPORTED),
       (dict(M=1 << 30, K=32), UNSUPPORTED), (dict(M=1 << 19, N=(1 << 18) + 1, ldy=1 << 20, ldr=1 << 20), UNSUPPORTED),
       (dict(ldy=1 << 62), UNSUPPORTED), (dict(ldr=1 << 62), UNSUPPORTED), (dict(ldy=(1 << 40) + 8), UNSUPPORTED)]
GRP = [(dict(packed=None), INVALID), (dict(scale=None), INVALID), (dict(Y=None), INVALID), (dict(offsets=None), INVALID),
       (dict(M=-1), INVALID), (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=40), INVALID), (dict(E=0), INVALID),
       (dict(E=1025), UNSUPPORTED), (dict(yt=2), INVALID), (dict(bt=3), INVALID), (dict(act=5), INVALID),
       (dict(rows=None, R=5), INVALID), (dict(rows=0x18002), UNSUPPORTED), (dict(offsets=0x38002), UNSUPPORTED),
       (dict(packed=0x20004), UNSUPPORTED), (dict(Y=0x60002), UNSUPPORTED), (dict(bias=0x40002), UNSUPPORTED),
       (dict(M=(1 << 24) + 1), UNSUPPORTED), (dict(E=1024, N=1 << 18, K=128), UNSUPPORTED), (dict(K=1 << 23), UNSUPPORTED),
       (dict(M=1 << 24, N=1 << 18), UNSUPPORTED)]
CASES = ([(n, kw, e) for n in ("ar_mxfp4_linear", "ar_mxfp4_linear_a4") for kw, e in LIN] +
         [(n, kw, e) for n in ("ar_mxfp4_grouped_gemm", "ar_mxfp4_grouped_gemm_a4") for kw, e in GRP] + [
    ("ar_mxfp4_linear", dict(X=None), INVALID), ("ar_mxfp4_linear", dict(X=0x10008), UNSUPPORTED),
    ("ar_mxfp4_linear_a4", dict(xp=None), INVALID), ("ar_mxfp4_linear_a4", dict(xs=None), INVALID),
    ("ar_mxfp4_linear_a4", dict(xp=0x10008), UNSUPPORTED),
    ("ar_mxfp4_grouped_gemm", dict(X=None), INVALID), ("ar_mxfp4_grouped_gemm", dict(X=0x10008), UNSUPPORTED),
    ("ar_mxfp4_grouped_gemm", dict(R=1 << 24), UNSUPPORTED),          # gathered X of 2^31 bytes
    ("ar_mxfp4_grouped_gemm_a4", dict(xp=None), INVALID), ("ar_mxfp4_grouped_gemm_a4", dict(xs=None), INVALID),
    ("ar_mxfp4_grouped_gemm_a4", dict(R=1 << 26), UNSUPPORTED),
    ("ar_moe_route", dict(T=-1), INVALID), ("ar_moe_route", dict(E=0), INVALID), ("ar_moe_route", dict(k=0), INVALID),
    ("ar_moe_route", dict(k=9), INVALID), ("ar_moe_route", dict(lt=2), INVALID), ("ar_moe_route", dict(score=2), INVALID),
    ("ar_moe_route", dict(E=1025), UNSUPPORTED), ("ar_moe_route", dict(E=100, k=65), UNSUPPORTED),
    ("ar_moe_route", dict(T=(1 << 23) + 1), UNSUPPORTED), ("ar_moe_route", dict(T=1 << 62), UNSUPPORTED),
    ("ar_moe_route", dict(logits=0x10002), UNSUPPORTED), ("ar_moe_route", dict(logits=0x10001, lt=1), UNSUPPORTED),
    *[("ar_moe_route", {p: None}, INVALID) for p in ("logits", "expert", "weight", "offsets", "token", "pos")],
    *[("ar_moe_route", {p: 0x10002 + 0x10000 * i}, UNSUPPORTED)
      for i, p in enumerate(("logits", "bias", "expert", "weight", "offsets", "token", "pos"))],
    ("ar_moe_route", dict(T=0, offsets=None), INVALID),
    ("ar_moe_combine", dict(T=-1), INVALID), ("ar_moe_combine", dict(P=-1), INVALID), ("ar_moe_combine", dict(N=0), INVALID),
    ("ar_moe_combine", dict(k=0), INVALID), ("ar_moe_combine", dict(k=65), UNSUPPORTED),
    ("ar_moe_combine", dict(zt=2), INVALID), ("ar_moe_combine", dict(yt=2), INVALID), ("ar_moe_combine", dict(rt=2), INVALID),
    ("ar_moe_combine", dict(T=(1 << 23) + 1), UNSUPPORTED), ("ar_moe_combine", dict(P=1 << 31), UNSUPPORTED),
    ("ar_moe_combine", dict(N=(1 << 33)), UNSUPPORTED), ("ar_moe_combine", dict(N=1 << 31, T=1, P=1), UNSUPPORTED),
    *[("ar_moe_combine", {p: None}, INVALID) for p in ("Z", "pos", "weight", "Y")],
    *[("ar_moe_combine", {p: 0x10002 + 0x10000 * i}, UNSUPPORTED)
      for i, p in enumerate(("Z", "pos", "weight", "residual", "Y"))],
])


@pytest.mark.parametrize("name,kw,expect", CASES)
def test_refused(ar, name, kw, expect):
    assert _call(ar, name, **kw) == expect
    assert ar.lib.ar_last_error().decode()


OVERLAPS = [   # (call, output, operand it meets, that operand's bytes)
    ("ar_mxfp4_linear", "Y", "X", 512), ("ar_mxfp4_linear", "Y", "packed", 256), ("ar_mxfp4_linear", "Y", "scale", 16),
    ("ar_mxfp4_linear", "Y", "bias", 32), ("ar_mxfp4_linear_a4", "Y", "xp", 128), ("ar_mxfp4_linear_a4", "Y", "xs", 8),
    ("ar_mxfp4_grouped_gemm", "Y", "X", 512), ("ar_mxfp4_grouped_gemm", "Y", "rows", 16),
    ("ar_mxfp4_grouped_gemm", "Y", "offsets", 16), ("ar_mxfp4_grouped_gemm", "Y", "packed", 768),
    ("ar_mxfp4_grouped_gemm", "Y", "scale", 48), ("ar_mxfp4_grouped_gemm", "Y", "bias", 96),
    ("ar_mxfp4_grouped_gemm_a4", "Y", "xp", 128), ("ar_mxfp4_grouped_gemm_a4", "Y", "xs", 8),
    ("ar_moe_route", "expert", "logits", 128), ("ar_moe_route", "token", "bias", 32), ("ar_moe_route", "weight", "expert", 32),
    ("ar_moe_route", "offsets", "weight", 32), ("ar_moe_route", "pos", "token", 32), ("ar_moe_route", "pos", "offsets", 36),
    ("ar_moe_combine", "Y", "Z", 512), ("ar_moe_combine", "Y", "pos", 32), ("ar_moe_combine", "Y", "weight", 32),
]


@pytest.mark.parametrize("name,out,other,size", OVERLAPS)
def test_overlaps_are_refused(ar, name, out, other, size):
    for at in (ORDER[name][other], ORDER[name][other] + max(0, (size - 1) // 16 * 16)):
        assert _call(ar, name, **{out: at}) == INVALID
        assert b"overlap" in ar.lib.ar_last_error()


@pytest.mark.parametrize("name,kw", [
    ("ar_mxfp4_linear", dict(Y=0x50000, yt=1)),             # the residual's address, another type
    ("ar_mxfp4_linear", dict(Y=0x50000, ldy=12)),           # another stride
    ("ar_mxfp4_linear", dict(Y=0x50004)), ("ar_mxfp4_linear", dict(Y=0x50000 + 124)), ("ar_mxfp4_linear", dict(Y=0x4FFFC)),
    ("ar_mxfp4_linear", dict(Y=0x50000 + 3 * 400 + 28, ldr=100)),   # the last element of a strided residual
    ("ar_moe_combine", dict(Y=0x40000, yt=1)), ("ar_moe_combine", dict(Y=0x40004)),
])
def test_a_residual_that_is_not_the_output_itself(ar, name, kw):
    assert _call(ar, name, **kw) == INVALID
    assert b"overlap" in ar.lib.ar_last_error()


@pytest.mark.parametrize("name,kw", [
    ("ar_mxfp4_linear", dict(M=0, X=None, Y=None, residual=None)),
    ("ar_mxfp4_linear_a4", dict(M=0, xp=None, xs=None, Y=None, bias=None)),
    ("ar_mxfp4_grouped_gemm", dict(M=0, Y=None, rows=None, R=0, X=None, offsets=None)),
    ("ar_mxfp4_grouped_gemm_a4", dict(M=0, Y=None, R=0, xp=None, xs=None)),
    ("ar_moe_combine", dict(T=0, Z=None, P=0, pos=None, weight=None, Y=None)),
])
def test_no_rows_is_an_empty_problem(ar, name, kw):
    assert _call(ar, name, **kw) == 0


def test_binding_refuses_host_tensors_and_names(ar):
    w = torch.zeros(4, 64, dtype=torch.bfloat16)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    g = torch.zeros(2, 4, 32, dtype=torch.uint8)
    i = torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(4, 2)
    for call in (lambda: ar.mxfp4_linear(w, u, u), lambda: ar.mxfp4_linear_a4(u, u, u, u),
                 lambda: ar.mxfp4_grouped_gemm(w, g, g, i), lambda: ar.mxfp4_grouped_gemm_a4(u, u, g, g, i),
                 lambda: ar.moe_route(f, 1), lambda: ar.moe_combine(f, i, f)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(TypeError):
        ar.mxfp4_linear([1.0], u, u)
    for table, name in ((ar.ACTIVATIONS, "tanh"), (ar.SCORES, None), (ar.SCORES, [])):
        with pytest.raises(ValueError, match="one of"):
            ar._named(table, name, "x")
