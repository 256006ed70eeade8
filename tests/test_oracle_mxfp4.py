"""Pins of the packed-MXFP4 oracle (CPU): worked blocks, the tensor-level
MXFP4 fake quantizer's oracle, the nibble order, and the norm and the gate
against torch in fp64."""
import numpy as np
import torch

from oracle import float_formats as ff
from oracle import mxfp4_ref as mx

F32 = np.float32


def test_worked_block():
    x = np.zeros((1, 32))
    # maximum 10: e = floor(log2 10) - 2 = 1; x / 2 = 5 (tie of 4 and 6: even code is 4), 0.25 (tie: 0), -0.75 (tie: -1)
    x[0, :5] = [10.0, 0.5, -1.5, -0.1, 7.0]
    codes, scale = mx.quantize(x)
    assert scale.tolist() == [[128]]
    assert codes[0, :5].tolist() == [6, 0, 8 | 2, 0, 6]     # 3.5 ties to 4
    v = mx.values(mx.pack(codes), scale)
    assert v[0, :5].tolist() == [8.0, 0.0, -2.0, 0.0, 8.0]


def test_nibble_order_and_round_trip():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (3, 64)).astype(np.uint8)
    p = mx.pack(codes)
    assert p[0, 0] == codes[0, 0] + 16 * codes[0, 1]
    np.testing.assert_array_equal(mx.unpack(p), codes)


def test_equals_the_tensor_level_oracle():
    rng = np.random.default_rng(1)
    W = (rng.standard_normal((40, 256)) * 0.02).astype(F32)
    W[3, :32] = 0.0
    alpha = rng.uniform(0.5, 1.0, (40, 8)).astype(F32)
    for al in (None, alpha):
        ref = ff.qdq_mxfp4(W, al)
        codes, scale = mx.quantize(W, al)
        np.testing.assert_array_equal(codes, ref["codes"])
        np.testing.assert_array_equal(scale, ref["scale_bits"])
        np.testing.assert_array_equal(mx.values(mx.pack(codes), scale), ref["w_hat"].astype(np.float64))


def test_nonfinite_and_tiny_blocks():
    x = np.ones((5, 32))
    x[0, 3] = np.nan
    x[1, 4] = -np.inf
    x[2, 5] = 1e39                      # finite, beyond fp32
    x[3] = 2.0 ** -140                  # exponent held at -127
    x[4] = 1e-60                        # zero in fp32
    codes, scale = mx.quantize(x)
    assert scale[:, 0].tolist() == [255, 255, 255, 0, 127]
    assert not codes.any()
    assert np.isnan(mx.values(mx.pack(codes), scale)[:3]).all()


def test_norm_and_gate_against_torch():
    rng = np.random.default_rng(2)
    r, w = rng.standard_normal((4, 96)), rng.standard_normal(96)
    t = torch.from_numpy(r)
    ref = torch.nn.functional.rms_norm(t, (96,), torch.from_numpy(w), eps=float(F32(1e-5))).numpy()
    np.testing.assert_allclose(mx.rmsnorm(r, w, 1e-5), ref, rtol=1e-13)
    ref = (torch.nn.functional.silu(t) * torch.from_numpy(w)).numpy()
    np.testing.assert_allclose(mx.swiglu(r, w[None]), ref, rtol=1e-13)
    x = mx.residual(F32([[1.0]]), F32([[3.0]]), 0.1)
    assert x[0, 0] == F32(1.0) + F32(F32(0.1) * F32(3.0))
