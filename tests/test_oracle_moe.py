"""Pins of the oracle of the operators around the packed-MXFP4 products (CPU):
activations, router and weighted sum against torch in fp64, worked cases of
masked and tied scores, and the order of the rows."""
import numpy as np
import pytest
import torch

from oracle import moe_ref as moe


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_activations_against_torch(act):
    a = np.concatenate([np.linspace(-40, 40, 2001), [0.0, 1e-300, -1e-300, np.inf, np.nan]])
    f = {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu, "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    # torch's (1 + erf) and (1 + tanh) cancel for negative values: absolute agreement
    np.testing.assert_allclose(moe.activate(a, act), f(torch.from_numpy(a)).numpy(), rtol=1e-13, atol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_against_torch(score, normalize):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 12))
    got = moe.route(x, 3, score, normalize, weight_scale=2.0)
    t = torch.from_numpy(x)
    s = torch.softmax(t, -1) if score == "softmax" else torch.sigmoid(t)
    w, e = torch.topk(s, 3)
    w = w / w.sum(-1, keepdim=True) if normalize else w
    assert (got["expert"] == e.numpy()).all()
    np.testing.assert_allclose(got["weight"], 2.0 * w.numpy(), rtol=1e-12)
    assert got["offsets"][0] == 0 and got["offsets"][-1] == 150
    for j in range(12):
        mine = got["token"][got["offsets"][j]:got["offsets"][j + 1]]
        assert (np.diff(mine) > 0).all() and (got["expert"][mine] == j).any(axis=1).all()
    assert (got["expert"].reshape(-1)[np.argsort(got["pos"].reshape(-1))] == np.repeat(np.arange(12), np.diff(got["offsets"]))).all()


def test_route_ties_masks_and_nan():
    inf = np.inf
    x = np.array([[1.0, 2.0, 2.0, 2.0], [-inf, 0.5, -inf, -inf], [-inf] * 4, [0.0, np.nan, 3.0, np.nan]])
    got = moe.route(x, 2)
    assert got["expert"].tolist() == [[1, 2], [1, -1], [-1, -1], [1, 3]]
    assert got["weight"][0].tolist() == [0.5, 0.5] and got["weight"][1].tolist() == [1.0, 0.0]
    assert got["weight"][2].tolist() == [0.0, 0.0] and np.isnan(got["weight"][3]).all()
    assert got["offsets"].tolist() == [0, 0, 3, 4, 5]
    assert got["token"].tolist() == [0, 1, 3, 0, 3, -1, -1, -1]
    assert got["pos"].tolist() == [[0, 3], [1, -1], [-1, -1], [2, 4]]
    biased = moe.route(np.zeros((1, 4)), 2, "sigmoid", False, bias=[0.0, -inf, 0.25, 0.25])
    assert biased["expert"].tolist() == [[2, 3]] and biased["weight"].tolist() == [[0.5, 0.5]]


def test_grouped_and_combine_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    w = np.stack([np.eye(2), 2 * np.eye(2)])
    y, written = moe.grouped(x, w, [0, 1, 2], rows=[1, 0, 0], bias=np.array([[0.0, 0.0], [1.0, 0.0]]))
    assert y[:2].tolist() == [[3.0, 4.0], [3.0, 4.0]] and written.tolist() == [True, True, False]
    z, mag = moe.combine(y, np.array([[0, 1], [-1, 1]]), np.array([[0.5, 0.25], [9.0, -1.0]]), residual=np.ones((2, 2)))
    assert z.tolist() == [[3.25, 4.0], [-2.0, -3.0]] and mag[1].tolist() == [4.0, 5.0]
