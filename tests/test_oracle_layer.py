"""The fp64 oracle of the projections, the feed-forward block, rotary positions
and the policy objective, pinned to closed forms and central differences (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import layer as ol

ACTS = ["none", "silu", "gelu", "gelu_tanh"]


def _diff(fn, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        up = fn()
        x[i] = keep - h
        g[i] = (up - fn()) / (2 * h)
        x[i] = keep
    return g


@pytest.mark.parametrize("name", ACTS)
def test_activations(name):
    z = np.linspace(-6, 6, 101)
    t = torch.from_numpy(z)
    want = {"none": t, "silu": torch.nn.functional.silu(t), "gelu": torch.nn.functional.gelu(t),
            "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}[name].numpy()
    value, slope = ol.act(z, name)
    np.testing.assert_allclose(value, want, atol=1e-14)
    np.testing.assert_allclose(slope, (ol.act(z + 1e-6, name)[0] - ol.act(z - 1e-6, name)[0]) / 2e-6, atol=1e-8)


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_are_differences(name):
    g = np.random.default_rng(1)
    x, w, b, dy = g.normal(size=(5, 3)), g.normal(size=(4, 3)), g.normal(size=4), g.normal(size=(5, 4))
    value = lambda: float((ol.linear(x, w, b, name) * dy).sum())
    for got, leaf in zip(ol.linear_bwd(x, w, dy, b, name), (x, w, b)):
        np.testing.assert_allclose(got, _diff(value, leaf), atol=1e-7)


@pytest.mark.parametrize("name", ACTS)
def test_ffn_gradients_are_differences(name):
    g = np.random.default_rng(2)
    x, w_in, w_out, dy = (g.normal(size=s) for s in ((4, 3), (10, 3), (6, 5), (4, 6)))
    value = lambda: float((ol.gated_ffn(x, w_in, w_out, name)[0] * dy).sum())
    for got, leaf in zip(ol.gated_ffn_bwd(x, w_in, w_out, dy, name), (x, w_in, w_out)):
        np.testing.assert_allclose(got, _diff(value, leaf), atol=1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_relative_distances(interleaved):
    g = np.random.default_rng(3)
    q, k = g.normal(size=(1, 1, 16)), g.normal(size=(1, 1, 16))
    f = 100.0 ** (-np.arange(4) / 4.0)
    at = lambda t, p: ol.rope(t, np.array([p]), f, interleaved)
    assert math.isclose((at(q, 7) * at(k, 3)).sum(), (at(q, 1007) * at(k, 1003)).sum(), rel_tol=1e-9)
    np.testing.assert_allclose(ol.rope(at(q, 9), np.array([9]), f, interleaved, inverse=True), q, atol=1e-12)
    assert np.array_equal(at(q, 5)[..., 8:], q[..., 8:])


@pytest.mark.parametrize("sequences", [False, True])
@pytest.mark.parametrize("dual", [0.0, 2.0])
def test_policy_gradient_is_differences(sequences, dual):
    g = np.random.default_rng(4)
    index = np.array([0, 1, 2, 0, 1, 3, 4, 0, 5, 6])
    offsets = np.array([0, 3, 7, 10]) if sequences else None
    loss, R = g.normal(size=7) + 2.0, len(index)
    old = -loss[index] + 0.6 * g.normal(size=R)
    ref = -loss[index] + 0.3 * g.normal(size=R)
    adv, weight = g.normal(size=R), g.random(R)
    weight[4] = 0.0
    call = lambda: ol.policy_loss(loss, old, adv, weight, index, ref, 0.2, 0.3, dual, 0.1, offsets)
    stats, grad, _, _ = call()
    np.testing.assert_allclose(grad, _diff(lambda: call()[0][0], loss), atol=1e-7)
    assert math.isclose(stats[4], weight.sum())


def test_policy_on_policy_is_the_plain_gradient():
    # ratio 1 everywhere: d objective / d loss = weight * advantage
    loss, index = np.array([1.0, 2.0, 0.5]), np.array([0, 1, 2, 0])
    adv, weight = np.array([1.0, -2.0, 0.5, 3.0]), np.array([0.1, 0.2, 0.3, 0.4])
    stats, grad, _, _ = ol.policy_loss(loss, -loss[index], adv, weight, index)
    np.testing.assert_allclose(grad, [0.1 + 1.2, -0.4, 0.15])
    assert math.isclose(stats[0], -(weight * adv).sum()) and stats[2] == 0.0
