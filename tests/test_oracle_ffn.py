"""Pins of the feed-forward oracle: closed forms and central differences (CPU only)."""
import math

import numpy as np
import pytest

import oracle
from oracle import ffn_oracle as F

XS = np.array([-30.0, -9.0, -4.0, -1.5, -0.75, -1e-3, 0.0, 1e-3, 0.3, 1.0, 2.5, 8.0, 40.0])


def test_activation_closed_forms():
    assert np.array_equal(F.act(XS, "none"), XS)
    assert np.array_equal(F.act(XS, "relu"), np.maximum(XS, 0))
    for x in XS:
        assert math.isclose(F.act(x, "silu"), x / (1 + math.exp(-x)), rel_tol=1e-12, abs_tol=0)
        assert math.isclose(F.act(x, "gelu"), 0.5 * x * math.erfc(-x / math.sqrt(2)), rel_tol=1e-10, abs_tol=1e-300)
        y = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        assert math.isclose(F.act(x, "gelu_tanh"), 0.5 * x * (1 + math.tanh(y)), rel_tol=1e-12, abs_tol=1e-15)


@pytest.mark.parametrize("name", F.ACTIVATIONS)
def test_activation_gradients_are_the_differences(name):
    x = XS[XS != 0]
    h = 1e-6
    d = (F.act(x + h, name) - F.act(x - h, name)) / (2 * h)
    # central difference: h^2/6 |f'''| + eps |f| / h
    assert np.all(np.abs(F.act_grad(x, name) - d) <= 1e-8 + 1e-15 / h * np.abs(x))


def _layer(rng, N, K):
    return oracle.quantize_pack((rng.standard_normal((N, K)) * 0.02).astype(np.float16))


@pytest.mark.parametrize("name", ("silu", "gelu", "gelu_tanh", "none"))
def test_block_gradient_is_the_difference(name):
    """The block's input gradient, chained from the operators, against central differences of
    sum(C * Y), Y the block's output."""
    rng = np.random.default_rng(5)
    M, D, F_ = 3, 128, 256
    gate, up, down = _layer(rng, F_, D), _layer(rng, F_, D), _layer(rng, D, F_)
    X, C = rng.standard_normal((M, D)), rng.standard_normal((M, D))

    def loss(x):
        H, _, _ = F.gated(x, gate, up, name)
        return float(np.sum(C * F.fused(H, down, residual=x)[0]))

    H, G, U = F.gated(X, gate, up, name)
    dG, dU = F.gate_backward(F.dx(C, down), G, U, name)
    dX = F.dx(dG, gate, dU, up) + C
    h = 1e-5
    for (m, k) in [(0, 0), (1, 77), (2, 127)]:
        e = np.zeros_like(X)
        e[m, k] = h
        assert abs((loss(X + e) - loss(X - e)) / (2 * h) - dX[m, k]) <= 1e-6 * (1 + abs(dX[m, k]))


def test_bias_and_activation_backward_are_the_differences():
    rng = np.random.default_rng(6)
    lay = _layer(rng, 16, 128)
    X, b, C = rng.standard_normal((5, 128)), rng.standard_normal(16), rng.standard_normal((5, 16))
    _, Z = F.fused(X, lay, b, "gelu")
    dZ, db = F.act_backward(C, Z, "gelu")
    h = 1e-5
    for n in (0, 7, 15):
        e = np.zeros(16)
        e[n] = h
        d = (np.sum(C * F.fused(X, lay, b + e, "gelu")[0]) - np.sum(C * F.fused(X, lay, b - e, "gelu")[0])) / (2 * h)
        assert abs(d - db[n]) <= 1e-6
    assert np.allclose(F.dx(dZ, lay), dZ @ F.weight(lay))
