"""Feed-forward operators on quantised layers, restated in 64 bits: the matrix product with bias,
activation and residual, the gated pair of projections, and the input gradients through them."""
import numpy as np
import torch

from .w4a16_oracle import dequantize

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _phi(x):
    return 0.5 * torch.special.erfc(torch.as_tensor(x) * -np.sqrt(0.5)).numpy()


def _sigmoid(x):
    return torch.sigmoid(torch.as_tensor(x)).numpy()


def act(x, name):
    x = np.asarray(x, np.float64)
    if name == "none":
        return x
    if name == "relu":
        return np.where(x < 0, 0.0, x)
    if name == "gelu":
        return x * _phi(x)
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))
    if name == "silu":
        return x * _sigmoid(x)
    raise ValueError(name)


def act_grad(x, name):
    x = np.asarray(x, np.float64)
    if name == "none":
        return np.ones_like(x)
    if name == "relu":
        return np.where(x > 0, 1.0, 0.0)
    if name == "gelu":
        return _phi(x) + x * np.exp(-0.5 * x * x) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        c = np.sqrt(2.0 / np.pi)
        t = np.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    if name == "silu":
        s = _sigmoid(x)
        return s * (1.0 + x * (1.0 - s))
    raise ValueError(name)


def weight(layer):
    """[N, K] float64 from (packed, scales, zeros)."""
    return np.asarray(dequantize(*layer), np.float64)


def fused(X, layer, bias=None, activation="none", residual=None):
    """(Y, Z)."""
    Z = np.asarray(X, np.float64) @ weight(layer).T
    if bias is not None:
        Z = Z + np.asarray(bias, np.float64)
    Y = act(Z, activation)
    if residual is not None:
        Y = Y + np.asarray(residual, np.float64)
    return Y, Z


def gated(X, gate, up, activation="silu"):
    """(H, G, U)."""
    X = np.asarray(X, np.float64)
    G, U = X @ weight(gate).T, X @ weight(up).T
    return act(G, activation) * U, G, U


def dx(dY, layer, dY2=None, layer2=None):
    out = np.asarray(dY, np.float64) @ weight(layer)
    if dY2 is not None:
        out = out + np.asarray(dY2, np.float64) @ weight(layer2)
    return out


def gate_backward(dH, G, U, activation="silu"):
    """(dG, dU)."""
    dH, G, U = (np.asarray(a, np.float64) for a in (dH, G, U))
    return dH * U * act_grad(G, activation), dH * act(G, activation)


def act_backward(dY, Z, activation):
    """(dZ, dbias)."""
    dZ = np.asarray(dY, np.float64) * act_grad(Z, activation)
    return dZ, dZ.sum(0)
