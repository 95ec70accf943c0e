"""The feed-forward operators' large-batch kernels against 64 bits: tiles of up to 256 rows whose ring of
stages wraps, several tiles a CTA pair, sums cut into slices, ragged edges, K/128 a multiple of 4 (vector
loads of the metadata) or not.

Tolerances, for products.  fp16 rounding of an output is at most half a step, and as a 2-norm over n outputs
R = sqrt(sum step_i^2 / 12), known from the 64-bit values; its spread is sqrt(0.8 / n) relative, below 1 %
for the n > 100,000 used here.  Before it:

  * forward: the products x (q - z) are exact and a group's fp32 sum of 128 takes eight steps, each off by a
    few 2^-24 of the partial sum, at most 8 * 2^-22 = 2^-19 of the group's size; the groups' sums are added in
    fp32, 2^-24 a step, in the random walk of up to 65 groups: 2^-21.  Together less than 2^-18 of the result's
    rms, held to 2^-17.  A kernel that rounded each weight to fp16 would be off by 1.5e-4 = 2^-12.7: seen.
  * input gradients: each weight is rounded once to fp16, relative error uniform in the weight's binade,
    2^-11 / sqrt(3) / 1.36 = 2.1e-4 at most in 2-norm; times independent gradients the same for the result.
    Together with R at most sqrt(R^2 + (2.1e-4)^2), and 1 % as above.

Single elements: five standard deviations of those 2-norms' parts, 2^-9 of the rms for the input
gradients (4.6 of 4.2e-4 rms), 2^-14 for the forward products, behind half a step of the output.  What
follows a product carries its error through its derivatives, at most 1.13 for every activation."""
import functools
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import ffn_oracle as F
from weight_only_int4_06_b200 import synth
from weight_only_int4_06_b200 import w4a16 as B

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -11
FWD_NORM, FWD_EACH = 2.0 ** -17, 2.0 ** -14
DX_NORM, DX_EACH = 2.1e-4, 2.0 ** -9
A = 2.0 ** -20  # of an activation or derivative of order one, in fp32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@functools.lru_cache(maxsize=4)
def layer(case, N, K):
    lay = oracle.quantize_pack(synth.layer_case(case, 1, K, N)[1])
    return lay, tuple(dev(t) for t in (lay[0].view(np.int32), lay[1], lay[2])), dev(F.weight(lay))


def normal(seed, M, N, std):
    """The same values on every run, on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(M, N, generator=gen, device="cuda") * std).half()


# The activations and their derivatives in 64 bits, on the GPU (oracle/ffn_oracle.py has them on the host).
def act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x * torch.sigmoid(x) if name == "silu" else x


def act_grad(x, name):
    if name == "relu":
        return (x > 0).double()
    if name == "gelu":
        return torch.special.ndtr(x) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    if name == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s))
    return torch.ones_like(x)


def test_the_formulas_here_are_the_oracles():
    x = np.linspace(-12, 12, 4001)
    for name in F.ACTIVATIONS:
        assert np.allclose(act(dev(x), name).cpu().numpy(), F.act(x, name), rtol=1e-9, atol=1e-13)
        assert np.allclose(act_grad(dev(x), name).cpu().numpy(), F.act_grad(x, name), rtol=1e-9, atol=1e-12)


def rms(a):
    return float(a.square().mean().sqrt())


def half_step(a):
    """Half an fp16 step at each value of a."""
    return torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -14))) - 11)


def check(got, ref, slack, what):
    assert got.shape == ref.shape, what
    assert bool(torch.isfinite(got).all()), what
    err = (got.double() - ref).abs()
    bound = HALF * (ref.abs() + slack) + 2.0 ** -25 + slack
    bad = err > bound
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:3].tolist()}; worst {float((err / bound).max()):.3g} bounds"


def check_product(got, ref, norm, each, what):
    check(got, ref, each * rms(ref), what)
    size, err = float(ref.norm()), float((got.double() - ref).norm())
    R = float((half_step(ref).square().sum() / 3).sqrt())
    limit = 1.01 * math.sqrt(R * R + (norm * size) ** 2)
    assert err <= limit, f"{what}: 2-norm {err / size:.3e}, limit {limit / size:.3e}"


def ok():
    assert B.w4_check_device_status() == 0


# M, N, K with the tile widths (fused, gated) that they take on 148 SMs
FORWARD = [
    (1100, 5000, 2176),   # 160 and 224 columns, 140 and 200 tiles for 74 pairs, 17 groups
    (512, 4096, 8192),    # 256 columns, 64 groups; fused in two slices
    (512, 2048, 8192),    # gated: 256 columns, two slices
    (1000, 10000, 1152),  # 224 and 256 columns, 316 gated tiles, 9 groups
    (513, 1032, 8320),    # four and two slices of 65 groups, a last row and eight last columns alone
    (777, 2056, 2688),    # 128 and 224 columns, 21 groups
    (130, 4104, 11008),   # 86 groups
]


@functools.lru_cache(maxsize=2)
def forward_case(M, N, K, gated):
    X = synth.layer_case(31, M, K, 8)[0]
    Xd = dev(X)
    a = layer(31, N, K)
    b = layer(32, N, K) if gated else None
    product = lambda lay: Xd.double() @ lay[2].t()
    return Xd, a[1], product(a), b and b[1], b and product(b)


@pytest.mark.parametrize("name", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_fused(M, N, K, name):
    Xd, lay, Z0, _, _ = forward_case(M, N, K, False)
    i = F.ACTIVATIONS.index(name)
    for bias, residual, pre in ((False, False, True), (True, True, i % 2 == 0), (i % 2 == 0, i % 2 == 1, True)):
        b = normal(1, 1, N, 0.5)[0] if bias else None
        r = normal(2, M, N, 2.0) if residual else None
        out = B.w4_gemm_fused(Xd, *lay, bias=b, activation=B.ACTIVATIONS[name], residual=r, save_pre=pre)
        ok()
        Y, Z = out if pre else (out, None)
        Zr = Z0 if b is None else Z0 + b.double()
        Yr = act(Zr, name) if r is None else act(Zr, name) + r.double()
        what = f"fused {M}x{N}x{K} {name} bias={bias} residual={residual}"
        # the fp32 sum's error, and the activation's and residual's own fp32 arithmetic on values of Z's size
        check(Y, Yr, (1.13 * FWD_EACH + A) * rms(Zr) + A * Zr.abs(), what)
        if pre:
            check_product(Z, Zr, FWD_NORM, FWD_EACH, what + " Z")


@pytest.mark.parametrize("name", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_gated(M, N, K, name):
    Xd, g, Gr, u, Ur = forward_case(M, N, K, True)
    Ga = act(Gr, name)
    eg, eu = FWD_EACH * rms(Gr), FWD_EACH * rms(Ur)
    slack = 1.13 * eg * (Ur.abs() + eu) + eu * Ga.abs() + A * (Gr * Ur).abs()
    H, G, U = B.w4_gemm_gated(Xd, g, u, activation=B.ACTIVATIONS[name], save_pre=True)
    H2 = B.w4_gemm_gated(Xd, g, u, activation=B.ACTIVATIONS[name])
    ok()
    what = f"gated {M}x{N}x{K} {name}"
    check(H, Ga * Ur, slack, what)
    assert torch.equal(H, H2)
    check_product(G, Gr, FWD_NORM, FWD_EACH, what + " G")
    check_product(U, Ur, FWD_NORM, FWD_EACH, what + " U")


# M, N, K of the layer(s): dY [M, N]
BACKWARD = [
    (1100, 5000, 2176),  # 256 columns, 40 and 80 steps, a step of 8 rows last, half a pair's tile past K
    (2500, 1160, 6400),  # 256 columns, 250 tiles for 74 pairs
    (700, 1000, 11008),  # 256 columns, 129 tiles
    (300, 4096, 1024),   # 128 columns, four and six slices
    (1000, 6000, 2048),  # 256 columns, two slices
    (600, 4096, 1408),   # 64 and 128 columns, an odd number of groups
]


@functools.lru_cache(maxsize=2)
def backward_case(M, N, K, pair):
    a = layer(51, N, K)
    dY = normal(3, M, N, 0.05)
    dX = dY.double() @ a[2]
    if not pair:
        return dY, a[1], dX, None, None
    b = layer(52, N, K)
    dY2 = normal(4, M, N, 0.05)
    return dY, a[1], dX + dY2.double() @ b[2], dY2, b[1]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_input_gradient(M, N, K, pair):
    dY, a, ref, dY2, b = backward_case(M, N, K, pair)
    out = B.w4_gemm_dx(dY, *a, dY2=dY2, weights2=b)
    ok()
    check_product(out, ref, DX_NORM, DX_EACH, f"dx {M}x{N}x{K} pair={pair}")


@pytest.mark.parametrize("name", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_input_gradient_through_the_gate(M, N, K, name):
    dY, a, dH, _, _ = backward_case(M, N, K, False)
    G, U = normal(6, M, K, 1.5), normal(7, M, K, 1.5)
    G64, U64 = G.double(), U.double()
    dG, dU = B.w4_gemm_dx_gated(dY, *a, G, U, activation=B.ACTIVATIONS[name])
    in_place = B.w4_gemm_dx_gated(dY, *a, G, U, activation=B.ACTIVATIONS[name], out=(G, U))
    ok()
    assert in_place[0] is G and torch.equal(dG, G) and torch.equal(dU, U)
    e = DX_EACH * rms(dH)
    what = f"dx_gated {M}x{N}x{K} {name}"
    check(dG, dH * U64 * act_grad(G64, name), e * (U64 * act_grad(G64, name)).abs() + A * (dH * U64).abs(), what + " dG")
    rU = dH * act(G64, name)
    check(dU, rU, e * act(G64, name).abs() + A * rU.abs(), what + " dU")


def test_static_weights_chain():
    """W4_FLAG_WEIGHTS_STATIC: the weights' first stages are fetched before the preceding call has finished."""
    D, Fi, M = 2048, 5504, 600
    g, u, d = (layer(82 + i, *s)[1] for i, s in enumerate(((Fi, D), (Fi, D), (D, Fi))))
    X = dev(synth.layer_case(82, M, D, 8)[0])

    def chain(flags):
        x = X
        for _ in range(3):
            x = B.w4_gemm_fused(B.w4_gemm_gated(X, g, u, flags=flags), *d, residual=x, flags=flags)
        return x

    plain = chain(0)
    assert bool(torch.isfinite(plain).all())
    for _ in range(4):
        assert torch.equal(plain, chain(B.FLAG_WEIGHTS_STATIC))
    ok()
