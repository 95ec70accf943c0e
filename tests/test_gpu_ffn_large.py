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
    return (np.random.default_rng(seed).standard_normal((M, N)) * std).astype(np.float16)


def rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def half_step(a):
    """Half an fp16 step at each value of a."""
    return 0.5 * np.spacing(np.minimum(np.abs(a), 65504.0).astype(np.float16)).astype(np.float64)


def check(got, ref, slack, what):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    bound = HALF * (np.abs(ref) + slack) + 2.0 ** -25 + slack
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[:3].tolist()}; worst {np.max(err / bound):.3g} bounds"
    return got


def check_product(got, ref, norm, each, what):
    got = check(got, ref, each * rms(ref), what)
    R = np.sqrt(np.sum(np.square(half_step(ref))) / 3.0)
    limit = 1.01 * np.sqrt(R * R + (norm * np.linalg.norm(ref)) ** 2)
    err = np.linalg.norm(got - ref)
    assert err <= limit, f"{what}: 2-norm {err / np.linalg.norm(ref):.3e}, limit {limit / np.linalg.norm(ref):.3e}"


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
    product = lambda lay: (Xd.double() @ lay[2].t()).cpu().numpy()
    return Xd, a[1], product(a), b and b[1], b and product(b)


@pytest.mark.parametrize("act", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_fused(M, N, K, act):
    Xd, lay, Z0, _, _ = forward_case(M, N, K, False)
    i = F.ACTIVATIONS.index(act)
    for bias, residual, pre in ((False, False, True), (True, True, i % 2 == 0), (i % 2 == 0, i % 2 == 1, True)):
        b = normal([31, 1], 1, N, 0.5)[0] if bias else None
        r = normal([31, 2], M, N, 2.0) if residual else None
        out = B.w4_gemm_fused(Xd, *lay, bias=None if b is None else dev(b), activation=B.ACTIVATIONS[act],
                              residual=None if r is None else dev(r), save_pre=pre)
        ok()
        Y, Z = out if pre else (out, None)
        Zr = Z0 if b is None else Z0 + b.astype(np.float64)
        Yr = F.act(Zr, act) if r is None else F.act(Zr, act) + r.astype(np.float64)
        what = f"fused {M}x{N}x{K} {act} bias={bias} residual={residual}"
        # the fp32 sum's error, and the activation's and residual's own fp32 arithmetic on values of Z's size
        check(Y, Yr, (1.13 * FWD_EACH + A) * rms(Zr) + A * np.abs(Zr), what)
        if pre:
            check_product(Z, Zr, FWD_NORM, FWD_EACH, what + " Z")


@pytest.mark.parametrize("act", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_gated(M, N, K, act):
    Xd, g, Gr, u, Ur = forward_case(M, N, K, True)
    Hr = F.act(Gr, act) * Ur
    eg, eu = FWD_EACH * rms(Gr), FWD_EACH * rms(Ur)
    slack = 1.13 * eg * (np.abs(Ur) + eu) + eu * np.abs(F.act(Gr, act)) + A * np.abs(Gr * Ur)
    H, G, U = B.w4_gemm_gated(Xd, g, u, activation=B.ACTIVATIONS[act], save_pre=True)
    H2 = B.w4_gemm_gated(Xd, g, u, activation=B.ACTIVATIONS[act])
    ok()
    what = f"gated {M}x{N}x{K} {act}"
    check(H, Hr, slack, what)
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
    dY = dev(normal([51, 3], M, N, 0.05))
    dX = dY.double() @ a[2]
    if not pair:
        return dY, a[1], dX.cpu().numpy(), None, None
    b = layer(52, N, K)
    dY2 = dev(normal([51, 4], M, N, 0.05))
    return dY, a[1], (dX + dY2.double() @ b[2]).cpu().numpy(), dY2, b[1]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_input_gradient(M, N, K, pair):
    dY, a, ref, dY2, b = backward_case(M, N, K, pair)
    out = B.w4_gemm_dx(dY, *a, dY2=dY2, weights2=b)
    ok()
    check_product(out, ref, DX_NORM, DX_EACH, f"dx {M}x{N}x{K} pair={pair}")


@pytest.mark.parametrize("act", F.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_input_gradient_through_the_gate(M, N, K, act):
    dY, a, dH, _, _ = backward_case(M, N, K, False)
    G, U = normal([61, 6], M, K, 1.5), normal([61, 7], M, K, 1.5)
    Gd, Ud = dev(G), dev(U)
    dG, dU = B.w4_gemm_dx_gated(dY, *a, Gd, Ud, activation=B.ACTIVATIONS[act])
    in_place = B.w4_gemm_dx_gated(dY, *a, Gd, Ud, activation=B.ACTIVATIONS[act], out=(Gd, Ud))
    ok()
    assert in_place[0] is Gd and torch.equal(dG, Gd) and torch.equal(dU, Ud)
    rG, rU = F.gate_backward(dH, G, U, act)
    e = DX_EACH * rms(dH)
    U64, G64 = U.astype(np.float64), G.astype(np.float64)
    what = f"dx_gated {M}x{N}x{K} {act}"
    check(dG, rG, e * np.abs(U64 * F.act_grad(G64, act)) + A * np.abs(dH * U64), what + " dG")
    check(dU, rU, e * np.abs(F.act(G64, act)) + A * np.abs(rU), what + " dU")


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
