"""How far the products are from 64 bits as a whole, at few activation rows.

An output's rounding to fp16 is known from the 64-bit values: half steps uniformly used, R = sqrt(sum step_i^2 / 12)
in 2-norm, with a spread of sqrt(0.8 / n) relative (2 % for n = 2000, the fewest here; 4 % allowed).  What a
kernel adds before that rounding has to stay below a share p of the result's 2-norm: the error's 2-norm is at
most 1.04 sqrt(R^2 + (p |Z|)^2).

  * GEMV (up to 8 rows, w4_gemm up to 16): operands 1024 + q and q - 1039, whose offsets cancel over a group
    of 128 up to the spread of the activations' differences.  A group's eight sums of 16 products grow as
    1024 sqrt(16 i) r (r the activations' rms), each cut off by less than one step, 2^-23 of it, uniformly:
    sqrt(sum_i (2^-23 1024 sqrt(16 i) r)^2 / 3) = 1.7e-3 r, against a group's own 2.9 sqrt(128) r = 33 r: 5.2e-5,
    and the same for the sum of all groups, whose errors have no common sign.  p = 2^-14.  fp16(x / 16)
    moves |x| < 2^-10 only (2^-21): nothing beside it.  With offsets of one sign, rows of one sign are off by
    1e-3 to 3e-3.
  * tensor-core products: p = 2^-17 (eight steps of a group's fp32 sum, 2^-22 of it each at most, and the
    groups' sums).  Weights rounded to fp16 would cost 1.5e-4 = 2^-12.7."""
import functools

import numpy as np
import pytest
import torch

import oracle
from oracle import ffn_oracle as F
from weight_only_int4_06_b200 import synth
from weight_only_int4_06_b200 import w4a16 as B

pytestmark = pytest.mark.gpu

GEMV, TC = 2.0 ** -14, 2.0 ** -17


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@functools.lru_cache(maxsize=4)
def layer(case, N, K):
    lay = oracle.quantize_pack(synth.layer_case(case, 1, K, N)[1])
    return tuple(dev(t) for t in (lay[0].view(np.int32), lay[1], lay[2])), F.weight(lay)


def check(got, ref, p, what):
    got = got.cpu().numpy().astype(np.float64)
    step = np.spacing(np.abs(ref).astype(np.float16)).astype(np.float64)
    size = np.linalg.norm(ref)
    limit = 1.04 * np.sqrt(np.sum(step * step) / 12.0 + (p * size) ** 2)
    err = np.linalg.norm(got - ref)
    assert err <= limit, f"{what}: {err / size:.3e} of the result, limit {limit / size:.3e}"


def rows(kind, M, K):
    X = np.random.default_rng([M, K]).standard_normal((M, K))
    if kind == "relu":  # behind a relu
        X = np.maximum(X, 0)
    elif kind == "negative":
        X = -np.abs(X)
    elif kind == "shifted":  # a mean well beside zero
        X = X + 3.0
    elif kind == "loud":  # one sign, 1 % of the channels twenty times larger
        X = np.abs(X)
        X[:, ::97] *= 20
    return X.astype(np.float16)


def ok():
    assert B.w4_check_device_status() == 0


@pytest.mark.parametrize("kind", ["normal", "relu", "negative", "shifted", "loud"])
@pytest.mark.parametrize("N,K", [(4096, 4096), (2048, 11008), (2048, 28672), (2056, 1152)])
def test_few_rows(N, K, kind):
    a, Wa = layer(41, N, K)
    b, Wb = layer(42, N, K)
    for M in (1, 2, 4, 8):
        X = rows(kind, M, K)
        Xd, X64 = dev(X), X.astype(np.float64)
        Gr, Ur = X64 @ Wa.T, X64 @ Wb.T
        what = f"{kind} {M}x{N}x{K}"
        check(B.w4_gemm_fused(Xd, *a), Gr, GEMV, "fused " + what)
        _, G, U = B.w4_gemm_gated(Xd, a, b, save_pre=True)
        check(G, Gr, GEMV, "gate " + what)
        check(U, Ur, GEMV, "up " + what)
        check(B.w4_gemm(Xd, *a), Gr, GEMV, "w4_gemm " + what)
    X = rows(kind, 16, K)
    check(B.w4_gemm(dev(X), *a), X.astype(np.float64) @ Wa.T, GEMV, f"w4_gemm {kind} 16x{N}x{K}")
    ok()


@pytest.mark.parametrize("kind", ["normal", "relu", "negative", "shifted", "loud"])
@pytest.mark.parametrize("N,K", [(4096, 4096), (2048, 1152)])
def test_gemv_with_weights_in_tensor_memory(N, K, kind):
    """The same operands in w4_gemm's other GEMV."""
    a, Wa = layer(41, N, K)
    for M in (1, 8):
        X = rows(kind, M, K)
        check(B.w4_gemm(dev(X), *a, variant=B.VARIANT_GEMV_TC), X.astype(np.float64) @ Wa.T, GEMV, f"{kind} {M}x{N}x{K}")
    ok()


@pytest.mark.parametrize("kind", ["normal", "relu", "negative", "shifted", "loud"])
@pytest.mark.parametrize("M,N,K", [(9, 2048, 4096), (24, 1032, 11008), (33, 4104, 2176), (64, 2048, 8192), (100, 520, 1152)])
def test_small_batches(M, N, K, kind):
    a, Wa = layer(43, N, K)
    b, Wb = layer(44, N, K)
    X = rows(kind, M, K)
    Xd, X64 = dev(X), X.astype(np.float64)
    Gr, Ur = X64 @ Wa.T, X64 @ Wb.T
    what = f"{kind} {M}x{N}x{K}"
    Y, Z = B.w4_gemm_fused(Xd, *a, activation=B.ACT_RELU, save_pre=True)
    check(Z, Gr, TC, "fused " + what)
    _, G, U = B.w4_gemm_gated(Xd, a, b, save_pre=True)
    check(G, Gr, TC, "gate " + what)
    check(U, Ur, TC, "up " + what)
    ok()


def test_metadata_without_alignment_takes_the_tensor_cores():
    M, N, K = 4, 2048, 4096
    (p, s, z), W = layer(45, N, K)
    s1 = torch.empty(s.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(s).copy_(s)
    z1 = torch.empty(z.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view_as(z).copy_(z)
    X = rows("relu", M, K)
    check(B.w4_gemm_fused(dev(X), p, s1, z1), X.astype(np.float64) @ W.T, TC, "misaligned metadata")
    ok()
