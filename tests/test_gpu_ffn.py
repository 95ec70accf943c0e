"""GPU parity of the feed-forward operators with the 64-bit oracle.

Tolerances.  Every output is rounded once to fp16: at most 2^-11 of its value (2^-25 absolute below
the normal range).  Before that, a product's fp32 sum is off by

  * accumulation: the GEMV sums x (1024 + q) and takes 1024 sum(x) off again, so a group of 128 of
    rms r_x carries rounding of eight steps of at most 2^-23 of its raw magnitude ~1031 sqrt(128) r_x s,
    0.011 r_x s, against a group's result rms of ~2.9 sqrt(128) r_x s = 33 r_x s: 3.4e-4 of the
    output's rms; three to six standard deviations over the few thousand outputs of a case: 2^-9 rms;
  * the input-gradient product rounds each weight once to fp16 (2^-11 of the weight at most, 2e-4 rms):
    below the same 2^-9 rms.

So a product z is within E = 2^-9 rms(z), and what follows carries E through its derivatives.  The
activations and their derivatives themselves are evaluated in fp32 to an absolute error of at most 2^-20
where they are of order one (the normal tail's fit: 6.4e-7 of Phi <= 1; exponential, division and the
multiply-adds behind them: a few 2^-24), which adds A = 2^-20 |factor|: it matters next to a derivative's
zero, where E times the derivative vanishes and the rounding alone may use all of its half step.  The
error's 2-norm is held to 2^-11 of the result's: fp16 rounding alone has 2^-11 / sqrt(3) / 1.36 = 2.1e-4,
the rest at most the same again (gate: two factors)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import ffn_oracle as F
from weight_only_int4_06_b200 import synth
from weight_only_int4_06_b200 import w4a16 as B

pytestmark = pytest.mark.gpu

E = 2.0 ** -9
A = 2.0 ** -20
HALF = 2.0 ** -11


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def layer(case, N, K):
    _, W = synth.layer_case(case, 1, K, N)
    return oracle.quantize_pack(W)


def dlayer(lay):
    p, s, z = lay
    return dev(p.view(np.int32)), dev(s), dev(z)


def normal(seed, M, N, std):
    return (np.random.default_rng(seed).standard_normal((M, N)) * std).astype(np.float16)


def rms(a):
    return float(np.sqrt(np.mean(np.square(a)))) if a.size else 0.0


def check(got, ref, slack, what, norm=True):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    bound = HALF * (np.abs(ref) + slack) + 2.0 ** -25 + slack
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off; worst {np.max(err / bound):.3g} bounds"
    if norm and ref.size >= 64 and np.linalg.norm(ref):
        assert np.linalg.norm(got - ref) <= HALF * np.linalg.norm(ref), (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))


def ok():
    assert B.w4_check_device_status() == 0


SHAPES = [  # M, N, K: one token, the GEMV's row bounds, odd rows, ragged tiles, one group, several waves
    (1, 8, 128), (1, 264, 384), (1, 4096, 4096), (2, 24, 11008), (3, 136, 2048), (5, 520, 1152), (8, 72, 11008),
    (8, 1024, 8192), (9, 40, 512), (13, 264, 4096), (16, 128, 8192), (16, 136, 1152), (17, 64, 256), (31, 200, 640),
    (33, 8, 2176), (48, 1000, 1152), (64, 256, 4096), (77, 392, 384), (100, 72, 128), (127, 520, 512), (129, 256, 1024),
    (192, 264, 768), (193, 384, 256), (255, 640, 384), (257, 136, 2048), (333, 1000, 1152), (600, 2056, 512),
    (16, 8, 28672), (1, 16, 65664), (40, 4104, 256),
]


def fused_case(M, N, K, act, bias, residual, pre, seed=31):
    X, _ = synth.layer_case(seed, M, K, 8)
    lay = layer(seed, N, K)
    b = normal([seed, 1], 1, N, 0.5)[0] if bias else None
    r = normal([seed, 2], M, N, 2.0) if residual else None
    out = B.w4_gemm_fused(dev(X), *dlayer(lay), bias=None if b is None else dev(b), activation=B.ACTIVATIONS[act],
                          residual=None if r is None else dev(r), save_pre=pre)
    ok()
    Y, Z = out if pre else (out, None)
    Yr, Zr = F.fused(X, lay, b, act, r)
    e = E * rms(Zr)
    what = f"fused {M}x{N}x{K} {act}"
    check(Y, Yr, 1.13 * e, what)  # |act'| <= 1.13
    if pre:
        check(Z, Zr, e, what + " Z")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_fused_shapes(M, N, K):
    i = SHAPES.index((M, N, K))
    acts = F.ACTIVATIONS
    fused_case(M, N, K, acts[i % 5], i % 2 == 0, i % 3 != 0, i % 4 == 1)


@pytest.mark.parametrize("M", [1, 7, 40, 300])
@pytest.mark.parametrize("act", F.ACTIVATIONS)
def test_fused_every_epilogue(M, act):
    for bias in (False, True):
        for residual in (False, True):
            fused_case(M, 200, 384, act, bias, residual, bias != residual)


def gated_case(M, N, K, act, pre, seed=41):
    X, _ = synth.layer_case(seed, M, K, 8)
    g, u = layer(seed, N, K), layer(seed + 1, N, K)
    out = B.w4_gemm_gated(dev(X), dlayer(g), dlayer(u), activation=B.ACTIVATIONS[act], save_pre=pre)
    ok()
    Hr, Gr, Ur = F.gated(X, g, u, act)
    H, G, U = out if pre else (out, None, None)
    eg, eu = E * rms(Gr), E * rms(Ur)
    what = f"gated {M}x{N}x{K} {act}"
    check(H, Hr, 1.13 * eg * (np.abs(Ur) + eu) + eu * np.abs(F.act(Gr, act)), what)
    if pre:
        check(G, Gr, eg, what + " G")
        check(U, Ur, eu, what + " U")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_shapes(M, N, K):
    i = SHAPES.index((M, N, K))
    gated_case(M, N, K, F.ACTIVATIONS[(i + 4) % 5], i % 2 == 0)


@pytest.mark.parametrize("M", [1, 6, 40, 300])
@pytest.mark.parametrize("act", F.ACTIVATIONS)
def test_gated_every_activation(M, act):
    gated_case(M, 136, 384, act, True)
    gated_case(M, 136, 384, act, False)


def dx_case(M, N, K, pair, seed=51):
    a, b = layer(seed, N, K), layer(seed + 1, N, K)
    dY, dY2 = normal([seed, 3], M, N, 0.05), normal([seed, 4], M, N, 0.05)
    if pair:
        out = B.w4_gemm_dx(dev(dY), *dlayer(a), dY2=dev(dY2), weights2=dlayer(b))
        ref = F.dx(dY, a, dY2, b)
    else:
        out = B.w4_gemm_dx(dev(dY), *dlayer(a))
        ref = F.dx(dY, a)
    ok()
    check(out, ref, E * rms(ref), f"dx {M}x{N}x{K} pair={pair}")


DX_SHAPES = [s for s in SHAPES if s[2] <= 28672] + [(1, 4104, 128), (200, 8, 1024), (2, 12000, 256), (513, 72, 640)]


@pytest.mark.parametrize("M,N,K", DX_SHAPES)
def test_dx_shapes(M, N, K):
    dx_case(M, N, K, DX_SHAPES.index((M, N, K)) % 2 == 0)
    dx_case(M, N, K, DX_SHAPES.index((M, N, K)) % 2 == 1)


def dx_gated_case(M, N, K, act, in_place=False, seed=61):
    lay = layer(seed, N, K)
    dY, G, U = normal([seed, 5], M, N, 0.05), normal([seed, 6], M, K, 1.5), normal([seed, 7], M, K, 1.5)
    Gd, Ud = dev(G), dev(U)
    dG, dU = B.w4_gemm_dx_gated(dev(dY), *dlayer(lay), Gd, Ud, activation=B.ACTIVATIONS[act],
                                out=(Gd, Ud) if in_place else None)
    ok()
    dH = F.dx(dY, lay)
    rG, rU = F.gate_backward(dH, G, U, act)
    e = E * rms(dH)
    U64, G64 = U.astype(np.float64), G.astype(np.float64)
    what = f"dx_gated {M}x{N}x{K} {act}"
    check(dG, rG, e * np.abs(U64 * F.act_grad(G64, act)) + A * np.abs(dH * U64), what + " dG")
    check(dU, rU, e * np.abs(F.act(G64, act)) + A * np.abs(rU), what + " dU")


@pytest.mark.parametrize("M,N,K", DX_SHAPES)
def test_dx_gated_shapes(M, N, K):
    i = DX_SHAPES.index((M, N, K))
    dx_gated_case(M, N, K, F.ACTIVATIONS[(i + 2) % 5], in_place=i % 3 == 0)


@pytest.mark.parametrize("act", F.ACTIVATIONS)
def test_dx_gated_every_activation(act):
    for M in (1, 40, 300):
        dx_gated_case(M, 136, 384, act)


@pytest.mark.parametrize("M,N", [(1, 8), (3, 2056), (17, 136), (333, 1000), (4097, 72), (9000, 8)])
@pytest.mark.parametrize("act", F.ACTIVATIONS)
def test_act_backward(M, N, act):
    dY, Z, U = normal([M, N, 1], M, N, 0.05), normal([M, N, 2], M, N, 1.5), normal([M, N, 3], M, N, 1.5)
    a = B.ACTIVATIONS[act]
    rZ, rb = F.act_backward(dY, Z, act)
    dZ = B.w4_act_backward(dev(dY), dev(Z), activation=a)
    check(dZ, rZ, 2.0 ** -20 * np.abs(dY.astype(np.float64)) * 1.13, f"dZ {act}")  # act' to a few fp32 ulps
    dZ2, db = B.w4_act_backward(dev(dY), dev(Z), activation=a, bias_grad=True)
    assert torch.equal(dZ, dZ2)
    # fp32 sums of M terms: at most M 2^-24 of the terms' magnitudes' sum, and act' to a few ulps
    mag = np.abs(rZ).sum(0) + np.abs(dY.astype(np.float64)).sum(0)
    assert np.all(np.abs(db.cpu().numpy() - rb) <= (M * 2.0 ** -24 + 2.0 ** -20) * mag)
    rG, rU = F.gate_backward(dY, Z, U, act)
    dG, dU = B.w4_act_backward(dev(dY), dev(Z), U=dev(U), activation=a)
    mag = np.abs(dY.astype(np.float64) * U)
    check(dG, rG, 2.0 ** -20 * mag * 1.13, f"dG {act}")
    check(dU, rU, 2.0 ** -20 * np.abs(rU) + 2.0 ** -40, f"dU {act}")
    ok()
    # in place: dZ on Z, dG on G and dU on U
    Zd, Ud = dev(Z), dev(U)
    assert torch.equal(B.w4_act_backward(dev(dY), Zd, activation=a, out=Zd), dZ)
    Zd = dev(Z)
    a1, a2 = B.w4_act_backward(dev(dY), Zd, U=Ud, activation=a, out=(Zd, Ud))
    assert torch.equal(a1, dG) and torch.equal(a2, dU)


def test_act_backward_identity():
    dY = dev(normal(1, 50, 136, 1.0))
    assert torch.equal(B.w4_act_backward(dY, None, activation=B.ACT_NONE), dY)
    _, db = B.w4_act_backward(dY, None, activation=B.ACT_NONE, bias_grad=True)
    assert torch.allclose(db.double(), dY.double().sum(0), atol=1e-4)


def test_bias_gradient_without_dz():
    """The C call with W4_ACT_NONE: no Z, no dZ, the bias gradient alone."""
    import ctypes
    M, N = 300, 520
    dY = dev(normal(2, M, N, 1.0))
    db = torch.empty(N, dtype=torch.float32, device="cuda")
    need = B.w4_act_backward_workspace_size(M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    st = B.lib().w4_act_backward(P(dY), None, None, M, N, B.ACT_NONE, None, None, P(db), P(ws), need,
                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    ref = dY.double().sum(0)
    # fp32 sums of M terms
    assert bool(((db.double() - ref).abs() <= M * 2.0 ** -24 * dY.double().abs().sum(0)).all())


def test_activation_extremes():
    """Saved pre-activations at the ends of fp16, infinite ones and NaN: finite inputs give finite
    gradients, infinities the limits, NaN stays NaN."""
    vals = np.array([65504.0, -65504.0, 1000.0, -1000.0, 89.0, -89.0, 15.0, -15.0, 6e-8, -6e-8, 0.0, -0.0, np.inf, -np.inf,
                     np.nan, 1.0], np.float16)
    Z = np.tile(vals, (3, 1))
    one = np.ones_like(Z)
    for act in F.ACTIVATIONS:
        dZ = B.w4_act_backward(dev(one), dev(Z), activation=B.ACTIVATIONS[act]).cpu().numpy().astype(np.float64)
        fin = np.isfinite(vals)
        ref = F.act_grad(vals[fin].astype(np.float64), act)
        assert np.all(np.abs(dZ[1][fin] - ref) <= HALF * np.abs(ref) + 2.0 ** -24), act
        assert dZ[0][12] == 1.0 and dZ[0][13] == (1.0 if act == "none" else 0.0), act
        if act != "none":
            assert np.isnan(dZ[0][14]), act
        dG, dU = B.w4_act_backward(dev(one), dev(Z), U=dev(one), activation=B.ACTIVATIONS[act])
        ref = F.act(vals[fin].astype(np.float64), act)
        got = dU.cpu().numpy()[2].astype(np.float64)[fin]
        assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + 2.0 ** -24), act
        assert torch.isnan(dU[0, 14])


# ------------------------------------------------------------------ edges of the shapes
def test_empty_sizes():
    one = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")
    empty = lambda N, K: (torch.empty(N, K // 8, dtype=torch.int32, device="cuda"),
                          torch.empty(N, K // 128, dtype=torch.float16, device="cuda"),
                          torch.empty(N, K // 128, dtype=torch.uint8, device="cuda"))
    assert B.w4_gemm_fused(one(0, 256), *empty(16, 256)).shape == (0, 16)
    assert B.w4_gemm_fused(one(5, 256), *empty(0, 256)).shape == (5, 0)
    # K == 0: act(bias) + residual
    b, r = one(16) * -2, one(5, 16) * 3
    Y, Z = B.w4_gemm_fused(one(5, 0), *empty(16, 0), bias=b, activation=B.ACT_RELU, residual=r, save_pre=True)
    assert torch.equal(Y, r) and torch.equal(Z, b.expand(5, 16))
    for t in B.w4_gemm_gated(one(5, 0), empty(16, 0), empty(16, 0), save_pre=True):
        assert t.shape == (5, 16) and not t.any()
    assert B.w4_gemm_gated(one(0, 256), empty(16, 256), empty(16, 256)).shape == (0, 16)
    # N == 0: the gradient of nothing
    dX = B.w4_gemm_dx(one(5, 0), *empty(0, 256), out=one(5, 256))
    assert dX.shape == (5, 256) and not dX.any()
    dG, dU = B.w4_gemm_dx_gated(one(5, 0), *empty(0, 256), one(5, 256), one(5, 256))
    assert not dG.any() and not dU.any()
    assert B.w4_gemm_dx(one(0, 16), *empty(16, 256)).shape == (0, 256)
    assert B.w4_gemm_dx(one(3, 16), *empty(16, 0)).shape == (3, 0)
    dZ, db = B.w4_act_backward(one(0, 16), one(0, 16), bias_grad=True)
    assert dZ.shape == (0, 16) and not db.any()
    ok()


def guarded(M, N, fill=7.0):
    """A [M, N] output inside a larger buffer whose surroundings must stay as they are."""
    buf = torch.full((M * N + 2048,), fill, dtype=torch.float16, device="cuda")
    return buf, buf[1024:1024 + M * N].view(M, N)


@pytest.mark.parametrize("M,N,K", [(1, 8, 128), (5, 24, 1152), (20, 200, 256), (130, 264, 384), (257, 72, 512)])
def test_nothing_outside_the_outputs_is_written(M, N, K):
    X, _ = synth.layer_case(71, M, K, 8)
    a, b = dlayer(layer(71, N, K)), dlayer(layer(72, N, K))
    dY = dev(normal(3, M, N, 0.05))
    GU = dev(normal(4, M, K, 1.0))
    bufs = []

    def out(m, n):
        buf, view = guarded(m, n)
        bufs.append((buf, m * n))
        return view

    B.w4_gemm_fused(dev(X), *a, activation=B.ACT_SILU, out=out(M, N))
    B.w4_gemm_gated(dev(X), a, b, out=out(M, N))
    B.w4_gemm_dx(dY, *a, out=out(M, K))
    B.w4_gemm_dx(dY, *a, dY2=dY, weights2=b, out=out(M, K))
    B.w4_gemm_dx_gated(dY, *a, GU, GU, out=(out(M, K), out(M, K)))
    B.w4_act_backward(dY, dY, out=out(M, N))
    ok()
    for buf, n in bufs:
        assert bool((buf[:1024] == 7).all()) and bool((buf[1024 + n:] == 7).all())
        assert bool(torch.isfinite(buf).all())


def test_misaligned_metadata():
    """scales and zeros need no alignment."""
    for M in (1, 4, 12, 40, 200):
        N, K = 136, 4096
        X, _ = synth.layer_case(73, M, K, 8)
        lay = layer(73, N, K)
        p, s, z = dlayer(lay)
        s1 = torch.empty(s.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(s).copy_(s)
        z1 = torch.empty(z.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view_as(z).copy_(z)
        Yr, _ = F.fused(X, lay)
        check(B.w4_gemm_fused(dev(X), p, s1, z1), Yr, E * rms(Yr), f"misaligned M={M}")
        Hr, Gr, Ur = F.gated(X, lay, lay, "silu")
        check(B.w4_gemm_gated(dev(X), (p, s1, z1), (p, s, z)), Hr,
              1.13 * E * rms(Gr) * np.abs(Ur) + E * rms(Ur) * np.abs(F.act(Gr, "silu")), f"misaligned gated M={M}",
              norm=False)  # H = act(g) g: the factors' errors add
        dY = normal(5, M, N, 0.05)
        ref = F.dx(dY, lay)
        check(B.w4_gemm_dx(dev(dY), p, s1, z1), ref, E * rms(ref), f"misaligned dx M={M}")
    ok()


def test_residual_in_place_and_determinism():
    for M, N, K in ((1, 4096, 4096), (4, 512, 28672), (24, 1024, 4096), (300, 520, 1152)):
        X, _ = synth.layer_case(74, M, K, 8)
        lay = dlayer(layer(74, N, K))
        r = dev(normal(8, M, N, 2.0))
        Y = B.w4_gemm_fused(dev(X), *lay, residual=r)
        Y2 = B.w4_gemm_fused(dev(X), *lay, residual=r)
        assert torch.equal(Y, Y2)
        assert B.w4_gemm_fused(dev(X), *lay, residual=r, out=r) is r
        assert torch.equal(Y, r)
        h = [B.w4_gemm_gated(dev(X), lay, lay) for _ in range(2)]
        assert torch.equal(*h)
        dY = dev(normal(9, M, N, 0.05))
        d = [B.w4_gemm_dx(dY, *lay, dY2=dY, weights2=lay) for _ in range(2)]
        assert torch.equal(*d)
    ok()


@pytest.mark.parametrize("M", [1, 4, 16, 40, 300])
def test_bad_values_stay_in_their_rows(M):
    """An infinity or NaN in one activation row or one gradient row changes no other row."""
    N, K = 136, 4096
    X, _ = synth.layer_case(75, M, K, 8)
    lay = dlayer(layer(75, N, K))
    rows = [0] if M == 1 else [0, M - 1]
    Xb = X.copy()
    Xb[rows[0], 5] = np.inf
    Xb[rows[-1], 77] = np.nan
    good = [m for m in range(M) if m not in rows]
    for f in (lambda t: B.w4_gemm_fused(t, *lay, activation=B.ACT_GELU), lambda t: B.w4_gemm_gated(t, lay, lay)):
        a, b = f(dev(X)), f(dev(Xb))
        assert torch.equal(a[good], b[good])
        assert not bool(torch.isfinite(b[rows]).all(1).any())
    dY = normal(10, M, N, 0.05)
    dYb = dY.copy()
    dYb[rows[-1], 3] = np.nan
    a, b = B.w4_gemm_dx(dev(dY), *lay), B.w4_gemm_dx(dev(dYb), *lay)
    assert torch.equal(a[good], b[good]) and bool(torch.isnan(b[rows[-1]]).any())
    ok()


def test_large_products_saturate_to_infinity():
    """Sums beyond fp16 become infinities of their sign; their rows' relu and gradients stay defined."""
    K, N = 256, 16
    W = np.full((N, K), 1.0, np.float16)
    W[1] = -1.0
    lay = oracle.quantize_pack(W)
    for M in (1, 20):
        X = np.full((M, K), 60000.0, np.float16)
        Y = B.w4_gemm_fused(dev(X), *dlayer(lay), activation=B.ACT_NONE)
        assert bool((Y[:, 0] == float("inf")).all()) and bool((Y[:, 1] == -float("inf")).all())
        Y = B.w4_gemm_fused(dev(X), *dlayer(lay), activation=B.ACT_SILU)
        assert bool((Y[:, 0] == float("inf")).all()) and bool((Y[:, 1] == 0).all())
    ok()


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_explicit_streams_and_shared_workspace():
    M, N, K = 24, 512, 4096
    X, _ = synth.layer_case(76, M, K, 8)
    Xd, a, b = dev(X), dlayer(layer(76, N, K)), dlayer(layer(77, N, K))
    need = max(B.w4_gemm_fused_workspace_size(M, N, K), B.w4_gemm_gated_workspace_size(M, N, K),
               B.w4_gemm_dx_workspace_size(M, N, K, 2), 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    Y, H = B.w4_gemm_fused(Xd, *a), B.w4_gemm_gated(Xd, a, b)
    dX = B.w4_gemm_dx(Y, *a, dY2=H, weights2=b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        Y1 = B.w4_gemm_fused(Xd, *a, workspace=ws, stream=stream)
        H1 = B.w4_gemm_gated(Xd, a, b, workspace=ws, stream=stream)
        dX1 = B.w4_gemm_dx(Y1, *a, dY2=H1, weights2=b, workspace=ws, stream=stream)
        side.synchronize()
        assert torch.equal(Y, Y1) and torch.equal(H, H1) and torch.equal(dX, dX1)
    ok()


@pytest.mark.parametrize("M", [1, 12, 48, 300])
def test_block_trains_and_serves_captured(M):
    """The whole block as it is used -- gated, down projection with the residual, and back -- against
    64 bits, then captured into a graph (with another eager pass in between) and replayed on new data."""
    D, Fi = 512, 1408
    g, u, d = layer(78, Fi, D), layer(79, Fi, D), layer(80, D, Fi)
    gd, ud, dd = dlayer(g), dlayer(u), dlayer(d)
    X = dev(synth.layer_case(78, M, D, 8)[0])
    dY = dev(normal(11, M, D, 0.05))

    def step():
        H, G, U = B.w4_gemm_gated(X, gd, ud, save_pre=True)
        Y = B.w4_gemm_fused(H, *dd, residual=X)
        dG, dU = B.w4_gemm_dx_gated(dY, *dd, G, U)
        dX = B.w4_gemm_dx(dG, *gd, dY2=dU, weights2=ud)
        return Y, dX

    def reference():
        x, dy = X.cpu().numpy(), dY.cpu().numpy()
        Hr, Gr, Ur = F.gated(x, g, u)
        Yr = F.fused(Hr, d, residual=x)[0]
        dGr, dUr = F.gate_backward(F.dx(dy, d), Gr, Ur)
        return Yr, F.dx(dGr, g, dUr, u)

    def compare(out):
        for got, ref, what in zip(out, reference(), ("Y", "dX")):
            err = got.cpu().numpy().astype(np.float64) - ref
            # intermediates rounded to fp16 (H; G, U, dG, dU): a few half steps in 2-norm
            assert np.linalg.norm(err) <= 4 * HALF * np.linalg.norm(ref), what

    compare(step())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    compare(out)
    X.copy_(dev(synth.layer_case(81, M, D, 8)[0]))
    dY.copy_(dev(normal(12, M, D, 0.05)))
    eager = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, out))
    compare(out)
    ok()


def test_concurrent_streams():
    """Calls that overlap on two streams, each with its own workspace, do not disturb each other."""
    M, N, K = 40, 1024, 4096
    w = [dlayer(layer(90 + i, N, K)) for i in range(2)]
    X = [dev(synth.layer_case(90 + i, M, K, 8)[0]) for i in range(2)]
    dY = [dev(normal([14, i], M, N, 0.05)) for i in range(2)]

    def step(i):
        return (B.w4_gemm_fused(X[i], *w[i], activation=B.ACT_SILU), B.w4_gemm_gated(X[i], w[i], w[1 - i]),
                B.w4_gemm_dx(dY[i], *w[i], dY2=dY[i], weights2=w[1 - i]))

    want = [step(0), step(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    ok()


def test_compiled_and_plain_binding_agree():
    """The binding's compiled usual case and its Python (taken with an explicit stream, parameters or a
    list of weights) give the same results and refuse the same arguments."""
    M, N, K = 5, 264, 512
    X = dev(synth.layer_case(92, M, K, 8)[0])
    a, b = dlayer(layer(92, N, K)), dlayer(layer(93, N, K))
    dY, G = dev(normal(15, M, N, 0.05)), dev(normal(16, M, K, 1.0))
    here = torch.cuda.current_stream()
    calls = [
        lambda **k: B.w4_gemm_fused(X, *a, bias=dY[0].contiguous(), activation=B.ACT_RELU, residual=dY, save_pre=True, **k),
        lambda **k: B.w4_gemm_gated(X, a, b, save_pre=True, **k),
        lambda **k: (B.w4_gemm_dx(dY, *a, dY2=dY, weights2=b, **k),),
        lambda **k: B.w4_gemm_dx_gated(dY, *a, G, G, **k),
        lambda **k: B.w4_act_backward(dY, dY, bias_grad=True, **k),
        lambda **k: B.w4_act_backward(dY, dY, U=dY, **k),
    ]
    for f in calls:
        assert all(torch.equal(x, y) for x, y in zip(f(), f(stream=here)))
    assert torch.equal(B.w4_gemm_gated(X, a, b), B.w4_gemm_gated(torch.nn.Parameter(X), list(a), b))
    for bad in (lambda: B.w4_gemm_fused(X, *a, bias=dY), lambda: B.w4_gemm_fused(X[:, ::2], *a),
                lambda: B.w4_gemm_fused(X, *a, residual=G), lambda: B.w4_gemm_fused(X, *a, out=G),
                lambda: B.w4_gemm_gated(X, a, (b[0], b[1], b[2].cpu())), lambda: B.w4_gemm_dx(dY, *a, dY2=dY),
                lambda: B.w4_gemm_dx_gated(dY, *a, G, G[:, :256]), lambda: B.w4_act_backward(dY, G),
                lambda: B.w4_gemm_fused(X, *a, workspace=torch.empty(4))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.w4_gemm_fused(X.float(), *a), lambda: B.w4_gemm_fused(X, a[0], a[1].float(), a[2]),
                lambda: B.w4_act_backward(dY, dY.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: B.w4_gemm_fused(X, *a, activation=9), lambda: B.w4_gemm_fused(X, *a, flags=3),
                lambda: B.w4_act_backward(dY, dY, U=dY, bias_grad=True),
                lambda: B.w4_act_backward(dY, None, activation=B.ACT_SILU)):
        with pytest.raises(B.W4Error):
            bad()
    ok()


def test_static_weights_chain():
    """W4_FLAG_WEIGHTS_STATIC: back-to-back dependent launches give the same bits."""
    D, Fi = 4096, 11008
    g, u, d = (dlayer(layer(82 + i, *s)) for i, s in enumerate(((Fi, D), (Fi, D), (D, Fi))))
    for M in (1, 4, 16, 40):
        X = dev(synth.layer_case(82, M, D, 8)[0])

        def chain(flags):
            x = X
            for _ in range(3):
                # each block reads X, so that the values stay within fp16; x is handed on as the residual
                x = B.w4_gemm_fused(B.w4_gemm_gated(X, g, u, flags=flags), *d, residual=x, flags=flags)
            return x

        plain = chain(0)
        assert bool(torch.isfinite(plain).all())
        assert torch.equal(plain, chain(B.FLAG_WEIGHTS_STATIC)), M
    ok()


@pytest.mark.parametrize("M", [1, 5])
def test_gradients_against_differences(M):
    """The GPU's input gradients against central differences of the 64-bit block's loss."""
    D, Fi = 128, 256
    g, u, d = layer(85, Fi, D), layer(86, Fi, D), layer(87, D, Fi)
    x, c = synth.layer_case(85, M, D, 8)[0], normal(13, M, D, 0.5)
    H, G, U = B.w4_gemm_gated(dev(x), dlayer(g), dlayer(u), save_pre=True)
    dG, dU = B.w4_gemm_dx_gated(dev(c), *dlayer(d), G, U)
    dX = B.w4_gemm_dx(dG, *dlayer(g), dY2=dU, weights2=dlayer(u)).cpu().numpy().astype(np.float64)
    ok()

    def loss(v):
        return float(np.sum(c.astype(np.float64) * F.fused(F.gated(v, g, u)[0], d)[0]))

    x64, h, diff = x.astype(np.float64), 1e-4, np.zeros((M, D))
    for m in range(M):
        for k in range(0, D, 5):
            e = np.zeros_like(x64)
            e[m, k] = h
            diff[m, k] = (loss(x64 + e) - loss(x64 - e)) / (2 * h)
    # G, U, dG and dU rounded to fp16: a few half steps of the gradient's rms, as a 2-norm
    err = (dX - diff)[:, ::5]
    assert np.linalg.norm(err) <= 4 * HALF * np.linalg.norm(diff[:, ::5])


@pytest.mark.parametrize("M", [1, 6, 40, 300])
def test_launches_wait_for_whatever_precedes_them(M):
    """Each call directly behind the work that makes its inputs -- the quantisation of its weights, a copy,
    a memset, a long kernel, another stream's joined work -- eagerly and captured: the bits of calls with a
    synchronisation before each."""
    N, K = 512, 1024
    W0, W1 = (dev(normal([17, i], N, K, 0.03)) for i in range(2))
    X0, dY0, G0 = dev(normal(18, M, K, 1.0)), dev(normal(19, M, N, 0.05)), dev(normal(20, M, K, 1.0))
    long = dev(normal(21, 2048, 2048, 0.01))
    side = torch.cuda.Stream()

    def step(between):
        out = []
        layers = []
        for W in (W0, W1):
            Wc = W.clone()
            between()
            layers.append(B.w4_quantize_pack(Wc))
        X, dY, G = torch.empty_like(X0), torch.empty_like(dY0), torch.zeros_like(G0)
        between()
        out.append(B.w4_gemm_fused(X.copy_(X0), *layers[0], activation=B.ACT_SILU))  # behind a copy
        between()
        out.append(B.w4_gemm_gated(X.zero_(), *layers, save_pre=True)[1])  # behind a memset
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.mm(long, long)
            dY.copy_(dY0)
        torch.mm(long, long)
        here.wait_stream(side)  # two predecessors
        between()
        out.append(B.w4_gemm_dx(dY, *layers[0], dY2=dY, weights2=layers[1]))
        between()
        out.append(B.w4_gemm_dx_gated(dY, *layers[0], G.copy_(G0), G)[0])
        between()
        out += B.w4_act_backward(out[0], out[0], bias_grad=True)
        between()
        out.append(B.w4_gemm_fused(X.copy_(X0), *layers[1], residual=out[0], out=torch.empty_like(out[0])))
        return out

    want = step(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, step(lambda: None)))
    graph, main = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=main):
        got = step(lambda: None)
    for _ in range(3):
        for t in got:
            t.fill_(7.0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    ok()


@pytest.mark.parametrize("M,N,K", [(9, 11008, 2176), (33, 11008, 4096), (40, 10000, 1152), (64, 5504, 7552), (24, 20000, 1024)])
def test_tiles_cut_into_equal_shares(M, N, K):
    """Small batches whose tiles do not fill whole waves: shares that end inside tiles, odd group counts."""
    fused_case(M, N, K, "gelu", True, True, True)
    gated_case(M, N // 16 * 8, K, "silu", True)
    ok()
