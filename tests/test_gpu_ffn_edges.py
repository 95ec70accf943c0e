"""Edges of the feed-forward operators on the GPU: empty batches and calls at the limits of their arguments."""
import numpy as np
import pytest
import torch

from weight_only_int4_06_b200 import w4a16 as B

pytestmark = pytest.mark.gpu


def ok():
    assert B.w4_check_device_status() == 0


def ones(*s):
    return torch.ones(*s, dtype=torch.float16, device="cuda")


def zero_layer(N, K):
    return (torch.zeros(N, K // 8, dtype=torch.int32, device="cuda"), ones(N, K // 128),
            torch.zeros(N, K // 128, dtype=torch.uint8, device="cuda"))


def halves():
    """The compiled half of the binding, then its Python half (an explicit stream)."""
    return {}, {"stream": torch.cuda.current_stream()}


@pytest.mark.parametrize("M,N,K", [(0, 16, 256), (3, 16, 0), (3, 0, 256), (0, 0, 256), (0, 16, 0)])
def test_input_gradient_of_an_empty_pair(M, N, K):
    for k in halves():
        dX = B.w4_gemm_dx(ones(M, N), *zero_layer(N, K), dY2=ones(M, N), weights2=zero_layer(N, K), out=ones(M, K), **k)
        assert dX.shape == (M, K) and not dX.any()
    ok()


@pytest.mark.parametrize("M,N", [(0, 16), (5, 0), (0, 0)])
def test_gated_activation_backward_of_an_empty_batch(M, N):
    """An empty U is still a U: a pair comes back, the outputs given are the ones returned, and it does not
    go with a bias gradient."""
    for k in halves():
        dG, dU = B.w4_act_backward(ones(M, N), ones(M, N), U=ones(M, N), **k)
        assert dG.shape == dU.shape == (M, N)
        out = ones(M, N), ones(M, N)
        got = B.w4_act_backward(ones(M, N), ones(M, N), U=ones(M, N), out=out, **k)
        assert got[0] is out[0] and got[1] is out[1]
        with pytest.raises(ValueError):
            B.w4_act_backward(ones(M, N), ones(M, N), U=ones(M, N), out=(out[0], ones(M + 1, N + 8)), **k)
        with pytest.raises(B.W4Error):
            B.w4_act_backward(ones(M, N), ones(M, N), U=ones(M, N), bias_grad=True, **k)
        dZ, db = B.w4_act_backward(ones(M, N), ones(M, N), bias_grad=True, **k)
        assert dZ.shape == (M, N) and db.shape == (N,) and not db.any()
    ok()


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 4, -2 ** 32, 2 ** 64, 2 ** 70, -2 ** 70])
def test_codes_beyond_an_int_are_refused(value):
    """activation, group and flags are C ints: a value whose low 32 bits are a valid code is still none."""
    N, K = 16, 128
    x, y, w = ones(2, K), ones(2, N), zero_layer(N, K)
    calls = [lambda **k: B.w4_gemm_fused(x, *w, activation=value, **k), lambda **k: B.w4_gemm_fused(x, *w, group=value + 128, **k),
             lambda **k: B.w4_gemm_fused(x, *w, flags=value, **k), lambda **k: B.w4_gemm_gated(x, w, w, activation=value, **k),
             lambda **k: B.w4_gemm_gated(x, w, w, group=value + 128, **k), lambda **k: B.w4_gemm_gated(x, w, w, flags=value, **k),
             lambda **k: B.w4_gemm_dx(y, *w, group=value + 128, **k),
             lambda **k: B.w4_gemm_dx_gated(y, *w, x, x, activation=value, **k),
             lambda **k: B.w4_gemm_dx_gated(y, *w, x, x, group=value + 128, **k),
             lambda **k: B.w4_act_backward(y, y, activation=value, **k)]
    for k in halves():
        for call in calls:
            with pytest.raises(B.W4Error):
                call(**k)
    assert torch.equal(B.w4_gemm_fused(x, *w, save_pre=2 ** 70)[1], B.w4_gemm_fused(x, *w))  # a truth value
    ok()


def test_null_stream_handle_is_the_default_stream():
    """A raw handle of 0 is the legacy default stream, as at the C entry points: the calls run behind the work
    queued there, and before the work queued after them."""
    N, K = 16, 128
    w = zero_layer(N, K)
    w[0].fill_(0x11111111)  # W = 1
    long = ones(4096, 4096) / 4096
    calls = [lambda x, y: B.w4_gemm_fused(x, *w, stream=0), lambda x, y: B.w4_gemm_gated(x, w, w, activation=B.ACT_NONE, stream=0),
             lambda x, y: B.w4_gemm_dx(y, *w, stream=0), lambda x, y: B.w4_gemm_dx_gated(y, *w, x, x, activation=B.ACT_NONE, stream=0)[0],
             lambda x, y: B.w4_act_backward(y, y, activation=B.ACT_NONE, stream=0), lambda x, y: B.w4_gemm(x, *w, stream=0)]
    for call, want in zip(calls, (1.5 * K, 2.25 * K * K, 1.5 * N, 2.25 * N, 1.5, 1.5 * K)):
        x, y = ones(2, K), ones(2, N)
        torch.cuda.synchronize()
        for _ in range(8):
            torch.mm(long, long)
        x.fill_(1.5)
        y.fill_(1.5)
        got = call(x, y)
        x.fill_(1)
        y.fill_(1)
        torch.cuda.synchronize()
        assert bool((got == want).all())
    ok()


def scaled_layer(N, K, code, zero, scale):
    """Every weight (code - zero) * scale."""
    w = zero_layer(N, K)
    w[0].fill_(int(np.array(code * 0x11111111, np.uint32).view(np.int32)))
    w[1].fill_(scale)
    w[2].fill_(zero)
    return w


# the largest weight that a code of the group can have: 15 * 4368 = 65520, 15 * 6000, 8 * 8192 are beyond fp16
@pytest.mark.parametrize("zero,scale", [(0, 4368.0), (15, 6000.0), (7, 8192.0), (8, 60000.0), (0, float("inf"))])
def test_weights_beyond_fp16_are_reported(zero, scale):
    """The input gradients round weights to fp16: a group whose weights may not fit is W4_ERR_RANGE, in any row,
    group and layer."""
    N, K, M = 264, 640, 5
    dY, X = ones(M, N), ones(M, K)
    good = scaled_layer(N, K, 1, 0, 1.0)
    for n, g in ((0, 0), (263, 4), (130, 3)):
        bad = [t.clone() for t in good]
        bad[1][n, g], bad[2][n, g] = scale, zero
        for call in (lambda: B.w4_gemm_dx(dY, *bad), lambda: B.w4_gemm_dx(dY, *good, dY2=dY, weights2=tuple(bad)),
                     lambda: B.w4_gemm_dx_gated(dY, *bad, X, X)):
            ok()
            call()
            assert B.STATUS_NAMES[B.w4_check_device_status()] == "W4_ERR_RANGE"
    ok()


@pytest.mark.parametrize("code,zero,scale", [(15, 0, 4364.0), (0, 15, 4364.0), (15, 7, 8184.0), (0, 8, 8184.0)])
def test_the_largest_weights_of_fp16_are_right(code, zero, scale):
    N, K, M = 264, 640, 5
    w, dY = scaled_layer(N, K, code, zero, scale), ones(M, N) / 4096
    want = (code - zero) * scale * N / 4096  # the weight rounds to fp16 (2^-11), the output too
    for got in (B.w4_gemm_dx(dY, *w), B.w4_gemm_dx_gated(dY, *w, ones(M, K), ones(M, K), activation=B.ACT_NONE)[0]):
        assert bool(((got.double() - want).abs() <= abs(want) * (2.0 ** -10 + 2.0 ** -20)).all())
    ok()


def test_identity_gate_has_derivative_one_everywhere():
    """Without an activation dG = dH U whatever G holds, as dZ = dY whatever Z holds."""
    M, N, K = 3, 264, 640
    w, dY, U = scaled_layer(N, K, 9, 8, 0.25), ones(M, N), ones(M, K) * 3
    G = ones(M, K)
    G[1, 5], G[2, 7], G[0, 9] = float("nan"), float("inf"), -float("inf")
    dG, dU = B.w4_gemm_dx_gated(dY, *w, G, U, activation=B.ACT_NONE)
    assert bool((dG == 3 * N / 4).all())
    assert torch.equal(torch.isnan(dU), torch.isnan(G)) and bool((dU[torch.isfinite(G)] == N / 4).all())
    dG, dU = B.w4_act_backward(U, G, U=U, activation=B.ACT_NONE)
    assert bool((dG == 9).all()) and torch.equal(torch.isnan(dU), torch.isnan(G))
    ok()
