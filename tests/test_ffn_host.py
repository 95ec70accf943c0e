"""The feed-forward entry points refuse bad arguments on the host (CPU only: every call is rejected
before anything is enqueued, or is a no-op)."""
import ctypes

import pytest
import torch

from weight_only_int4_06_b200 import w4a16 as B

P = ctypes.c_void_p
GOOD = P(1 << 20)        # never dereferenced
BAD = P((1 << 20) + 2)
BIG = 1 << 40
OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def L():
    return B.lib()


def fused(L, **k):
    g = lambda n, d: k.get(n, d)
    return L.w4_gemm_fused(g("X", GOOD), g("M", 4), g("N", 16), g("K", 256), g("packed", GOOD), g("scales", GOOD),
                           g("zeros", GOOD), g("group", 128), g("bias", None), g("act", 0), g("residual", None),
                           g("Y", GOOD), g("Z", None), g("ws", GOOD), g("ws_bytes", BIG), g("flags", 0), None)


def gated(L, **k):
    g = lambda n, d: k.get(n, d)
    return L.w4_gemm_gated(g("X", GOOD), g("M", 4), g("N", 16), g("K", 256), g("gp", GOOD), g("gs", GOOD), g("gz", GOOD),
                           g("up", GOOD), g("us", GOOD), g("uz", GOOD), g("group", 128), g("act", 4), g("H", GOOD),
                           g("G", None), g("U", None), g("ws", GOOD), g("ws_bytes", BIG), g("flags", 0), None)


def dx(L, **k):
    g = lambda n, d: k.get(n, d)
    return L.w4_gemm_dx(g("dY", GOOD), g("M", 4), g("N", 16), g("K", 256), g("p", GOOD), g("s", GOOD), g("z", GOOD),
                        g("dY2", None), g("p2", None), g("s2", None), g("z2", None), g("group", 128), g("dX", GOOD),
                        g("ws", GOOD), g("ws_bytes", BIG), None)


def dx_gated(L, **k):
    g = lambda n, d: k.get(n, d)
    return L.w4_gemm_dx_gated(g("dY", GOOD), g("M", 4), g("N", 16), g("K", 256), g("p", GOOD), g("s", GOOD), g("z", GOOD),
                              g("group", 128), g("G", GOOD), g("U", GOOD), g("act", 4), g("dG", GOOD), g("dU", GOOD),
                              g("ws", GOOD), g("ws_bytes", BIG), None)


def act_backward(L, **k):
    g = lambda n, d: k.get(n, d)
    return L.w4_act_backward(g("dY", GOOD), g("Z", GOOD), g("U", None), g("M", 4), g("N", 16), g("act", 4),
                             g("dZ", GOOD), g("dU", None), g("dbias", None), g("ws", GOOD), g("ws_bytes", BIG), None)


@pytest.mark.parametrize("call", (fused, gated, dx, dx_gated))
def test_shapes_and_groups(L, call):
    assert call(L, group=64) == UNSUPPORTED
    assert call(L, K=200) == SHAPE
    assert call(L, N=12) == SHAPE
    assert call(L, M=-1) == SHAPE
    assert call(L, N=1 << 31) == SHAPE
    assert call(L, M=(1 << 31) - 1, N=(1 << 31) - 8) == SHAPE  # over 2^40 elements
    assert call(L, M=0) == OK                                   # nothing to write


def test_fused_refusals(L):
    assert fused(L, N=0) == OK
    for n in ("X", "packed", "scales", "zeros", "Y"):
        assert fused(L, **{n: None}) == NULL, n
    for n in ("X", "packed", "Y", "Z", "bias", "residual"):
        assert fused(L, **{n: BAD}) == ALIGN, n
    assert fused(L, act=5) == UNSUPPORTED
    assert fused(L, act=-1) == UNSUPPORTED
    assert fused(L, flags=1) == UNSUPPORTED
    assert fused(L, flags=-1) == UNSUPPORTED


def test_gated_refusals(L):
    assert gated(L, N=0) == OK
    for n in ("X", "gp", "gs", "gz", "up", "us", "uz", "H"):
        assert gated(L, **{n: None}) == NULL, n
    assert gated(L, G=GOOD) == NULL and gated(L, U=GOOD) == NULL  # both or neither
    for n in ("X", "gp", "up", "H"):
        assert gated(L, **{n: BAD}) == ALIGN, n
    assert gated(L, G=BAD, U=GOOD) == ALIGN and gated(L, G=GOOD, U=BAD) == ALIGN
    assert gated(L, act=5) == UNSUPPORTED
    assert gated(L, flags=2) == UNSUPPORTED


def test_dx_refusals(L):
    assert dx(L, K=0) == OK
    for n in ("dY", "p", "s", "z", "dX"):
        assert dx(L, **{n: None}) == NULL, n
    two = dict(dY2=GOOD, p2=GOOD, s2=GOOD, z2=GOOD)
    for n in two:
        assert dx(L, **{**two, n: None}) == NULL, n     # the second layer in part
        assert dx(L, **{n: GOOD}) == NULL, n
    for n in ("dY", "p", "dX"):
        assert dx(L, **{n: BAD}) == ALIGN, n
    assert dx(L, **{**two, "dY2": BAD}) == ALIGN and dx(L, **{**two, "p2": BAD}) == ALIGN


def test_dx_gated_refusals(L):
    assert dx_gated(L, K=0) == OK
    for n in ("dY", "p", "s", "z", "G", "U", "dG", "dU"):
        assert dx_gated(L, **{n: None}) == NULL, n
    for n in ("dY", "p", "G", "U", "dG", "dU"):
        assert dx_gated(L, **{n: BAD}) == ALIGN, n
    assert dx_gated(L, act=9) == UNSUPPORTED


def test_act_backward_refusals(L):
    assert act_backward(L, M=0) == OK and act_backward(L, N=0) == OK
    assert act_backward(L, N=12) == SHAPE and act_backward(L, M=-1) == SHAPE
    assert act_backward(L, act=5) == UNSUPPORTED
    assert act_backward(L, U=GOOD, dU=GOOD, dbias=GOOD) == UNSUPPORTED
    for n in ("dY", "Z", "dZ"):
        assert act_backward(L, **{n: None}) == NULL, n
        assert act_backward(L, **{n: BAD}) == ALIGN, n
    assert act_backward(L, U=GOOD) == NULL and act_backward(L, dU=GOOD) == NULL
    assert act_backward(L, U=GOOD, dU=BAD) == ALIGN and act_backward(L, dbias=BAD) == ALIGN
    assert act_backward(L, dbias=GOOD, ws=None, ws_bytes=0) == WORKSPACE
    assert act_backward(L, dbias=GOOD, ws=BAD) == ALIGN
    assert act_backward(L, act=0, Z=None, dZ=None) == OK  # nothing asked for


def test_workspace_queries(L):
    n = ctypes.c_size_t(7)
    for f, dims in ((L.w4_gemm_fused_workspace_size, (4, 16, 256, 128)), (L.w4_gemm_gated_workspace_size, (4, 16, 256, 128)),
                    (L.w4_gemm_dx_workspace_size, (4, 16, 256, 2, 128)), (L.w4_act_backward_workspace_size, (4, 16))):
        assert f(*dims, ctypes.byref(n)) == OK
        assert f(*dims, None) == NULL
        assert f(-1, *dims[1:], ctypes.byref(n)) == SHAPE
    assert L.w4_gemm_dx_workspace_size(4, 16, 256, 3, 128, ctypes.byref(n)) == UNSUPPORTED
    assert L.w4_gemm_fused_workspace_size(4, 16, 256, 64, ctypes.byref(n)) == UNSUPPORTED


def _short_workspaces(L):
    """(call, dims) whose query asks for a workspace."""
    found = []
    for call, f, extra in ((fused, L.w4_gemm_fused_workspace_size, ()), (gated, L.w4_gemm_gated_workspace_size, ()),
                           (dx, L.w4_gemm_dx_workspace_size, (1,)), (dx_gated, L.w4_gemm_dx_workspace_size, (1,))):
        for M, N, K in ((1, 4096, 28672), (8, 4096, 28672), (32, 4096, 4096), (64, 512, 8192), (300, 1024, 4096)):
            n = ctypes.c_size_t(0)
            assert f(M, N, K, *extra, 128, ctypes.byref(n)) == OK
            if n.value:
                found.append((call, dict(M=M, N=N, K=K), n.value))
    return found


def test_short_missing_and_misaligned_workspaces(L):
    for call, dims, need in _short_workspaces(L):
        assert call(L, ws_bytes=need - 1, **dims) == WORKSPACE
        assert call(L, ws=None, **dims) == NULL
        assert call(L, ws=BAD, **dims) == ALIGN


# ------------------------------------------------------------------ the binding
H = torch.float16
X = torch.zeros(4, 256, dtype=H)
W = (torch.zeros(64, 32, dtype=torch.int32), torch.zeros(64, 2, dtype=H), torch.zeros(64, 2, dtype=torch.uint8))
Y = torch.zeros(4, 64, dtype=H)

HOST_CALLS = {
    "w4_gemm_fused": lambda: B.w4_gemm_fused(X, *W),
    "w4_gemm_gated": lambda: B.w4_gemm_gated(X, W, W),
    "w4_gemm_dx": lambda: B.w4_gemm_dx(Y, *W),
    "w4_gemm_dx_gated": lambda: B.w4_gemm_dx_gated(Y, *W, X, X),
    "w4_act_backward": lambda: B.w4_act_backward(Y, Y),
}


@pytest.mark.parametrize("name", sorted(HOST_CALLS))
def test_host_tensors_are_rejected(name):
    with pytest.raises(ValueError):
        HOST_CALLS[name]()


def test_argument_checks():
    dev = torch.device("cpu")
    with pytest.raises(TypeError):
        B._arg(X.float(), H, (4, 256), dev, "X")
    with pytest.raises(ValueError, match="shape"):
        B._arg(X, H, (4, 255), dev, "X")
    with pytest.raises(ValueError):
        B._matrix(torch.zeros(3), "X")
    with pytest.raises(ValueError):
        B._matrix(torch.zeros(2, 3, 4), "X")
