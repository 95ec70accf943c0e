"""Edges of the feed-forward entry points that need no GPU: every call is a no-op or is refused before
anything is enqueued."""
import ctypes

import pytest
import torch

from weight_only_int4_06_b200 import w4a16 as B

P = ctypes.c_void_p
GOOD = P(1 << 20)  # never dereferenced
OK, NULL = 0, 1


@pytest.fixture(scope="module")
def L():
    return B.lib()


# What torch hands over for a pair of layers of these sizes: the address of an empty tensor is null.
@pytest.mark.parametrize("M,N,K", [(0, 16, 256), (4, 16, 0), (0, 16, 0), (0, 0, 256), (4, 0, 0), (0, 0, 0)])
def test_input_gradient_of_an_empty_pair(L, M, N, K):
    ptr = lambda *s: GOOD if all(s) else None
    y, layer = ptr(M, N), (ptr(N, K), ptr(N, K), ptr(N, K))
    assert L.w4_gemm_dx(y, M, N, K, *layer, None, None, None, None, 128, ptr(M, K), None, 0, None) == OK
    assert L.w4_gemm_dx(y, M, N, K, *layer, y, *layer, 128, ptr(M, K), None, 0, None) == OK
    # arrays without elements may have any address
    assert L.w4_gemm_dx(GOOD, M, N, K, GOOD, GOOD, GOOD, None, GOOD, None, GOOD, 128, GOOD, None, 0, None) == OK


def test_input_gradient_of_a_pair_given_in_part(L):
    """With something to compute the second layer is whole or absent."""
    second = [GOOD] * 4
    for i in range(4):
        part = second[:i] + [None] + second[i + 1:]
        for s in (part, [GOOD if p is None else None for p in part]):
            assert L.w4_gemm_dx(GOOD, 4, 16, 256, GOOD, GOOD, GOOD, *s, 128, GOOD, GOOD, 1 << 40, None) == NULL


def test_workspace_size_is_that_of_the_call_at_hand(monkeypatch):
    """The plans depend on the current device's SM count: a size found on one device is not kept for another."""
    sizes = iter((0, 4096, 64))

    class Lib:
        @staticmethod
        def w4_gemm_fused_workspace_size(M, N, K, group, out):
            out._obj.value = next(sizes)
            return OK

    monkeypatch.setattr(B, "lib", lambda: Lib)
    like = torch.empty(0, dtype=torch.float16)
    for need in (0, 4096, 64):
        address, have, tensor = B._ffn_workspace("w4_gemm_fused_workspace_size", (4, 16, 256, 128), None, like)
        assert have == need and (tensor is None) == (need == 0)
