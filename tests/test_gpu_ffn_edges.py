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
