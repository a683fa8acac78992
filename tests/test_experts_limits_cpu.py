"""Sizes that spear_w4_experts takes: those that its header states, and the
workspace query answers for the same ones (no GPU)."""
import ctypes

import pytest

from quantized_gemm_w4a16_amd import spear as sp

A = 0x10000            # fake, aligned device address: never dereferenced
E_SHAPE, E_WS = -2, -5


def status(M, topk, E, K, I, N, glu=1):
    """The call with a workspace that is too small: E_WS if the sizes are taken."""
    s = sp._Experts(A, A, None, None, A, A, None, None, K, I, N, E, 2, glu)
    return sp.load().spear_w4_experts(A, M, ctypes.byref(s), A, A, topk, None, A, A, 256, None)


MOST = 1 << 25


@pytest.mark.parametrize("M,topk,E,K,I,N", [
    (1 << 19, 8, 64, 4096, 8192, 4096), (1 << 30, 1, 1, 32, 32, 1), (1 << 25, 32, 512, 32, 32, 64),
    (1 << 27, 8, 128, 7168, 4096, 7168), (1, 1, 1, 32, MOST, 1), (1, 1, 1, 32, 32, MOST), (4096, 8, 512, 32, MOST, MOST),
    (1, 1, 1, 1 << 31, 32, 1)])
def test_sizes_of_the_header_are_taken(M, topk, E, K, I, N):
    assert sp.spear_w4_experts_workspace_size(M, topk, E, I, N) > 0
    for glu in (0, 1):
        assert status(M, topk, E, K, I, N, glu) == E_WS


@pytest.mark.parametrize("M,topk,E,K,I,N", [
    ((1 << 30) + 1, 1, 1, 32, 32, 1), ((1 << 25) + 1, 32, 512, 32, 32, 64), (1, 1, 1, 32, MOST + 32, 1),
    (1, 1, 1, 32, 32, MOST + 1), (1, 1, 1, 32, 48, 64)])
def test_sizes_beyond_are_refused_by_both(M, topk, E, K, I, N):
    assert sp.spear_w4_experts_workspace_size(M, topk, E, I, N) == 0
    for glu in (0, 1):
        assert status(M, topk, E, K, I, N, glu) == E_SHAPE
