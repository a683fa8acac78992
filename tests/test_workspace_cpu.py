"""Sizes of the linear's workspace, which callers keep (no GPU)."""
import pytest

from quantized_gemm_w4a16_amd import spear as sp


@pytest.mark.parametrize("M,N,K,r,size", [
    (1, 2048, 2048, 32, 4410368), (16, 16384, 2048, 32, 2313216), (16, 2048, 8192, 32, 7887872),
    (77, 1000, 4128, 16, 6859520), (401, 14336, 14336, 64, 50310144), (2048, 4096, 4096, 64, 41059072),
    (1, 64, 32, 8, 2247936), (16, 4096, 4096, 96, 12356608), (1, 2048, 2048, 0, 2105856)])
def test_sizes_stay(M, N, K, r, size):
    """A workspace of a size that was enough stays enough (ABI version 2)."""
    assert sp.spear_abi_version() == 2
    assert sp.spear_w4_linear_workspace_size(M, N, K, r) <= size


def test_the_static_scratch_still_serves():
    """Rank 64, 14336 x 14336, 401 tokens fits the allocation-free entry point."""
    assert sp.spear_w4_linear_workspace_size(401, 14336, 14336, 64) <= sp.NOALLOC_MAX_WORKSPACE
