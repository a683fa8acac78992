"""Layers of fewer than 128 input channels through the MFMA GEMM, whose stages
are 128 deep."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from test_gpu_epilogue import Case, check
from test_gpu_experts import Case as Experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [32, 64, 96, 160])
@pytest.mark.parametrize("M", [20, 150])
@pytest.mark.parametrize("r", [0, 16])
def test_prefill_paths(K, M, r):
    c = Case(M, 70, K, r, 0, K + M, False, True, False, sp.OUT_F32)
    ref, tol = c.reference(ref64.SILU)
    for path in (sp.PATH_AUTO, sp.PATH_PREFILL_LARGE):
        y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_SILU), c.ec, path=path)
        check(y, ref, tol, f"K={K} M={M} r={r} path={path}")


@pytest.mark.parametrize("K", [32, 64, 96])
def test_weights_that_fill_an_allocation(K):
    """Weights of an allocation of their own: the first rows have nothing before
    them."""
    N, M = (24 << 20) // (K // 2) // 64 * 64, 17
    c = Case(M, 128, K, 0, 0, K, False, False, False, sp.OUT_F32)
    packed = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(N, device="cuda")
    packed[:64], packed[-64:] = c.w.packed[:64], c.w.packed[64:]
    scales[:64], scales[-64:] = c.w.scales[:64], c.w.scales[64:]
    zeros = torch.full((N,), 8, dtype=torch.uint8, device="cuda")
    zeros[:64], zeros[-64:] = c.w.zeros[:64], c.w.zeros[64:]
    ref, tol = c.reference(ref64.NONE)
    for path in (sp.PATH_PREFILL, sp.PATH_PREFILL_LARGE):
        y = sp.spear_w4_linear(c.x, sp.W4(packed, scales, zeros, N, K), path=path)
        check(torch.cat((y[:, :64], y[:, -64:]), 1), ref, tol, f"K={K} path={path}")


@pytest.mark.parametrize("K,I", [(32, 32), (96, 64)])
def test_experts_in_tiles_of_128_rows(K, I):
    c = Experts(41000 // (I // 32), 1, 1, K, I, 72, bias=True, seed=K, ids=None)
    c.check(c.run(), f"K={K} I={I}")
