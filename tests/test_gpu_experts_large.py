"""Products over so many row tiles that they take several launches."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from test_gpu_epilogue import bf16, to64
from test_gpu_experts import w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,E,K,I,N,glu", [(300000, 8, 32, 32, 28704, True), (1 << 20, 1, 32, 16544, 40, True)])
def test_more_blocks_than_a_launch(M, E, K, I, N, glu):
    """64-row tiles over wide outputs (second product), 128-row tiles over wide
    inner layers (first product): tokens of the first, middle and last tiles
    against the reference, every row finite."""
    rng = np.random.default_rng(N)
    (uc, us, uz), up = w4(rng, E, 2 * I if glu else I, K)
    (dc, ds, dz), down = w4(rng, E, N, I)
    some = np.unique(np.concatenate([np.arange(40), M // 2 + np.arange(40), M - 40 + np.arange(40),
                                     rng.integers(0, M, 60)]))
    base, base64 = bf16(rng.normal(0, 1, (997, K)))
    x = base[torch.arange(M, device="cuda") % 997].contiguous()
    ids = torch.from_numpy(rng.integers(0, E, (M, 1)).astype(np.int32)).cuda()
    weights = torch.rand(M, 1, device="cuda")
    y = sp.spear_w4_experts(x, sp.Experts(*up, *down, glu=glu), ids, weights)
    pick = torch.from_numpy(some).cuda()
    ref, err = ref64.experts(base64[some % 997], (uc, us, uz), (dc, ds, dz), ids[pick].cpu().numpy(),
                             weights[pick].cpu().numpy(), ref64.SILU, glu)
    tol = ref64.rounded(ref, err, ref64.HALF_BF16)
    worst = float(np.max(np.abs(to64(y[pick]) - ref) / tol))
    print(f"[experts] M={M} N={N} I={I}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0
    # rows of the same token and expert are the same but for their weight
    for i in range(0, M, 1 << 16):
        assert bool(torch.isfinite(y[i: i + (1 << 16)]).all())
