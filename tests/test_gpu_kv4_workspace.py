"""Attention on a workspace of which only the counters were zeroed."""
import pytest
import torch

from quantized_gemm_w4a16_amd import spear as sp
from kv4_util import Step
from test_gpu_kv4_attention import room

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_what_lies_behind_the_counters_does_not_count(D):
    """Chunks of both kernels, joined in the kernel, by groups and by a launch."""
    for s in (Step([6000, 40], [1, 1], 8, 1, D, 64, seed=D), Step([700, 90, 2500], [1, 3, 1], 6, 2, D, 16, seed=D),
              Step([3000, 900], [70, 2], 2, 1, D, 16, seed=D, width=room(16, True))):
        n = sp.spear_kv4_attention_workspace_size(s.T, len(s.kv), max(s.fresh), s.Hq, s.heads, D, s.width, s.P)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")           # NaN, were it read
        ws[: sp.KV4_COUNTER_BYTES] = 0
        s.check(f"workspace of anything, D={D}", workspace=ws)
        s.check(f"the same once more, D={D}", workspace=ws)
        assert not ws[: sp.KV4_COUNTER_BYTES].any()
