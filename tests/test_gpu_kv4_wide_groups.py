"""A token whose query heads share a key head fills up to 64 rows, and takes the kernel
for few rows as every token does, with its two terms of a probability."""
import pytest
import torch

from kv4_util import Step
from test_gpu_kv4_attention import room
from test_gpu_kv4_precision import TWO

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("G,heads", [(33, 1), (40, 2), (64, 1)])
def test_one_token(G, heads, D):
    kv = [1, 2, 17, 64, 129, 300]
    Step(kv, [1] * len(kv), G * heads, heads, D, 16, seed=G, q_sd=0.3, width=room(16, True)).check(f"groups of {G}, D={D}", p_round=TWO)


@pytest.mark.parametrize("G", [33, 64])
def test_tokens_beside_a_prompt(G):
    """... and beside requests that take the kernel for many rows."""
    kv, fresh = [300, 90, 1, 40, 2000], [1, 90, 1, 3, 1]
    s = Step(kv, fresh, G, 1, 128, 16, seed=G, q_sd=0.3, width=room(16, True))
    y = s.check(f"groups of {G} beside a prompt")
    one = Step(kv, fresh, G, 1, 128, 16, seed=G, q_sd=0.3)
    s2 = one.run(max_fresh=0)                             # (the kernel for few rows alone)
    for b in (0, 2, 4):
        t = int(s.q_start[b])
        off = (y[t].double() - s2[t].double()).abs()
        # two roundings to bf16, of values that are 2^-13 apart at most: 2^-17 each, |v| <= 6
        assert bool((off <= 2.1 * 2.0 ** -8 * s2[t].double().abs() + 2.0 ** -13).all()), (b, float(off.max()))
    assert torch.isfinite(y).all()
