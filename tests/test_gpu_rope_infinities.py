"""Infinities, NaN and the largest numbers among the rotated channels: what
m (x_a cos t - x_b sin t) and m (x_b cos t + x_a sin t) give for them."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import bf16
from rope_util import check_rotated

pytestmark = pytest.mark.gpu
INF = np.inf


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (256, 22), (24, 24)])
@pytest.mark.parametrize("scale", [1.0, -1.25])
def test_infinite_channels(D, rot, layout, scale):
    rng = np.random.default_rng(D + rot)
    pos = np.array([0, 0, 1, 2, 3, 1000, 1 << 20, 7], np.int32)
    T, H = len(pos), 9
    a = rng.normal(0, 1, (T, H, D))
    for h, special in enumerate((INF, -INF, np.nan, 3e38)):
        for t in range(T):
            for c in rng.permutation(D)[:6]:
                a[t, h, c] = special
    a[:, 4] = np.where(rng.random((T, D)) < 0.5, INF, -INF)
    a[:, 5, ::3] = INF
    a[:, 6, 1::3] = -INF
    x, x64 = bf16(a)
    f = sp.spear_rope_frequencies(rot)
    rope = sp.Rope(f.cuda(), layout, scale)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref_kv4.rotate(x64, pos, f.numpy(), layout, scale)
    assert np.isinf(want).any() and np.isnan(want).any()
    check_rotated(sp.spear_rope(x, dev(pos), rope), want, x64, rot // 2, layout, scale)
    if D % 32 == 0:
        kv = sp.new_kv4(1, 1, D, 16)
        k = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
        q = sp.spear_rope_kv4_write(x, k, k, dev(pos), dev(np.arange(T)), rope, kv)
        check_rotated(q, want, x64, rot // 2, layout, scale)


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
def test_an_infinity_at_position_0_stays_one(layout):
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3] = float("inf")
    y = sp.spear_rope(x, dev(np.zeros(1, np.int32)), sp.Rope(sp.spear_rope_frequencies(64).cuda(), layout))
    assert y[0, 0, 3] == float("inf")


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
def test_sums_that_pass_the_largest_number_on_their_way(layout):
    """Products beyond fp32 whose difference is not, and rotated values beyond bf16."""
    T, D = 50, 64
    rng = np.random.default_rng(5)
    x, x64 = bf16(np.where(rng.random((T, 3, D)) < 0.5, 1.0, -1.0) * rng.choice([3e38, 2.5e38, 1.0], (T, 3, D)))
    pos = rng.integers(0, 1 << 16, T).astype(np.int32)
    f = sp.spear_rope_frequencies(D)
    f[5], f[9] = np.pi / 4, -np.pi / 4                    # (position 1: cosine and sine alike)
    pos[:10] = 1
    for m in (1.0, 2.0, 2.0 ** 20, 2.0 ** -20):
        want = ref_kv4.rotate(x64, pos, f.numpy(), layout, m)
        check_rotated(sp.spear_rope(x, dev(pos), sp.Rope(f.cuda(), layout, m)), want, x64, D // 2, layout, m)
