"""Rotation: the error's bound channel by channel, with factors of all sizes."""
import numpy as np
import pytest

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import bf16
from rope_util import check_rotated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
@pytest.mark.parametrize("m", [0.0, 1.0, -1.25, 1e4, 2.0 ** 100, -2.0 ** -100, 3e-7])
def test_bound_of_every_channel(m, layout):
    """Channels of sizes far apart in one head, and angles next to a quarter turn, where
    y is small beside its terms."""
    T, H, D, rot = 300, 5, 128, 112
    rng = np.random.default_rng(7)
    x, x64 = bf16(rng.normal(0, 1, (T, H, D)) * np.exp2(rng.integers(-60, 20, (T, H, D))))
    f = sp.spear_rope_frequencies(rot)
    f[3], f[11], f[12] = np.pi / 2, np.pi / 4, np.pi
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[:40] = np.arange(40)
    want = ref_kv4.rotate(x64, pos, f.numpy(), layout, m)
    rope = sp.Rope(f.cuda(), layout, m)
    worst = check_rotated(sp.spear_rope(x, dev(pos), rope), want, x64, rot // 2, layout, m)
    kv = sp.new_kv4(-(-T // 16), 1, D, 16)
    k = x[:, :1].contiguous()
    check_rotated(sp.spear_rope_kv4_write(x, k, k, dev(pos), dev(np.arange(T)), rope, kv), want, x64, rot // 2, layout, m)
    print(f"[rope] factor {m}: worst {worst:.3f} of the bound", flush=True)


def test_smallest_channels():
    """Channels below fp32's smallest normal number."""
    rng = np.random.default_rng(8)
    x, x64 = bf16(rng.integers(-200, 200, (64, 4, 64)) * 2.0 ** -133)
    f = sp.spear_rope_frequencies(64)
    pos = rng.integers(0, 1 << 10, 64).astype(np.int32)
    for m in (1.0, 0.25, 64.0):
        want = ref_kv4.rotate(x64, pos, f.numpy(), 0, m)
        check_rotated(sp.spear_rope(x, dev(pos), sp.Rope(f.cuda(), 0, m)), want, x64, 32, 0, m)
