"""Keys and values at the top of the range: held at 6 * 2^125, never as NaN."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import bf16, to64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
@pytest.mark.parametrize("m", [1.0, 1.5, 2.0 ** 60])
def test_rotated_keys_beyond_fp32(layout, m):
    """Two channels of 3e38 turned by 45 degrees make 4.2e38."""
    T, heads, D, P = 60, 2, 128, 16
    rng = np.random.default_rng(1)
    k, k64 = bf16(np.where(rng.random((T, heads, D)) < 0.5, 1.0, -1.0) * rng.choice([3e38, 3.38e38, 1e38, 2.0 ** -20], (T, heads, D)))
    f = sp.spear_rope_frequencies(D)
    f[7] = np.pi / 4
    pos = rng.integers(0, 1 << 16, T).astype(np.int32)
    pos[:20] = 1
    turned = ref_kv4.rotate(k64, pos, f.numpy(), layout, m)
    assert (np.abs(turned) > np.finfo(np.float32).max).any() and np.isfinite(turned).all()
    slots = np.arange(T, dtype=np.int64)
    cache = ref_kv4.Cache(-(-T // P), heads, D, P, rng)
    kv = sp.KV4(*(dev(a[n].copy()) for n in "kv" for a in (cache.codes, cache.scales)))
    sp.spear_rope_kv4_write(k, k, k, dev(pos), dev(slots), sp.Rope(f.cuda(), layout, m), kv)
    cache.write("k", slots, turned)
    cache.write("v", slots, k64)
    gk, gv = sp.spear_kv4_read(kv, dev(slots))
    assert bool(torch.isfinite(gk).all()) and bool(torch.isfinite(gv).all())
    assert np.array_equal(to64(gk), cache.read("k", slots)) and np.array_equal(to64(gv), cache.read("v", slots))
    for name, codes, scales in (("k", kv.k_codes, kv.k_scales), ("v", kv.v_codes, kv.v_scales)):
        assert np.array_equal(scales.cpu().numpy(), cache.scales[name]) and np.array_equal(codes.cpu().numpy(), cache.codes[name])


def test_an_infinite_key_is_still_nan():
    """An infinity that is rotated is none that a sum made: its blocks read NaN."""
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 5] = float("inf")
    kv = sp.new_kv4(1, 1, 64, 16)
    slots = dev(np.arange(2))
    sp.spear_rope_kv4_write(x, x, x, dev(np.array([3, 3], np.int32)), slots, sp.Rope(sp.spear_rope_frequencies(32).cuda()), kv)
    k, v = sp.spear_kv4_read(kv, slots)
    for t in (k, v):
        assert bool(t[0, 0, :32].isnan().all()) and bool(torch.isfinite(t[0, 0, 32:]).all()) and bool(torch.isfinite(t[1]).all())
