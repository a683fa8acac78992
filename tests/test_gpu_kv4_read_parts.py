"""Keys or values of the cache read by themselves."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import to64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,heads,D", [(1, 1, 64), (700, 3, 96), (3000, 8, 128)])
def test_one_of_them(T, heads, D):
    rng = np.random.default_rng(T)
    cache = ref_kv4.Cache(20, heads, D, 16, rng)
    for a in cache.scales.values():
        a[a == 255] = 128
    kv = sp.KV4(*(dev(a[n]) for n in "kv" for a in (cache.codes, cache.scales)))
    slots = rng.integers(-2, 20 * 16 + 2, T).astype(np.int64)
    for i, part in enumerate("kv"):
        got = sp.spear_kv4_read(kv, dev(slots), parts=part)
        assert got[1 - i] is None and np.array_equal(to64(got[i]), cache.read(part, slots))
        own = torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda")
        got = sp.spear_kv4_read(kv, dev(slots), parts=part, **{part: own})
        assert got[i] is own and got[1 - i] is None and np.array_equal(to64(own), cache.read(part, slots))
