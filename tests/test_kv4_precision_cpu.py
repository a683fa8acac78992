"""What a bound of 2^-17 for the probabilities sees: planted in the reference, one
bf16 in place of two fails it (CPU only)."""
import numpy as np
import pytest
import torch

import ref_kv4


def rounded(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()


def with_probabilities(q, cache, slots, scale, held):
    """One token on the cached keys, fp64 but for the probabilities, which are held as `held` has them."""
    k, v = cache.read("k", slots), cache.read("v", slots)
    G = q.shape[0] // cache.heads
    y = np.zeros(q.shape)
    for h in range(q.shape[0]):
        z = scale * (k[:, h // G] @ q[h])
        p = np.exp(z - z.max())
        y[h] = held(p) @ v[:, h // G] / p.sum()
    return y


@pytest.mark.parametrize("D,Hq,heads,n", [(64, 8, 8, 33), (128, 8, 2, 65), (128, 16, 1, 300), (256, 4, 1, 129)])
def test_one_bf16_is_seen_and_two_are_not(D, Hq, heads, n):
    rng = np.random.default_rng(n)
    cache = ref_kv4.Cache(-(-n // 16), heads, D, 16, rng)
    slots = np.arange(n)
    for name in "kv":
        cache.write(name, slots, rng.normal(0, 1, (n, heads, D)))
    q = rounded(rng.normal(0, 0.3, (Hq, D)))
    scale = D ** -0.5
    want, err, _, _ = ref_kv4.attention(q[None], cache, np.arange(-(-n // 16))[None], [0, 1], [n], scale, p_round=2.0 ** -17)
    tol = err + ref_kv4.HALF_BF16 * (np.abs(want) + err)

    def share(held):
        return float((np.abs(rounded(with_probabilities(q, cache, slots, scale, held)) - want[0]) / tol[0]).max())

    def two(p):
        hi = rounded(p)
        return hi + rounded(p - hi)

    p = np.exp(-rng.random(1 << 16) * 40)
    assert np.max(np.abs(two(p) - p) / p) <= 2.0 ** -17 and 2.0 ** -9 < np.max(np.abs(rounded(p) - p) / p) <= 2.0 ** -8
    assert share(two) <= 1.0
    assert share(rounded) > 1.5, share(rounded)
    assert share(lambda p: rounded(p) + rounded(p - rounded(p))[::-1]) > 1.5     # the low terms in another order
