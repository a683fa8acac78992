"""How far a rotated channel in fp32 may be from fp64's, and the comparison."""
import numpy as np
import torch

import ref_kv4
from kv4_util import to64


def off(x, want, n, layout, m):
    """Bound of the error before the rounding to bf16, channel by channel: of a channel
    that is rotated with the factors m cos t and m sin t,
      2^-23 |y| + 2^-37 |m| (|x_a| + |x_b|) + 2^-147.
    A factor c is c0 + c1, c0 its first 16 bits: |c1| <= 2^-15 |c|, rounded to 2^-40 |c|.
    x c0 + p s0 is rounded once (2^-24 of it), the second terms' product and sum are
    rounded (2^-39 of the terms each), then the sum of both (2^-24 of y): with the terms
    |x c| + |p s| <= |m| (|x_a| + |x_b|), 2^-23 |y| + (2^-40 + 2^-39 + 2^-39 + 2^-39) of
    these.  Four results below fp32's smallest normal number are off by 2^-150 each."""
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == ref_kv4.HALF else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    e = np.zeros(x.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        e[..., a] = e[..., b] = abs(m) * 2.0 ** -37 * (np.abs(x[..., a]) + np.abs(x[..., b])) + 2.0 ** -147
        e[..., : 2 * n] += 2.0 ** -23 * np.abs(want[..., : 2 * n])
    return e


def check_rotated(got, want, x, n, layout, m):
    """NaN where the formula has it, infinities of the same sign (bf16's own overflow
    among them), the others within the bound and a rounding; -> the worst's share of it."""
    g = to64(got)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan)
    r = torch.from_numpy(np.clip(np.where(nan, 0.0, want), -1e300, 1e300)).bfloat16().double().numpy()
    inf = np.isinf(r)
    assert np.array_equal(g[~nan & inf], r[~nan & inf])
    fine = ~nan & ~inf
    before = off(x, want, n, layout, m)[fine]
    w = want[fine]
    tol = before + np.maximum(ref_kv4.HALF_BF16 * (np.abs(w) + before), 2.0 ** -134)
    err = np.abs(g[fine] - w)
    assert (err <= tol).all(), float((err / tol).max())
    return float((err / tol).max(initial=0.0))
