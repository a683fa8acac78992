"""Finite scores that pass fp32's range when they are scaled: the softmax is one of
the differences, which say which keys count."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from kv4_util import Step, bf16, to64
from test_gpu_kv4_attention import room

pytestmark = pytest.mark.gpu
FLT_MAX = float(np.finfo(np.float32).max)


def large_step(kv, fresh, Hq, heads, D, P, sign, seed, **kw):
    """Scores q . k of one product each, exact: a level times 2^125, 0 where it is 0."""
    s = Step(kv, fresh, Hq, heads, D, P, seed=seed, **kw)
    rng = np.random.default_rng(seed)
    q = np.zeros((s.T, Hq, D))
    q[..., 5] = sign * 2.0 ** 63
    s.q, s.q64 = bf16(q)
    for b, n in enumerate(kv):
        k = np.zeros((n, heads, D))
        k[..., 5] = rng.choice([0.0, 1.0, 3.0, 6.0], (n, heads), p=[0.1, 0.5, 0.3, 0.1]) * 2.0 ** 62
        if n > 10:
            k[: n // 2, :, 5] = np.minimum(k[: n // 2, :, 5], 2.0 ** 62)         # the largest come late
            if sign < 0:
                k[..., 5] = np.maximum(k[..., 5], 2.0 ** 61)                     # and no score is 0
        slots = s.table[b][np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        s.cache.write("k", slots, k)
    s.to_device()
    return s


def check_large(s, scale, window=0):
    y = to64(s.run(scale=scale, window=window))
    want, _, lse, _ = ref_kv4.attention(s.q64, s.cache, s.table, s.q_start, s.kv, scale, window)
    n = int(s.q_start[-1])
    assert np.isfinite(want[:n]).all()
    # equal weights: rounded once, behind a sum in fp32 and its quotient
    size = 6.0 * 2.0 ** -20
    worst = np.abs(y - want)[:n] - ref_kv4.HALF_BF16 * np.abs(want[:n]) - size
    assert worst.max() <= 0, worst.max()
    gl, empty = to64(s.lse)[:n], np.isneginf(lse[:n])
    assert np.array_equal(np.isneginf(gl) & (lse[:n] > -FLT_MAX), empty & (lse[:n] > -FLT_MAX))
    with np.errstate(over="ignore"):
        held = lse[:n].astype(np.float32).astype(np.float64)
    big = ~np.isfinite(held)
    assert np.array_equal(gl[big], held[big])
    assert (np.abs(gl[~big] - held[~big]) <= 8 * ref_kv4.HALF_F32 * np.abs(held[~big]) + 2.0 ** -18).all()


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_scaled_scores_beyond_fp32(D, many, sign):
    s = large_step([1, 70, 200, 64, 33], [1, 40, 2, 64, 33], 4, 2, D, 16, sign, seed=D, pad=2, width=room(16, many))
    for scale in (2.0 ** -101, 1.0, 4.0, 1e20):
        check_large(s, scale)
    check_large(s, 4.0, window=30)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,Hq,heads,n", [(64, 2, 1, 700), (128, 8, 1, 20000), (256, 3, 3, 6000)])
def test_in_chunks(D, Hq, heads, n, sign):
    s = large_step([n, 9], [1, 1], Hq, heads, D, 64, sign, seed=n)
    for scale in (2.0 ** -101, 1.0, 4.0, 1e20):
        check_large(s, scale)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_many_rows_in_chunks(D, sign):
    s = large_step([3000], [70], 2, 1, D, 16, sign, seed=3, width=room(16, True))
    for scale in (2.0 ** -101, 1.0, 4.0, 1e20):
        check_large(s, scale)


def test_ordinary_rows_beside_large_ones():
    """A row's own scores decide: neighbours in its tile keep every bit."""
    for many in (False, True):
        s = Step([50, 40], [20, 30], 4, 2, 128, 16, seed=8, width=room(16, many))
        want = s.run(scale=3.0)
        s.q[7, 1] *= 2.0 ** 100
        s.q[33, 2] *= 2.0 ** 110
        got = s.run(scale=3.0)
        large = torch.zeros(s.T, 4, dtype=torch.bool, device="cuda")
        large[7, 1] = large[33, 2] = True
        assert torch.equal(got[~large], want[~large]) and bool(torch.isfinite(got).all())


def near_step(base, step, kv, fresh, Hq, heads, D, P, sign, seed, **kw):
    """Scores base + step * (a level), exact in fp32, so that several keys count."""
    s = Step(kv, fresh, Hq, heads, D, P, seed=seed, **kw)
    rng = np.random.default_rng(seed)
    q = np.zeros((s.T, Hq, D))
    for i in range(4):                                   # base in pieces of 8 bits
        q[..., i] = sign * (base & (255 << 8 * i))
    q[..., 40] = sign * step
    s.q, s.q64 = bf16(q)
    for b, n in enumerate(kv):
        k = np.zeros((n, heads, D))
        k[..., :4] = 1.0
        k[..., 40] = rng.choice(ref_kv4.LEVELS[[0, 2, 4, 5, 6, 7]], (n, heads))
        slots = s.table[b][np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        s.cache.write("k", slots, k)
    s.to_device()
    return s


def check_near(s, scale, p_round):
    """A product is exact, a difference too; its product with the scale, the scale's own
    rounding and the exponential's argument are 2^-24 each of 40 at most (24 log2 e),
    a sum of n probabilities depth(n) roundings."""
    y = to64(s.run(scale=scale))
    want, _, lse, _ = ref_kv4.attention(s.q64, s.cache, s.table, s.q_start, s.kv, scale)
    n = int(s.q_start[-1])
    err = (2 * (3 * 40 + 2 + ref_kv4.depth(max(s.kv))) * ref_kv4.HALF_F32 + p_round) * 6.0     # |v| <= 6
    assert (np.abs(y - want)[:n] <= err + ref_kv4.HALF_BF16 * (np.abs(want[:n]) + err)).all(), np.abs(y - want)[:n].max() / err
    assert (np.abs(to64(s.lse) - lse)[:n] <= 8 * ref_kv4.HALF_F32 * np.abs(lse[:n])).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("base,step", [(1 << 23, 1), (11629072, 2), (1 << 24, 4), ((1 << 30) + (1 << 23), 256)])
@pytest.mark.parametrize("many", [False, True])
def test_scores_whose_exponents_have_no_bits_behind_the_point(base, step, sign, many):
    """11629072 log2 e is 2^24 - 11: some keys are on either side of where the maximum is
    taken off the products."""
    scale = 1.0 if step < 256 else 2.0 ** -4
    p_round = ref_kv4.HALF_BF16 if many else 2.0 ** -17
    for D in (64, 128, 256):
        s = near_step(base, step, [1, 70, 200, 64, 33], [1, 40, 2, 64, 33], 4, 2, D, 16, sign, seed=D, width=room(16, many))
        check_near(s, scale, p_round)
    if not many:
        check_near(near_step(base, step, [6000, 9], [1, 1], 4, 1, 128, 64, sign, seed=1), scale, p_round)
    else:
        for D in (64, 96, 192):
            check_near(near_step(base, step, [2000], [70], 2, 1, D, 16, sign, seed=2, width=room(16, True)), scale, p_round)
