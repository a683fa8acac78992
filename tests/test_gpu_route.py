"""The expert router against the fp64 reference: the choice has to be the
same, expert for expert, and the weights within the bound of fp32 logits."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev, host
from test_gpu_epilogue import bf16

pytestmark = pytest.mark.gpu



def rtol(x64, w64):
    """Relative error of a token's weights.  The weights come of fp32 logits: a
    product passes through at most D roundings of a step (2^-23) each: 32 in a
    matrix instruction, 8 along a chain of them, one for each further chain
    (256 depths), one for each of 16 K slices at most, so a logit is off by at most zd = D 2^-23 |x| |w|.  A sigmoid
    is then off by zd relative, an exponential by zd and the sum that it is
    divided by (softmax, renorm) by zd again, 2 zd (1 + zd) in all; then one
    rounding to fp32."""
    K = x64.shape[1]
    zd = (32 + 8 + 2 + K / 256 + 16) * 2.0 ** -23 * np.linalg.norm(x64, axis=1) * \
        np.linalg.norm(w64, axis=1).max()
    return (2.0 * zd * (1.0 + zd) + 2.0 ** -24 * (1 + 1e-5))[:, None]


def run(x, w, **kw):
    r = sp.Router(w, **kw)
    weights, ids = sp.spear_route(x, r)
    torch.cuda.synchronize()
    return host(weights).astype(np.float64), host(ids)


def compare(x, x64, w, w64, bias=None, topk=2, score=sp.SCORE_SOFTMAX, **kw):
    got_w, got_i = run(x, w, bias=None if bias is None else dev(bias), topk=topk, score=score, **kw)
    ref_w, ref_i = ref64.route(x64, w64, topk, score == sp.SCORE_SIGMOID, bias, **kw)
    assert np.array_equal(got_i, ref_i), (np.argwhere(got_i != ref_i)[:5], x.shape, w.shape)
    assert np.all(np.abs(got_w - ref_w) <= rtol(x64, w64) * np.abs(ref_w) + 1e-45)
    return got_w, got_i


def draw(M, E, K, seed, gain=1.0):
    rng = np.random.default_rng(seed)
    return (*bf16(rng.normal(0, gain, (M, K))), *bf16(rng.normal(0, 1 / np.sqrt(K), (E, K))), rng)


@pytest.mark.parametrize("M,E,K,topk", [(1, 1, 32, 1), (1, 8, 64, 8), (1, 64, 2048, 8), (3, 60, 96, 4),
                                        (7, 2, 4096, 1), (8, 512, 512, 32), (9, 65, 1056, 6),
                                        (16, 128, 2080, 8), (33, 256, 1024, 8), (130, 100, 288, 3),
                                        (517, 16, 160, 2), (1030, 64, 256, 8)])
@pytest.mark.parametrize("score", [sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID])
def test_route_parity(M, E, K, topk, score):
    x, x64, w, w64, rng = draw(M, E, K, M + E + K)
    bias = rng.normal(0, 0.1, E).astype(np.float32)
    for renorm in (True, False):
        compare(x, x64, w, w64, None, topk, score, renorm=renorm, scale=2.5)
        compare(x, x64, w, w64, bias, topk, score, renorm=renorm)


@pytest.mark.parametrize("E,G,kept,best,topk", [(64, 8, 4, 2, 8), (64, 8, 1, 1, 8), (256, 8, 4, 2, 8),
                                                (60, 4, 3, 2, 5), (64, 64, 6, 2, 6), (512, 64, 9, 1, 32),
                                                (24, 3, 2, 2, 16), (7, 7, 7, 2, 7)])
@pytest.mark.parametrize("M", [1, 5, 70, 290])
def test_groups(E, G, kept, best, topk, M):
    for score in (sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID):
        x, x64, w, w64, rng = draw(M, E, 256, E + G + M)
        bias = rng.normal(0, 0.2, E).astype(np.float32)
        compare(x, x64, w, w64, bias, topk, score, n_group=G, topk_group=kept, group_best=best)


@pytest.mark.parametrize("M", [1, 37, 200, 300])
def test_near_ties_are_decided_in_fp64(M):
    """Experts whose logits differ in the 8th digit and beyond: the small
    components decide behind large ones that cancel nothing, and copies of an
    expert come in index order."""
    rng = np.random.default_rng(M)
    K, E = 512, 96
    base = rng.integers(-8, 9, K) / 8.0
    w = np.repeat(base[None], E, 0)
    w[:, K - 64:] = 0.0
    # one small component an expert: logits 2^-20 .. apart, many equal
    for e in range(E):
        w[e, K - 1 - e % 24] = 2.0 ** -18
    x = rng.integers(-8, 9, (M, K)) / 8.0
    (xt, x64), (wt, w64) = bf16(x), bf16(w)
    for score in (sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID):
        # sums of these are exact, so equal logits are equal in any order
        compare(xt, x64, wt, w64, None, 12, score)
        compare(xt, x64, wt, w64, None, 12, score, n_group=8, topk_group=3)


def test_exact_ties_go_to_the_lowest_index():
    x, x64 = bf16(np.ones((5, 32)))
    w, w64 = bf16(np.ones((40, 32)) / 8)
    _, ids = compare(x, x64, w, w64, None, 8)
    assert np.array_equal(ids, np.tile(np.arange(8), (5, 1)))
    _, ids = compare(x, x64, w, w64, None, 6, sp.SCORE_SIGMOID, n_group=10, topk_group=2)
    assert np.array_equal(ids, np.tile(np.arange(6), (5, 1)))


@pytest.mark.parametrize("M", [4, 150, 310])
def test_left_out_experts_empty_slots_and_nan(M):
    """A bias of -inf takes experts out; slots left over are -1 with weight 0;
    a token with NaN in it has no experts; scores of zero sum to zero weights."""
    x, x64, w, w64, rng = draw(M, 32, 128, 5)
    bias = np.full(32, -np.inf, np.float32)
    bias[[3, 17, 30]] = [0.1, 0.0, -0.2]
    for score in (sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID):
        got_w, got_i = compare(x, x64, w, w64, bias, 6, score)
        assert np.all(got_i[:, 3:] == -1) and np.all(got_w[:, 3:] == 0) and np.all(got_i[:, :3] >= 0)
        compare(x, x64, w, w64, bias, 2, score, n_group=8, topk_group=2, group_best=1)
    x64[1, 7] = np.nan
    x[1, 7] = float("nan")
    got_w, got_i = run(x, w, topk=4)
    assert np.all(got_i[1] == -1) and np.all(got_w[1] == 0)
    keep = np.arange(M) != 1
    ref_w, ref_i = ref64.route(x64[keep], w64, 4, False)
    assert np.array_equal(got_i[keep], ref_i)
    # sigmoid of -1e4 is 0 in fp64: ties by index, weights 0
    x, x64 = bf16(np.full((M, 128), -1e4))
    w, w64 = bf16(np.ones((32, 128)))
    got_w, got_i = run(x, w, topk=4, score=sp.SCORE_SIGMOID)
    assert np.all(got_w == 0) and np.array_equal(got_i, np.tile(np.arange(4), (M, 1)))


@pytest.mark.parametrize("M", [2, 64, 260])
def test_large_logits(M):
    """Softmax of logits far apart neither overflows nor loses its choice."""
    x, x64, w, w64, _ = draw(M, 48, 1024, 9, gain=1000.0)
    compare(x, x64, w, w64, None, 4, renorm=False)
    compare(x, x64, w, w64, None, 1, sp.SCORE_SIGMOID)


def test_no_tokens_and_rows_behind():
    x, x64, w, w64, _ = draw(3, 16, 64, 1)
    weights, ids = sp.spear_route(x[:0], sp.Router(w, topk=2))
    assert weights.shape == ids.shape == (0, 2)
    bw = torch.full((5, 2), 7.0, device="cuda")
    bi = torch.full((5, 2), 7, dtype=torch.int32, device="cuda")
    sp.spear_route(x, sp.Router(w, topk=2), weights=bw[:3], ids=bi[:3])
    assert bool((bw[3:] == 7).all()) and bool((bi[3:] == 7).all())
    assert np.array_equal(host(bi[:3]), ref64.route(x64, w64, 2, False)[1])


@pytest.mark.parametrize("E,G,kept,topk,copies", [(64, 1, 1, 8, 5), (128, 1, 1, 32, 24), (256, 8, 4, 8, 20),
                                                  (256, 1, 1, 8, 100), (512, 16, 3, 32, 40), (60, 6, 2, 4, 60)])
@pytest.mark.parametrize("score", [sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID])
def test_many_ties_in_a_long_batch(E, G, kept, topk, copies, score):
    """Whole groups of equal experts, rows of zeros among the tokens, a batch that
    ends inside four tokens.  Small integers over 16: every sum is exact whatever
    its order, so ties are ties, and go to the lowest index."""
    rng = np.random.default_rng(E + copies)
    M, K = 303, 2112
    x = rng.integers(-3, 4, (M, K)) * (rng.random((M, K)) < 0.02)
    x[rng.random(M) < 0.2] = 0
    w = rng.integers(-3, 4, (E, K)) / 16.0
    w[rng.choice(E, copies, replace=False)] = w[0]
    xt, x64 = bf16(x.astype(np.float64))
    wt, w64 = bf16(w)
    assert np.array_equal(x64, x) and np.array_equal(w64, w)
    compare(xt, x64, wt, w64, None, topk, score, n_group=G, topk_group=kept)
    bias = (rng.integers(-1, 2, E) / 8.0).astype(np.float32)
    compare(xt, x64, wt, w64, bias, topk, score, n_group=G, topk_group=kept, renorm=False)


@pytest.mark.parametrize("M,E,K", [(64, 48, 288), (65, 48, 288), (256, 48, 288), (257, 48, 288), (64, 300, 992),
                                   (65, 300, 992), (128, 300, 992), (129, 300, 992), (3, 511, 4128), (1, 12, 8224)])
def test_where_the_launches_change(M, E, K):
    x, x64, w, w64, rng = draw(M, E, K, M + E)
    bias = rng.normal(0, 0.1, E).astype(np.float32)
    G = 4 if E % 4 == 0 else 7
    compare(x, x64, w, w64, bias, 6, sp.SCORE_SIGMOID, n_group=G, topk_group=2)
    compare(x, x64, w, w64, None, 6, sp.SCORE_SOFTMAX)


def test_rows_past_32_bit_offsets():
    """A batch of more than 2^32 bytes: its last tokens against the reference."""
    M, E, K = 1100003, 16, 2048
    _, _, w, w64, _ = draw(1, E, K, 3)
    tail, t64 = bf16(np.random.default_rng(4).normal(0, 1, (40, K)))
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-40:] = tail
    assert x.numel() * 2 > 1 << 32
    weights, ids = sp.spear_route(x, sp.Router(w, topk=3))
    ref_w, ref_i = ref64.route(t64, w64, 3, False)
    assert np.array_equal(host(ids[-40:]), ref_i)
    assert np.all(np.abs(host(weights[-40:]) - ref_w) <= rtol(t64, w64) * ref_w)
    assert bool((ids[:-40] == torch.arange(3, dtype=torch.int32, device="cuda")).all())
