"""The experts' streaming products at depths on both sides of every change of
their loops (prologue, counted waits over the ring, tail), against the fp64
reference: N is small, so that the depths are cheap."""
import numpy as np
import pytest

from test_gpu_experts import Case

pytestmark = pytest.mark.gpu


def spread(counts, seed):
    """Ids of one slot a token: counts[e] tokens for expert e, in mixed order."""
    ids = np.repeat(np.arange(len(counts)), counts)
    return np.random.default_rng(seed).permutation(ids).reshape(-1, 1)


# chunks of 256 depths in a ring of two: the loop runs from four chunks on
@pytest.mark.parametrize("K,I", [(736, 1056), (768, 800), (800, 768), (992, 1024), (1024, 992), (1056, 736),
                                 (1312, 1280), (2080, 2304), (2304, 2080)])
def test_tiles_of_64_rows(K, I):
    """Experts that fill one to four fragments of a tile, and several tiles."""
    counts = [9, 27, 41, 64, 150, 0, 16]
    c = Case(sum(counts), len(counts), 1, K, I, 72, bias=True, residual=True, seed=K + I, ids=spread(counts, K))
    c.check(c.run(), f"64 rows K={K} I={I}")


# chunks of 512 depths in a ring of two
@pytest.mark.parametrize("K,I", [(1536, 1568), (1568, 1536), (2048, 512), (2080, 3104), (3104, 2080), (4608, 1024)])
def test_planned_tiles_of_16_rows(K, I):
    counts = [1, 16, 17, 5, 0, 2]
    c = Case(sum(counts), len(counts), 1, K, I, 40, bias=True, seed=K + I, ids=spread(counts, K))
    c.check(c.run(), f"16 rows K={K} I={I}")


# chunks of 512 depths in a ring of four; the second product takes 1024 at a time
@pytest.mark.parametrize("K,I", [(3584, 1024), (3616, 1056), (4096, 2048), (4128, 2080), (6176, 3104), (8224, 544)])
@pytest.mark.parametrize("M,topk,E", [(1, 2, 5), (2, 8, 20), (16, 1, 3), (1, 1, 1)])
def test_few_slots(K, I, M, topk, E):
    rng = np.random.default_rng(K + M)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)])
    c = Case(M, E, topk, K, I, 24, bias=True, residual=True, seed=K + M, ids=ids)
    c.check(c.run(), f"few slots K={K} I={I} M={M} topk={topk}")
