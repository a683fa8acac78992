"""Attention over the cache of 4 bits: group sizes above 32 in both kernels, keys cut
into chunks under a window, the join of heads of 96 and 192, and the cut of steps of
many requests, against plain fp64."""
import numpy as np
import pytest

from kv4_util import Step
from test_gpu_kv4_attention import room

pytestmark = pytest.mark.gpu
DIMS = [64, 96, 128, 192, 256]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("G,heads", [(33, 1), (40, 2), (64, 1)])
@pytest.mark.parametrize("many", [False, True])
def test_wide_groups(G, heads, D, many):
    """One token (which fills 33 to 64 rows) and several, either kernel for all."""
    kv = [1, 2, 17, 64, 65, 129, 200]
    Step(kv, [1] * len(kv), G * heads, heads, D, 16, seed=D + G, width=room(16, many)).check(f"one token, groups of {G}, D={D} many={many}")
    Step([90, 33, 5, 150], [1, 5, 5, 3], G * heads, heads, D, 32, seed=D + G, pad=2, width=room(32, many)).check(
        f"some tokens, groups of {G}, D={D} many={many}", window=40)


@pytest.mark.parametrize("G", [33, 64])
def test_wide_groups_in_chunks(G):
    Step([3000, 20], [1, 1], G, 1, 64, 64, seed=G).check(f"few rows in chunks, groups of {G}")
    Step([3000, 20], [1, 2], G, 1, 64, 64, seed=G, width=room(64, True)).check(f"many rows in chunks, groups of {G}")


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("window", [777, 4000])
def test_chunks_under_a_window(D, window):
    """The first step that a request's rows see is not its first, and several chunks
    follow it: of the kernel for few rows, then of the one for many."""
    Step([9000, 5000, 30], [1, 1, 1], 4, 1, D, 64, seed=window).check(f"tokens on a window of {window}, D={D}", window=window)
    # (many padded rows: the step takes both kernels, whatever the window leaves of the keys)
    Step([6000, 4500], [40, 3], 2, 1, D, 64, seed=window, pad=12000).check(f"rows on a window of {window}, D={D}", window=window, max_fresh=150)


@pytest.mark.parametrize("D", DIMS)
def test_chunks_of_many_rows(D):
    """Tiles that end inside a wave's rows, joined by the launch behind."""
    Step([4000], [67], 2, 1, D, 64, seed=D, width=room(64, True)).check(f"67 rows x 2 on 4000 keys, D={D}")
    Step([2500, 1800], [129, 40], 1, 1, D, 64, seed=D + 1, width=room(64, True)).check(f"129 and 40 rows, D={D}")


@pytest.mark.parametrize("B", [65, 90, 128, 300])
@pytest.mark.parametrize("D,heads", [(64, 1), (128, 2)])
def test_cut_steps_of_many_requests(B, D, heads):
    """More requests than a wave has lanes, long ones among them in each sixty-four."""
    rng = np.random.default_rng(B + D)
    kv = rng.integers(1, 60, B)
    kv[:: max(7, B // 12)] = rng.integers(1500, 4000, len(kv[:: max(7, B // 12)]))
    Step(kv.tolist(), [1] * B, heads * 2, heads, D, 64, seed=B).check(f"{B} requests, long ones among them, D={D}")
    fresh = [min(int(n), 1 + i % 3) for i, n in enumerate(kv)]
    fresh[B // 2], kv[B // 2] = 40, 64
    Step(kv.tolist(), fresh, heads * 2, heads, D, 64, seed=B + 1, width=room(64, True)).check(f"{B} requests, both kernels, D={D}")


@pytest.mark.parametrize("B", [1000, 4096])
def test_as_many_requests_as_a_step_may_have(B):
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 40, B)
    kv[B - 3] = 900
    Step(kv.tolist(), rng.integers(0, 2, B).tolist(), 4, 2, 64, 16, seed=B, pad=1).check(f"{B} requests")
    Step(kv.tolist(), [1] * B, 2, 1, 64, 16, seed=B + 1, pad=1).check(f"{B} requests of one token")
