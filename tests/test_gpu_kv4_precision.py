"""The kernel for few rows holds probabilities as two bf16, 2^-17 of their size (what
rounding x to hi leaves is half a step of it, 2^(e-8) for x in [2^e, 2^(e+1)), and half
a step of that 2^(e-17)): checked with that bound where no other kernel runs.  Flat
rows, so that sums cancel and y's own rounding is small beside a probability's."""
import pytest

from kv4_util import Step

pytestmark = pytest.mark.gpu
TWO = 2.0 ** -17
DIMS = [64, 96, 128, 192, 256]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("Hq,heads,P", [(8, 8, 64), (8, 2, 128), (16, 1, 16), (24, 1, 256)])
def test_one_token(D, Hq, heads, P):
    kv = [1, 2, 17, 63, 64, 65, 129, 300]
    Step(kv, [1] * len(kv), Hq, heads, D, P, seed=D + Hq, q_sd=0.3).check(f"two terms, D={D} {Hq}/{heads}", p_round=TWO)


@pytest.mark.parametrize("D", DIMS)
def test_a_few_tokens(D):
    fresh, kv = [1, 2, 17, 5, 30], [90, 64, 17, 128, 200]
    Step(kv, fresh, 6, 2, D, 32, seed=D, q_sd=0.3).check(f"two terms, some tokens, D={D}", p_round=TWO)
    Step(kv, fresh, 6, 2, D, 32, seed=D, q_sd=0.3).check(f"two terms, window, D={D}", p_round=TWO, window=40)


@pytest.mark.parametrize("D,Hq,heads,n", [(64, 4, 1, 700), (128, 8, 1, 6000), (256, 5, 1, 2500), (96, 3, 1, 1500), (192, 2, 2, 1500)])
def test_in_chunks(D, Hq, heads, n):
    Step([n, 40], [1, 1], Hq, heads, D, 64, seed=n, q_sd=0.3).check(f"two terms, {n} keys of D={D}", p_round=TWO)
