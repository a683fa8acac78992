"""The router where values are not ordinary numbers: the choice is the one of
the fp64 formula whatever the number of tokens."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev, host
from test_gpu_epilogue import bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 64, 65, 200, 300])
@pytest.mark.parametrize("K", [32, 2048, 2080, 4128])
@pytest.mark.parametrize("score", [sp.SCORE_SOFTMAX, sp.SCORE_SIGMOID])
def test_infinite_router_weights(M, K, score):
    """Logits of +inf and -inf, by the token's sign at one depth: a sigmoid is 1
    or 0, a softmax without an answer leaves the token without experts, one
    expert at -inf leaves the others as they are."""
    rng = np.random.default_rng(M + K)
    E, topk = 40, 5
    x, w = rng.normal(0, 1, (M, K)), rng.normal(0, 1 / np.sqrt(K), (E, K))
    x[:, 3] = np.where(rng.random(M) < 0.5, 1.5, -1.5)
    w[[2, 17], 3] = np.inf, -np.inf
    for rows in ([2], [17], [2, 17]):
        wr = w.copy()
        wr[[e for e in (2, 17) if e not in rows], 3] = 0.25
        (xt, x64), (wt, w64) = bf16(x), bf16(wr)
        weights, ids = sp.spear_route(xt, sp.Router(wt, topk, score))
        with np.errstate(invalid="ignore"):
            ref_w, ref_i = ref64.route(x64, w64, topk, score == sp.SCORE_SIGMOID)
        assert np.array_equal(host(ids), ref_i), (rows, np.argwhere(host(ids) != ref_i)[:4])
        # fp32 logits of norm-1 rows over tokens of norm sqrt(K): far below this
        np.testing.assert_allclose(host(weights), ref_w, rtol=2 * (58 + K / 256) * 2.0 ** -23 * 1.1 *
                                   np.linalg.norm(x64, axis=1).max() + 2.0 ** -23, atol=1e-45)
