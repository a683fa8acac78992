"""The router's choice whatever the size of the logits: with larger ones more
tokens lie inside the bounds of the fp32 logits and are settled in fp64."""
import numpy as np
import pytest

from quantized_gemm_w4a16_amd import spear as sp
from test_gpu_route import compare
from test_gpu_epilogue import bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gain", [0.25, 1.0, 2.0, 4.0, 8.0, 16.0, 300.0])
@pytest.mark.parametrize("M,E,K,topk,G,kept", [(700, 256, 1024, 8, 8, 4), (700, 256, 1024, 8, 1, 1), (450, 60, 2080, 4, 6, 3),
                                               (300, 512, 544, 16, 16, 5)])
def test_choice(gain, M, E, K, topk, G, kept):
    rng = np.random.default_rng(E + M)
    x, x64 = bf16(rng.normal(0, 1, (M, K)))
    w, w64 = bf16(rng.normal(0, gain / np.sqrt(K), (E, K)))
    bias = rng.normal(0, 0.05, E).astype(np.float32)
    for score in (sp.SCORE_SIGMOID, sp.SCORE_SOFTMAX):
        compare(x, x64, w, w64, bias, topk, score, n_group=G, topk_group=kept, scale=2.5)
        compare(x, x64, w, w64, None, topk, score, n_group=G, topk_group=kept)
