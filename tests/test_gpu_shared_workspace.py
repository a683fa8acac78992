"""One workspace for several calls of a layer: what one leaves there is taken by
no other."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from test_gpu_epilogue import Case, check

pytestmark = pytest.mark.gpu


# (wide layers, and 14 tokens or more at depths of 4096 to 8192, take that pre-pass)
@pytest.mark.parametrize("M,N,K,r", [(1, 10242, 32, 8), (1, 16384, 2048, 32), (2, 10250, 96, 64), (16, 2048, 8192, 64),
                                     (14, 4096, 4160, 40), (12, 12288, 544, 16)])
def test_partials_of_the_epilogues_pre_pass_carry_no_tag(M, N, K, r):
    """Launches know their own partial results by the upper half of a 64-bit word,
    which counts launches from one; the chosen path's pre-pass writes words of
    upper half zero, so that no layout of the workspace finds a tag in them."""
    c = Case(M, N, K, r, 0, M + K, False, True, False, sp.OUT_F32)
    ref, tol = c.reference(ref64.SILU)
    ws = sp.new_workspace(M, N, K, r)
    y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_SILU), c.ec, workspace=ws)
    check(y, ref, tol, f"M={M} N={N} K={K} r={r}")
    # behind the counters; sums of K ranges joined inside the launch have its tag, 1
    # (at 16 tokens a range holds 18 steps of 128)
    upper = (ws.view(torch.int64)[(256 + 64 * 128) // 8:] >> 32) & 0xFFFFFFFF
    assert int(upper.max()) <= 1


@pytest.mark.parametrize("r", [32, 64])
def test_calls_of_many_token_counts_in_turn(r):
    N, K, most = 10304, 1056, 2040
    ws = sp.new_workspace(most, N, K, r)
    cases = {M: Case(M, N, K, r, 0, M, False, True, False, sp.OUT_F32) for M in (1, 5, 16, 40, 300, most)}
    for M in (1, most, 5, 300, 16, 1, 40, most, 5, 16):
        c = cases[M]
        ref, tol = c.reference(ref64.GELU)
        for path in ([sp.PATH_AUTO, sp.PATH_DECODE] if M <= 16 else [sp.PATH_AUTO]):
            y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_GELU), c.ec, workspace=ws, path=path)
            check(y, ref, tol, f"M={M} r={r} path={path}")
    assert sp.spear_workspace_timeouts(ws) == 0


@pytest.mark.parametrize("M,N,K,r", [(1, 10242, 32, 8), (1, 16384, 2048, 32), (2, 10240, 96, 64), (5, 10256, 4128, 40),
                                     (8, 11008, 1056, 16), (16, 2048, 8192, 32), (15, 4100, 5120, 64), (13, 14336, 288, 48)])
@pytest.mark.parametrize("hard", [0, 1])
@pytest.mark.parametrize("out", [sp.OUT_F32, sp.OUT_BF16])
def test_wide_layers_where_the_path_is_chosen(M, N, K, r, hard, out):
    """Outputs, gates and selected tokens, with the gated pair and a residual, on a
    workspace that other calls of the layer use in between."""
    c = Case(M, N, K, r, hard, M + N + K, True, True, True, out)
    ref, tol = c.reference(ref64.SILU)
    ws = sp.new_workspace(M, N, K, r)
    g, idx, n = sp.spear_gate(c.x, c.ec.w_gate, c.ec.b, c.ec.tau, hard)
    k = int(n.item())
    for path in (sp.PATH_DECODE, sp.PATH_PREFILL):
        c.ec.g_out = torch.full((M,), -1.0, device="cuda")
        c.ec.idx_out = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        c.ec.n_active_out = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_SILU), c.ec, out_dtype=out, workspace=ws)
        check(y, ref, tol, f"wide M={M} N={N} K={K} r={r} hard={hard}")
        assert int(c.ec.n_active_out.item()) == k and torch.equal(c.ec.idx_out[:k], idx[:k])
        # two fp64 sums of a logit, an exponential and a rounding to fp32 each
        assert bool(((c.ec.g_out - g).abs() <= 2.0 ** -23 * g).all())
        sp.spear_w4_linear(c.x, c.w, c.ec, workspace=ws, path=path)
    assert sp.spear_workspace_timeouts(ws) == 0


def test_the_static_scratch_holds_a_layer_close_to_its_size():
    M, N, K, r = 401, 14336, 14336, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    packed = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    w = sp.W4(packed, torch.full((N,), 0.01, device="cuda"), None, N, K)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    ec = sp.EC(rand(r, K) * 0.01, rand(N, r) * 0.01, rand(K) * 0.01)
    x = rand(M, K)
    y = sp.spear_w4_linear_noalloc(x, w, ec)
    assert torch.equal(y, sp.spear_w4_linear(x, w, ec))
