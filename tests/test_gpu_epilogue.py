"""The W4 linear with bias, activation (plain and gated pair) and residual in
its epilogue, on every path, against the fp64 reference."""
import numpy as np
import pytest
import torch

import oracle
import ref64
from quantized_gemm_w4a16_amd import inputs as gen
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

DECODE = [sp.PATH_AUTO, sp.PATH_DECODE, sp.PATH_DECODE_2PASS, sp.PATH_PREFILL,
          sp.PATH_PREFILL_LARGE]
PREFILL = [sp.PATH_PREFILL, sp.PATH_PREFILL_LARGE]


def bf16(a):
    """numpy float -> (torch bf16 on the GPU, the same values as float64)."""
    bits = gen.bf16_bits(np.asarray(a, np.float32))
    return (torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16),
            gen.bf16_to_f32(bits).astype(np.float64))


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Case:
    def __init__(self, M, N, K, r, hard, seed, glu, bias, residual, out):
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.glu, self.out = M, N, K, glu, out
        self.codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
        self.scales = (rng.uniform(0.5, 2.0, N) * 0.2 / np.sqrt(K)).astype(np.float32)
        self.zeros = rng.integers(0, 16, N, dtype=np.uint8)
        self.x, self.x64 = bf16(rng.normal(0, 1, (M, K)))
        self.w = sp.W4(sp.spear_pack_w4(dev(self.codes), sp.CODES_U4), dev(self.scales),
                       dev(self.zeros), N, K)
        self.ec = self.ec64 = None
        if r:
            A, A64 = bf16(rng.normal(0, 1 / np.sqrt(K), (r, K)))
            B, B64 = bf16(rng.normal(0, 0.5 / np.sqrt(r), (N, r)))
            g, g64 = bf16(rng.normal(0, 1 / np.sqrt(K), K))
            self.ec = sp.EC(A, B, g, 0.25, 0.55, hard)
            self.ec64 = dict(A=A64, B=B64, w_g=g64, b=0.25, tau=float(np.float32(0.55)), hard=hard)
        self.bias = rng.normal(0, 0.5, N).astype(np.float32) if bias else None
        self.res, self.res64 = None, None
        if residual:
            v = rng.normal(0, 1, (M, N // 2 if glu else N)).astype(np.float32)
            if out == sp.OUT_F32:
                self.res, self.res64 = dev(v), v.astype(np.float64)
            else:
                self.res, self.res64 = bf16(v)

    def epilogue(self, kind):
        return sp.Epilogue(dev(self.bias) if self.bias is not None else None, kind, self.glu,
                           self.res)

    def reference(self, kind):
        t, err = ref64.linear(self.x64, self.codes, self.scales, self.zeros, self.ec64)
        y, err = ref64.finish(t, err, kind, self.glu, self.bias, self.res64)
        return y, ref64.rounded(y, err, ref64.HALF_F32 if self.out == sp.OUT_F32 else ref64.HALF_BF16)


def check(y, ref, tol, what):
    d = np.abs(to64(y) - ref)
    worst = float(np.max(d / tol)) if d.size else 0.0
    print(f"[epilogue] {what}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, what


# one token, ragged K and N, both outputs' vector widths (N / 2 odd, N odd),
# K split over decode workgroups (long K), K slices of the GEMM (few tiles),
# 64 x 64 and 256 x 128 tiles with partial ones, ranks of one and of several blocks
SHAPES = [(1, 64, 128, 0), (1, 258, 416, 16), (2, 77, 96, 8), (5, 300, 2080, 64), (16, 130, 1056, 32),
          (13, 64, 22016, 32), (17, 34, 512, 32), (40, 200, 1056, 96), (129, 258, 4096, 32),
          (150, 515, 544, 0), (300, 1030, 256, 64)]


@pytest.mark.parametrize("M,N,K,r", SHAPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("out", [sp.OUT_F32, sp.OUT_BF16])
def test_epilogue_parity(M, N, K, r, glu, out):
    if glu and N % 2:
        N += 1
    kind = (M + N) % 5
    c = Case(M, N, K, r, M % 2, M * 7 + N, glu, True, True, out)
    ref, tol = c.reference(kind)
    for path in (DECODE if M <= 16 else PREFILL):
        y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(kind), c.ec, out_dtype=out, path=path)
        check(y, ref, tol, f"M={M} N={N} K={K} r={r} glu={glu} out={out} act={kind} path={path}")


@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("M", [1, 3, 70])
def test_activations(M, kind):
    """Every activation, small to large arguments of both signs."""
    for glu in (False, True):
        c = Case(M, 96, 256, 0, 0, kind + M, glu, False, False, sp.OUT_F32)
        scales = c.scales * np.repeat([0.05, 1.0, 30.0], 32).astype(np.float32)
        c.scales, c.w.scales = scales, dev(scales)
        ref, tol = c.reference(kind)
        for path in (DECODE if M <= 16 else PREFILL):
            y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(kind), None, path=path)
            check(y, ref, tol, f"act={kind} M={M} glu={glu} path={path}")


@pytest.mark.parametrize("M", [1, 6, 100])
def test_no_epilogue_is_the_layer_bit_for_bit(M):
    """No bias, no activation, no residual: the plain entry point's bits, on
    every path and, without an error compensator, where the path is chosen."""
    c = Case(M, 274, 1024, 32, 1, M, False, False, False, sp.OUT_F32)
    for out in (sp.OUT_F32, sp.OUT_BF16):
        for path in (DECODE if M <= 16 else PREFILL):
            for ec in ([c.ec, None] if path != sp.PATH_AUTO else [None]):
                a = sp.spear_w4_linear(c.x, c.w, ec, out_dtype=out, path=path)
                b = sp.spear_w4_linear_epilogue(c.x, c.w, sp.Epilogue(), ec, out_dtype=out, path=path)
                assert torch.equal(a, b), (M, out, path)


@pytest.mark.parametrize("M,N,K,r", [(1, 64, 32, 8), (1, 2048, 2048, 32), (2, 100, 96, 64), (5, 48, 9000 // 32 * 32, 40),
                                     (16, 300, 1056, 64), (16, 64, 12288, 32), (11, 4112, 512, 16)])
@pytest.mark.parametrize("hard", [0, 1])
def test_chosen_path_with_the_compensator(M, N, K, r, hard):
    """The path that the call chooses: the gates and the selected tokens are the
    gate entry point's, and the outputs hold on a workspace that other calls of
    the layer have used."""
    c = Case(M, N, K, r, hard, M + N + K, False, True, False, sp.OUT_F32)
    ref, tol = c.reference(ref64.SILU)
    ws = sp.new_workspace(M, N, K, r)
    g, idx, n = sp.spear_gate(c.x, c.ec.w_gate, c.ec.b, c.ec.tau, hard)
    for i in range(3):
        c.ec.g_out = torch.full((M,), -1.0, device="cuda")
        c.ec.idx_out = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        c.ec.n_active_out = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        y = sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_SILU), c.ec, workspace=ws)
        check(y, ref, tol, f"chosen M={M} N={N} K={K} r={r} hard={hard} call {i}")
        k = int(n.item())
        assert int(c.ec.n_active_out.item()) == k and torch.equal(c.ec.idx_out[:k], idx[:k])
        np.testing.assert_allclose(host(c.ec.g_out), host(g), rtol=2e-7)
        sp.spear_w4_linear(c.x, c.w, c.ec, workspace=ws, path=[sp.PATH_DECODE, sp.PATH_PREFILL, sp.PATH_AUTO][i])
    assert sp.spear_workspace_timeouts(ws) == 0


@pytest.mark.parametrize("M", [1, 9, 65, 200])
@pytest.mark.parametrize("glu", [False, True])
def test_residual_in_place_and_rows_behind(M, glu):
    """y may be the residual; what lies behind the last row stays as it was."""
    c = Case(M, 196, 640, 16, 0, 40 + M, glu, True, True, sp.OUT_BF16)
    ref, tol = c.reference(ref64.SILU)
    ep = c.epilogue(sp.ACT_SILU)
    NO = 98 if glu else 196
    for path in (DECODE if M <= 16 else PREFILL):
        buf = torch.full(((M + 3) * NO,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[: M * NO].view(M, NO)
        y.copy_(c.res)
        ep.residual = y
        out = sp.spear_w4_linear_epilogue(c.x, c.w, ep, c.ec, y=y, out_dtype=sp.OUT_BF16, path=path)
        assert out is y
        check(y, ref, tol, f"in place M={M} glu={glu} path={path}")
        assert bool((buf[M * NO:] == 7.0).all())


def test_special_values_pass_as_in_the_formula():
    """Infinite and NaN biases: relu, silu and gelu go to 0 at -inf, NaN stays."""
    c = Case(2, 64, 64, 0, 0, 3, False, False, False, sp.OUT_F32)
    b = np.zeros(64, np.float32)
    b[0], b[1], b[2], b[3] = np.inf, -np.inf, np.nan, -3e38
    for kind in range(1, 5):
        for path in DECODE:
            y = host(sp.spear_w4_linear_epilogue(c.x, c.w, sp.Epilogue(dev(b), kind), path=path))
            assert np.all(np.isposinf(y[:, 0])) and np.all(y[:, 1] == 0) and np.all(np.isnan(y[:, 2]))
            assert np.all(y[:, 3] == 0) and np.all(np.isfinite(y[:, 4:]))


def test_no_tokens_and_signed_codes():
    c = Case(0, 64, 64, 0, 0, 3, True, True, True, sp.OUT_F32)
    assert sp.spear_w4_linear_epilogue(c.x, c.w, c.epilogue(sp.ACT_SILU)).shape == (0, 32)
    rng = np.random.default_rng(8)
    q = rng.integers(-8, 8, (96, 256), dtype=np.int8)
    s = rng.uniform(0.005, 0.02, 96).astype(np.float32)
    w = sp.W4(sp.spear_pack_w4(dev(q), sp.CODES_S4), dev(s), None, 96, 256)
    for M in (1, 4, 33):
        x, x64 = bf16(rng.normal(0, 1, (M, 256)))
        t, err = ref64.linear(x64, q.astype(np.int16) + 8, s, np.full(96, 8))
        y, err = ref64.finish(t, err, ref64.GELU, False)
        got = sp.spear_w4_linear_epilogue(x, w, sp.Epilogue(act=sp.ACT_GELU))
        check(got, y, ref64.rounded(y, err, ref64.HALF_F32), f"signed M={M}")


def test_expired_wait_gives_nan_through_the_activation():
    """A bounded wait that expires leaves NaN behind relu and the gated pair too."""
    c = Case(4, 256, 4096, 32, 0, 11, True, True, False, sp.OUT_F32)
    ws = sp.new_workspace(4, 256, 4096, 32)
    ep = c.epilogue(sp.ACT_RELU)
    ref, tol = c.reference(ref64.RELU)
    sp.spear_set_wait_limit(1)
    try:
        y = sp.spear_w4_linear_epilogue(c.x, c.w, ep, c.ec, workspace=ws, path=sp.PATH_DECODE)
        torch.cuda.synchronize()
        expired = sp.spear_workspace_timeouts(ws)
    finally:
        sp.spear_set_wait_limit(0)
    got = to64(y)
    bad = np.isnan(got)
    assert bad.any() == (expired > 0)
    assert np.all((np.abs(got - ref) <= tol) | bad)
    y = sp.spear_w4_linear_epilogue(c.x, c.w, ep, c.ec, workspace=ws, path=sp.PATH_DECODE)
    check(y, ref, tol, "after an expired wait")


@pytest.mark.parametrize("M", [1, 7, 16, 90])
@pytest.mark.parametrize("r,h", [(32, 12), (72, 0), (256, 0)])
def test_compensators_that_keep_the_layers_own_launch(M, r, h):
    """A gate vector, ranks above 64: the plain entry point's bits where the path
    is chosen, and its gates."""
    c = Case(M, 140, 1056, r, 0, M + r + h, False, False, False, sp.OUT_F32)
    if h:
        rng = np.random.default_rng(r)
        for name, shape in (("gate_w1", (h, r)), ("gate_c1", (h,)), ("gate_w2", (r, h)), ("gate_c2", (r,))):
            setattr(c.ec, name, dev(rng.normal(0, 0.4, shape).astype(np.float32)))
        c.ec.alpha = 0.7
    a = sp.spear_w4_linear(c.x, c.w, c.ec)
    assert torch.equal(a, sp.spear_w4_linear_epilogue(c.x, c.w, sp.Epilogue(), c.ec))


def test_outputs_past_32_bit_offsets():
    """An output of more than 2^32 bytes: its last rows against the reference."""
    M, N, K = 40000, 32768, 64
    c = Case(8, N, K, 0, 0, 5, False, True, False, sp.OUT_F32)
    ref, tol = c.reference(ref64.SILU)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-8:] = c.x
    y = sp.spear_w4_linear_epilogue(x, c.w, c.epilogue(sp.ACT_SILU), None)
    assert y.numel() * 4 > 1 << 32
    check(y[-8:], ref, tol, "last rows")
