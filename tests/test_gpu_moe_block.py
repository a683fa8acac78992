"""A decoder's mixture-of-experts block as it is used: the router, the experts
and a shared expert through the linear's epilogue, eager, on another stream,
from two streams at once, and captured into a graph that is replayed."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from test_gpu_epilogue import bf16, to64
from test_gpu_experts import w4

pytestmark = pytest.mark.gpu
D, FF, E, TOPK, INNER = 256, 192, 16, 3, 64


class Block:
    """y = x + shared(x) + sum over the routed experts."""

    def __init__(self, M, seed=0):
        rng = np.random.default_rng(seed)
        self.M = M
        self.router_w, self.router64 = bf16(rng.normal(0, 1 / np.sqrt(D), (E, D)))
        self.bias = rng.normal(0, 0.1, E).astype(np.float32)
        self.router = sp.Router(self.router_w, TOPK, sp.SCORE_SIGMOID, dev(self.bias), n_group=4, topk_group=2)
        self.up, up = w4(rng, E, 2 * INNER, D)
        self.down, down = w4(rng, E, D, INNER)
        self.experts = sp.Experts(*up, *down)
        self.su, su = w4(rng, 1, 2 * FF, D)
        self.sd, sd = w4(rng, 1, D, FF)
        self.shared_up = sp.W4(su[0][0], su[1][0], su[2][0], 2 * FF, D)
        self.shared_down = sp.W4(sd[0][0], sd[1][0], sd[2][0], D, FF)
        self.buffers()

    def buffers(self):
        M = self.M
        self.weights = torch.empty(M, TOPK, device="cuda")
        self.ids = torch.empty(M, TOPK, dtype=torch.int32, device="cuda")
        self.h = torch.empty(M, FF, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
        self.ws = (sp.new_route_workspace(M, self.router), sp.new_experts_workspace(M, TOPK, self.experts),
                   sp.new_workspace(M, 2 * FF, D, 0), sp.new_workspace(M, D, FF, 0))

    def __call__(self, x, stream=None):
        s = stream
        sp.spear_route(x, self.router, self.weights, self.ids, self.ws[0], stream=s)
        sp.spear_w4_experts(x, self.experts, self.ids, self.weights, residual=x, y=self.y, workspace=self.ws[1],
                            stream=s)
        sp.spear_w4_linear_epilogue(x, self.shared_up, sp.Epilogue(act=sp.ACT_SILU, glu=True), y=self.h,
                                    out_dtype=sp.OUT_BF16, workspace=self.ws[2], stream=s)
        sp.spear_w4_linear_epilogue(self.h, self.shared_down, sp.Epilogue(residual=self.y), y=self.y,
                                    out_dtype=sp.OUT_BF16, workspace=self.ws[3], stream=s)
        return self.y

    def reference(self, x64):
        weights, ids = ref64.route(x64, self.router64, TOPK, True, self.bias, n_group=4, topk_group=2)
        y, err = ref64.experts(x64, self.up, self.down, ids, weights, ref64.SILU, True, residual=x64)
        err = ref64.rounded(y, err, ref64.HALF_BF16) + 2 * ref64.HALF_F32 * np.abs(y)
        t, te = ref64.linear(x64, self.su[0][0], self.su[1][0], self.su[2][0])
        h, he = ref64.finish(t, te, ref64.SILU, True)
        he = ref64.rounded(h, he, ref64.HALF_BF16)
        d, de = ref64.linear(h, self.sd[0][0], self.sd[1][0], self.sd[2][0])
        dw = (self.sd[0][0].astype(np.float64) - self.sd[2][0][:, None]) * self.sd[1][0][:, None]
        y, err = y + d, err + de + he @ np.abs(dw).T
        return y, ref64.rounded(y, err, ref64.HALF_BF16)


def tokens(M, seed):
    return bf16(np.random.default_rng(seed).normal(0, 1, (M, D)))


@pytest.mark.parametrize("M", [1, 4, 16, 47, 200, 420])
def test_block_parity(M):
    b = Block(M)
    x, x64 = tokens(M, M)
    ref, tol = b.reference(x64)
    worst = float(np.max(np.abs(to64(b(x)) - ref) / tol))
    print(f"[block] M={M}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("M", [1, 8, 90, 420])
def test_block_in_a_graph(M):
    """Captured once, replayed on new tokens with eager work of its own buffers
    in between, each replay the eager result bit for bit."""
    b, eager = Block(M, 1), Block(M, 1)
    x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    x.copy_(tokens(M, 0)[0])
    b(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b(x)
    for seed in range(4):
        x.copy_(tokens(M, 10 + seed)[0])
        b.y.fill_(float("nan"))
        g.replay()
        want = eager(x)
        torch.cuda.synchronize()
        assert torch.equal(b.y, want), seed
        assert torch.equal(b.ids, eager.ids) and torch.equal(b.weights, eager.weights)


def test_block_on_other_streams():
    """Given as a stream object, as a raw handle and as the current stream; the
    calls' own allocations belong to that stream."""
    b, M = Block(20, 2), 20
    x, _ = tokens(M, 3)
    want = b(x).clone()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0, None):
        torch.cuda.synchronize()
        assert torch.equal(b(x, stream).clone() if stream is None else _done(b(x, stream)), want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        weights, ids = sp.spear_route(x, b.router)                # allocates
        y = sp.spear_w4_experts(x, b.experts, ids, weights, residual=x)
    s.synchronize()
    assert torch.equal(ids, b.ids) and torch.equal(weights, b.weights)
    weights, ids = sp.spear_route(x, b.router, stream=s)
    z = sp.spear_w4_experts(x, b.experts, ids, weights, residual=x, stream=s)
    s.synchronize()
    assert torch.equal(y, z)


def _done(y):
    torch.cuda.synchronize()
    return y.clone()


def test_two_blocks_at_once():
    """Two blocks with workspaces of their own on two streams."""
    M = 64
    blocks = [Block(M, 4), Block(M, 5)]
    xs = [tokens(M, 6)[0], tokens(M, 7)[0]]
    want = [_done(b(x)) for b, x in zip(blocks, xs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, x, s in zip(blocks, xs, streams):
            b(x, s)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert torch.equal(b.y, w)
