"""A decoder's attention block as it is used: the W4 q/k/v projection, a step's
plan, rotation and write into the cache of 4 bits, the attention over it, and the
W4 output projection onto the residual; prompts in chunks, then token by token,
eager and from a captured graph, against plain fp64."""
import numpy as np
import pytest
import torch

import ref64
import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import bf16, to64
from test_gpu_experts import w4

pytestmark = pytest.mark.gpu
HID, HQ, HEADS, D, P, WIDTH, PAGES, B = 256, 4, 2, 64, 16, 8, 30, 3
ROW = (HQ + 2 * HEADS) * D


class Block:
    def __init__(self, T, seed=0):
        rng = np.random.default_rng(seed)
        q, qkv = w4(rng, 1, ROW, HID)
        o, out = w4(rng, 1, HID, HQ * D)
        self.qkv64, self.o64 = [a[0] for a in q], [a[0] for a in o]
        self.qkv = sp.W4(qkv[0][0], qkv[1][0], qkv[2][0], ROW, HID)
        self.out = sp.W4(out[0][0], out[1][0], out[2][0], HID, HQ * D)
        self.freqs = sp.spear_rope_frequencies(D, kind=sp.ROPE_PARTS, factor=4.0, original=64.0)
        self.rope = sp.Rope(self.freqs.cuda())
        self.kv = sp.new_kv4(PAGES, HEADS, D, P)
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = dev(rng.permutation(PAGES).astype(np.int32))
        self.n_free = torch.full((1,), PAGES, dtype=torch.int32, device="cuda")
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.fresh = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.plan = sp.new_kv4_plan(B, T)
        self.rows = torch.empty(T, ROW, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(T, HID, dtype=torch.bfloat16, device="cuda")
        self.a = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.ws = (sp.new_workspace(T, ROW, HID, 0), sp.new_workspace(T, HID, HQ * D, 0), sp.new_kv4_workspace(T, B, T, HQ, self.kv, WIDTH))
        self.T = T

    def __call__(self, x):
        T, p = self.T, self.plan
        sp.spear_w4_linear(x, self.qkv, y=self.rows, out_dtype=sp.OUT_BF16, workspace=self.ws[0])
        sp.spear_kv4_plan(self.cached, self.fresh, self.table, self.free, self.n_free, T, P, plan=p)
        q, k, v = self.rows.view(T, -1, D).split((HQ, HEADS, HEADS), 1)
        sp.spear_rope_kv4_write(q, k, v, p.positions, p.slots, self.rope, self.kv, q_out=q)
        sp.spear_kv4_attention(q, self.kv, self.table, p.q_start, p.kv_len, T, y=self.a, workspace=self.ws[2])
        sp.spear_w4_linear_epilogue(self.a.view(T, -1), self.out, sp.Epilogue(residual=x), y=self.y, out_dtype=sp.OUT_BF16, workspace=self.ws[1])
        self.cached.copy_(p.kv_len)                       # the next step's
        self.n_free.copy_(p.n_left)
        return self.y


def reference(block, history, x64, fresh):
    """history: each request's x so far, in order -> y of the fresh rows, from the
    exact bf16 q/k/v rows that the library's projection gives (read back)."""
    rows = to64(block.rows_read).reshape(block.T, -1, D)
    start = np.concatenate(([0], np.cumsum(fresh)))
    out = np.zeros((block.T, HQ, D))
    err = np.zeros((block.T, HQ, D))
    for b, n in enumerate(fresh):
        r = rows[start[b]:start[b + 1]]
        pos = np.arange(len(history[b]["k"]), len(history[b]["k"]) + n)
        turn = lambda a: ref_kv4.rotate(a, pos, block.freqs.numpy(), 0)
        for name, a in (("k", turn(r[:, HQ:HQ + HEADS])), ("v", r[:, HQ + HEADS:])):
            history[b][name] += list(ref_kv4.value(*ref_kv4.hold(a)))
        q = torch.from_numpy(turn(r[:, :HQ])).bfloat16().double().numpy()
        k, v = np.array(history[b]["k"]), np.array(history[b]["v"])
        for i in range(n):
            m = pos[i] + 1
            for h in range(HQ):
                z = k[:m, h // 2] @ q[i, h] * D ** -0.5
                w = np.exp(z - z.max())
                w /= w.sum()
                out[start[b] + i, h] = w @ v[:m, h // 2]
                az = np.abs(k[:m, h // 2]) @ np.abs(q[i, h]) * D ** -0.5
                dz = (ref64.depth(D) + 12) * ref64.HALF_F32 * az.max() + 8 * ref64.HALF_F32 * (1 + 2 * np.abs(z).max())
                err[start[b] + i, h] = (2 * dz + 2 * ref64.depth(m) * ref64.HALF_F32 + ref64.HALF_BF16) * (w @ np.abs(v[:m, h // 2]))
    err += ref64.HALF_BF16 * (np.abs(out) + err)
    a = out.reshape(block.T, -1)
    t, te = ref64.linear(a, *block.o64)
    wo = np.abs((block.o64[0].astype(np.float64) - block.o64[2][:, None]) * block.o64[1][:, None])
    te = te + err.reshape(block.T, -1) @ wo.T
    y, ye = ref64.finish(t, te, ref64.NONE, False, residual=x64)
    return y, ref64.rounded(y, ye, ref64.HALF_BF16)


# two prompts, one of them in two chunks, and a request that comes later; then tokens
STEPS = [[21, 0, 9], [0, 17, 30], [1, 1, 1], [1, 2, 1], [0, 1, 1], [1, 1, 1]]
T = 47


@pytest.mark.parametrize("captured", [False, True])
def test_block(captured):
    block, history = Block(T), [{"k": [], "v": []} for _ in range(B)]
    x = torch.zeros(T, HID, dtype=torch.bfloat16, device="cuda")
    if captured:
        block(x)                                          # fresh is all zeros: nothing is taken or written
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block(x)
    worst = 0.0
    for i, fresh in enumerate(STEPS):
        n = sum(fresh)
        xi, x64 = bf16(np.random.default_rng(50 + i).normal(0, 1, (T, HID)))
        x.copy_(xi)
        block.fresh.copy_(dev(np.array(fresh, np.int32)))
        block.rows_read = sp.spear_w4_linear(x, block.qkv, out_dtype=sp.OUT_BF16)
        y = (g.replay(), block.y)[1] if captured else block(x)
        torch.cuda.synchronize()
        want, tol = reference(block, history, x64, fresh)
        worst = max(worst, float(np.max(np.abs(to64(y)[:n] - want[:n]) / tol[:n])))
        assert [len(h["k"]) for h in history] == block.cached.tolist()
    used = sum(-(-len(h["k"]) // P) for h in history)
    assert int(block.n_free) == PAGES - used and block.plan.status.tolist() == [0, 0]
    print(f"[block] captured={captured}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0
