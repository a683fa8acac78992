"""The routed tokens through their experts' two W4 layers, against the fp64
reference."""
import numpy as np
import pytest
import torch

import ref64
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from test_gpu_epilogue import bf16, to64

pytestmark = pytest.mark.gpu

# y and h are rounded to bf16, each off by at most 2^-8 relative; over many
# outputs the errors of h's independent roundings add in squares, as the terms do
RTOL_L2 = 2 * ref64.HALF_BF16


def w4(rng, E, N, K):
    codes = rng.integers(0, 16, (E, N, K), dtype=np.uint8)
    scales = (rng.uniform(0.5, 1.5, (E, N)) * 0.2 / np.sqrt(K)).astype(np.float32)
    zeros = rng.integers(5, 11, (E, N), dtype=np.uint8)
    packed = sp.spear_pack_w4(dev(codes.reshape(E * N, K)), sp.CODES_U4).view(E, N, K // 2)
    return (codes, scales, zeros), (packed, dev(scales), dev(zeros))


class Case:
    def __init__(self, M, E, topk, K, I, N, kind=sp.ACT_SILU, glu=True, bias=False, residual=False,
                 seed=0, ids=None):
        rng = np.random.default_rng(seed)
        self.rng, self.kind, self.glu = rng, kind, glu
        self.x, self.x64 = bf16(rng.normal(0, 1, (M, K)))
        NU = 2 * I if glu else I
        self.up, up = w4(rng, E, NU, K)
        self.down, down = w4(rng, E, N, I)
        self.ub = rng.normal(0, 0.3, (E, NU)).astype(np.float32) if bias else None
        self.db = rng.normal(0, 0.3, (E, N)).astype(np.float32) if bias else None
        self.experts = sp.Experts(*up, *down, up_bias=dev(self.ub) if bias else None,
                                  down_bias=dev(self.db) if bias else None, act=kind, glu=glu)
        if ids is None:
            ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]) if M else np.zeros((0, topk))
        self.ids = np.asarray(ids, np.int32).reshape(M, topk)
        self.weights = rng.uniform(-0.2, 1.0, (M, topk)).astype(np.float32)
        self.res, self.res64 = bf16(rng.normal(0, 1, (M, N))) if residual else (None, None)

    def run(self, **kw):
        kw.setdefault("residual", self.res)
        return sp.spear_w4_experts(self.x, self.experts, dev(self.ids), dev(self.weights), **kw)

    def reference(self):
        y, err = ref64.experts(self.x64, self.up, self.down, self.ids, self.weights, self.kind,
                               self.glu, self.ub, self.db, self.res64)
        return y, ref64.rounded(y, err, ref64.HALF_BF16)

    def check(self, y, what=""):
        ref, tol = self.reference()
        d = np.abs(to64(y) - ref)
        worst = float(np.max(d / tol)) if d.size else 0.0
        rel = float(np.linalg.norm(d) / max(np.linalg.norm(ref), 1e-300))
        print(f"[experts] {what}: worst {worst:.3f} of the bound, rel_l2 {rel:.2e}", flush=True)
        assert worst <= 1.0 and rel <= RTOL_L2, what


SHAPES = [  # M, E, topk, K, I, N
    (1, 1, 1, 32, 32, 1), (1, 8, 8, 64, 32, 64), (1, 64, 8, 512, 96, 130), (2, 4, 2, 96, 64, 33),
    (5, 300, 6, 160, 32, 48), (16, 16, 4, 416, 160, 200), (17, 3, 2, 128, 96, 66),
    (40, 8, 3, 1056, 64, 257), (64, 2, 1, 256, 288, 64), (130, 5, 2, 544, 128, 300),
    (300, 4, 4, 256, 192, 128), (700, 6, 2, 128, 64, 100)]


@pytest.mark.parametrize("M,E,topk,K,I,N", SHAPES)
@pytest.mark.parametrize("glu", [True, False])
def test_experts_parity(M, E, topk, K, I, N, glu):
    c = Case(M, E, topk, K, I, N, kind=(M + I) % 5, glu=glu, bias=N % 2 == 0, residual=K % 64 == 0,
             seed=M + E + K)
    c.check(c.run(), f"M={M} E={E} topk={topk} K={K} I={I} N={N} glu={glu} act={c.kind}")


@pytest.mark.parametrize("M", [1, 6, 33, 200])
def test_slots_without_an_expert(M):
    """Ids outside [0, E) add nothing, whatever their weight (NaN, inf); a token
    without any expert gives its residual, or zero."""
    for residual in (False, True):
        c = Case(M, 6, 3, 128, 64, 72, residual=residual, seed=M)
        away = c.rng.random((M, 3)) < 0.4
        away[0] = True
        c.ids[away] = c.rng.choice([-1, 6, 1 << 30, -(1 << 31)], int(away.sum()))
        clean = c.weights.copy()
        c.weights[away] = c.rng.choice([np.nan, np.inf], int(away.sum()))
        y = c.run()
        c.weights = clean
        c.check(y, f"away M={M} residual={residual}")
        first = to64(y)[0]
        assert np.array_equal(first, c.res64[0] if residual else np.zeros(72))


def test_all_slots_away():
    c = Case(9, 4, 2, 64, 32, 40, residual=True, ids=np.full((9, 2), -1))
    assert torch.equal(c.run(), c.res)


@pytest.mark.parametrize("M", [3, 50])
def test_one_expert_twice_and_one_for_all(M):
    """The same expert twice in a token; every token at one expert (the other
    experts empty)."""
    c = Case(M, 5, 4, 96, 64, 64, seed=2, ids=np.tile([[2, 2, 4, 2]], (M, 1)))
    c.check(c.run(), f"twice M={M}")
    c = Case(M, 7, 1, 96, 64, 64, seed=3, ids=np.full((M, 1), 6))
    c.check(c.run(), f"one expert M={M}")


def test_uneven_experts():
    """One expert with most tokens, several with one, some with none."""
    rng = np.random.default_rng(4)
    ids = np.where(rng.random((400, 1)) < 0.9, 3, rng.integers(0, 12, (400, 1)))
    c = Case(400, 12, 1, 128, 96, 80, seed=5, ids=ids)
    c.check(c.run(), "uneven")


@pytest.mark.parametrize("M", [2, 90])
def test_in_place_residual_and_rows_behind(M):
    c = Case(M, 4, 2, 128, 64, 96, residual=True, seed=6)
    buf = torch.full((M + 2, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:M]
    y.copy_(c.res)
    c.run(residual=y, y=y)
    c.check(y, f"in place M={M}")
    assert bool((buf[M:] == 7.0).all())


def test_signed_codes_have_zero_point_8():
    rng = np.random.default_rng(7)
    E, K, I, N, M = 3, 64, 32, 48, 10
    up, down = rng.integers(-8, 8, (E, 2 * I, K), dtype=np.int8), rng.integers(-8, 8, (E, N, I), dtype=np.int8)
    us, ds = np.full((E, 2 * I), 0.02, np.float32), np.full((E, N), 0.02, np.float32)
    ex = sp.Experts(sp.spear_pack_w4(dev(up.reshape(-1, K)), sp.CODES_S4).view(E, 2 * I, K // 2), dev(us), None,
                    sp.spear_pack_w4(dev(down.reshape(-1, I)), sp.CODES_S4).view(E, N, I // 2), dev(ds), None)
    x, x64 = bf16(rng.normal(0, 1, (M, K)))
    ids = rng.integers(0, E, (M, 2)).astype(np.int32)
    weights = rng.random((M, 2)).astype(np.float32)
    y = sp.spear_w4_experts(x, ex, dev(ids), dev(weights))
    ref, err = ref64.experts(x64, (up.astype(np.int16) + 8, us, np.full((E, 2 * I), 8)),
                             (down.astype(np.int16) + 8, ds, np.full((E, N), 8)), ids, weights, ref64.SILU, True)
    assert np.all(np.abs(to64(y) - ref) <= ref64.rounded(ref, err, ref64.HALF_BF16))


def test_one_workspace_for_many_sizes_and_no_tokens():
    """A workspace for the most tokens serves fewer; what an earlier call left
    there does not matter."""
    big = Case(120, 6, 2, 128, 64, 64, seed=8)
    ws = sp.new_experts_workspace(120, 2, big.experts)
    ws.fill_(0xFF)
    a = big.run(workspace=ws)
    for M in (1, 20, 119):
        c = Case(M, 6, 2, 128, 64, 64, seed=9 + M)
        c.check(c.run(workspace=ws), f"shared workspace M={M}")
    assert torch.equal(a, big.run(workspace=ws))
    c = Case(0, 6, 2, 128, 64, 64)
    assert c.run(workspace=ws).shape == (0, 64)


def test_a_row_does_not_depend_on_its_neighbours():
    """A token's result is the same bits alone, in a batch and after a shuffle."""
    c = Case(150, 6, 2, 256, 64, 96, seed=10)
    y = c.run()
    assert torch.equal(y, c.run())
    p = c.rng.permutation(150)
    z = sp.spear_w4_experts(c.x[torch.from_numpy(p).cuda()].contiguous(), c.experts, dev(c.ids[p]), dev(c.weights[p]))
    assert torch.equal(z, y[torch.from_numpy(p).cuda()])


@pytest.mark.parametrize("M,E,topk", [(16, 9, 1), (17, 9, 1), (2, 64, 8), (3, 40, 6), (4, 1, 4), (33, 2, 1),
                                      (31, 2, 1), (32, 2, 1)])
def test_where_the_launches_change(M, E, topk):
    """Slots on both sides of the two-launch form and of the 64-row tiles."""
    c = Case(M, E, topk, 160, 96, 72, bias=True, residual=True, seed=M + E,
             ids=None if E >= topk else np.zeros((M, topk)))
    c.check(c.run(), f"M={M} E={E} topk={topk}")


@pytest.mark.parametrize("K,I", [(2048, 2048), (2080, 2112)])
def test_tiles_of_128_rows(K, I):
    """Many slots an expert at depths long enough for the largest tiles; the last
    tile of an expert ragged, one expert empty, some slots elsewhere."""
    rng = np.random.default_rng(K)
    E, M, N = 3, 2200, 136
    ids = rng.choice([0, 2, 2, 2, -1], (M, 1))
    c = Case(M, E, 1, K, I, N, bias=True, residual=True, seed=K, ids=ids)
    c.check(c.run(), f"128 rows K={K} I={I}")


@pytest.mark.parametrize("M", [2, 40])
def test_weights_past_32_bit_offsets(M):
    """More than 2^32 bytes of weights: the last expert's rows are those of an
    experts' handle that has it alone."""
    E, K, I, N = 512, 8192, 1056, 64
    packed = torch.randint(0, 256, (E, 2 * I, K // 2), dtype=torch.uint8, device="cuda")
    assert packed.numel() > 1 << 32
    us = torch.full((E, 2 * I), 0.002, device="cuda")
    down = torch.randint(0, 256, (E, N, I // 2), dtype=torch.uint8, device="cuda")
    ds = torch.full((E, N), 0.01, device="cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    weights = torch.rand(M, 1, device="cuda")
    ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
    y = sp.spear_w4_experts(x, sp.Experts(packed, us, None, down, ds, None), ids, weights)
    # (8 copies, of which the fourth is asked for)
    alone = sp.Experts(packed[-1:].expand(8, -1, -1).contiguous(), us[:8], None,
                       down[-1:].expand(8, -1, -1).contiguous(), ds[:8], None)
    z = sp.spear_w4_experts(x, alone, torch.full_like(ids, 3), weights)
    assert torch.equal(y, z) and bool(torch.isfinite(y.float()).all())
