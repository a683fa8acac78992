"""A step's plan, rotary positions, and the cache of 4 bits written and read,
against plain fp64 references."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import bf16, to64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ plan
def check_plan(cached, fresh, width, n_pages, n_free, T, P, seed=0, plan=None):
    rng = np.random.default_rng(seed)
    B = len(cached)
    free = rng.permutation(n_pages).astype(np.int32)
    table = rng.integers(0, 1000, (B, width)).astype(np.int32)
    want = ref_kv4.plan(cached, fresh, table, free, n_free, T, P)
    dt = dev(table)
    got = sp.spear_kv4_plan(dev(np.array(cached, np.int32)), dev(np.array(fresh, np.int32)), dt, dev(free),
                            dev(np.array([n_free], np.int32)), T, P, plan=plan)
    for name, g, w in zip(("q_start", "kv_len", "positions", "slots", "table", "n_left", "status"),
                          (got.q_start, got.kv_len, got.positions, got.slots, dt, got.n_left, got.status), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w), name
    return got


@pytest.mark.parametrize("B", [0, 1, 2, 63, 64, 65, 511, 513, 1000, 4096])
@pytest.mark.parametrize("P", [16, 1024])
def test_plan(B, P):
    rng = np.random.default_rng(B + P)
    cached = rng.integers(0, 3 * P, B)
    fresh = np.where(rng.random(B) < 0.1, rng.integers(0, 2 * P, B), rng.integers(0, 2, B))
    T = int(fresh.sum())
    check_plan(cached, fresh, 6, 3 * B + T // P + 5, 3 * B + T // P + 5, T + 3, P, seed=B)


@pytest.mark.parametrize("case", [
    dict(cached=[0, 15, 16, 17, 0], fresh=[1, 1, 1, 1, 0], T=4),
    dict(cached=[-5, 3], fresh=[2, -7], T=6),                            # negative lengths count as none
    dict(cached=[5, 5, 5], fresh=[10, 10, 10], T=17),                    # the second request is cut, the third gets nothing
    dict(cached=[5], fresh=[3], T=0),
    dict(cached=[0, 0, 40], fresh=[40, 40, 9], T=100, n_free=3),         # not enough pages
    dict(cached=[0], fresh=[40], T=40, n_free=0),
    dict(cached=[0], fresh=[40], T=40, n_free=-3),
    dict(cached=[0], fresh=[40], T=40, n_free=99999),                    # more than the list is long
    dict(cached=[60, 64, 200], fresh=[10, 10, 10], T=40, width=4),       # the table's rows are full, or were
    dict(cached=[0], fresh=[2 ** 31 - 1], T=50, width=9),
    dict(cached=[0] * 70, fresh=[2 ** 31 - 1] * 70, T=50, width=9),      # sums beyond 32 bits
])
def test_plan_at_its_edges(case):
    c = dict(width=12, n_pages=40, P=16)
    c.update(case)
    c.setdefault("n_free", c["n_pages"])
    check_plan(**c)


def test_plan_of_many_rows():
    check_plan([100, 0, 7], [20000, 1, 60000], 5000, 6000, 5999, 80100, 16)


def test_plan_in_a_graph():
    B, T, P, width = 20, 64, 16, 8
    cached, fresh = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    table, plan = torch.zeros(B, width, dtype=torch.int32, device="cuda"), sp.new_kv4_plan(B, T)
    free, nf = torch.arange(200, dtype=torch.int32, device="cuda").flip(0).contiguous(), torch.full((1,), 200, dtype=torch.int32, device="cuda")
    call = lambda p, t: sp.spear_kv4_plan(cached, fresh, t, free, nf, T, P, plan=p)
    call(plan, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(plan, table)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        cached.copy_(dev(rng.integers(0, 50, B).astype(np.int32)))
        fresh.copy_(dev(rng.integers(0, 4, B).astype(np.int32)))
        table.fill_(-9)
        other = table.clone()
        g.replay()
        e = call(sp.new_kv4_plan(B, T), other)
        torch.cuda.synchronize()
        assert torch.equal(table, other)
        for name in ("q_start", "kv_len", "positions", "slots", "n_left", "status"):
            assert torch.equal(getattr(plan, name), getattr(e, name)), name


# ------------------------------------------------------------------------ rope
def same_bf16(got, want64):
    """got is want64 rounded to bf16, from a value that is off by 2^-23 |y| + 2^-38 |x|:
    the factors are held as c0 + c1 with c1 2^-16 of c0 and rounded (2^-41); x c0 +
    p s0 is rounded once (2^-24 of its size), so are the small terms' product and sum
    (2^-40 each) and the last sum (2^-24)."""
    w = torch.from_numpy(want64)
    err = (got.double().cpu() - w).abs().numpy()
    before = 2.0 ** -23 * np.abs(want64) + 2.0 ** -38 * np.abs(want64).max() * 4
    assert (err <= ref_kv4.HALF_BF16 * (np.abs(want64) + before) + before).all()


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 8, 2), (1, 32, 128, 128), (3, 5, 64, 64), (2, 7, 96, 24), (5, 3, 192, 96), (4, 2, 256, 256),
                                       (4, 9, 256, 6), (2, 3, 40, 22), (700, 16, 128, 64), (4100, 3, 24, 24), (1, 1024, 64, 64)])
def test_rope(T, H, D, rot, layout):
    rng = np.random.default_rng(T * D + rot)
    x, x64 = bf16(rng.normal(0, 2, (T, H, D)))
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[0] = rng.choice([0, 2 ** 31 - 1, -7])
    f = sp.spear_rope_frequencies(rot)
    rope = sp.Rope(f.cuda(), layout, 1.25)
    want = ref_kv4.rotate(x64, pos, f.numpy(), layout, 1.25)
    y = sp.spear_rope(x, dev(pos), rope)
    same_bf16(y, want)
    # a part of a wider row, into another, and in place
    wide = torch.full((T, H + 3, D), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:H + 1] = x
    if D % 8 == 0:
        out = torch.full((T, H + 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
        sp.spear_rope(wide[:, 1:H + 1], dev(pos), rope, y=out[:, 1:])
        assert torch.equal(out[:, 1:], y) and bool((out[:, 0] == 5.0).all())
    part = wide[:, 1:H + 1]
    assert sp.spear_rope(part, dev(pos), rope, y=part) is part
    assert torch.equal(part, y) and bool((wide[:, 0] == 3.0).all()) and bool((wide[:, H + 1:] == 3.0).all())


def test_rope_leaves_the_other_channels_alone():
    """An infinity or a NaN beside the rotated channels stays where it is."""
    x = torch.ones(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 1, 40], x[1, 2, 63] = float("inf"), float("nan")
    y = sp.spear_rope(x, dev(np.array([5, 9], np.int32)), sp.Rope(sp.spear_rope_frequencies(32).cuda()))
    assert torch.equal(torch.isfinite(y), torch.isfinite(x)) and y[0, 1, 40] == float("inf")


# ------------------------------------------------------------- write and read
@pytest.mark.parametrize("T,Hq,heads,D,P,rot,layout", [
    (1, 1, 1, 64, 16, 64, 0), (1, 32, 8, 128, 64, 128, 0), (5, 6, 3, 96, 16, 24, 0), (7, 4, 2, 192, 32, 192, 1), (9, 2, 2, 256, 1024, 64, 1),
    (300, 10, 5, 64, 16, 32, 1), (1500, 8, 8, 128, 128, 128, 0), (3, 5, 1, 256, 16, 18, 0), (4, 3, 3, 128, 32, 0, 0)])
def test_write_and_read(T, Hq, heads, D, P, rot, layout):
    rng = np.random.default_rng(T + D)
    pages = -(-T // P) + 3
    row = Hq + 2 * heads
    qkv, x64 = bf16(rng.normal(0, 1, (T, row, D)) * np.exp2(rng.integers(-9, 9, (T, row, D // 32))).repeat(32, -1))
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:]
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = rng.choice([-1, pages * P, -(1 << 40), 1 << 40])
    f = sp.spear_rope_frequencies(max(rot, 2))
    rope = sp.Rope(f.cuda(), layout) if rot else None
    want = ref_kv4.rotate(x64, pos, f.numpy(), layout) if rot else x64
    cache = ref_kv4.Cache(pages, heads, D, P, rng)
    kv = sp.KV4(*(dev(a[n].copy()) for n in "kv" for a in (cache.codes, cache.scales)))
    qo = sp.spear_rope_kv4_write(q, k, v, dev(pos) if rot else None, dev(slots), rope, kv)
    same_bf16(qo, want[:, :Hq])
    cache.write("k", slots, want[:, Hq:Hq + heads])
    cache.write("v", slots, x64[:, Hq + heads:])
    # every byte of the cache, those that nothing was written to among them
    for name, codes, scales in (("k", kv.k_codes, kv.k_scales), ("v", kv.v_codes, kv.v_scales)):
        assert np.array_equal(scales.cpu().numpy(), cache.scales[name]), name
        assert np.array_equal(codes.cpu().numpy(), cache.codes[name]), name
    rk, rv = sp.spear_kv4_read(kv, dev(slots))
    assert np.array_equal(to64(rk), cache.read("k", slots)) and np.array_equal(to64(rv), cache.read("v", slots))
    # in place
    assert sp.spear_rope_kv4_write(q, k, v, dev(pos) if rot else None, dev(slots), rope, kv, q_out=q) is q
    assert torch.equal(q, qo) and np.array_equal(kv.k_codes.cpu().numpy(), cache.codes["k"])


def test_values_at_the_borders():
    """Ties, the exponent's step at 1.75, its two ends, zeros of both signs, and blocks
    with an infinity or a NaN: every bit as the definition has it."""
    rows = []
    ties = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for e in (-130, -127, -126, -125, -124, -20, 0, 20, 120, 124):
        for top in (4.0, 6.0, 6.96875, 7.0, 7.96875):
            x = np.concatenate(([top], ties[1:], -ties[1:], [0.0, -0.0], np.zeros(15)))
            rows.append(x * 2.0 ** e)
    rows.append(np.array([np.inf] + [1.0] * 31))
    rows.append(np.array([1.0] * 31 + [np.nan]))
    rows.append(np.full(32, 2.0 ** -133))
    rows.append(np.full(32, -0.0))
    while len(rows) % 2:
        rows.append(np.zeros(32))
    x, x64 = bf16(np.array(rows).reshape(-1, 1, 64))
    T = len(x64)
    kv, cache = sp.new_kv4(T, 1, 64, 16), ref_kv4.Cache(T, 1, 64, 16, np.random.default_rng(0))
    slots = np.arange(T, dtype=np.int64) * 16 + 3
    sp.spear_rope_kv4_write(x, x, x, None, dev(slots), None, kv)
    cache.write("v", slots, x64)
    for codes, scales in ((kv.k_codes, kv.k_scales), (kv.v_codes, kv.v_scales)):
        s = scales.cpu().numpy()[:, 0, :, 3]
        assert np.array_equal(s, cache.scales["v"][:, 0, :, 3])
        c, w = codes.cpu().numpy()[:, 0, 3].reshape(T, 2, 16), cache.codes["v"][:, 0, 3].reshape(T, 2, 16)
        fine = s != 255
        assert np.array_equal(c[fine], w[fine])
    k, _ = sp.spear_kv4_read(kv, dev(slots))
    got, want = to64(k), cache.read("v", slots)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_write_behind_4_gib():
    """Codes that lie beyond 2^32 bytes of the cache."""
    P, heads, D = 1024, 8, 256
    pages = (1 << 32) // (heads * P * D // 2) + 3
    kv = sp.new_kv4(pages, heads, D, P)
    rng = np.random.default_rng(5)
    x, x64 = bf16(rng.normal(0, 1, (4, heads, D)))
    slots = np.array([0, pages * P - 1, (pages - 2) * P + 17, pages * P], np.int64)
    sp.spear_rope_kv4_write(x, x, x, None, dev(slots), None, kv)
    k, v = sp.spear_kv4_read(kv, dev(slots))
    want = ref_kv4.value(*ref_kv4.hold(x64))
    want[3] = 0.0
    assert np.array_equal(to64(k), want) and np.array_equal(to64(v), want)


@pytest.mark.parametrize("layout", [sp.ROPE_HALF, sp.ROPE_PAIRS])
def test_rotated_keys_next_to_the_borders(layout):
    """Keys made so that many rotated channels lie within a few fp32 steps of a tie or
    of the exponent's step: the codes are those of the exact rotation."""
    rng = np.random.default_rng(3)
    T, D, heads, P = 400, 128, 2, 64
    f = sp.spear_rope_frequencies(D)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    target = rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.0]), (T, heads, D)) * rng.choice([-1.0, 1.0], (T, heads, D))
    k, k64 = bf16(ref_kv4.rotate(target, -pos.astype(np.int64), f.numpy(), layout) * np.exp2(rng.integers(-8, 8, (T, heads, 1))))
    small = rng.random((T, heads, 1)) < 0.2              # and pairs of very different size
    k = torch.where(torch.from_numpy(small).cuda() & (torch.arange(D, device="cuda") % 7 == 0), k * 2.0 ** -20, k)
    k64 = to64(k)
    slots = np.arange(T, dtype=np.int64)
    kv, cache = sp.new_kv4(-(-T // P), heads, D, P), ref_kv4.Cache(-(-T // P), heads, D, P, rng)
    sp.spear_rope_kv4_write(k, k, k, dev(pos), dev(slots), sp.Rope(f.cuda(), layout), kv)
    cache.write("k", slots, ref_kv4.rotate(k64, pos, f.numpy(), layout))
    got, _ = sp.spear_kv4_read(kv, dev(slots))
    assert np.array_equal(to64(got), cache.read("k", slots))
