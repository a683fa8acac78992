"""Attention over the cache of 4 bits against plain fp64."""
import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev
from kv4_util import Step, bf16, to64

pytestmark = pytest.mark.gpu
DIMS = [64, 96, 128, 192, 256]


def room(P, many):
    """Table columns behind the pages.  A step of few rows and keys takes the kernel
    for few rows alone, and the keys are what the table has room for: with room for
    2^24, requests of more than 32 rows take the kernel for many."""
    return (1 << 24) // P if many else 0


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("Hq,heads,P", [(1, 1, 16), (8, 8, 64), (8, 2, 128), (5, 1, 32), (16, 1, 1024), (24, 1, 256)])
def test_one_token(D, Hq, heads, P):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300]
    Step(kv, [1] * len(kv), Hq, heads, D, P, seed=D + Hq).check(f"one token D={D} {Hq}/{heads} P={P}")


@pytest.mark.parametrize("n", [1, 255, 257, 1000, 2500])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_request(n, D):
    """A long axis cut into chunks for a single request."""
    Step([n], [1], 4, 1, D, 16, seed=n).check(f"one request of {n} D={D}")


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("Hq,heads", [(1, 1), (6, 2), (7, 1)])
@pytest.mark.parametrize("many", [False, True])
def test_few_and_many_tokens(D, Hq, heads, many):
    """Requests of one token, of a few and of whole prompts side by side."""
    fresh = [1, 2, 3, 17, 40, 5, 70, 1]
    kv = [90, 2, 64, 17, 101, 128, 70, 1]
    Step(kv, fresh, Hq, heads, D, 32, seed=D + Hq, pad=5, width=room(32, many)).check(f"mixed D={D} {Hq}/{heads} many={many}")


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("fresh,G", [(33, 1), (64, 2), (65, 4), (130, 2), (257, 1), (300, 3)])
def test_chunks_of_a_prompt(D, fresh, G):
    """Rows that end inside a tile of 128 or 256, on keys that end inside a step."""
    Step([fresh + 3, fresh, fresh + 200], [fresh, fresh, 1], G, 1, D, 16, seed=fresh, pad=1, width=room(16, True)).check(
        f"{fresh} rows x {G}, D={D}")


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 1 << 30])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pad", [2, 1 << 18])
def test_windows(window, D, pad):
    """(with many padded rows, requests of more than 32 take the kernel for many)"""
    s = Step([5, 64, 200, 333, 90, 1], [1, 64, 3, 50, 1, 1], 4, 2, D, 16, seed=window % 97, pad=2)
    s.check(f"window {window} D={D}", window=window)
    if pad > 2:
        q = torch.zeros(pad, 4, D, dtype=torch.bfloat16, device="cuda")
        q[: s.T] = s.q
        y = sp.spear_kv4_attention(q, s.kv4, s.dtable, s.dstart, s.dkv, 64, window=window, y=torch.full_like(q, 7.0))
        s.check(f"window {window} D={D} of {pad} rows", y=y[: s.T], window=window)
        assert bool((y[s.T:] == 7.0).all())


@pytest.mark.parametrize("fresh", [[1, 1, 1], [0, 5, 40]])
@pytest.mark.parametrize("many", [False, True])
def test_rows_that_see_nothing(fresh, many):
    """No keys at all, fewer keys than rows, requests without rows."""
    s = Step([0, 3, 20], fresh, 4, 2, 128, 16, seed=3, pad=3, width=room(16, many))
    y = s.check("rows without keys")
    for b, n in enumerate(s.kv):
        t0, t1 = s.q_start[b], s.q_start[b + 1]
        blind = t0 + max(0, (t1 - t0) - n)
        assert bool((y[t0:blind] == 0).all())


def test_no_rows_no_requests():
    s = Step([5, 9], [0, 0], 2, 2, 64, 16, pad=4)
    s.check("no rows")
    kv = s.kv4
    e = lambda *n: torch.empty(*n, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert sp.spear_kv4_attention(q, kv, s.dtable, torch.zeros(3, dtype=torch.int32, device="cuda"), s.dkv, 1).shape == (0, 2, 64)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(q, 7.0)
    sp.spear_kv4_attention(q, kv, e(0, 4), torch.zeros(1, dtype=torch.int32, device="cuda"), e(0), 1, y=y)
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("window,many", [(0, False), (0, True), (40, False)])
def test_masked_places_may_hold_anything(window, many):
    """NaN in keys and values that some rows see and others do not: only the
    rows that see them are NaN; pages that were let go are as if masked."""
    for seed, D in enumerate(DIMS):
        s = Step([70, 130, 200, 33], [20, 1, 60, 2], 4, 2, D, 16, seed=seed, pad=2, width=room(16, many))
        c = s.cache
        def spoil(b, key, name, head, block):
            c.scales[name][s.table[b, key // 16], head, block, key % 16] = 255
        spoil(0, 60, "v", 0, 0)                          # seen by the last ten rows of the request
        spoil(0, 55, "v", 1, D // 32 - 1)
        spoil(0, 66, "k", 1, 1)
        spoil(2, 150, "v", 0, 1)
        spoil(2, 171, "k", 0, 0)
        s.table[1, 2] = -1
        s.table[2, 4] = c.pages
        s.table[2, 5] = 2 ** 31 - 1
        s.table[3, 0] = -2 ** 31
        s.to_device()
        s.check(f"masked places D={D} window={window} many={many}", window=window)


@pytest.mark.parametrize("n", [700, 6000])
@pytest.mark.parametrize("D,Hq,heads", [(64, 2, 1), (128, 8, 1), (256, 3, 3)])
def test_nan_among_keys_that_count_for_nothing(n, D, Hq, heads):
    """A long axis in chunks: a NaN that a row sees makes it NaN, from a chunk whose
    other scores lie far below the rest as well."""
    for where in ("q", "k", "v"):
        s = Step([n], [1], Hq, heads, D, 16, seed=n + D)
        if where == "q":
            s.q[0, 0, 5] = float("nan")
            s.q64[0, 0, 5] = np.nan
        else:
            s.cache.scales[where][s.table[0, n // 2 // 16], 0, 1, n // 2 % 16] = 255
        s.to_device()
        want, _, _, _ = ref_kv4.attention(s.q64, s.cache, s.table, s.q_start, s.kv, 40.0)
        assert np.isnan(want).any() and (heads == 1 or not np.isnan(want).all())
        # scores of some hundreds: outside the chunk of the largest, probabilities are 0
        got = to64(s.run(scale=40.0))
        assert (np.isnan(got) == np.isnan(want)).all(), where


@pytest.mark.parametrize("many", [False, True])
def test_every_page_let_go(many):
    s = Step([40, 70], [1, 30], 2, 1, 64, 16, seed=1, width=room(16, many))
    s.table[:] = -1
    s.to_device()
    y = s.check("no pages")
    assert bool((y == 0).all())


def test_lengths_beyond_the_table_are_held():
    """kv_len past the table's room and q_start past the rows read nothing outside."""
    s = Step([48, 20], [1, 2], 2, 1, 64, 16, seed=2)
    want = s.run()
    s.dkv = dev(np.array([1 << 30, 20], np.int32))
    s.dstart = dev(np.array([0, 1, 3], np.int32))
    got = s.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1:], want[1:])
    s.dstart = dev(np.array([-4, 1, 1 << 20], np.int32))
    s.dkv = dev(np.array([-3, 20], np.int32))
    got = s.run()
    assert torch.equal(got[1:], want[1:]) and bool((got[0] == 0).all())


@pytest.mark.parametrize("q_sd,scale", [(40.0, None), (1e-3, None), (1.0, 3.0), (1.0, 1e-20), (1e18, 1e-18)])
@pytest.mark.parametrize("many", [False, True])
def test_sharp_and_flat_rows(q_sd, scale, many):
    Step([200, 90], [1, 33], 4, 2, 128, 32, seed=9, q_sd=q_sd, width=room(32, many)).check(f"q of {q_sd}, scale {scale}", scale=scale)


@pytest.mark.parametrize("many", [False, True])
def test_infinite_queries_stay_in_their_rows(many):
    s = Step([50, 40], [1, 30], 2, 1, 64, 16, seed=4, width=room(16, many))
    want = s.run()
    s.q[3, 1, 7], s.q[9, 0, 0] = float("inf"), float("nan")
    got = s.run()
    spoilt = torch.zeros(s.T, 2, dtype=torch.bool, device="cuda")
    spoilt[3, 1] = spoilt[9, 0] = True
    assert bool(got[spoilt].isnan().all()) and torch.equal(got[~spoilt], want[~spoilt])


@pytest.mark.parametrize("many", [False, True])
def test_strided_queries_in_place_and_without_lse(many):
    s = Step([50, 40, 200], [1, 30, 2], 6, 2, 128, 16, seed=6, width=room(16, many))
    want = s.check("whole rows")
    wide = torch.full((s.T, 10, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = s.q
    assert torch.equal(s.run(q=wide[:, 2:8]), want)
    assert torch.equal(s.run(lse=False), want)
    q = s.q.clone()
    assert s.run(q=q, y=q) is q and torch.equal(q, want)


@pytest.mark.parametrize("most", [0, 1, 3, 30, 1 << 40])
def test_max_fresh_is_only_a_hint(most):
    Step([50, 40, 200, 64], [1, 30, 2, 7], 6, 2, 128, 16, seed=7, width=room(16, True)).check(f"max_fresh {most}, wide", max_fresh=most)
    s = Step([50, 40, 200, 64], [1, 30, 2, 7], 6, 2, 128, 16, seed=7)
    s.check(f"max_fresh {most}", max_fresh=most)


@pytest.mark.parametrize("B", [64, 65, 300])
def test_many_requests(B):
    rng = np.random.default_rng(B)
    kv = rng.integers(1, 40, B).tolist()
    Step(kv, [min(n, int(f)) for n, f in zip(kv, rng.integers(0, 3, B))], 2, 1, 64, 16, seed=B, pad=1).check(f"{B} requests")


def test_behind_4_gib():
    """Codes beyond 2^32 bytes of the cache, scales beyond 2^28."""
    P, heads, D = 1024, 8, 256
    pages = (1 << 32) // (heads * P * D // 2) + 2
    kv = sp.new_kv4(pages, heads, D, P)
    rng = np.random.default_rng(8)
    n = 100
    x, x64 = bf16(rng.normal(0, 1, (n, heads, D)))
    q, q64 = bf16(rng.normal(0, 1, (1, heads, D)))
    table = np.array([[pages - 1]], np.int32)
    slots = (pages - 1) * P + np.arange(n)
    sp.spear_rope_kv4_write(x, x, x, None, dev(slots), None, kv)
    small = ref_kv4.Cache(1, heads, D, P, rng)
    for name in "kv":
        small.write(name, np.arange(n), x64)
    y = sp.spear_kv4_attention(q, kv, dev(table), dev(np.array([0, 1], np.int32)), dev(np.array([n], np.int32)), 1)
    want, err, _, _ = ref_kv4.attention(q64, small, np.zeros((1, 1), np.int32), [0, 1], [n], D ** -0.5)
    assert (np.abs(to64(y) - want) <= err + ref_kv4.HALF_BF16 * (np.abs(want) + err)).all()


def test_repeats_bit_for_bit():
    s = Step([900, 2000, 333], [1, 70, 2], 8, 2, 128, 16, seed=11, width=room(16, True))
    want, lse = s.run(), s.lse
    for _ in range(3):
        assert torch.equal(s.run(), want) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("D,Hq,heads,n", [(64, 1, 1, 6000), (128, 8, 1, 20000), (96, 16, 1, 12000), (128, 2, 2, 33000), (256, 5, 1, 9000)])
def test_many_chunks(D, Hq, heads, n):
    """Chunks joined by groups, and groups joined."""
    Step([n, 40], [1, 1], Hq, heads, D, 64, seed=n).check(f"{n} keys of D={D}, {Hq}/{heads}")


def test_chunks_of_many_rows():
    """A few dozen rows over a long context: cut, and joined by a second launch."""
    Step([9000, 700], [40, 9], 4, 1, 64, 64, seed=12, width=room(64, True)).check("40 rows on 9000 keys")
    Step([5000], [70], 2, 1, 256, 16, seed=13, width=room(16, True)).check("70 rows on 5000 keys, D=256")
    Step([4000, 300], [130, 20], 2, 1, 128, 16, seed=14, width=room(16, True)).check("130 rows on 4000 keys, eight waves")


def test_one_workspace_for_calls_of_all_sizes():
    """Calls of other sizes in between leave the counters as they found them."""
    big = Step([6000, 300, 1, 900], [1, 60, 1, 2], 8, 2, 128, 16, seed=14, width=room(16, True))
    small = Step([2500], [1], 8, 2, 128, 16, seed=15)
    wide = Step([4000, 17], [1, 9], 16, 1, 256, 16, seed=16)
    ws = max((sp.new_kv4_workspace(s.T, len(s.kv), max(s.fresh), s.Hq, s.kv4, s.width) for s in (big, small, wide)), key=len)
    want = [s.run() for s in (big, small, wide)]
    for _ in range(3):
        for s, w in zip((big, small, wide), want):
            assert torch.equal(s.run(workspace=ws), w)


@pytest.mark.parametrize("width", [120, 1 << 20])
def test_in_a_graph(width):
    """Captured once for the largest step and replayed on others: lengths, pages and
    rows change, the launches do not."""
    B, T, Hq, heads, D, P = 6, 40, 8, 2, 128, 16
    steps = [Step(kv, fresh, Hq, heads, D, P, seed=20 + i, pad=T - sum(fresh), width=width - max([1] + [-(-n // P) for n in kv]))
             for i, (kv, fresh) in enumerate([([1900, 30, 1, 400, 64, 17], [1, 1, 1, 1, 1, 1]), ([50, 60, 20, 16, 0, 5], [30, 1, 3, 0, 0, 5]),
                                              ([1, 1900, 1900, 3, 3, 3], [1, 1, 1, 1, 1, 1]), ([0] * 6, [0] * 6)])]
    pages = max(s.cache.pages for s in steps)
    kv = sp.new_kv4(pages, heads, D, P)
    e = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    q, table, start, n = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"), e(B, width), e(B + 1), e(B)
    y, lse = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    ws = sp.new_kv4_workspace(T, B, 30, Hq, kv, width)
    call = lambda y, lse, ws: sp.spear_kv4_attention(q, kv, table, start, n, 30, y=y, lse=lse, workspace=ws)

    def put(s):
        for mine, theirs in ((kv.k_codes, s.kv4.k_codes), (kv.k_scales, s.kv4.k_scales), (kv.v_codes, s.kv4.v_codes), (kv.v_scales, s.kv4.v_scales)):
            mine[: theirs.shape[0]].copy_(theirs)
        q.copy_(s.q), table.copy_(s.dtable), start.copy_(s.dstart), n.copy_(s.dkv)

    put(steps[0])
    call(y, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y, lse, ws)
    for s in steps + steps[:2]:
        put(s)
        y.fill_(7.0), lse.fill_(7.0)
        g.replay()
        y2, lse2 = torch.full_like(y, 7.0), torch.full_like(lse, 7.0)
        call(y2, lse2, None)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(lse, lse2)
        s.lse = lse
        s.check("replayed", y=y)


def test_two_streams_at_once():
    steps = [Step([3000, 70], [1, 40], 8, 2, 128, 16, seed=31, width=room(16, True)), Step([40, 2500, 9], [9, 1, 1], 4, 4, 64, 32, seed=32)]
    want = [s.run() for s in steps]
    ws = [sp.new_kv4_workspace(s.T, len(s.kv), max(s.fresh), s.Hq, s.kv4, s.width) for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(6):
        for i, s in enumerate(steps):
            got[i] = sp.spear_kv4_attention(s.q, s.kv4, s.dtable, s.dstart, s.dkv, max(s.fresh), y=got[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for s, g, w in zip(steps, got, want):
        n = int(s.q_start[-1])
        assert torch.equal(g[:n], w[:n])


def test_many_short_requests_around_a_long_one():
    """Parts of a request cut into chunks behind a thousand whole tiles: each request's
    rows are those of a call of its own."""
    heads, D, P, fresh, n_long = 8, 64, 64, 17, 40000
    kv_len = np.full(512, 30, np.int32)
    kv_len[[3, 509]] = n_long
    counts = np.full(512, fresh, np.int32)
    counts[100] = 40
    kv_len[100] = 64
    pages = -(-kv_len // P)
    width = int(pages.max()) + room(P, True)
    table = torch.full((512, width), -1, dtype=torch.int32, device="cuda")
    first = np.concatenate(([0], np.cumsum(pages)))
    for b in (3, 509, 100):
        table[b, : pages[b]] = torch.arange(first[b], first[b + 1], dtype=torch.int32, device="cuda")
    one = pages == 1
    table[torch.from_numpy(np.flatnonzero(one)).cuda(), 0] = dev(first[:-1][one].astype(np.int32))
    kv = sp.new_kv4(int(first[-1]), heads, D, P)
    g = torch.Generator(device="cuda").manual_seed(4)
    places = int(first[-1]) * P
    k, v = (torch.randn(places, heads, D, device="cuda", generator=g, dtype=torch.float32).bfloat16() for _ in "kv")
    sp.spear_rope_kv4_write(k, k, v, None, torch.arange(places, device="cuda"), None, kv)
    start = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    q = torch.randn(int(start[-1]), heads, D, device="cuda", generator=g, dtype=torch.float32).bfloat16()
    y = sp.spear_kv4_attention(q, kv, table, dev(start), dev(kv_len), 40)
    for b in (0, 3, 100, 300, 508, 509, 510, 511):
        t0, t1 = int(start[b]), int(start[b + 1])
        alone = sp.spear_kv4_attention(q[t0:t1].contiguous(), kv, table[b : b + 1, : pages[b]].contiguous(),
                                       dev(np.array([0, t1 - t0], np.int32)), dev(kv_len[b : b + 1]), t1 - t0)
        # two roundings to bf16, and in the kernel for many rows P's, with |v| <= 6
        off = (y[t0:t1].double() - alone.double()).abs()
        bound = 2.1 * ref_kv4.HALF_BF16 * alone.double().abs() + (6 * ref_kv4.HALF_BF16 if b == 100 else 2 ** -14)
        assert bool((off <= bound).all()), (b, float(off.max()))
