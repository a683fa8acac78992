"""The cache of 4 bits without a GPU: the oracle's rounding, the rotation's
frequencies, refusals of the entry points before any HIP call, and the binding's
checks of its tensors."""
import ctypes
import math

import numpy as np
import pytest
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp

E_NULL, E_SHAPE, E_ALIGN, E_ARG, E_WS = -1, -2, -3, -4, -5
A = 0x10000            # fake, aligned device addresses: never dereferenced


def test_oracle_levels_and_ties():
    x = np.zeros(64)
    x[:10] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 0.2500001]
    x[32:36] = [7.0, 3.0, 1.0, -0.5]                     # 7 = 1.75 * 4: the next power of two
    codes, bytes_ = ref_kv4.hold(x)
    assert list(codes[:10]) == [7, 0, 2, 2, 4, 4, 6, 6, 14, 1] and bytes_[0] == 127
    assert bytes_[1] == 128 and list(codes[32:36]) == [6, 3, 1, 8]
    v = ref_kv4.value(codes, bytes_)
    assert list(v[32:36]) == [8.0, 3.0, 1.0, 0.0] and v[0] == 6.0
    codes, bytes_ = ref_kv4.hold(np.array([np.nan] + [1.0] * 31 + [np.inf] + [0.0] * 31 + [0.0] * 32))
    assert list(bytes_) == [255, 255, 2]


@pytest.mark.parametrize("rot", [2, 4, 24, 64, 128, 256])
def test_frequencies(rot):
    base, s, ctx = 10000.0, 8.0, 2048.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    get = lambda kind: sp.spear_rope_frequencies(rot, base, kind, s, ctx, 1.0, 32.0).numpy()
    np.testing.assert_allclose(get(sp.ROPE_PLAIN), f, rtol=1e-14)
    np.testing.assert_allclose(get(sp.ROPE_LINEAR), f / s, rtol=1e-14)
    if rot > 2:
        g = get(sp.ROPE_BASE)
        assert g[0] == 1.0 and abs(g[-1] * s / f[-1] - 1) < 1e-12       # fastest as before, slowest s times slower
    turns = ctx * f / (2 * math.pi)
    g = get(sp.ROPE_PARTS)
    for a, b, t in zip(g, f, turns):
        want = b if t >= 32 else b / s if t <= 1 else ((t - 1) / 31) * b + (1 - (t - 1) / 31) * b / s
        assert abs(a / want - 1) < 1e-13


def test_frequencies_refusals():
    lib, out = sp.load(), (ctypes.c_double * 128)()
    f = lambda rot=8, base=1e4, kind=0, factor=1.0, ctx=1.0, low=1.0, high=2.0, o=out: lib.spear_rope_frequencies(
        rot, base, kind, factor, ctx, low, high, o)
    assert f() == 0 and f(o=None) == E_NULL
    assert f(rot=0) == f(rot=7) == f(rot=258) == f(rot=2, kind=2) == E_SHAPE
    assert f(kind=4) == f(kind=-1) == f(base=1.0) == f(factor=0.0) == f(base=float("nan")) == E_ARG
    assert f(kind=3, ctx=0.0) == f(kind=3, low=2.0) == f(kind=3, high=float("inf")) == E_ARG


def kv4(**kw):
    p = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, pages=4, heads=2, D=128, P=16)
    p.update(kw)
    return ctypes.byref(sp._KV4(*p.values()))


BAD_KV4 = ((dict(k_codes=None), E_NULL), (dict(v_scales=None), E_NULL), (dict(pages=0), E_SHAPE), (dict(pages=1 << 31), E_SHAPE),
           (dict(heads=0), E_SHAPE), (dict(heads=1025), E_SHAPE), (dict(D=32), E_SHAPE), (dict(D=80), E_SHAPE), (dict(P=8), E_SHAPE),
           (dict(P=48), E_SHAPE), (dict(P=2048), E_SHAPE), (dict(k_scales=A + 4), E_ALIGN), (dict(v_codes=A + 8), E_ALIGN))


def test_plan_refusals():
    lib = sp.load()

    def f(cached=A, fresh=A, B=2, table=A, width=4, free=A, n_pages=8, n_free=A + 4, T=4, P=16, step=True, **kw):
        s = dict(q_start=A, kv_len=2 * A, positions=A, slots=A, n_left=2 * A, status=A)
        s.update(kw)
        return lib.spear_kv4_plan(cached, fresh, B, table, width, free, n_pages, n_free, T, P,
                                  ctypes.byref(sp._Step(*s.values())) if step else None, None)

    assert f(step=False) == E_NULL
    for k in ("cached", "fresh", "table", "free", "n_free", "q_start", "kv_len", "positions", "slots", "n_left", "status"):
        assert f(**{k: None}) == E_NULL, k
    assert f(B=-1) == f(B=4097) == f(T=-1) == f(T=(1 << 23) + 1) == f(P=24) == f(P=8) == f(width=0) == E_SHAPE
    assert f(width=(1 << 26) + 1) == f(n_pages=-1) == f(n_pages=1 << 31) == E_SHAPE
    for k in ("cached", "table", "free", "n_free", "positions", "status"):
        assert f(**{k: A + 2}) == E_ALIGN, k
    assert f(slots=A + 4) == E_ALIGN
    assert f(kv_len=A) == f(n_left=A + 4) == E_ARG       # the lengths' and the free list's own words


def test_rope_refusals():
    lib = sp.load()

    def f(x=A, xs=256, T=4, H=2, D=128, pos=A, y=2 * A, ys=256, rope=True, freqs=A, scale=1.0, rot=128, layout=0):
        r = sp._Rotation(freqs, scale, rot, layout)
        return lib.spear_rope(x, xs, T, H, D, pos, ctypes.byref(r) if rope else None, y, ys, None)

    assert f(rope=False) == f(freqs=None) == f(x=None) == f(pos=None) == f(y=None) == E_NULL
    assert f(T=-1) == f(T=(1 << 23) + 1) == f(H=0) == f(H=1025, xs=1 << 20, ys=1 << 20) == f(D=12) == f(D=264, xs=528, ys=528) == E_SHAPE
    assert f(xs=248) == f(xs=260) == f(ys=128) == f(rot=0) == f(rot=130) == f(rot=3) == f(y=A, ys=512) == E_SHAPE
    assert f(layout=2) == f(scale=float("inf")) == f(scale=float("nan")) == E_ARG
    assert f(x=A + 8) == f(y=A + 2) == f(pos=A + 2) == f(freqs=A + 4) == E_ALIGN


def test_write_and_read_refusals():
    lib = sp.load()

    def f(q=A, qs=512, k=A, ks=256, v=A, vs=256, T=4, Hq=4, pos=A, slots=A, rope=True, rot=64, freqs=A, y=2 * A, ys=512, **kw):
        r = sp._Rotation(freqs, 1.0, rot, 0)
        return lib.spear_rope_kv4_write(q, qs, k, ks, v, vs, T, Hq, pos, slots, ctypes.byref(r) if rope else None, kv4(**kw), y, ys,
                                        None)

    for k in ("q", "k", "v", "slots", "pos", "y", "freqs"):
        assert f(**{k: None}) == E_NULL, k
    assert f(rope=False, pos=None, qs=8) == E_SHAPE      # without a rotation no positions are wanted
    assert f(T=-1) == f(Hq=0) == f(qs=504) == f(ks=128) == f(vs=257) == f(ys=8) == f(rot=130) == f(y=A, ys=1024) == E_SHAPE
    assert f(q=A + 8) == f(v=A + 2) == f(slots=A + 4) == f(y=A + 8) == E_ALIGN
    read = lambda slots=A, T=4, k=A, v=A, **kw: lib.spear_kv4_read(kv4(**kw), slots, T, k, v, None)
    assert read(slots=None) == E_NULL and read(T=-1) == E_SHAPE and read(k=A + 8) == read(slots=A + 4) == E_ALIGN
    for kw, st in BAD_KV4:
        assert f(**kw, qs=4096, ks=1 << 20, vs=1 << 20, ys=4096) == st and read(**kw) == st, kw
    assert lib.spear_kv4_read(None, A, 4, A, A, None) == E_NULL


def test_attention_refusals():
    lib = sp.load()

    def f(q=A, qs=512, T=4, Hq=4, table=A, width=4, q_start=A, kv_len=A, B=2, most=2, scale=1.0, window=0, y=2 * A, lse=None, ws=A,
          wsb=1 << 30, **kw):
        return lib.spear_kv4_attention(q, qs, T, Hq, kv4(**kw), table, width, q_start, kv_len, B, most, scale, window, y, lse, ws, wsb,
                                       None)

    for k in ("q", "table", "q_start", "kv_len", "y", "ws"):
        assert f(**{k: None}) == E_NULL, k
    for kw, st in BAD_KV4:
        assert f(**kw) == st, kw
    assert f(T=-1) == f(B=-1) == f(B=4097) == f(Hq=3) == f(Hq=0) == f(Hq=256, qs=1 << 16) == f(width=0) == f(most=-1) == E_SHAPE
    assert f(qs=504) == f(qs=516) == f(window=-1) == f(width=1 << 30) == f(T=1 << 23, Hq=32, qs=4096) == E_SHAPE
    assert f(q=A, y=A, qs=1024) == E_SHAPE
    for s in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert f(scale=s) == E_ARG
    assert f(q=A + 8) == f(y=A + 8) == f(lse=A + 2) == f(ws=A + 64) == f(kv_len=A + 2) == E_ALIGN
    need = sp.spear_kv4_attention_workspace_size(4, 2, 2, 4, 2, 128, 4, 16)
    assert need > 0 and f(wsb=need - 1) == E_WS
    assert sp.spear_kv4_attention_workspace_size(4, 2, 2, 3, 2, 128, 4, 16) == 0


def test_attention_workspace_serves_smaller_steps():
    f = sp.spear_kv4_attention_workspace_size
    for Hq, heads, D in ((8, 8, 64), (32, 8, 128), (40, 1, 256)):
        whole = f(2048, 64, 2048, Hq, heads, D, 100, 64)
        for T in (1, 2, 16, 63, 64, 65, 500, 2047):
            for B in (1, 3, 64):
                for most in (1, 5, T):
                    assert 0 < f(T, B, most, Hq, heads, D, 100, 64) <= whole, (T, B, most)


def refused(status, f, *a, **kw):
    with pytest.raises(sp.SpearError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value


def test_binding_checks_its_tensors():
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    kv = sp.new_kv4(4, 2, 64, 16, device="cpu")
    refused(E_ARG, sp.KV4, kv.k_codes.int(), kv.k_scales, kv.v_codes, kv.v_scales)
    refused(E_SHAPE, sp.KV4, kv.k_codes, kv.k_scales, kv.v_codes[:3], kv.v_scales)
    refused(E_SHAPE, sp.KV4, kv.k_codes[0], kv.k_scales, kv.v_codes, kv.v_scales)
    rope = sp.Rope(sp.spear_rope_frequencies(64))
    refused(E_ARG, sp.Rope, torch.zeros(4))
    x, pos, slots = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i64)
    refused(E_ARG, sp.spear_rope, x, pos, rope)                                    # on the CPU
    refused(E_ARG, sp.spear_rope, x.float(), pos, rope)
    refused(E_SHAPE, sp.spear_rope, x[0], pos, rope)
    refused(E_SHAPE, sp.spear_rope, x, pos[:2], rope)
    refused(E_ARG, sp.spear_rope, x, pos.long(), rope)
    refused(E_ARG, sp.spear_rope, x.transpose(1, 2), pos, rope)                    # gaps within a row
    refused(E_SHAPE, sp.spear_rope, x, pos, rope, y=x[:, :2])
    k = torch.zeros(3, 2, 64, dtype=bf)
    refused(E_ARG, sp.spear_rope_kv4_write, x, k, k, pos, slots, rope, kv)         # on the CPU
    refused(E_NULL, sp.spear_rope_kv4_write, x, k, k, None, slots, rope, kv)
    refused(E_SHAPE, sp.spear_rope_kv4_write, x, x, k, pos, slots, rope, kv)
    refused(E_ARG, sp.spear_rope_kv4_write, x, k, k, pos, slots.int(), rope, kv)
    refused(E_ARG, sp.spear_kv4_read, kv, slots)
    refused(E_SHAPE, sp.spear_kv4_read, kv, slots, k=x)
    table, start, n = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    refused(E_ARG, sp.spear_kv4_attention, x, kv, table, start, n, 2)
    refused(E_SHAPE, sp.spear_kv4_attention, x, kv, table, start[:2], n, 2)
    refused(E_SHAPE, sp.spear_kv4_attention, x, kv, table[:1], start, n, 2)
    refused(E_SHAPE, sp.spear_kv4_attention, x[..., :32], kv, table, start, n, 2)
    refused(E_ARG, sp.spear_kv4_attention, x, kv, table.t().contiguous().t(), start, n, 2)
    refused(E_SHAPE, sp.spear_kv4_attention, x, kv, table, start, n, 2, lse=torch.zeros(3, 2))
    refused(E_ARG, sp.spear_kv4_attention, x, kv, table, start, n, 2, workspace=torch.zeros(64))
    free, nf = torch.zeros(5, dtype=i32), torch.zeros(1, dtype=i32)
    refused(E_ARG, sp.spear_kv4_plan, n, n, table, free, nf, 4, 16)
    refused(E_SHAPE, sp.spear_kv4_plan, n, n[:1], table, free, nf, 4, 16)
    refused(E_SHAPE, sp.spear_kv4_plan, n, n, table, free, nf, 4, 16, plan=sp.new_kv4_plan(2, 5, device="cpu"))
    refused(E_ARG, sp.spear_kv4_plan, n, n.long(), table, free, nf, 4, 16)


def test_numbers_beyond_32_bits_are_refused():
    i32 = torch.int32
    kv, x = sp.new_kv4(4, 2, 64, 16, device="cpu"), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, start, n, one = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    refused(E_SHAPE, sp.spear_kv4_attention, x, kv, table, start, n, 2, window=(1 << 32) + 5)
    refused(E_SHAPE, sp.spear_kv4_plan, n, n, table, one, one, 4, (1 << 32) + 16)
    refused(E_SHAPE, sp.spear_rope_frequencies, (1 << 32) + 64)


def test_attention_workspace_is_bounded():
    """Parts are of 8192 tiles and two rounds of chunks at most, however many requests."""
    f = sp.spear_kv4_attention_workspace_size
    for B, heads, D in ((4096, 8, 128), (4096, 64, 256), (300, 1, 64)):
        n = f(1 << 15, B, 1 << 15, heads, heads, D, 1000, 64)
        few, many = 8192 + (2 * (768 + heads) + 16 * heads), 8192 + (512 + heads) + 16 * heads
        assert 0 < n <= 4 * (few * 16 * (D + 4) + many * 256 * (D + 2) + 8192 + 32768)
