"""What the attention's workspace takes: as much as its parts need, growing with the
rows and requests of a step alone."""
import itertools
import os
import re

import torch

from quantized_gemm_w4a16_amd import spear as sp

size = sp.spear_kv4_attention_workspace_size
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "spear.h")


def test_decode_steps_hold_no_room_for_prompts_of_each_request():
    """256 requests of one token, 32 heads over 8 of 128, can have 31 of more than 32 rows."""
    n = size(256, 256, 1, 32, 8, 128, 1000, 64)
    few = ((1024 // 16 + 256) + 2 * 96 + 16) * 8 * 16 * (128 + 4) * 4
    many = (1024 // 128 + 1024 // 33 + 64 + 16) * 8 * 256 * (128 + 2) * 4
    assert n <= few + many + 4 * (8192 + 32768)


def test_one_for_the_largest_step_serves_the_others():
    steps = list(itertools.product((1, 2, 16, 33, 64, 100, 513, 2048), (1, 2, 31, 64, 300)))
    for Hq, heads, D in ((8, 8, 64), (32, 8, 128), (64, 1, 128), (40, 1, 256), (96, 2, 96)):
        n = {s: size(*s, 1, Hq, heads, D, 100, 64) for s in steps}
        for (t, b), (t2, b2) in itertools.product(steps, steps):
            if t <= t2 and b <= b2:
                assert 0 < n[t, b] <= n[t2, b2], (t, b, t2, b2)
        for (t, b), most in itertools.product(steps, (0, 7, 1 << 40)):
            assert size(t, b, most, Hq, heads, D, 1, 16) == n[t, b]


def test_only_the_counters_are_zeroed(monkeypatch):
    """A call without a workspace clears 160 KB, not all of it."""
    assert int(re.search(r"SPEAR_KV4_COUNTER_BYTES \(\(size_t\)(\d+)\)", open(HEADER).read()).group(1)) == sp.KV4_COUNTER_BYTES
    monkeypatch.setattr(torch, "empty", lambda *n, **kw: torch.full(n, 255, **kw))
    kv = sp.KV4(*(torch.full(s, 0, dtype=torch.uint8) for s in ((4, 2, 16, 32), (4, 2, 2, 16)) * 2))
    ws = sp.new_kv4_workspace(3, 2, 2, 4, kv, 5)
    assert ws.numel() == size(3, 2, 2, 4, 2, 64, 5, 16)
    assert not ws[: sp.KV4_COUNTER_BYTES].any() and bool((ws[sp.KV4_COUNTER_BYTES:] == 255).all())
