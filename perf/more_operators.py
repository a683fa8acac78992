"""Cases and plain forms of attention over a cache held in 4 bits, and of what
stands between a decoder's q/k/v projection and it: the plan of a serving step
(block table, slots), rotary positions, and the write into the cache.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the library (``quantized_gemm_w4a16_amd.spear``).

The cache holds a channel in 4 bits (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6 and a
sign) and a power of two (its exponent plus 127 in a byte) for every block of
32 channels, in pages of ``page`` tokens:
  codes  [pages][heads][page][dim / 2]    two codes a byte, the lower channel low
  scales [pages][heads][dim / 32][page]
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One request's next token: lengths to positions, slots and a page now and then.
        _plan("plan_b1", 1, 900, 900, 1, 1, 16),
        # A serving step: 250 running requests with one token each, six prompts in chunks, a padded row count.
        _plan("plan_mixed", 256, 1, 30000, 1, 700, 64, pad=500),
        # One token's query heads between two projections.
        _rope("rope_t1", 1, 32, 128, 128, "half", "none", 40000),
        # A prefill chunk of wide heads, the first quarter of each rotated in pairs, far positions.
        _rope("rope_t6000", 6000, 24, 256, 64, "pairs", "parts", 500000),
        # Sixteen running requests: q, k and v of one token each, some rows padding.
        _write("write_t16", 16, 32, 8, 128, 128, "half", "none", 30000, 64, away=0.2),
        # An odd prompt over small heads, half of each rotated in pairs.
        _write("write_t777", 777, 15, 5, 64, 32, "pairs", "linear", 9000, 16),
        # A prefill chunk of a large model.
        _write("write_t8192", 8192, 32, 8, 128, 128, "half", "parts", 130000, 64),
        # One request, one token: launches and round trips count.
        _attention("attend_b1", 1, 16, 8, 128, 16, 1021, 1021, 1, 1),
        # A batch of running requests of mixed lengths.
        _attention("attend_b48", 48, 32, 8, 128, 64, 300, 16000, 1, 1),
        # Two long documents, one token each, few key heads.
        _attention("attend_long", 2, 32, 4, 128, 256, 120001, 131000, 1, 1),
        # Drafted tokens and short chunks beside each other under a sliding window, wide heads.
        _attention("attend_window", 24, 10, 2, 256, 32, 40, 9000, 1, 150, window=1500),
        # A prefill chunk on a cached prefix.
        _attention("attend_prefill", 1, 32, 8, 128, 64, 16384, 16384, 8192, 8192),
    ]


def _plan(name, b, ctx_lo, ctx_hi, fresh_lo, fresh_hi, page, pad=0):
    c = dict(op="plan", b=b, ctx_lo=ctx_lo, ctx_hi=ctx_hi, fresh_lo=fresh_lo, fresh_hi=fresh_hi, page=page, pad=pad)
    return dict(c, name=name) if name else c


def _rope(name, t, h, d, rot, layout, scaling, far):
    c = dict(op="rope", t=t, h=h, d=d, rot=rot, layout=layout, scaling=scaling, far=far)
    return dict(c, name=name) if name else c


def _write(name, t, hq, hkv, d, rot, layout, scaling, far, page, away=0.0):
    c = dict(op="write", t=t, hq=hq, hkv=hkv, d=d, rot=rot, layout=layout, scaling=scaling, far=far, page=page, away=away)
    return dict(c, name=name) if name else c


def _attention(name, b, hq, hkv, d, page, ctx_lo, ctx_hi, fresh_lo, fresh_hi, window=0, lse=True):
    c = dict(op="attention", b=b, hq=hq, hkv=hkv, d=d, page=page, ctx_lo=ctx_lo, ctx_hi=ctx_hi, fresh_lo=fresh_lo, fresh_hi=fresh_hi,
             window=window, lse=lse)
    return dict(c, name=name) if name else c


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(("plan", "rope", "write", "attention", "attention", "attention"))
    page = rng.choice((16, 32, 64, 128, 256))
    d = rng.choice((64, 96, 128, 128, 192, 256))
    if op == "plan":
        lo, hi = sorted((size(1, 30000), size(1, 30000)))
        return _plan("", size(1, 256), lo, hi, 1, size(1, 700), page, pad=rng.choice((0, 0, size(1, 500))))
    if op in ("rope", "write"):
        t, rot = size(1, 8192), rng.choice((d, d, d // 2, d // 4))
        more = (rng.choice(("half", "pairs")), rng.choice(("none", "linear", "base", "parts")), size(1000, 500000))
        if op == "rope":
            return _rope("", t, rng.randint(1, max(1, 4096 // d)), d, rot, *more)
        hkv = rng.randint(1, 8)
        return _write("", t, hkv * rng.randint(1, max(1, min(8, 4096 // (hkv * d)))), hkv, d, rot, *more, page, away=rng.choice((0.0, 0.0, 0.3)))
    hkv, group = rng.randint(1, 8), rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    while hkv * group > 40:
        hkv -= 1
    lo, hi = sorted((size(1, 24000), size(1, 24000)))
    most = rng.choice((1, 1, 1, 6, 60, 2000))
    b = size(1, max(1, min(64, 2 ** 19 // hi, 6000 // most)))
    return _attention("", b, hkv * group, hkv, d, page, lo, hi, 1, min(hi, size(1, most)), window=rng.choice((0, 0, 0, size(16, 4000))),
                      lse=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _spread(b, lo, hi, turn):
    """b lengths from lo to hi, even in their logarithm, out of order."""
    step = next(s for s in range(max(2, b // 2 + 1), b + 3) if math.gcd(s, b) == 1)
    return [round(lo * (hi / lo) ** (((i * step + turn) % b + 0.5) / b)) for i in range(b)]


def _lengths(c):
    """-> (tokens in the cache after the step, fresh ones among them) of each request."""
    kv = _spread(c["b"], c["ctx_lo"], c["ctx_hi"], 0)
    fresh = _spread(c["b"], c["fresh_lo"], c["fresh_hi"], c["b"] // 3)
    if c["op"] == "plan":          # most requests run with one token, some are prompts
        fresh = [f if i % 40 == 0 else 1 for i, f in enumerate(fresh)]
        return [k + f for k, f in zip(kv, fresh)], fresh
    return kv, [min(f, k) for f, k in zip(fresh, kv)]


def _frequencies(c):
    """Angle of a position in each rotated pair, in 64 bits, and the factor of the rotated channels."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    base, scaling = 10000.0, c["scaling"]
    if scaling == "base":
        base *= 8.0 ** (c["rot"] / (c["rot"] - 2))
    f = base ** (-2.0 * i / c["rot"])
    if scaling == "linear":
        f = f / 4.0
    if scaling == "parts":
        keep = ((4096.0 * f / (2.0 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - keep) * f / 16.0 + keep * f
    return f, (1.2772588722239782 if scaling == "parts" else 1.0)


class _Random:
    """Seeded numbers on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def whole(self, lo, hi, *shape, dtype=torch.int64):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda", dtype=dtype)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")

    def heads(self, t, h, d):
        """q, k or v rows: normal, some channels of each head larger than the rest."""
        x = torch.randn((t, h, d), generator=self.g, device="cuda")
        x *= torch.where(torch.rand((h, d), generator=self.g, device="cuda") < 0.03, 6.0, 1.0)
        return x.bfloat16()


def prepare(case, seed):
    c, r = dict(case), _Random(seed)
    s = {"case": c}
    if c["op"] == "plan":
        kv, fresh = _lengths(c)
        p = c["page"]
        cached = [k - f for k, f in zip(kv, fresh)]
        width = -(-max(kv) // p) + 3
        held = [-(-n // p) for n in cached]
        total = sum(held) + sum(-(-k // p) for k in kv)
        order = r.order(total).int()
        table = torch.full((c["b"], width), -1, dtype=torch.int32, device="cuda")
        place = torch.arange(width, device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]
        table[place] = order[: sum(held)]
        s.update(cached=torch.tensor(cached, dtype=torch.int32, device="cuda"), fresh=torch.tensor(fresh, dtype=torch.int32, device="cuda"),
                 table=table, free=order[sum(held):].contiguous(), rows=sum(fresh) + c["pad"])
        s["n_free"] = torch.tensor([len(s["free"])], dtype=torch.int32, device="cuda")
    elif c["op"] == "rope":
        s["x"], s["positions"] = r.heads(c["t"], c["h"], c["d"]), r.whole(0, c["far"], c["t"], dtype=torch.int32)
        s["freqs"], s["factor"] = _frequencies(c)
    elif c["op"] == "write":
        t, hq, hkv, d = c["t"], c["hq"], c["hkv"], c["d"]
        # q, k and v come side by side out of one projection
        s["qkv"] = torch.cat((r.heads(t, hq, d), r.heads(t, hkv, d), r.heads(t, hkv, d)), 1)
        s["positions"] = r.whole(0, c["far"], t, dtype=torch.int32)
        s["freqs"], s["factor"] = _frequencies(c)
        s["pages"] = -(-2 * t // c["page"]) + 2
        slots = r.order(s["pages"] * c["page"])[:t]
        s["slots"] = torch.where(torch.rand(t, generator=r.g, device="cuda") < c["away"], -1, slots)
    else:
        kv, fresh = _lengths(c)
        p, h, d = c["page"], c["hkv"], c["d"]
        need = [-(-n // p) for n in kv]
        pages = sum(need) + 1
        s["table"] = torch.full((c["b"], max(need)), -1, dtype=torch.int32, device="cuda")
        place = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
        s["table"][place] = r.order(pages)[: sum(need)].int()
        start = [0]
        for f in fresh:
            start.append(start[-1] + f)
        s["q"] = r.heads(start[-1], c["hq"], d)
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["lengths"] = kv, fresh
        s["k"], s["v"] = (_cache(r, pages, h, p, d, hi) for hi in (127, 129))
    if own:
        s.update(_kept(s))
    return s


def _cache(r, pages, h, p, d, hi):
    """Codes and scales as they lie in the cache, those behind the last token of a request among them."""
    return r.whole(0, 256, pages, h, p, d // 2, dtype=torch.uint8), r.whole(hi - 3, hi, pages, h, d // 32, p, dtype=torch.uint8)


def _kept(s):
    """What a program keeps between calls: the cache's and the rotation's
    handles, the workspace and the output buffers."""
    from quantized_gemm_w4a16_amd import spear as sp
    c = s["case"]
    if c["op"] == "plan":
        return {"sp": sp, "plan": sp.new_kv4_plan(c["b"], s["rows"])}
    if c["op"] == "attention":
        kv = sp.KV4(*s["k"], *s["v"])
        t, most = s["q"].shape[0], max(s["lengths"][1])
        return {"sp": sp, "kv": kv, "most": most, "y": torch.empty_like(s["q"]),
                "lse": torch.empty(t, c["hq"], device="cuda") if c["lse"] else None,
                "ws": sp.new_kv4_workspace(t, c["b"], most, c["hq"], kv, s["table"].shape[1])}
    kind = {"none": sp.ROPE_PLAIN, "linear": sp.ROPE_LINEAR, "base": sp.ROPE_BASE, "parts": sp.ROPE_PARTS}[c["scaling"]]
    factor = {"none": 1.0, "linear": 4.0, "base": 8.0, "parts": 16.0}[c["scaling"]]
    freqs = sp.spear_rope_frequencies(c["rot"], 10000.0, kind, factor, original=4096.0, low=1.0, high=32.0)
    rope = sp.Rope(freqs.cuda(), sp.ROPE_HALF if c["layout"] == "half" else sp.ROPE_PAIRS, s["factor"])
    if c["op"] == "rope":
        return {"sp": sp, "rope": rope, "y": torch.empty_like(s["x"])}
    row = (c["t"], c["hkv"], c["d"])
    return {"sp": sp, "rope": rope, "kv": sp.new_kv4(s["pages"], c["hkv"], c["d"], c["page"]),
            "q_out": torch.empty(c["t"], c["hq"], c["d"], dtype=torch.bfloat16, device="cuda"),
            "k_out": torch.empty(row, dtype=torch.bfloat16, device="cuda"), "v_out": torch.empty(row, dtype=torch.bfloat16, device="cuda")}


# --------------------------------------------------------------- one pass

def run(state):
    return {"plan": _run_plan, "rope": _run_rope, "write": _run_write, "attention": _run_attention}[state["case"]["op"]](state)


def _run_plan(s):
    p, rows = s["case"]["page"], s["rows"]
    if own:
        plan = s["sp"].spear_kv4_plan(s["cached"], s["fresh"], s["table"], s["free"], s["n_free"], rows, p, plan=s["plan"])
        return plan.q_start, plan.kv_len, plan.positions, plan.slots, s["table"], plan.n_left, plan.status
    width = s["table"].shape[1]
    start = torch.zeros(len(s["fresh"]) + 1, dtype=torch.int64, device="cuda")
    start[1:] = s["fresh"].long().clamp(min=0).cumsum(0).clamp(max=rows)
    cached = s["cached"].long().clamp(min=0)
    kv = cached + start[1:] - start[:-1]
    held, full = (cached + p - 1) // p, (kv + p - 1) // p
    take = full.clamp(max=width) - held.clamp(max=width)
    before = take.cumsum(0) - take
    free = s["n_free"].long().clamp(0, len(s["free"]))
    entry = torch.arange(width, device="cuda")[None] - held[:, None]
    kth = before[:, None] + entry
    page = torch.where(kth < free, s["free"][(free - 1 - kth).clamp(0, max(len(s["free"]) - 1, 0))], -1)
    table = torch.where((entry >= 0) & (entry < take[:, None]), page, s["table"])
    row = torch.arange(rows, device="cuda")
    of = torch.searchsorted(start[1:], row, right=True)
    real = of < len(kv)
    of = of.clamp(max=len(kv) - 1)
    position = cached[of] + row - start[of]
    there = table[of, (position // p).clamp(max=width - 1)].long()
    slots = torch.where(real & (position // p < width) & (there >= 0), there * p + position % p, -1)
    wanted = take.sum()
    status = torch.stack(((wanted - free[0]).clamp(min=0), (full - torch.maximum(held, torch.full_like(held, width))).clamp(min=0).sum()))
    return (start.int(), kv.int(), torch.where(real, position, 0).int(), slots, table, (free - wanted).clamp(min=0).int(), status.int())


def _turned(x, positions, freqs, factor, layout):
    """Rows [T][H][D] with the first channels of each head rotated, in 64 bits."""
    angle = positions.double()[:, None, None] * freqs
    cos, sin = torch.cos(angle) * factor, torch.sin(angle) * factor
    n = len(freqs)
    x = x.double()
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * n:]), -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., 2 * n:]), -1)


def _run_rope(s):
    if own:
        return s["sp"].spear_rope(s["x"], s["positions"], s["rope"], y=s["y"])
    return _turned(s["x"], s["positions"], s["freqs"], s["factor"], s["case"]["layout"]).bfloat16()


def _held(x):
    """The values that a cache of 4 bits holds of rows [..., D]."""
    x = x.double().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = (e - 3 + (m >= 0.875).int()).clamp(-125, 125)
    e = torch.where(amax > 0, e, -125)
    y = torch.ldexp(x.abs(), -e)
    step = torch.where(y < 2.0, 0.5, torch.where(y < 4.0, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    return (torch.ldexp(y, e) * torch.sign(x)).flatten(-2)


def _run_write(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
    if own:
        sp = s["sp"]
        q = sp.spear_rope_kv4_write(q, k, v, s["positions"], s["slots"], s["rope"], s["kv"], q_out=s["q_out"])
        # the cache's rows as the values they stand for
        k, v = sp.spear_kv4_read(s["kv"], s["slots"], k=s["k_out"], v=s["v_out"])
        return q, k, v
    q, k = (_turned(x, s["positions"], s["freqs"], s["factor"], c["layout"]) for x in (q, k))
    kept = (s["slots"] >= 0)[:, None, None]
    return q.bfloat16(), torch.where(kept, _held(k), 0.0).bfloat16(), torch.where(kept, _held(v), 0.0).bfloat16()


def _rows(codes, scales, pages, n):
    """The first n tokens [H][n][D] of the listed pages."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    b = codes[pages]
    x = levels[torch.stack((b & 15, b >> 4), -1).flatten(-2).long()]
    x = x * torch.exp2(scales[pages].float() - 127.0).transpose(2, 3).repeat_interleave(32, -1)
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _run_attention(s):
    c = s["case"]
    if own:
        y = s["sp"].spear_kv4_attention(s["q"], s["kv"], s["table"], s["q_start"], s["kv_len"], s["most"], window=c["window"], y=s["y"],
                                        lse=s["lse"], workspace=s["ws"])
        return (y, s["lse"]) if c["lse"] else y
    group, p, scale = c["hq"] // c["hkv"], c["page"], 1.0 / math.sqrt(c["d"])
    y = torch.empty(s["q"].shape, device="cuda")
    lse = torch.empty(y.shape[:2], device="cuda")
    first = 0
    for i, (n, f) in enumerate(zip(*s["lengths"])):
        # nothing before the window of the first fresh token is read
        page0 = max(0, n - f + 1 - c["window"]) // p if c["window"] else 0
        pages = s["table"][i, page0: -(-n // p)].long()
        k, v = (_rows(*s[x], pages, n - page0 * p) for x in ("k", "v"))
        at = torch.arange(n - f, n, device="cuda")[:, None]
        seen = torch.arange(page0 * p, n, device="cuda")[None]
        mask = seen > at
        if c["window"]:
            mask |= seen <= at - c["window"]
        # [key heads][fresh tokens x group][D], as many heads at a time as 1 GB of scores holds
        q = s["q"][first:first + f].float().unflatten(1, (c["hkv"], group)).transpose(0, 1).flatten(1, 2)
        for some in torch.arange(c["hkv"]).split(max(1, 2 ** 28 // (group * f * k.shape[1]))):
            h = slice(int(some[0]), int(some[-1]) + 1)
            z = q[h] @ k[h].transpose(1, 2).contiguous() * scale
            z = z.unflatten(1, (f, group)).masked_fill_(mask[:, None], -math.inf).flatten(1, 2)
            top = z.max(2, keepdim=True).values
            e = torch.exp(z - top)
            total = e.sum(2, keepdim=True)
            heads = slice(h.start * group, h.stop * group)
            y[first:first + f, heads] = (e @ v[h] / total).unflatten(1, (f, group)).transpose(0, 1).flatten(1, 2)
            lse[first:first + f, heads] = (top + torch.log(total))[..., 0].unflatten(1, (f, group)).transpose(0, 1).flatten(1, 2)
        first += f
    return (y.bfloat16(), lse) if c["lse"] else y.bfloat16()


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "plan":
        kv, fresh = _lengths(c)
        new = sum(-(-k // c["page"]) - -(-(k - f) // c["page"]) for k, f in zip(kv, fresh))
        rows = sum(fresh) + c["pad"]
        return {"bytes": 16 * c["b"] + 8 * new + 12 * rows + 24, "flops": 4.0 * (c["b"] + rows)}
    if c["op"] == "rope":
        n = c["t"] * c["h"] * c["d"]
        return {"bytes": 4 * n + 4 * c["t"] + 4 * c["rot"], "flops": 3.0 * c["t"] * c["h"] * c["rot"]}
    if c["op"] == "write":
        t, q, kv = c["t"], c["hq"] * c["d"], c["hkv"] * c["d"]
        return {"bytes": t * (4 * q + 4 * kv) + 2 * t * kv * (17.0 / 32.0 + 2.0) * (1.0 - c["away"]) + 12 * t,
                "flops": 3.0 * t * (c["hq"] + c["hkv"]) * c["rot"] + 4.0 * t * kv}
    kv, fresh = _lengths(c)
    w = c["window"]
    pairs = sum(min(p + 1, w) if w else p + 1 for n, f in zip(kv, fresh) for p in range(n - f, n))
    read = sum(min(n, f - 1 + w) if w else n for n, f in zip(kv, fresh))
    return {"bytes": 4 * sum(fresh) * c["hq"] * c["d"] + read * c["hkv"] * c["d"] * 17.0 / 16.0 + (4 * sum(fresh) * c["hq"] if c["lse"] else 0),
            "flops": 4.0 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------ exact

def _e2m1(y):
    """The nearest level of each |y|, the even code where two are as near."""
    up = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), dtype=torch.float64, device=y.device)
    a = y.abs()
    low, high = torch.bucketize(a, up), torch.bucketize(a, up, right=True)   # ties differ: low rounds down
    code = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return torch.tensor(LEVELS, dtype=torch.float64, device=y.device)[code] * torch.where(y < 0, -1.0, 1.0)


def _exact_held(x):
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().max(-1, keepdim=True).values.clamp(min=2.0 ** -140)
    e = torch.floor(torch.log2(top))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    e = torch.where(top * torch.exp2(-e) >= 1.75, e - 1, e - 2).clamp(-125, 125)
    return (_e2m1(b * torch.exp2(-e)) * torch.exp2(e)).reshape(x.shape)


def _exact_turned(x, positions, freqs, factor, layout):
    n = len(freqs)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    turn = torch.polar(torch.full((len(positions), 1, n), factor, dtype=torch.float64, device="cuda"), positions[:, None, None].double() * freqs)
    y = x.double().clone()
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    if case["op"] == "plan":
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c = s["case"]
    if c["op"] == "rope":
        return _exact_turned(s["x"], s["positions"], s["freqs"], s["factor"], c["layout"])
    if c["op"] == "write":
        q, k, v = s["qkv"].split((c["hq"], c["hkv"], c["hkv"]), 1)
        q, k = (_exact_turned(x, s["positions"], s["freqs"], s["factor"], c["layout"]) for x in (q, k))
        k, v = _exact_held(k), _exact_held(v.double())
        lost = s["slots"] < 0
        k[lost], v[lost] = 0.0, 0.0
        return q, k, v
    group, page = c["hq"] // c["hkv"], c["page"]
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(y.shape[:2], dtype=torch.float64, device="cuda")
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, f) in enumerate(zip(*s["lengths"])):
        token = torch.arange(n, device="cuda")
        where, slot = s["table"][b].long()[token // page], token % page
        for h in range(c["hkv"]):
            kept = []
            for codes, scales in (s["k"], s["v"]):
                x = torch.empty(n, c["d"], dtype=torch.float64, device="cuda")
                raw = codes[where, h, slot].long()
                for place in (0, 1):
                    nibble = (raw >> (4 * place)) & 15
                    x[:, place::2] = level[nibble & 7] * (1.0 - 2.0 * (nibble >> 3).double())
                for block in range(c["d"] // 32):
                    x[:, 32 * block:32 * block + 32] *= torch.pow(2.0, scales[where, h, block, slot].double()[:, None] - 127.0)
                kept.append(x)
            for j in range(h * group, h * group + group):
                z = torch.matmul(s["q"][row:row + f, j].double(), kept[0].t()) / math.sqrt(c["d"])
                ahead = (token[None] - (n - f) - torch.arange(f, device="cuda")[:, None])
                z[(ahead > 0) | (ahead <= -c["window"] if c["window"] else ahead > 0)] = -math.inf
                lse[row:row + f, j] = torch.logsumexp(z, 1)
                y[row:row + f, j] = torch.matmul(torch.exp(z - lse[row:row + f, j, None]), kept[1])
        row += f
    return (y, lse) if c["lse"] else y
