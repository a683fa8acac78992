"""Cases and plain forms of the layer-level operators around the W4A16 linear:
the linear with bias, activation (plain or gated), and residual in its
epilogue; the router that picks a token's experts; and the experts' W4
products over the routed tokens.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the library (``quantized_gemm_w4a16_amd.spear``).
"""
import math

import torch

own = False

# Position p of a packed 32-bit word holds code PERM[p] of its eight.
PERM = (0, 2, 4, 6, 1, 3, 5, 7)
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def listed():
    return [
        # One token of a chat through a decoder's merged gate and up projection
        # (rows interleaved), its error compensator on: launch latency counts.
        _linear("gate_up_m1", 1, 16384, 2048, "silu", True, rank=32, hard=True),
        # Sixteen running requests through the down projection, added onto the
        # residual stream.
        _linear("down_m16", 16, 2048, 8192, "none", False, rank=32, residual=True),
        # A short ragged prompt through an odd-sized layer with a bias, fp32 out.
        _linear("bias_gelu_m77", 77, 1000, 4128, "gelu", False, bias=True, f32=True),
        # A prefill chunk through a large model's merged gate and up projection.
        _linear("gate_up_m4096", 4096, 28672, 4096, "silu", True, rank=32),
        # One token choosing 8 of 64 experts.
        _route("route_m1", 1, 64, 2048, 8, "softmax", renorm=True),
        # A ragged batch, an expert count that fills no tile, biased sigmoid scores.
        _route("route_m777", 777, 60, 2080, 4, "sigmoid", bias=True, renorm=True, scale=2.5),
        # A long prefill chunk over 256 experts in 8 groups of which 4 are kept.
        _route("route_m8192", 8192, 256, 4096, 8, "sigmoid", bias=True, groups=8, kept=4, renorm=True, scale=2.5),
        # One token through its 8 of 64 experts.
        _experts("experts_m1", 1, 64, 8, 2048, 1024, "silu", True),
        # Sixteen running requests, most experts busy with one or two tokens.
        _experts("experts_m16", 16, 64, 8, 2048, 1024, "silu", True, residual=True),
        # A short prompt on a device that holds most of the experts: some slots are elsewhere.
        _experts("experts_m300", 300, 32, 4, 2048, 1408, "silu", True, away=0.1),
        # A prefill chunk through 8 large experts, two a token.
        _experts("experts_m4096", 4096, 8, 2, 4096, 8192, "silu", True, residual=True),
    ]


def _linear(name, m, n, k, act, glu, rank=0, hard=False, bias=False, residual=False, f32=False):
    c = dict(op="linear", m=m, n=n, k=k, act=act, glu=glu, rank=rank, hard=hard, bias=bias, residual=residual, f32=f32)
    return dict(c, name=name) if name else c


def _route(name, m, e, k, topk, score, bias=False, groups=1, kept=1, renorm=True, scale=1.0):
    c = dict(op="route", m=m, e=e, k=k, topk=topk, score=score, bias=bias, groups=groups, kept=kept, renorm=renorm, scale=scale)
    return dict(c, name=name) if name else c


def _experts(name, m, e, topk, k, i, act, glu, residual=False, bias=False, away=0.0):
    c = dict(op="experts", m=m, e=e, topk=topk, k=k, i=i, act=act, glu=glu, residual=residual, bias=bias, away=away)
    return dict(c, name=name) if name else c


def draw(rng):
    def size(lo, hi, step):
        return step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) or step

    op = rng.choice(("linear", "route", "experts"))
    if op == "linear":
        k, n = size(256, 8192, 32), size(64, 28672, 2)
        m = size(1, max(1, min(4096, 2 ** 38 // (n * k))), 1)
        glu = rng.random() < 0.5
        return _linear("", m, n, k, rng.choice(list(ACTS)), glu, rank=rng.choice((0, 16, 32, 64)), hard=rng.random() < 0.5,
                       bias=rng.random() < 0.5, residual=rng.random() < 0.5, f32=rng.random() < 0.3)
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        e = groups * rng.randint(3, 256 // groups)
        k, topk = size(256, 4096, 32), min(e, rng.choice((1, 2, 4, 6, 8)))
        kept = rng.randint(-(-topk * groups // e), groups)
        return _route("", size(1, 8192, 1), e, k, topk, rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, kept=kept,
                      renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)))
    e, topk = rng.randint(4, 64), rng.randint(1, 8)
    k, i = size(256, 4096, 32), size(128, 2048, 32)
    return _experts("", size(1, 4096, 1), e, min(topk, e), k, i, rng.choice(("silu", "gelu", "relu")), rng.random() < 0.7,
                    residual=rng.random() < 0.5, bias=rng.random() < 0.3, away=rng.choice((0.0, 0.0, 0.2)))


# ------------------------------------------------------------------ inputs

class _Random:
    """Seeded numbers on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, sd=1.0):
        return torch.randn(shape, generator=self.g, device="cuda") * sd

    def uniform(self, lo, hi, *shape):
        return torch.rand(shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def whole(self, lo, hi, *shape, dtype=torch.uint8):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda", dtype=dtype)

    def tokens(self, m, k):
        """Activations with a few outlier channels, as decoders have them."""
        x = self.normal(m, k)
        x[:, self.whole(0, k, max(1, k // 200), dtype=torch.int64)] *= 10.0
        return x.bfloat16()

    def w4(self, *shape):
        """Packed 4-bit codes [..., N, K/2], scales and zero points [..., N]."""
        *lead, n, k = shape
        return self.whole(0, 256, *lead, n, k // 2), self.uniform(0.005, 0.02, *lead, n) * (16.0 / math.sqrt(k)), self.whole(6, 10, *lead, n)


def prepare(case, seed):
    c, r = dict(case), _Random(seed)
    s = {"case": c, "x": r.tokens(c["m"], c["k"])}
    if c["op"] == "linear":
        s["packed"], s["scales"], s["zeros"] = r.w4(c["n"], c["k"])
        s["bias"] = r.normal(c["n"], sd=0.3) if c["bias"] else None
        wide = c["n"] // 2 if c["glu"] else c["n"]
        s["residual"] = r.normal(c["m"], wide).to(torch.float32 if c["f32"] else torch.bfloat16) if c["residual"] else None
        if c["rank"]:
            s["a"] = r.normal(c["rank"], c["k"], sd=0.02).bfloat16()
            s["b"] = r.normal(c["n"], c["rank"], sd=0.02).bfloat16()
            s["w_gate"] = r.normal(c["k"], sd=1.0 / math.sqrt(c["k"])).bfloat16()
    elif c["op"] == "route":
        s["w"] = r.normal(c["e"], c["k"], sd=1.0 / math.sqrt(c["k"])).bfloat16()
        s["bias"] = r.normal(c["e"], sd=0.05) if c["bias"] else None
    else:
        nu = 2 * c["i"] if c["glu"] else c["i"]
        s["up"], s["down"] = r.w4(c["e"], nu, c["k"]), r.w4(c["e"], c["k"], c["i"])
        s["up_bias"] = r.normal(c["e"], nu, sd=0.3) if c["bias"] else None
        s["down_bias"] = r.normal(c["e"], c["k"], sd=0.3) if c["bias"] else None
        s["residual"] = r.normal(c["m"], c["k"]).bfloat16() if c["residual"] else None
        # some experts are chosen more often than others
        liking = r.normal(c["m"], c["e"]) + r.normal(c["e"], sd=0.5)
        ids = liking.topk(c["topk"], dim=1).indices.to(torch.int32)
        s["ids"] = torch.where(r.uniform(0, 1, c["m"], c["topk"]) < c["away"], -1, ids).contiguous()
        s["weights"] = torch.softmax(r.normal(c["m"], c["topk"]), 1)
    if own:
        s.update(_kept(s))
    return s


def _kept(s):
    """What a program keeps between calls: the weights' handles, the workspace
    and the output buffers."""
    from quantized_gemm_w4a16_amd import spear as sp
    c = s["case"]
    if c["op"] == "linear":
        ec = sp.EC(s["a"], s["b"], s["w_gate"], 0.0, 0.5, int(c["hard"])) if c["rank"] else None
        return {"sp": sp, "layer": sp.W4(s["packed"], s["scales"], s["zeros"], c["n"], c["k"]), "ec": ec,
                "epilogue": sp.Epilogue(bias=s["bias"], act=ACTS[c["act"]], glu=c["glu"]),
                "y": torch.empty(c["m"], c["n"] // 2 if c["glu"] else c["n"], device="cuda", dtype=torch.float32 if c["f32"] else torch.bfloat16),
                "ws": sp.new_workspace(c["m"], c["n"], c["k"], c["rank"])}
    if c["op"] == "route":
        router = sp.Router(s["w"], topk=c["topk"], score=sp.SCORE_SIGMOID if c["score"] == "sigmoid" else sp.SCORE_SOFTMAX, bias=s["bias"],
                           n_group=c["groups"], topk_group=c["kept"], renorm=c["renorm"], scale=c["scale"])
        return {"sp": sp, "router": router, "weights": torch.empty(c["m"], c["topk"], device="cuda"),
                "ids": torch.empty(c["m"], c["topk"], device="cuda", dtype=torch.int32), "ws": sp.new_route_workspace(c["m"], router)}
    experts = sp.Experts(*s["up"], *s["down"], up_bias=s["up_bias"], down_bias=s["down_bias"], act=ACTS[c["act"]], glu=c["glu"])
    return {"sp": sp, "experts": experts, "y": torch.empty_like(s["x"]), "ws": sp.new_experts_workspace(c["m"], c["topk"], experts)}


# --------------------------------------------------------------- one pass

def run(state):
    return {"linear": _run_linear, "route": _run_route, "experts": _run_experts}[state["case"]["op"]](state)


def _codes(packed):
    """The codes [..., K] of packed bytes [..., K/2]."""
    b = packed.unflatten(-1, (-1, 4))
    nibbles = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    order = [PERM.index(i) for i in range(8)]
    return nibbles[..., order].flatten(-2)


def _weights(packed, scales, zeros):
    return (_codes(packed).float() - zeros.float()[..., None]) * scales[..., None]


def _act(t, name):
    if name == "relu":
        return torch.clamp(t, min=0.0)
    if name == "silu":
        return t / (1.0 + torch.exp(-t))
    if name == "gelu":
        return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _finish(t, act, glu):
    return _act(t[..., 0::2], act) * t[..., 1::2] if glu else _act(t, act)


def _run_linear(s):
    c = s["case"]
    if own:
        ep = s["epilogue"]
        ep.residual = s["residual"]
        return s["sp"].spear_w4_linear_epilogue(s["x"], s["layer"], ep, s["ec"], y=s["y"], out_dtype=s["sp"].OUT_F32 if c["f32"] else s["sp"].OUT_BF16,
                                                workspace=s["ws"])
    x = s["x"].float()
    t = x @ _weights(s["packed"], s["scales"], s["zeros"]).t()
    if c["rank"]:
        z = s["x"].double() @ s["w_gate"].double()
        gate = (1.0 / (1.0 + torch.exp(-z))).float() * ((z > 0) if c["hard"] else 1.0)
        t = t + (gate[:, None] * (x @ s["a"].float().t())) @ s["b"].float().t()
    if s["bias"] is not None:
        t = t + s["bias"]
    y = _finish(t, c["act"], c["glu"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if c["f32"] else y.bfloat16()


def _run_route(s):
    c = s["case"]
    if own:
        return s["sp"].spear_route(s["x"], s["router"], weights=s["weights"], ids=s["ids"], workspace=s["ws"])
    # scores in 64 bits: which expert comes next can hang on the last digits
    z = s["x"].double() @ s["w"].double().t()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        score = torch.exp(z - z.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    choice = score + s["bias"].double() if s["bias"] is not None else score
    if c["groups"] > 1:
        g = choice.unflatten(1, (c["groups"], -1))
        best = g.sort(dim=2, descending=True).values[..., :2].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, : c["kept"]]
        mask = torch.zeros_like(best).scatter_(1, keep, 1.0) > 0
        choice = torch.where(mask[..., None], g, -math.inf).flatten(1)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, : c["topk"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (w * c["scale"]).float(), ids.int()


def _each(x, w):
    """x [E][M][K] w [E][N][K] -> [E][M][N]"""
    return torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)


def _run_experts(s):
    c = s["case"]
    if own:
        return s["sp"].spear_w4_experts(s["x"], s["experts"], s["ids"], s["weights"], residual=s["residual"], y=s["y"], workspace=s["ws"])
    # the tokens of each expert in use, side by side and padded to the longest list
    m, topk = c["m"], c["topk"]
    slots = s["ids"].flatten().long()
    held = (slots >= 0).nonzero()[:, 0]
    used, which, count = slots[held].unique(return_inverse=True, return_counts=True)
    y = torch.zeros(m, c["k"], device="cuda") if s["residual"] is None else s["residual"].float()
    if len(held):
        order = which.sort(stable=True).indices
        first = count.cumsum(0) - count
        place = torch.empty_like(which)
        place[order] = torch.arange(len(held), device="cuda") - first[which[order]]
        rows = torch.zeros(len(used), int(count.max()), c["k"], device="cuda")
        rows[which, place] = s["x"].float()[held // topk]
        h = _each(rows, _weights(*(v[used] for v in s["up"])))
        if s["up_bias"] is not None:
            h = h + s["up_bias"][used][:, None]
        h = _finish(h, c["act"], c["glu"])
        out = _each(h, _weights(*(v[used] for v in s["down"])))
        if s["down_bias"] is not None:
            out = out + s["down_bias"][used][:, None]
        each = torch.zeros(m * topk, c["k"], device="cuda")
        each[held] = out[which, place] * s["weights"].flatten()[held][:, None]
        y = y + each.unflatten(0, (m, topk)).sum(1)
    return y.bfloat16()


# ------------------------------------------------------------------- work

def work(case):
    c = case
    m, k = c["m"], c["k"]
    if c["op"] == "linear":
        n, r = c["n"], c["rank"]
        wide = n // 2 if c["glu"] else n
        size = 4 if c["f32"] else 2
        return {"bytes": n * k / 2 + 5 * n + (4 * n if c["bias"] else 0) + (2 * (r * k + n * r + k) if r else 0) + 2 * m * k + size * m * wide * (2 if c["residual"] else 1),
                "flops": 2.0 * m * n * k + (2.0 * m * r * (n + k) if r else 0)}
    if c["op"] == "route":
        return {"bytes": 2 * c["e"] * k + 2 * m * k + 8 * m * c["topk"], "flops": 2.0 * m * c["e"] * k}
    nu = 2 * c["i"] if c["glu"] else c["i"]
    slots = m * c["topk"] * (1.0 - c["away"])
    used = c["e"] * (1.0 - (1.0 - c["topk"] * (1.0 - c["away"]) / c["e"]) ** m)
    per = (nu * k + k * c["i"]) / 2 + (9 if c["bias"] else 5) * (nu + k)
    return {"bytes": used * per + 2 * m * k * (3 if c["residual"] else 2) + 8 * m * c["topk"], "flops": 2.0 * slots * (nu * k + k * c["i"])}


# ------------------------------------------------------------------ exact

def _dense(packed, scales, zeros):
    """One matrix of weights in 64 bits, from its 32-bit words."""
    words = packed.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    out = torch.empty(packed.shape[0], packed.shape[1] * 2, dtype=torch.float64, device=packed.device)
    for place, code in enumerate(PERM):
        out[:, code::8] = ((words >> (4 * place)) & 15).double()
    return out.sub_(zeros.double()[:, None]).mul_(scales.double()[:, None])


def _exact_act(t, name):
    if name == "relu":
        return t * (t > 0)
    if name == "silu":
        return t * torch.special.expit(t)
    if name == "gelu":
        return t * 0.5 * torch.special.erfc(-t / math.sqrt(2.0))
    if name == "gelu_tanh":
        return t * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3))
    return t


def _exact_ffn(t, act, glu):
    if not glu:
        return _exact_act(t, act)
    pair = t.unflatten(1, (-1, 2))
    return _exact_act(pair[:, :, 0], act) * pair[:, :, 1]


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c, x = s["case"], s["x"].double()
    if c["op"] == "linear":
        t = torch.matmul(x, _dense(s["packed"], s["scales"], s["zeros"]).t())
        if c["rank"]:
            z = (x * s["w_gate"].double()).sum(1)
            u = torch.matmul(x, s["a"].double().t()) * torch.special.expit(z)[:, None]
            if c["hard"]:
                u[z <= 0] = 0.0
            t += torch.matmul(u, s["b"].double().t())
        if c["bias"]:
            t += s["bias"].double()
        y = _exact_ffn(t, c["act"], c["glu"])
        return y + s["residual"].double() if c["residual"] else y
    if c["op"] == "route":
        z = torch.matmul(x, s["w"].double().t())
        p = torch.special.expit(z) if c["score"] == "sigmoid" else (z - torch.logsumexp(z, 1, keepdim=True)).exp()
        q = p + s["bias"].double() if c["bias"] else p.clone()
        if c["groups"] > 1:
            of = torch.arange(c["e"], device="cuda") // (c["e"] // c["groups"])
            total = torch.stack([q[:, of == g].topk(min(2, c["e"] // c["groups"]), 1).values.sum(1) for g in range(c["groups"])], 1)
            lost = torch.ones_like(total, dtype=torch.bool).scatter_(1, total.topk(c["kept"], 1).indices, False)
            q[lost[:, of]] = -math.inf
        w = p.gather(1, q.topk(c["topk"], 1).indices)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return w * c["scale"], None
    y = s["residual"].double() if c["residual"] else torch.zeros_like(x)
    for e in range(c["e"]):
        token, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if not len(token):
            continue
        t = torch.matmul(x[token], _dense(*(v[e] for v in s["up"])).t())
        if c["bias"]:
            t += s["up_bias"][e].double()
        t = torch.matmul(_exact_ffn(t, c["act"], c["glu"]), _dense(*(v[e] for v in s["down"])).t())
        if c["bias"]:
            t += s["down_bias"][e].double()
        y.index_add_(0, token, t * s["weights"][token, slot].double()[:, None])
    return y
