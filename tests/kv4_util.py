"""Seeded steps over a cache of 4 bits, in numpy and on the device."""
import numpy as np
import torch

import ref_kv4
from quantized_gemm_w4a16_amd import spear as sp
from gpu_util import dev


def bf16(a):
    """-> (bf16 tensor on the device, its values in fp64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


def to64(t):
    return t.detach().double().cpu().numpy()


class Step:
    """Requests with kv tokens in the cache of which the last fresh ones are this
    step's rows; `pad` rows more than that; the pages lie in any order."""

    def __init__(self, kv, fresh, Hq, heads, D, P, seed=0, pad=0, width=0, spare=2, q_sd=1.0):
        rng = np.random.default_rng(seed)
        self.kv, self.fresh, self.P, self.D, self.Hq, self.heads = list(kv), list(fresh), P, D, Hq, heads
        need = [-(-n // P) for n in kv]
        pages = sum(need) + spare
        self.width = max(need + [1]) + width
        order = rng.permutation(pages)
        self.table = np.full((len(kv), self.width), -1, np.int32)
        self.cache = ref_kv4.Cache(pages, heads, D, P, rng)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            slots = self.table[b][np.arange(kv[b]) // P].astype(np.int64) * P + np.arange(kv[b]) % P
            for name in "kv":
                self.cache.write(name, slots, rng.normal(0, 1.0, (kv[b], heads, D)))
        self.q_start = np.concatenate(([0], np.cumsum(fresh))).astype(np.int32)
        self.T = int(self.q_start[-1]) + pad
        self.q, self.q64 = bf16(rng.normal(0, q_sd, (self.T, Hq, D)))
        self.to_device()

    def to_device(self):
        c = self.cache
        self.kv4 = sp.KV4(dev(c.codes["k"]), dev(c.scales["k"]), dev(c.codes["v"]), dev(c.scales["v"]))
        self.dtable, self.dstart = dev(self.table), dev(self.q_start)
        self.dkv = dev(np.array(self.kv, np.int32))

    def run(self, lse=True, **kw):
        self.lse = torch.full((self.T, self.Hq), 7.0, device="cuda") if lse else None
        kw.setdefault("y", torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda"))
        kw.setdefault("max_fresh", max(self.fresh + [0]))
        q = kw.pop("q", self.q)
        return sp.spear_kv4_attention(q, self.kv4, self.dtable, self.dstart, self.dkv, lse=self.lse, **kw)

    def check(self, what, y=None, scale=None, window=0, p_round=ref_kv4.HALF_BF16, **kw):
        y = self.run(scale=scale, window=window, **kw) if y is None else y
        want, err, lse, le = ref_kv4.attention(self.q64, self.cache, self.table, self.q_start, self.kv,
                                               self.D ** -0.5 if scale is None else scale, window, p_round)
        n = int(self.q_start[-1])
        got, tol = to64(y), err + ref_kv4.HALF_BF16 * (np.abs(want) + err) + 1e-30
        assert (got[n:] == 7.0).all(), "rows behind the last request were written"
        nan = np.isnan(want[:n])
        assert (np.isnan(got[:n]) == nan).all()
        worst = np.max(np.where(nan, 0.0, np.abs(got - want)[:n] / tol[:n]), initial=0.0)
        gl = to64(self.lse)
        assert (gl[n:] == 7.0).all()
        empty = np.isneginf(lse[:n])
        assert (np.isneginf(gl[:n]) == empty).all()
        ln = np.isnan(lse[:n])
        assert (np.isnan(gl[:n]) == ln).all()
        with np.errstate(invalid="ignore"):
            off = np.max(np.where(empty | ln, 0.0, np.abs(gl - lse)[:n] / (le[:n] + 1e-30)), initial=0.0)
        print(f"[kv4] {what}: worst {worst:.3f} of the bound, lse {off:.3f}", flush=True)
        assert worst <= 1.0 and off <= 1.0, what
        return y
