"""Plain fp64 references of the epilogue, the router and the experts, with
bounds for what fp32 sums and roundings may differ (numpy, CPU).

Bounds.  A product that takes part in an fp32 sum passes through at most
D = 32 + K / 32 + 24 roundings (within a 32-deep matrix instruction, along the
chain of them, and where waves and K slices are joined), each off by at most
half a step, 2^-24 relative.  The kernels sum x (16 + u) and remove
(16 + z) sum x, so the terms of an output are s |x| (16 + u) and
s |x| (16 + z)."""
import math

import numpy as np

HALF_F32 = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
_erf = np.vectorize(math.erf, otypes=[np.float64])

NONE, RELU, SILU, GELU, GELU_TANH = range(5)
# |act'| is at most 1.13 (gelu); an activation is computed within 16 fp32 steps
ACT_SLOPE = 1.13
ACT_ULP = 16 * HALF_F32


def act(t, kind):
    if kind == RELU:
        return np.where(t > 0, t, np.where(np.isnan(t), t, 0.0))
    if kind == SILU:
        return t / (1.0 + np.exp(-np.clip(t, -700.0, None)))
    if kind == GELU:
        return 0.5 * t * (1.0 + _erf(t / math.sqrt(2.0)))
    if kind == GELU_TANH:
        return 0.5 * t * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def depth(K):
    return 32 + K / 32 + 24


def linear(x, codes, scales, zeros, ec=None):
    """-> (t, bound of t's error): the layer in fp64.  x [M][K] float64, codes
    [N][K] 0..15, ec a dict of float64 arrays A, B, w_g and b, tau, hard."""
    s, z = scales.astype(np.float64), zeros.astype(np.float64)
    u = codes.astype(np.float64)
    t = (x @ (u - z[:, None]).T) * s
    ax = np.abs(x)
    err = depth(x.shape[1]) * HALF_F32 * s * (ax @ (16.0 + u).T + ax.sum(1)[:, None] * (16.0 + z))
    if ec is not None:
        logit = ec["b"] + x @ ec["w_g"]
        g = 1.0 / (1.0 + np.exp(-logit))
        if ec["hard"]:
            g = np.where(logit > math.log(ec["tau"] / (1.0 - ec["tau"])), g, 0.0)
        d = x @ ec["A"].T
        t = t + (g[:, None] * d) @ ec["B"].T
        # g A x is held as two bf16 (2^-16 relative), B's products in fp32
        de = 2.0 ** -16 * np.abs(d) + depth(x.shape[1]) * HALF_F32 * (ax @ np.abs(ec["A"]).T)
        err = err + (g[:, None] * (de + 64 * HALF_F32 * np.abs(d))) @ np.abs(ec["B"]).T
        err = err + 4 * HALF_F32 * np.abs(t)
    return t, err + 4 * HALF_F32 * np.abs(t)


def finish(t, err, kind, glu, bias=None, residual=None):
    """-> (y before its rounding, bound): what follows the layer."""
    if bias is not None:
        t = t + bias
        err = err + HALF_F32 * np.abs(t)
    if glu:
        a, b, ea, eb = t[:, 0::2], t[:, 1::2], err[:, 0::2], err[:, 1::2]
        f = act(a, kind)
        ef = ACT_SLOPE * ea + (ACT_ULP * np.abs(f) if kind else 0.0)
        y, err = f * b, ef * np.abs(b) + np.abs(f) * eb + ef * eb
        err = err + HALF_F32 * np.abs(y)
    else:
        y = act(t, kind)
        err = (ACT_SLOPE if kind else 1.0) * err + (ACT_ULP * np.abs(y) if kind else 0.0)
    if residual is not None:
        y = y + residual
        err = err + HALF_F32 * np.abs(y)
    return y, err


def rounded(y, err, half):
    """The bound after y is rounded to a type of that half step; 1e-37 for
    results below fp32's normal range."""
    return err + half * (np.abs(y) + err) + 1e-37


def route(x, w, topk, sigmoid, bias=None, n_group=1, topk_group=1, group_best=2, renorm=True,
          scale=1.0):
    """-> (weights float64, ids)."""
    with np.errstate(all="ignore"):
        z = x @ w.T
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-z))
        else:
            s = np.exp(z - z.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
        c = s if bias is None else s + bias.astype(np.float64)
    M, E = s.shape
    gs = E // n_group
    ids = np.full((M, topk), -1, np.int32)
    weights = np.zeros((M, topk))
    for m in range(M):
        cm = [v if v == v else -math.inf for v in c[m]]
        best = []
        for g in range(n_group):
            top = sorted(cm[g * gs:(g + 1) * gs], reverse=True)[:group_best]
            v = sum(top)
            best.append(v if v == v else -math.inf)
        kept = set(sorted(range(n_group), key=lambda g: (-best[g], g))[:topk_group])
        order = sorted((e for e in range(E) if e // gs in kept and cm[e] > -math.inf),
                       key=lambda e: (-cm[e], e))[:topk]
        got = [s[m, e] for e in order]
        total = sum(got)
        for j, e in enumerate(order):
            ids[m, j] = e
            weights[m, j] = scale * (got[j] if not renorm else got[j] / total if total else 0.0)
    return weights, ids


def experts(x, up, down, ids, weights, kind, glu, up_bias=None, down_bias=None, residual=None):
    """-> (y before its rounding, bound).  up and down are (codes [E][N][K],
    scales, zeros [E][N])."""
    M, topk = ids.shape
    E, N = down[0].shape[:2]
    y = np.zeros((M, N)) if residual is None else residual.astype(np.float64).copy()
    err = np.zeros((M, N))
    for e in range(E):
        m, j = np.nonzero(ids == e)
        if not len(m):
            continue
        t, te = linear(x[m], up[0][e], up[1][e], up[2][e])
        h, he = finish(t, te, kind, glu, None if up_bias is None else up_bias[e])
        he = rounded(h, he, HALF_BF16)                    # h is held in bf16
        dw = (down[0][e].astype(np.float64) - down[2][e][:, None]) * down[1][e][:, None]
        d, de = linear(h, down[0][e], down[1][e], down[2][e])
        de = de + he @ np.abs(dw).T
        if down_bias is not None:
            d = d + down_bias[e]
        w = weights[m, j].astype(np.float64)[:, None]
        np.add.at(y, m, w * d)
        np.add.at(err, m, np.abs(w) * (de + (topk + 2) * HALF_F32 * np.abs(d)))
    return y, err + (topk + 2) * HALF_F32 * np.abs(y)
