"""Refusals of the epilogue, router and experts entry points: the documented
status before any HIP call, and the binding's checks of its tensors (no GPU)."""
import ctypes

import pytest
import torch

from quantized_gemm_w4a16_amd import spear as sp

E_NULL, E_SHAPE, E_ALIGN, E_ARG, E_WS = -1, -2, -3, -4, -5
A = 0x10000            # fake, aligned device addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    return sp.load()


def epilogue(lib, x=A, M=4, N=64, K=128, bias=None, residual=None, act=0, glu=0, y=A, out=1, ws=A,
             wsb=1 << 20, path=0, ep=True):
    w = sp._W4(A, A, None, N, K)
    e = sp._Epilogue(bias, residual, act, glu)
    return lib.spear_w4_linear_epilogue(x, M, ctypes.byref(w), None, ctypes.byref(e) if ep else None,
                                        y, out, ws, wsb, path, None)


def test_epilogue_refusals(lib):
    assert epilogue(lib, ep=False) == E_NULL
    assert epilogue(lib, x=None) == E_NULL
    assert epilogue(lib, act=5) == E_ARG
    assert epilogue(lib, act=-1) == E_ARG
    assert epilogue(lib, glu=2) == E_ARG
    assert epilogue(lib, N=63, glu=1) == E_SHAPE
    assert epilogue(lib, M=-1) == E_SHAPE
    assert epilogue(lib, K=48) == E_SHAPE
    assert epilogue(lib, M=17, path=sp.PATH_DECODE) == E_SHAPE
    assert epilogue(lib, bias=A + 2) == E_ALIGN
    assert epilogue(lib, residual=A + 8) == E_ALIGN
    assert epilogue(lib, y=A + 8) == E_ALIGN
    assert epilogue(lib, out=2) == E_ARG
    assert epilogue(lib, wsb=16) == E_WS


def route(lib, x=A, M=4, K=64, w=A, bias=None, E=8, topk=2, score=0, G=1, kept=1, best=2, renorm=1,
          scale=1.0, weights=A, ids=A, ws=A, wsb=1 << 20, router=True):
    r = sp._Router(w, bias, E, topk, score, G, kept, best, renorm, scale)
    return lib.spear_route(x, M, K, ctypes.byref(r) if router else None, weights, ids, ws, wsb, None)


def test_route_refusals(lib):
    assert route(lib, router=False) == E_NULL
    for k in ("x", "w", "weights", "ids", "ws"):
        assert route(lib, **{k: None}) == E_NULL, k
    assert route(lib, M=-1) == E_SHAPE
    assert route(lib, K=40) == E_SHAPE and route(lib, K=0) == E_SHAPE
    assert route(lib, E=0) == E_SHAPE and route(lib, E=513, wsb=1 << 30) == E_SHAPE
    assert route(lib, topk=0) == E_SHAPE and route(lib, topk=9) == E_SHAPE
    assert route(lib, E=64, topk=33) == E_SHAPE
    assert route(lib, G=3) == E_SHAPE and route(lib, G=0) == E_SHAPE
    assert route(lib, E=512, G=128) == E_SHAPE
    assert route(lib, G=4, kept=5) == E_SHAPE and route(lib, G=4, kept=0) == E_SHAPE
    assert route(lib, G=4, kept=1, topk=3) == E_SHAPE
    assert route(lib, score=2) == E_ARG and route(lib, best=3) == E_ARG and route(lib, best=0) == E_ARG
    assert route(lib, renorm=2) == E_ARG and route(lib, scale=float("nan")) == E_ARG
    for k in ("x", "w", "ws"):
        assert route(lib, **{k: A + 8}) == E_ALIGN, k
    for k in ("weights", "ids", "bias"):
        assert route(lib, **{k: A + 2}) == E_ALIGN, k
    assert route(lib, wsb=sp.spear_route_workspace_size(4, 8) - 1) == E_WS


def test_route_workspace_size():
    f = sp.spear_route_workspace_size
    assert f(-1, 8) == 0 and f(1, 0) == 0 and f(1, 513) == 0
    for E in (1, 60, 64, 512):
        sizes = [f(M, E) for M in (0, 1, 2, 16, 17, 127, 128, 129, 5000, 1 << 20)]
        assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:])), sizes


def experts(lib, x=A, M=4, topk=2, E=8, K=64, I=32, N=64, act=2, glu=1, ids=A, weights=A, res=None,
            y=A, ws=A, wsb=1 << 24, w=True, **kw):
    p = dict(up=A, up_scales=A, up_zeros=None, up_bias=None, down=A, down_scales=A, down_zeros=None,
             down_bias=None)
    p.update(kw)
    s = sp._Experts(*(p[k] for k in ("up", "up_scales", "up_zeros", "up_bias", "down", "down_scales",
                                     "down_zeros", "down_bias")), K, I, N, E, act, glu)
    return lib.spear_w4_experts(x, M, ctypes.byref(s) if w else None, ids, weights, topk, res, y, ws,
                                wsb, None)


def test_experts_refusals(lib):
    assert experts(lib, w=False) == E_NULL
    for k in ("x", "ids", "weights", "y", "ws", "up", "up_scales", "down", "down_scales"):
        assert experts(lib, **{k: None}) == E_NULL, k
    assert experts(lib, M=-1) == E_SHAPE
    assert experts(lib, topk=0) == E_SHAPE and experts(lib, topk=33) == E_SHAPE
    assert experts(lib, E=0) == E_SHAPE and experts(lib, E=513) == E_SHAPE
    for k in ("K", "I"):
        assert experts(lib, **{k: 0}) == E_SHAPE and experts(lib, **{k: 48}) == E_SHAPE
        assert experts(lib, **{k: 1 << 40}) == E_SHAPE
    assert experts(lib, N=0) == E_SHAPE and experts(lib, N=1 << 40) == E_SHAPE
    assert experts(lib, M=1 << 31, topk=1) == E_SHAPE and experts(lib, M=1 << 28, topk=32) == E_SHAPE
    assert experts(lib, act=9) == E_ARG and experts(lib, glu=-1) == E_ARG
    for k in ("x", "y", "up", "down", "res"):
        assert experts(lib, **{k: A + 8}) == E_ALIGN, k
    for k in ("ids", "weights", "up_scales", "down_scales", "up_bias", "down_bias"):
        assert experts(lib, **{k: A + 2}) == E_ALIGN, k
    assert experts(lib, ws=A + 64) == E_ALIGN
    need = sp.spear_w4_experts_workspace_size(4, 2, 8, 32, 64)
    assert experts(lib, wsb=need - 1) == E_WS


def test_experts_workspace_size():
    f = sp.spear_w4_experts_workspace_size
    assert f(-1, 2, 8, 32, 64) == 0 and f(1, 0, 8, 32, 64) == 0 and f(1, 2, 513, 32, 64) == 0
    for (topk, E, I, N) in [(1, 1, 32, 1), (2, 8, 512, 256), (8, 64, 1024, 2048), (32, 512, 32, 64)]:
        sizes = [f(M, topk, E, I, N) for M in list(range(0, 70)) + [100, 127, 128, 129, 500, 1000, 4096, 5000]]
        assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:])), (topk, E, sizes)


def refused(status, f, *a, **kw):
    with pytest.raises(sp.SpearError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value


def test_binding_checks_its_tensors():
    """Wrong types, shapes, gaps and CPU tensors are refused before the library
    sees a pointer."""
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x = torch.zeros(4, 64, dtype=bf)
    router = sp.Router(torch.zeros(8, 64, dtype=bf), 2)
    refused(E_ARG, sp.spear_route, x, router)                          # on the CPU
    refused(E_ARG, sp.spear_route, x.float(), router)
    refused(E_SHAPE, sp.spear_route, torch.zeros(4, 96, dtype=bf), router)
    refused(E_ARG, sp.spear_route, torch.zeros(64, 4, dtype=bf).t(), router)
    refused(E_ARG, sp.spear_route, x, router, ids=torch.zeros(4, 2, dtype=torch.int64))
    refused(E_SHAPE, sp.spear_route, x, router, weights=torch.zeros(4, 3))
    refused(E_ARG, sp.spear_route, x, router, workspace=torch.zeros(4096, dtype=torch.int32))
    refused(E_ARG, sp.Router, torch.zeros(8, 64), 2)
    refused(E_SHAPE, sp.Router, torch.zeros(8, 64, dtype=bf), 2, bias=torch.zeros(7))
    w = [torch.zeros(3, 64, 32, dtype=u8), torch.zeros(3, 64), None, torch.zeros(3, 64, 16, dtype=u8),
         torch.zeros(3, 64), None]
    ex = sp.Experts(*w)
    ids, weights = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    refused(E_ARG, sp.spear_w4_experts, x, ex, ids, weights)           # on the CPU
    refused(E_ARG, sp.spear_w4_experts, x, ex, ids.long(), weights)
    refused(E_SHAPE, sp.spear_w4_experts, x, ex, ids, weights[:3])
    refused(E_SHAPE, sp.spear_w4_experts, x, ex, ids, weights, residual=torch.zeros(4, 32, dtype=bf))
    refused(E_ARG, sp.spear_w4_experts, x, ex, ids, weights, y=torch.zeros(4, 64, dtype=f32))
    refused(E_SHAPE, sp.Experts, *w, glu=False)
    refused(E_SHAPE, sp.Experts, *w, up_bias=torch.zeros(3, 32))
    layer = sp.W4(torch.zeros(64, 32, dtype=u8), torch.zeros(64), None, 64, 64)
    refused(E_ARG, sp.spear_w4_linear_epilogue, x, layer, sp.Epilogue())   # on the CPU
    refused(E_SHAPE, sp.spear_w4_linear_epilogue, x, layer, sp.Epilogue(bias=torch.zeros(32)))
    refused(E_ARG, sp.spear_w4_linear_epilogue, x, layer, sp.Epilogue(residual=torch.zeros(4, 64, dtype=bf)))
    refused(E_SHAPE, sp.spear_w4_linear_epilogue, x, layer, sp.Epilogue(glu=True), y=torch.zeros(4, 64))


def test_packed_structs_are_the_ctypes_ones():
    """The byte strings that the binding passes have the C structs' layout."""
    t = [torch.zeros(8, 32) for _ in range(10)]
    w = sp.W4(t[0], t[1], None, 8, 32)
    assert sp._PACK_W4(t[0].data_ptr(), t[1].data_ptr(), 0, 8, 32) == bytes(w._c())
    e = sp.EC(t[0], t[1], t[2], 0.5, 0.25, 1, t[3], t[4], t[5], t[6], t[7], t[8], t[9], 0.75)
    assert e._packed() == bytes(e._c())
    e = sp.EC(t[0], t[1], t[2])
    assert e._packed() == bytes(e._c())
    assert sp._PACK_EPILOGUE(5, 7, 2, True) == bytes(sp._Epilogue(5, 7, 2, 1))
