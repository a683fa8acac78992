"""The epilogue entry point's binding refuses weights and compensators that do
not fit the call, before the library sees a pointer (no GPU: the tensors are on
the meta device, which stands for one device and its other memory)."""
import pytest
import torch

from quantized_gemm_w4a16_amd import spear as sp

E_NULL, E_SHAPE, E_ARG = -1, -2, -4
M, N, K, R, H = 3, 64, 96, 16, 5
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def z(*shape, dtype=F32, device="meta"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def call(weights=None, ec=None, vector=False):
    w = dict(packed=z(N, K // 2, dtype=U8), scales=z(N), zeros=z(N, dtype=U8))
    w.update(weights or {})
    e = dict(A=z(R, K, dtype=BF), B=z(N, R, dtype=BF), w_gate=z(K, dtype=BF), g_out=z(M), idx_out=z(M, dtype=I32),
             n_active_out=z(1, dtype=I32))
    if vector:
        e.update(gate_w1=z(H, R), gate_c1=z(H), gate_w2=z(R, H), gate_c2=z(R))
    e.update(ec or {})
    with pytest.raises(sp.SpearError) as err:
        sp.spear_w4_linear_epilogue(z(M, K, dtype=BF), sp.W4(**w, N=N, K=K), sp.Epilogue(), sp.EC(**e))
    return err.value


def test_fitting_arguments_get_to_the_device_check():
    for vector in (False, True):
        assert "not on a GPU" in str(call(vector=vector))
    assert "not on a GPU" in str(call(weights=dict(zeros=None)))
    assert "not on a GPU" in str(call(ec=dict(g_out=z(M + 5))))       # outputs may be longer


@pytest.mark.parametrize("name,good", [("packed", (N, K // 2)), ("scales", (N,)), ("zeros", (N,))])
def test_weights(name, good):
    t = {"packed": U8, "scales": F32, "zeros": U8}[name]
    assert call({name: z(*good[:-1], good[-1] - 1, dtype=t)}).status == E_SHAPE
    assert call({name: z(*good, dtype=torch.float64)}).status == E_ARG
    assert call({name: z(*good, dtype=t, device="cpu")}).status == E_ARG


@pytest.mark.parametrize("name,good,t", [("A", (R, K), BF), ("B", (N, R), BF), ("w_gate", (K,), BF), ("g_out", (M,), F32),
                                         ("idx_out", (M,), I32), ("n_active_out", (1,), I32), ("gate_w1", (H, R), F32),
                                         ("gate_c1", (H,), F32), ("gate_w2", (R, H), F32), ("gate_c2", (R,), F32)])
def test_compensator(name, good, t):
    assert call(ec={name: z(*good[:-1], good[-1] - 1, dtype=t)}, vector=True).status == E_SHAPE
    assert call(ec={name: z(*good, dtype=torch.float64)}, vector=True).status == E_ARG
    assert call(ec={name: z(*good, dtype=t, device="cpu")}, vector=True).status == E_ARG
    if name.startswith("gate_") and name != "gate_w1":
        assert call(ec={name: None}, vector=True).status == E_NULL


def test_gaps_between_elements():
    assert call({"packed": z(K // 2, N, dtype=U8).t()}).status == E_ARG
    assert call(ec={"A": z(R, 2 * K, dtype=BF)[:, ::2]}).status == E_ARG
