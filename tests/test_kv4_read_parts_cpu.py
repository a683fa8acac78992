"""spear_kv4_read: which parts may be asked for, checked before the device is."""
import pytest
import torch

from quantized_gemm_w4a16_amd import spear as sp


def test_parts_that_are_none():
    kv = sp.new_kv4(4, 2, 64, 16, device="cpu")
    slots, x = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(parts=""), dict(parts="vk"), dict(parts="x"), dict(parts="k", v=x), dict(parts="v", k=x)):
        with pytest.raises(sp.SpearError, match="parts") as e:
            sp.spear_kv4_read(kv, slots, **kw)
        assert e.value.status == sp.E_ARG
