"""Factors of a rotation whose two terms in fp32 cannot hold the stated bound are
refused, before any HIP call."""
import ctypes

import pytest

from quantized_gemm_w4a16_amd import spear as sp

E_ARG = -4
A = 0x10000            # fake, aligned device addresses: never dereferenced
OUT = (2.0 ** 101, -1e31, 1e39, -1e300, 1.7e308, 2.0 ** -101, -2.0 ** -120, 1e-40, 5e-324, float("inf"), float("nan"))
IN = (0.0, -0.0, 1.0, -1.25, 2.0 ** 100, -2.0 ** 100, 2.0 ** -100)


def rope(scale, T=4):
    r = sp._Rotation(A, scale, 128, 0)
    return sp.load().spear_rope(A, 256, T, 2, 128, A, ctypes.byref(r), 2 * A, 256, None)


def write(scale, T=4):
    r = sp._Rotation(A, scale, 128, 0)
    kv = sp._KV4(A, A, A, A, 4, 2, 128, 16)
    return sp.load().spear_rope_kv4_write(A, 512, A, 256, A, 256, T, 4, A, A, ctypes.byref(r), ctypes.byref(kv), 2 * A, 512, None)


@pytest.mark.parametrize("scale", OUT)
def test_factors_out_of_range(scale):
    assert rope(scale) == E_ARG and write(scale) == E_ARG


@pytest.mark.parametrize("scale", IN)
def test_factors_in_range(scale):
    """Without rows nothing is launched; what is left to refuse is the device."""
    assert rope(scale, T=0) != E_ARG and write(scale, T=0) != E_ARG
