"""Where the GEMM reads packed weights: inside the row, whatever K (no GPU).  The
offsets are the kernel's own function, compiled for the host."""
import os
import shutil
import subprocess

import pytest

from quantized_gemm_w4a16_amd import build

SOURCE = r"""
#include "spear_internal.hpp"
#include <stdio.h>
int main()
{
    int bad = 0;
    for (int64_t K = 32; K <= 4160; K += 32)
        for (int c = 0; c < 4; c++)
            for (int64_t st = 0; st < (K + 127) / 128 + 3; st++) {
                const int64_t o = spear::w_offset(K, c, st), in = 128 * st + 32 * c < K;
                if (o < 0 || o + 16 > K / 2 || (in && o != 64 * st + 16 * c))
                    bad += printf("K %ld piece %d stage %ld: offset %ld\n", (long)K, c, (long)st, (long)o) > 0;
            }
    return bad != 0;
}
"""


def test_offsets_stay_inside_the_row(tmp_path):
    hipcc = build._hipcc()
    if shutil.which(hipcc) is None:
        pytest.skip("hipcc not found")
    (tmp_path / "a.hip").write_text(SOURCE)
    subprocess.run([hipcc, "-O1", "-std=c++17", "--cuda-host-only", "-I", build.CSRC, str(tmp_path / "a.hip"), "-o",
                    str(tmp_path / "a")], check=True, capture_output=True)
    r = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[:2000]
