"""No vector instruction meets a matrix instruction's result before it is there
(CPU only, on the assembly that the build's own flags give).

The hardware does not wait: 8 wait states have to pass behind a matrix instruction
of 16 x 16 x 32 and 12 behind one of 32 x 32 x 16 before its result is read or
written by anything but a matrix instruction that adds to it.  The compiler puts
them in, but where branches rejoin it has counted the longer path only.
"""
import os
import re
import shutil
import subprocess

import pytest

from quantized_gemm_w4a16_amd import build
from test_lds_reads_cpu import kernels, pending_at_barriers

STATES = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_32x32x16_bf16": 12}


def registers(text):
    out = set()
    for m in re.finditer(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        lo, hi = (m.group(2), m.group(3)) if m.group(2) else (m.group(4), m.group(4))
        out |= {(m.group(1), i) for i in range(int(lo), int(hi) + 1)}
    return out


def operands(args):
    return [registers(a) for a in re.split(r",\s*(?![^\[]*\])", args)]


def too_early(code, labels):
    """[(matrix instruction, the one that meets its result, states between)] over all paths."""
    bad = []
    for k, (op, args) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        need, result = STATES[op], operands(args)[0]
        seen, work = {}, [(k + 1, 0)]
        while work:
            i, n = work.pop()
            while i < len(code) and n < need and seen.get(i, need) > n:
                seen[i] = n
                op2, args2 = code[i]
                if op2 == "s_nop":
                    n += int(args2, 0)
                elif op2.startswith("v_mfma"):
                    to, a, b, c = operands(args2)
                    if (a | b) & result:
                        bad.append((k, i, n))
                    if to & result:                       # adds to it; its own result is walked by itself
                        break
                elif re.match(r"v_|ds_|global_|buffer_|flat_|scratch_", op2) and registers(args2) & result:
                    bad.append((k, i, n))
                    break
                n += 1
                if op2 == "s_branch":
                    i = labels[args2]
                    continue
                if op2.startswith("s_cbranch"):
                    work.append((labels[args2], n))
                if op2 in ("s_endpgm", "s_setpc_b64"):
                    break
                i += 1
    return bad


def test_the_walk_itself():
    mf = "v_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], v[0:15]\n"
    for between, n in (("", 1), ("s_nop 11\n", 0), ("s_nop 10\n", 1), ("s_nop 10\ns_mov_b32 s0, 0\n", 0),
                       ("s_cbranch_scc0 .LBB1\ns_nop 15\n.LBB1:\n", 1),
                       ("s_nop 10\ns_cbranch_scc0 .LBB1\ns_nop 15\n.LBB1:\n", 0)):
        (found,) = kernels("_Zk:\n" + mf + between + "v_max_f32_e32 v30, v15, v15\ns_endpgm\n").values()
        assert len(too_early(*found)) == n, between
    for use, n in (("v_mfma_f32_32x32x16_bf16 v[0:15], v[24:27], v[20:23], v[0:15]", 0),
                   ("v_mfma_f32_32x32x16_bf16 v[32:47], v[12:15], v[20:23], v[32:47]", 1),
                   ("v_mov_b32_e32 v3, v40", 1), ("v_mov_b32_e32 v16, v40", 0), ("ds_write_b64 v50, v[14:15]", 1)):
        (found,) = kernels("_Zk:\n" + mf + use + "\ns_endpgm\n").values()
        assert len(too_early(*found)) == n, use


def test_attention_waits(tmp_path):
    hipcc = build._hipcc()
    if shutil.which(hipcc) is None:
        pytest.skip("hipcc not found")
    out = tmp_path / "a.s"
    subprocess.run([hipcc, *build.CFLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, "kv_attention.hip"), "-o",
                    str(out)], check=True, capture_output=True)
    found = kernels(out.read_text())
    assert sum(op.startswith("v_mfma") for code, _ in found.values() for op, _ in code) > 200
    early = {name: [(*code[k], *code[i], n) for k, i, n in bad] for name, (code, labels) in found.items()
             if (bad := too_early(code, labels))}
    assert not early, early
    late = {name: len(b) for name, k in found.items() if (b := pending_at_barriers(*k))}
    assert not late, late
