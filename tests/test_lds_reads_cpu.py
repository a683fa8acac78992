"""No LDS read is in flight where a workgroup meets (CPU only, on the assembly
that the build's own flags give).

The kernels that stream through ring buffers in LDS refill a buffer by DMA right
behind a barrier.  A read of that buffer which a wave issued before the barrier
and has not waited for may then return the new bytes, so every path to an
s_barrier has to pass a wait for the LDS reads before it.
"""
import os
import re
import shutil
import subprocess

import pytest

from quantized_gemm_w4a16_amd import build

LDS_READ = re.compile(r"^ds_(read|load|permute|bpermute|swizzle)")


def kernels(text):
    """-> {name: (instructions [(op, operands)], labels {label: index})}"""
    found, name, code, labels = {}, None, None, None
    for line in text.splitlines():
        s = line.split(";")[0].strip()
        m = re.match(r"^(_Z\w+):", s)
        if m:
            name, code, labels = m.group(1), [], {}
            found[name] = (code, labels)
        elif name and re.match(r"^\.L\w+:", s):
            labels[s[:-1]] = len(code)
        elif name and s.startswith(".section"):
            name = None
        elif name and s and not s.startswith("."):
            op, _, args = s.partition(" ")
            code.append((op, args.strip()))
    return {k: v for k, v in found.items() if any(op == "s_endpgm" for op, _ in v[0])}


def pending_at_barriers(code, labels):
    """Indices of the barriers that some path reaches with LDS reads in flight.
    The state of a path is how many LDS reads are younger than its last wait, 15
    at most (the counter has four bits, and more is no worse)."""
    bad, seen, work = set(), {}, [(0, 0)]
    while work:
        i, n = work.pop()
        while i < len(code) and seen.get(i, -1) < n:
            seen[i] = n
            op, args = code[i]
            if LDS_READ.match(op):
                n = min(n + 1, 15)
            elif op == "s_waitcnt":
                m = re.search(r"lgkmcnt\((\d+)\)", args)
                if m:
                    n = min(n, int(m.group(1)))
                elif re.fullmatch(r"(0x[0-9a-f]+|\d+)", args):
                    n = min(n, int(args, 0) >> 8 & 15)
            elif op == "s_barrier" and n:
                bad.add(i)
            if op == "s_branch":
                i = labels[args]
                continue
            if op.startswith("s_cbranch"):
                work.append((labels[args], n))
            if op in ("s_endpgm", "s_setpc_b64"):
                break
            i += 1
    return bad


def test_the_walk_itself():
    loop = "k:\n.LBB0:\nds_read_b128 v[0:3], v4\n{}\ns_barrier\ns_cbranch_scc0 .LBB0\ns_endpgm\n"
    for wait, n in (("s_nop 0", 1), ("s_waitcnt lgkmcnt(0)", 0), ("s_waitcnt vmcnt(0)", 1),
                    ("s_waitcnt vmcnt(3) lgkmcnt(0)", 0), ("s_waitcnt lgkmcnt(1)", 1)):
        (found,) = kernels("_Z" + loop.format(wait)).values()
        assert len(pending_at_barriers(*found)) == n, wait
    around = ("_Zk:\nds_read_b32 v0, v1\ns_cbranch_scc0 .LBB1\ns_waitcnt lgkmcnt(0)\n"
              ".LBB1:\ns_barrier\ns_endpgm\n")
    (found,) = kernels(around).values()
    assert pending_at_barriers(*found)


@pytest.mark.parametrize("source", ["experts.hip", "route.hip", "prefill.hip"])
def test_no_lds_read_in_flight_at_a_barrier(source, tmp_path):
    hipcc = build._hipcc()
    if shutil.which(hipcc) is None:
        pytest.skip("hipcc not found")
    out = tmp_path / "a.s"
    subprocess.run([hipcc, *build.CFLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, source), "-o",
                    str(out)], check=True, capture_output=True)
    found = kernels(out.read_text())
    assert len(found) >= 5 and any("s_barrier" == op for code, _ in found.values() for op, _ in code)
    late = {name: len(b) for name, k in found.items() if (b := pending_at_barriers(*k))}
    assert not late, late
