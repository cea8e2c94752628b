"""Inline assembly beside matrix instructions (CPU only: reads the assembly of
the kernels built here).

An MFMA goes on reading its addend and writing its result for some cycles after
it was issued.  The compiler keeps vector instructions of its own away from
those registers for that long, but it does not look into inline assembly, so no
vector instruction of an assembly block may write a register that an MFMA just
before it names as addend or result."""

import concurrent.futures
import os
import re
import subprocess

import pytest

from bit_nf4_quantized_21_amd import build as B

WINDOW = 24     # instructions: more than the wait states of the longest MFMA (18)


def _sources():
    return [f for f in sorted(os.listdir(B.CSRC)) if f.endswith(".hip") and "mfma" in open(os.path.join(B.CSRC, f)).read()]


def _registers(text):
    text = text.strip()
    m = re.match(r"([va])\[(\d+):(\d+)\]", text)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([va])(\d+)$", text)
    return {(m[1], int(m[2]))} if m else set()


def _conflicts(listing):
    """(matrix instructions, [(kernel, assembly instruction)] that write a register in use)."""
    kernel, inside, recent, matrix, found = "", False, [], 0, []
    for line in listing.splitlines():
        s = line.strip()
        if re.match(r"_Z\S+:", s):
            kernel, recent = s.split(":")[0], []
        if "#ASMSTART" in s or "#ASMEND" in s:
            inside = "#ASMSTART" in s
            continue
        s = s.split(";")[0].strip()
        if not s or s[0] == "." or s.endswith(":"):
            continue
        op, _, rest = s.partition(" ")
        args = rest.split(",")
        in_use = set()
        if op.startswith("v_mfma"):
            matrix += 1
            in_use = _registers(args[0]) | _registers(args[3].split()[0])
        elif inside and op.startswith("v_") and any(_registers(args[0]) & r for r in recent):
            found.append((kernel, s))
        recent = (recent + [in_use])[-WINDOW:]
    return matrix, found


def test_the_scan_sees_a_conflict():
    good = "_Zk:\n v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[4:7]\n ;;#ASMSTART\n v_mov_b32 {}, v20\n ;;#ASMEND\n"
    assert _conflicts(good.format("v16")) == (1, [])
    assert _conflicts(good.format("v5"))[1] and _conflicts(good.format("v0"))[1]
    assert _conflicts(good.format("v5").replace(";;#ASM", ";"))[1] == []       # the compiler's own: not ours to check


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="needs hipcc")
def test_no_assembly_writes_a_register_of_a_running_matrix_instruction(tmp_path):
    def listing(f):
        out = str(tmp_path / (f + ".s"))
        subprocess.run([B.HIPCC, *B.HIP_FLAGS, *B.FILE_FLAGS.get(f, []), "-S", "--cuda-device-only", os.path.join(B.CSRC, f),
                        "-o", out], check=True, capture_output=True, text=True, timeout=300)
        return _conflicts(open(out).read())
    files = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        results = dict(zip(files, ex.map(listing, files)))
    assert {"gemm_fwd.hip", "gemm_dx.hip", "gemv.hip", "attend.hip", "attend_tile.hip"} <= set(files)
    assert sum(n for n, _ in results.values()) > 1000
    assert {f: found for f, (_, found) in results.items() if found} == {}
