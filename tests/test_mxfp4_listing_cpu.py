"""The loads that MXFP4's tiles make in inline assembly, in the listing of the built kernels:
five instructions or as long a pause lie between a vector instruction that writes a scalar
register and a load that takes it, which the compiler does not see to inside assembly."""
import os
import re
import subprocess

import pytest

from w4a16_dequant_gemv_amd import build

LOAD = re.compile(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\], s(\d+) offen lds")
WRITES = re.compile(r"v_\w+ (?:s(\d+)|s\[(\d+):(\d+)\])(?:,|$)")


def faults(lines):
    """(line, what) of every load that comes too early behind such a write."""
    bad, loads = [], 0
    code = [l.split(";")[0].strip() for l in lines]
    code = [l for l in code if l and not l.startswith(".") and not l.endswith(":")]
    for i, l in enumerate(code):
        m = LOAD.match(l)
        if not m:
            continue
        loads += 1
        takes = {*range(int(m[1]), int(m[2]) + 1), int(m[3])}
        states, j = 0, i - 1
        while states < 5 and j >= 0:
            w = WRITES.match(code[j])
            if w:
                lo = int(w[1] or w[2])
                if takes & set(range(lo, int(w[3] or lo) + 1)):
                    bad.append((l, code[j]))
            nop = re.match(r"s_nop (\d+)", code[j])
            states += int(nop[1]) + 1 if nop else 1
            j -= 1
    return bad, loads


def test_the_search_finds_one():
    load = "\tbuffer_load_dwordx4 v3, s[4:7], s22 offen lds"
    for gap, bad in (["\ts_nop 0"], 1), (["\ts_nop 3"], 1), (["\ts_nop 4"], 0), (["\ts_mov_b32 s9, 0"] * 5, 0):
        assert len(faults(["\tv_readfirstlane_b32 s5, v17", *gap, load])[0]) == bad
    assert faults(["\tv_readfirstlane_b32 s8, v17", load]) == ([], 1)
    assert len(faults(["\tv_readlane_b32 s22, v1, 3", ";;#ASMSTART", "\ts_nop 0", load])[0]) == 1


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")
def test_loads_in_assembly(tmp_path):
    out = tmp_path / "mx4_matmul.s"
    subprocess.run([build.HIPCC, *build.COMMON, *build.PER_FILE.get("mx4_matmul.hip", []), "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "mx4_matmul.hip"), "-o", str(out)], check=True, capture_output=True)
    text = out.read_text()
    bad, loads = faults(text.split("\n"))
    assert loads > 100 and not bad, bad[:3]
    for what in ("sgpr_spill_count", "vgpr_spill_count", "private_segment_fixed_size"):
        counts = re.findall(rf"\.{what}:\s+(\d+)", text)
        assert counts and set(counts) == {"0"}, what
