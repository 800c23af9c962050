"""Kernels that load from memory straight to LDS order those loads themselves:
at a barrier none of a wavefront's reads of LDS may be unfinished, as another
wavefront may ask for the next piece in their place right behind it.  Read from
the assembly of the kernels' sources, along the order of its lines (no GPU)."""
import os
import re
import subprocess

import pytest

from clebsch_gordan_tensor_amd import build as B


def _open_reads(lines):
    """{kernel: reads of LDS that are unfinished at each of its barriers}, of
    the kernels that load to LDS."""
    out, direct, name, pending = {}, set(), None, 0
    for line in lines:
        label = re.match(r"(_Z\w+):", line)
        if label:
            name, pending = label.group(1), 0
        t = line.strip()
        if re.match(r"(global|buffer)_load_lds|buffer_load\w* .* lds\b", t):
            direct.add(name)
        elif t.startswith("ds_read"):
            pending += 1
        elif t.startswith("s_waitcnt"):
            left = re.search(r"lgkmcnt\((\d+)\)", t)
            pending = min(pending, int(left.group(1))) if left else pending
        elif t.startswith("s_barrier"):
            out.setdefault(name, []).append(pending)
    return {k: out.get(k, []) for k in direct}


def test_the_reading_of_the_assembly():
    text = ["_Zk:", " global_load_lds_dwordx4 v[0:1], off", " ds_read_b128 v[0:3], v4",
            " ds_read_b128 v[4:7], v4", " s_waitcnt lgkmcnt(1)", " s_barrier",
            " s_waitcnt vmcnt(0) lgkmcnt(0)", " s_barrier", "_Zother:", " ds_read_b32 v0, v1",
            " s_barrier"]
    assert _open_reads(text) == {"_Zk": [1, 0]}


@pytest.mark.parametrize("source,kernels", [("grouped", 3), ("fp8", 2)])
def test_no_read_is_open_at_a_barrier(tmp_path, source, kernels):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    asm = str(tmp_path / "k.s")
    flags = [f for f in B.HIP_FLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, "-S", "--cuda-device-only", "-o", asm,
                    os.path.join(B.CSRC, "kernels", source + ".hip")], check=True,
                   capture_output=True)
    with open(asm) as f:
        found = _open_reads(f)
    assert len(found) == kernels, sorted(found)
    for name, reads in found.items():
        assert reads and not any(reads), (name, reads)
