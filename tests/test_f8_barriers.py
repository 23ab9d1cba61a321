"""Synchronisation of the f8 kernels, read from the gfx950 assembly that their
sources compile to (no GPU needed)."""
import os
import re
import subprocess

import pytest

from quantized_weight_gemv_amd import build


def _assembly(unit, tmp_path):
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path / (unit + ".s")
    subprocess.run([hipcc, *build.COMMON, "--cuda-device-only", "-S", os.path.join(build.CSRC, unit), "-o", str(out)],
                   check=True, capture_output=True)
    return out.read_text().splitlines()


def _reads_at_barriers(lines):
    """{kernel: [LDS reads that may be in flight at each barrier]}, counted along the code: the count of
    s_waitcnt is an upper bound of what is left."""
    found, kernel, reads = {}, None, 0
    for line in lines:
        label = re.match(r"^(_Z\S+):", line)
        if label:
            kernel, reads = label.group(1), 0
            found[kernel] = []
            continue
        op = line.strip()
        if op.startswith("ds_read"):
            reads += 1
        elif op.startswith("s_waitcnt"):
            left = re.search(r"lgkmcnt\((\d+)\)", op)
            if left:
                reads = min(reads, int(left.group(1)))
        elif op.startswith("s_barrier"):
            found[kernel].append(reads)
        elif op.startswith("s_endpgm"):
            reads = 0
    return {k: v for k, v in found.items() if v}


@pytest.mark.parametrize("unit,kernels", [("qgemv_f8_gemm.hip", 2), ("qgemv_f8_skinny.hip", 7),
                                          ("qgemv_f8_wgrad.hip", 6)])
def test_no_lds_read_is_in_flight_at_a_barrier(unit, kernels, tmp_path):
    """Behind a barrier other waves copy into the buffers that were read in front of it, with loads that write
    LDS: a read that still waits in the LDS queue would return what they bring."""
    found = _reads_at_barriers(_assembly(unit, tmp_path))
    assert len(found) >= kernels
    bad = {k: v for k, v in found.items() if any(v)}
    assert not bad, bad


def _waits_in_loops(lines):
    """{kernel: [vmcnt of each wait in the loop that multiplies]}."""
    found, kernel, labels = {}, None, {}
    for n, line in enumerate(lines):
        name = re.match(r"^(_Z\S+):", line)
        if name:
            kernel, labels = name.group(1), {}
        label = re.match(r"^(\.LBB\S+):", line)
        if label:
            labels[label.group(1)] = n
        back = re.match(r"\s+s_c?branch\S*\s+(\.LBB\S+)", line)
        if back and back.group(1) in labels:
            body = lines[labels[back.group(1)]:n]
            if any("v_mfma" in op for op in body):
                found[kernel] = [int(w) for op in body for w in re.findall(r"s_waitcnt.*vmcnt\((\d+)\)", op)]
    return found


def test_gemm_loops_keep_their_copies_in_flight(tmp_path):
    """The loop waits for the copies that a step reads, by count; a wait for all of them would empty the ring."""
    found = _waits_in_loops(_assembly("qgemv_f8_gemm.hip", tmp_path))
    assert len(found) >= 12
    drained = {k: v for k, v in found.items() if 0 in v or not v}
    assert not drained, drained


def test_the_count_sees_a_missing_wait():
    """The counting itself, on a loop with and without the wait."""
    code = ["_Zk:", "ds_read_b128 v[0:3], v9", "s_waitcnt vmcnt(4)", "s_barrier", "s_waitcnt lgkmcnt(0)", "s_endpgm"]
    assert _reads_at_barriers(code) == {"_Zk": [1]}
    code[2] = "s_waitcnt vmcnt(4) lgkmcnt(0)"
    assert _reads_at_barriers(code) == {"_Zk": [0]}
