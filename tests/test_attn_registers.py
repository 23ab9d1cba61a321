"""The attention step's kernels keep what a lane holds in registers, read from the gfx950 assembly that their sources
compile to (no GPU needed)."""
import re

import pytest

from test_f8_barriers import _assembly


# two tiles of rows at 256 dimensions in 16 bits have more operands than registers, and are faster all the same
SPILLS = "attend_kernelINS_4(Fp|Bf)16ELb0ELi256ELi2E"


@pytest.mark.parametrize("unit,kernels", [("qgemv_heads.hip", 90), ("qgemv_attend.hip", 40)])
def test_nothing_goes_through_private_memory(unit, kernels, tmp_path):
    """An array that is indexed under a branch moves to memory: every head's values went there and back, and the
    waits for them emptied the queue of loads made ahead."""
    found, kernel = {}, None
    for line in _assembly(unit, tmp_path):
        label = re.match(r"^(_Z\S+):", line)
        if label:
            kernel = label.group(1)
            found[kernel] = 0
        elif line.strip().startswith("scratch_"):
            found[kernel] += 1
    assert len(found) >= kernels
    bad = {k: n for k, n in found.items() if n and not re.search(SPILLS, k)}
    assert not bad, bad
