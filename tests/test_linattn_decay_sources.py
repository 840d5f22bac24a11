"""Properties of the decayed attention's sources that no run shows (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rwkv_linear_rnn_b200", "csrc")


@pytest.mark.parametrize("name", ["linattn_decay_rec.cu", "linattn_rotary.cu"])
def test_shared_arrays_read_by_vectors_are_aligned(name):
    """A shared array that is read as float4 says so in its declaration: its place among the others is the
    compiler's choice, and a plain float array is only aligned to 4 bytes."""
    src = open(os.path.join(CSRC, name), encoding="utf-8").read()
    declared = re.findall(r"(?:extern )?__shared__ ([^;]+);", src)
    assert declared
    for line in declared:
        for array in re.findall(r"(\w+)\[", line.replace("__align__", "")):
            vector = re.search(r"reinterpret_cast<(?:const )?(?:float4|ulonglong2|uint4) \*>\(%s\b" % array, src)
            assert not vector or "__align__(16)" in line, (name, line)
