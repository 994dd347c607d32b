"""Guards on the generated gfx950 code of the decoding kernels (no GPU needed)."""

import os
import re

from test_build_guards import CSRC, _assembly


def test_no_scalar_instruction_with_a_64_bit_literal():
    """gfx950 has no encoding for a scalar instruction with a 64-bit literal. The compiler
    may form one all the same from an fp64 constant that is uniform over a wavefront; it
    prints the literal, and writes 0 into the object. So no kernel may contain one."""
    for src in sorted(os.listdir(CSRC)):
        if src.endswith(".hip"):
            found = re.findall(r"^\s*s_\w+_b64 .*0x[0-9a-f]{9,}.*$", _assembly(os.path.join(CSRC, src)), re.M)
            assert not found, (src, found)


def test_attention_keeps_its_sums_in_registers():
    """The sums over keys stay in registers: a kernel that spills them to scratch memory computes the same, slower."""
    found = {}
    for block in re.split(r"\n\s+- \.", _assembly(os.path.join(CSRC, "attend_kernels.hip"))):
        name = re.search(r"\.name:\s+(\S+)", block)
        size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", block)
        if name and size and "k_attend" in name.group(1):
            found[name.group(1)] = int(size.group(1))
    assert len(found) >= 48, sorted(found)
    assert not any(found.values()), {k: v for k, v in found.items() if v}
