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
