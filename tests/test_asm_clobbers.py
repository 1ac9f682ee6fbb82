"""Inline assembly of the kernels names the registers that it overwrites by
name (CPU only: reads the sources)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_post_weight_amd", "csrc")


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            end = text.index(");", m.end())
            yield os.path.basename(path), text[m.end():end]


def test_named_registers_are_clobbers():
    found = 0
    for path, body in _statements():
        parts = re.split(r'(?<![:"]):(?![:"])', re.sub(r"::", " : : ", body))
        for reg in set(re.findall(r"s_mov_b32 (m0)", parts[0])):
            found += 1
            assert len(parts) == 4 and f'"{reg}"' in parts[3], (path, body)
    assert found == 2  # the 16- and 4-byte transfers to LDS
