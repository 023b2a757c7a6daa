"""Wait states in hand-written assembly (CPU only, read from the sources)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "flatquant_transform_quant_amd", "csrc")
SOURCES = [f for f in glob.glob(os.path.join(CSRC, "**", "*"), recursive=True) if f.endswith((".hip", ".h"))]


def _blocks(text):
    """The instruction texts of the file's asm statements."""
    for m in re.finditer(r'asm\s+volatile\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text):
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m[1])).replace("\\n", "\n").replace("\\t", "\t")


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.relpath(f, CSRC) for f in SOURCES])
def test_a_load_placed_by_m0_waits_for_m0(path):
    """A memory instruction that takes its LDS place from m0 needs a wait state after a scalar write of m0; the compiler adds it
    to its own code, not inside an asm statement."""
    with open(path, encoding="utf-8") as fh:
        for block in _blocks(fh.read()):
            lines = [l.strip() for l in block.splitlines() if l.strip()]
            for a, b in zip(lines, lines[1:]):
                if re.match(r"s_mov_b32\s+m0\b", a):
                    assert not re.search(r"\blds\b", b), (os.path.basename(path), a, b)


def test_the_blocks_are_found():
    found = [b for f in SOURCES for b in _blocks(open(f, encoding="utf-8").read()) if "m0" in b]
    assert len(found) == 2 and all("offen lds" in b for b in found)
