"""Inline assembly names what it writes."""
import glob
import os
import re

from bit_gradient_compression_amd import build as B


def asm_blocks(text):
    """The statements `asm ... ( ... );` of a source, with their parentheses balanced."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b[^(;]*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def test_m0_is_declared():
    """Assembly that writes m0 lists it as clobbered, so that the compiler keeps nothing there, or
    saves it first and restores it last."""
    seen = 0
    for path in glob.glob(os.path.join(B.CSRC, "*.h*")):
        for block in asm_blocks(open(path).read()):
            if re.search(r"s_mov_b32\s+m0", block):
                seen += 1
                restored = re.search(r"s_mov_b32 (%\d), m0.*s_mov_b32 m0, \1\"", block, re.S)
                assert restored or '"m0"' in block.rsplit(":", 1)[1], path
    assert seen
