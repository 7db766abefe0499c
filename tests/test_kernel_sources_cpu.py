"""Rules for the kernels' inline assembly that a compiler does not check."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_rotations_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))
MEMORY = r"\b(?:buffer|global|flat|scratch)_(?:load|store|atomic)"


def asm_blocks(text):
    """Every asm statement, its parentheses matched."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.start():i]


def instructions(block):
    """Its instructions, one a string."""
    code = ""
    for text, end in re.findall(r'"((?:[^"\\]|\\.)*)"|(:)', block):
        if end:                                                   # what follows are operands
            break
        code += text
    return [x.strip() for x in re.split(r"\\n(?:\\t)?", code) if x.strip()]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_memory_instructions_wait_for_scalar_registers(path):
    """A memory instruction has to be five wait states behind a vector
    instruction (v_readlane, v_readfirstlane) that wrote a scalar register which
    it reads.  The compiler inserts them for its own memory instructions only,
    and may put such a write right in front of assembly."""
    for block in asm_blocks(open(path).read()):
        states = 0                                                # since the assembly's beginning
        for code in instructions(block):
            if re.match(MEMORY, code):
                assert states >= 5, block
            states += int(code.split()[1]) + 1 if code.startswith("s_nop") else 1


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_m0_is_named_where_it_is_written(path):
    """The compiler uses m0 for itself and takes no clobber of it: assembly that
    writes it names it as a result."""
    for block in asm_blocks(open(path).read()):
        if any(re.match(r"s_\w+ m0,", code) for code in instructions(block)):
            assert '"={m0}"(' in block, block


def test_the_rules_see_what_they_are_for():
    found = [b for p in SOURCES for b in asm_blocks(open(p).read()) if any(re.match(MEMORY, c) for c in instructions(b))]
    assert len(found) == 7
