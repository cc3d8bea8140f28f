"""What the kernels' inline assembly may hold.  The compiler puts the wait states between a matrix instruction and the reader
of its result, but does not look into inline assembly: so that computes nothing and only waits, or only marks a value."""
import os
import re

import pytest

from canvas_rope_rotary_amd.build import CSRC

SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".hip")))
ASM = re.compile(r'\basm\s*(?:volatile\s*)?\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)')
WAITS = ("s_waitcnt", "s_barrier", "s_nop")


def instructions(text):
    """Mnemonics of every asm statement of a source."""
    out = []
    for m in ASM.finditer(text):
        body = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))
        out += [line.split()[0] for line in re.split(r"\\n|\\t|;", body) if line.strip()]
    return out


def test_the_search_finds_instructions():
    assert instructions('asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x));') == ["v_max3_f32"]
    assert instructions('asm volatile("s_waitcnt vmcnt(0)\\n\\ts_barrier" ::: "memory");') == ["s_waitcnt", "s_barrier"]
    assert instructions('asm volatile("" : "+v"(y));') == []


@pytest.mark.parametrize("name", SOURCES)
def test_inline_assembly_only_waits(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert len(ASM.findall(text)) == len(re.findall(r"\basm\b", re.sub(r"//.*", "", text)))
    assert all(i in WAITS for i in instructions(text)), instructions(text)
