"""No instruction in inline assembly next to matrix instructions: the compiler keeps
the waits between a matrix instruction and the next access of its registers for its
own instructions only."""
import os
import re

import pytest

from dequant_matmul_int3_amd import build as qbuild


def _with_includes(name, seen):
    if name in seen or not os.path.exists(os.path.join(qbuild.CSRC, name)):
        return seen
    with open(os.path.join(qbuild.CSRC, name)) as f:
        seen[name] = re.sub(r"//[^\n]*", "", f.read())
    for inc in re.findall(r'#include "([^"]+)"', seen[name]):
        _with_includes(inc, seen)
    return seen


def _instructions(text):
    """Templates of inline assembly that are not empty."""
    return [t for t in re.findall(r'\basm\b[\w\s]*\(\s*"([^"]*)"', text) if t.strip()]


def test_what_counts():
    assert _instructions('asm volatile("s_nop 0" :: ); asm("" : "+v"(x)); asm(\n "v_mov %0, 0"') == \
        ["s_nop 0", "v_mov %0, 0"]


@pytest.mark.parametrize("src", [s for s in qbuild.SOURCES if s.endswith(".hip")])
def test_no_instruction_in_assembly_next_to_matrix_instructions(src):
    files = _with_includes(src, {})
    if any("__builtin_amdgcn_mfma" in t for t in files.values()):
        assert not {n: a for n, t in files.items() for a in _instructions(t)}
