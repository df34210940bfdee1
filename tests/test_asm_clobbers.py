"""Inline assembly of the kernels that writes M0 lists it among its clobbers: a value that the
compiler kept there across the statement would be lost without a word."""
import glob
import os
import re

import pytest

import precision_moe_amd as pm

CSRC = os.path.join(os.path.dirname(os.path.abspath(pm.__file__)), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


def _statements(text):
    """The inside of each asm statement's parentheses, comments and line breaks within taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield " ".join(text[m.end():i - 1].split())


def _parts(statement):
    """(template, names of clobbers) of an asm statement: the parts between colons outside quotes and parentheses."""
    parts, depth, quoted = [""], 0, False
    for i, c in enumerate(statement):
        if c == '"' and statement[i - 1] != "\\":
            quoted = not quoted
        elif not quoted:
            depth += (c in "([") - (c in ")]")
            if c == ":" and depth == 0:
                parts.append("")
                continue
        parts[-1] += c
    return parts[0], re.findall(r'"([^"]+)"', parts[3]) if len(parts) > 3 else []


def test_parts_of_a_statement():
    template, clobbers = _parts('"s_mov_b32 m0, %0" ::"s"(f(a)), "v"(b[1]) : "m0", "memory"')
    assert "m0, %0" in template and clobbers == ["m0", "memory"]
    assert _parts('"s_nop 0"') == ('"s_nop 0"', [])
    assert _parts('"" : "+v"(v)')[1] == []


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_statements_that_write_m0_say_so(path):
    with open(path) as f:
        for s in _statements(f.read()):
            template, clobbers = _parts(s)
            if re.search(r"\b\w+\s+m0\s*,", template):
                assert "m0" in clobbers, s


def test_there_are_such_statements():
    found = [s for p in SOURCES for s in _statements(open(p).read()) if re.search(r"\b\w+\s+m0\s*,", _parts(s)[0])]
    assert found
