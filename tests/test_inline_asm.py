"""Inline assembly names what it changes: a statement that writes m0 lists it, so that the compiler
keeps no value of its own there across it."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_kla_amd", "csrc")


def statements(path):
    """The text of every asm statement, up to its closing bracket."""
    text = open(path).read()
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            depth += 0 if quoted else (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*"))), ids=os.path.basename)
def test_writers_of_m0_say_so(path):
    for s in statements(path):
        if re.search(r"s_\w+ m0\b", s):
            assert '"m0"' in s.rsplit(":", 1)[1], s
