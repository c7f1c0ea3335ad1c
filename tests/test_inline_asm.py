"""Inline assembly names the special registers that it writes: the compiler keeps
nothing in a register that a statement clobbers, and may in one that it does not name."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scaled_fp8_casting_amd", "csrc")
SPECIAL = re.compile(r"\b[sv]_\w+ (m0|vcc|exec|vcc_lo|vcc_hi|exec_lo|exec_hi)\b")


def statements(text):
    """Every asm statement: what its parentheses hold."""
    for m in re.finditer(r"\b(?:__asm__|asm)\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


def unnamed(text):
    """(register, statement) of each special register written and not named after the last colon."""
    found = []
    for s in statements(text):
        strings = re.findall(r'"((?:[^"\\]|\\.)*)"', s)
        for reg in {r for code in strings for r in SPECIAL.findall(code.replace("\\n", "\n").replace("\\t", " "))}:
            if reg not in strings:
                found.append((reg, s))
    return found


def test_the_scan():
    bad = '__asm__ volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" ::"s"(f(1)) : "memory");'
    assert [r for r, _ in unnamed(bad)] == ["m0"]
    assert unnamed(bad.replace('"memory"', '"memory", "m0"')) == []
    assert unnamed('__asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(3) : "memory");') == []


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".hip"))))
def test_sources(name):
    with open(os.path.join(CSRC, name)) as f:
        assert unnamed(f.read()) == []
