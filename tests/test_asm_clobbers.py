"""Inline assembly in the kernel sources names the special registers it writes
(CPU only: the sources are read, nothing is run)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rotation_int4_weight_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h*")))
# an instruction's first operand is what it writes
WRITES = re.compile(r"\b[sv]_\w+\s+(m0|vcc|exec|scc)\b")


def statements(text):
    """(template, rest of the operands) of every asm statement."""
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        body = text[m.end():i - 1]
        strings = [s for s in re.finditer(r'"((?:[^"\\]|\\.)*)"', body)]
        template, end = "", 0
        for s in strings:  # adjacent literals are one template
            if template and body[end:s.start()].strip():
                break
            template, end = template + s.group(1), s.end()
        yield template.replace("\\n", "\n").replace("\\t", " "), body[end:]


def unnamed(text):
    return [(w, t) for t, rest in statements(text) for w in WRITES.findall(t) if f'"{w}"' not in rest]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_written_registers_are_named(path):
    with open(path) as f:
        assert unnamed(f.read()) == []


def test_a_missing_name_is_found():
    line = 'asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 4\\n\\t" "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at) : "memory"{});'
    assert [w for w, _ in unnamed(line.format(""))] == ["m0"] and unnamed(line.format(', "m0"')) == []
    assert unnamed('asm("s_waitcnt vmcnt(0)" ::: "memory"); asm volatile("v_mov_b32 %0, 0" : "=v"(x));') == []
