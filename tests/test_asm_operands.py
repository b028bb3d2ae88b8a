"""Checks of the operands of the kernels' inline assembly (no GPU needed)."""
import glob
import os
import re

import pytest

from deepseek_sparse_attention_lightning_gb300 import build
from test_kernel_sources import _code

SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(build.CSRC, "*.cu*")))


def _statements(text):
    """(template, output constraints, number of inputs) of each asm statement."""
    found = []
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        parts, depth, i, literal = [""], 1, m.end(), ""
        while depth:
            c = text[i]
            if c == '"':
                j = i + 1
                while text[j] != '"':
                    j += 2 if text[j] == "\\" else 1
                parts[-1] += text[i:j + 1]
                i = j + 1
                continue
            depth += (c == "(") - (c == ")")
            if depth == 1 and text[i:i + 2] == "::":
                parts += ["", ""]
                i += 2
                continue
            if depth == 1 and c == ":":
                parts.append("")
            elif depth:
                parts[-1] += c
            i += 1
        literals = lambda s: re.findall(r'"((?:[^"\\]|\\.)*)"', s)
        parts += [""] * (3 - len(parts))
        found.append(("".join(literals(parts[0])).replace("\\n", "\n"), literals(parts[1]), len(literals(parts[2]))))
    return found


def _late_reads(template, outputs, inputs):
    """Outputs that are written before an input is read, and are not marked so."""
    written, late = set(), set()
    for line in template.split(";"):
        named = [int(n) for n in re.findall(r"%(\d+)", line)]
        if any(len(outputs) <= n < len(outputs) + inputs for n in named):
            late |= written
        written |= {n for n in named if n < len(outputs)}
    return sorted(n for n in late if "&" not in outputs[n])


@pytest.mark.parametrize("name", SOURCES)
def test_outputs_written_before_an_input_is_read_say_so(name):
    """An output without "&" may be given the register of an input.  Where one instruction of a statement
    writes it and a later one reads the input (a load's address, say), the input would be gone."""
    for template, outputs, inputs in _statements(_code(name)):
        assert _late_reads(template, outputs, inputs) == [], template


def test_the_check_sees_a_late_read():
    text = 'f(); asm volatile("ld %0, [%2];\\n" "ld %1, [%3];\\n" : "=r"(a[0]), "=r"(b) : "r"(x), "r"(y + g(1)) : "memory"); h();'
    (statement,) = _statements(text)
    assert statement == ("ld %0, [%2];\nld %1, [%3];\n", ["=r", "=r"], 2)
    assert _late_reads(*statement) == [0]
    assert _late_reads(statement[0], ["=&r", "=&r"], 2) == []
    assert _statements('asm volatile("st [%0], %1;" ::"r"(p), "r"(v) : "memory");') == [("st [%0], %1;", [], 2)]
