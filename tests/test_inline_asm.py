"""Inline assembly names every register it uses to the compiler: as an operand, or among
the clobbered ones (CPU only: the sources are read)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_collective_payloads_amd", "csrc")
REGISTER = r"(?<![\w%.])(?:m0|vcc(?:_lo|_hi)?|exec(?:_lo|_hi)?|scc|flat_scratch|[sva]\d+|[sva]\[\d+:\d+\])(?!\w)"
# instructions that write scc or vcc without saying so in their operands
IMPLICIT = r"\b(s_(?:add|sub|addc|subb|and|or|xor|andn2|orn2|nand|nor|xnor|lshl|lshr|ashr|not|min|max|abs|bfe|cmp|cmpk|bitcmp)\w*|v_div_fmas\w*)"


def statements(text):
    """(template, the rest) of each asm statement."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\s+volatile\s*\(|\basm\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if quoted and c == "\\":
                i += 1
            elif c == '"':
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        body = text[m.end():i - 1]
        template = re.match(r'(?:\s*"(?:[^"\\]|\\.)*")+', body).group(0)
        yield template, body[len(template):]


def unnamed(template, rest):
    code = template.replace("\\n", "\n").replace("\\t", " ")
    return [r for r in re.findall(REGISTER, code) if f'"{r}"' not in rest] + re.findall(IMPLICIT, code)


SOURCES = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".hip", ".h"))]


@pytest.mark.parametrize("name", SOURCES)
def test_no_register_is_used_behind_the_compilers_back(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        for template, rest in statements(f.read()):
            assert not unnamed(template, rest), (template, rest)


def test_the_scan_sees_them():
    seen = list(statements('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" :: "s"(f(x)) : "memory"); // asm("v0")\n'
                           'asm("v_mov_b32 v7, %0" :: "v"(x) : "v7"); asm volatile("" : "+v"(y));'))
    assert [unnamed(*s) for s in seen] == [["m0"], [], []]
