"""A memory instruction in inline assembly that reads scalar registers comes after the five
wait states that it needs behind a vector instruction which wrote one of them (CPU only: the
sources are read).  The compiler counts no wait states into an asm statement."""
import os
import re

import pytest

from tests.test_inline_asm import CSRC, SOURCES, statements

MEMORY = r"\b(?:buffer|global|flat|scratch|tbuffer)_\w+"


def wait_states(template, rest):
    """What the statement waits before each of its memory instructions that read scalar operands."""
    if not re.search(r'"s"\s*\(', rest):
        return []
    code = template.replace('"', "").replace("\\n", "\n").replace("\\t", " ")
    got, waited = [], 0
    for line in (part.strip() for part in re.split(r"[\n;]", code)):
        nop = re.match(r"s_nop\s+(\d+)", line)
        if re.match(MEMORY, line):
            got.append(waited)
        waited += int(nop.group(1)) + 1 if nop else 1 if line else 0
    return got


@pytest.mark.parametrize("name", SOURCES)
def test_scalar_operands_are_waited_for(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        for template, rest in statements(f.read()):
            assert all(n >= 5 for n in wait_states(template, rest)), (template, rest)


def test_the_scan_sees_them():
    seen = [wait_states(*s) for s in statements(
        'asm volatile("s_nop 0\\n\\tbuffer_load_dword %0, %1, 0 offen lds" :: "v"(a), "s"(b)); '
        'asm volatile("s_nop 4\\n\\tbuffer_load_dwordx4 %0, %1, %2 offen lds" :: "v"(a), "s"(b), "s"(c)); '
        'asm volatile("global_load_dword %0, %1, off" : "=v"(x) : "v"(a)); asm volatile("s_waitcnt vmcnt(0)");')]
    assert seen == [[1], [5], [], []]
