"""A copy to LDS whose addresses may pass the end of its buffer leaves it to the range check to read
zeros there, and passes no scalar offset: whether that check counts one is not for the code to rely
on.  Other copies may pass one; their addresses end within the buffer by themselves (CPU only: the
sources are read)."""
import os
import re

import pytest

from tests.test_inline_asm import CSRC, SOURCES

# copies of whole rows, whose offsets end within a row; every other kernel's copies may pass the end
WITHIN = {"qcp_int8_matmul.hip", "qcp_mxfp4_matmul.hip"}


def scalar_offsets(text):
    """The last argument of each call of copy_to_lds."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\bcopy_to_lds\s*\((?!\s*uint32_t\b)", text):
        depth, i, last = 1, m.end(), m.end()
        while depth:
            depth += (text[i] in "([{") - (text[i] in ")]}")
            if depth == 1 and text[i] == ",":
                last = i + 1
            i += 1
        yield text[last:i - 1].strip()


@pytest.mark.parametrize("name", [f for f in SOURCES if f not in WITHIN])
def test_copies_that_may_pass_the_end_pass_no_scalar_offset(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        assert set(scalar_offsets(f.read())) <= {"0"}


def test_the_scan_sees_them():
    got = scalar_offsets("void copy_to_lds(uint32_t lds, uint32_t soff) {} // copy_to_lds(a, b, c, d)\n"
                         "copy_to_lds(to + f(i, j), at, buffer_of(p, (uint64_t)(m - 1) * 2), (uint32_t)k * 2); copy_to_lds(a, b, c, 0);")
    assert list(got) == ["(uint32_t)k * 2", "0"]
