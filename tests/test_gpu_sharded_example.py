"""The sharded training step with 4-bit weights and 8-bit moments
(examples/sharded_mxfp4.py): it learns, repeats itself bit for bit, and its
weights do not depend on how many ranks share them beyond the gradients' rounding."""
import importlib.util
import os

import pytest
import torch

import quantized_collective_payloads_amd as qcp

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sharded_mxfp4.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    qcp.library()
    spec = importlib.util.spec_from_file_location("sharded_mxfp4", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_it_learns_and_repeats(example):
    first = example.train(4, 60, 0, log=None)
    assert first == example.train(4, 60, 0, log=None)
    start, end = sum(first[:5]) / 5, sum(first[-5:]) / 5
    # the student starts at the teacher's own variance; it has to lose half of it
    assert end < 0.5 * start, (start, end)


def test_gathered_rows_are_the_owners_rows(example):
    total = sum(r * c for r, c in example.SHAPES)
    flat = torch.randn(total, device="cuda")
    for n in (1, 2, 4, 8):
        ranks = [example.Rank(flat, r * (total // n), total // n) for r in range(n)]
        for r in ranks:
            r.copy.copy_(r.master)
        at = 0
        for w, (rows, cols) in zip(example.gather(ranks), example.SHAPES):
            mine = flat[at:at + rows * cols].view(rows, cols).to(torch.bfloat16)
            want = qcp.mxfp4_dequantize(*qcp.mxfp4_quantize(mine), cols, torch.bfloat16)
            assert torch.equal(w, want), n
            at += rows * cols


def test_ranks_that_do_not_divide_the_rows_are_refused(example):
    with pytest.raises(ValueError):
        example.train(5, 1, 0, log=None)
