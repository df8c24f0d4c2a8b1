"""A frozen weight's payload holds rows of whole 128s; given with its row length, an x of another one is
refused, as with a weight tensor."""
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests.test_int8 import GPU, gpu, layer_on_cpu, values  # noqa: F401


def test_a_payload_given_with_its_row_length_refuses_other_inputs(layer_on_cpu):  # noqa: F811
    payload = torch.zeros(4, 640, dtype=torch.uint8), torch.ones(4)
    x = lambda n: torch.ones(3, n, dtype=torch.bfloat16)  # noqa: E731
    for n in (513, 520, 639, 640):
        assert qcp.int8_linear(x(n), (*payload, n)).shape == (3, 4)
        assert qcp.int8_linear(x(n), [*payload, n]).shape == (3, 4)
        assert qcp.int8_linear(x(n), payload).shape == (3, 4)            # not told: to whole 128s
    for n in (513, 519, 521, 640):
        with pytest.raises(ValueError, match=f"last dimension {n}, weight's 520"):
            qcp.int8_linear(x(n), (*payload, 520))
    for n in (512, 641, 0, -1):
        with pytest.raises(ValueError, match=f"codes: rows of 640 values for {n} columns"):
            qcp.int8_linear(x(520), (*payload, n))
    for odd in (None, "520", 520.0, torch.tensor(520)):
        with pytest.raises(ValueError, match="weight: expected a tensor or a payload"):
            qcp.int8_linear(x(520), (*payload, odd))
    for many in (payload[:1], (*payload, 520, 4), ()):
        with pytest.raises(ValueError, match="weight: expected a tensor or a payload"):
            qcp.int8_linear(x(520), many)


@GPU
def test_a_payload_given_with_its_row_length_is_the_payload(gpu):  # noqa: F811
    w, dy = values(70, 520, "bf16", 1), values(20, 70, "bf16", 2)
    payload = qcp.int8_quantize(w)
    for rows in (3, 20):
        x = values(rows, 520, "bf16", 3).requires_grad_()
        y, z = qcp.int8_linear(x, payload), qcp.int8_linear(x, (*payload, 520))
        assert torch.equal(y, z)
        assert torch.equal(torch.autograd.grad(y, x, dy[:rows])[0], torch.autograd.grad(z, x, dy[:rows])[0])
        with torch.no_grad():
            assert torch.equal(qcp.int8_linear(x, (*payload, 520)), y)
