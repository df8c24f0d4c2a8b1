"""Which captured backward passes of the 8-bit integer layer are refused: those that give a gradient to
a leaf whose graph from the default stream lives, whatever lies between the two, and no others."""
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from quantized_collective_payloads_amd import int8
from tests.test_int8 import GPU, gpu, layer_on_cpu, values  # noqa: F401

REFUSED = "default stream, lives"


@pytest.fixture()
def stream(monkeypatch, layer_on_cpu):  # noqa: F811
    """The current stream's number, 9 in a capture."""
    now = {"is": 0}
    monkeypatch.setattr(int8, "_raw_stream", lambda index: now["is"])
    monkeypatch.setattr(int8, "_captured", lambda index: now["is"] == 9)
    return now


def leaf(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype, requires_grad=True)


def test_a_leaf_without_a_gradient_in_the_pass_does_not_count(stream):
    x, v, w = leaf(6, 32), leaf(6, 32), leaf(4, 32)
    alive = qcp.int8_linear(v, w)
    stream["is"] = 9
    layer = lambda: qcp.int8_linear(x, w)  # noqa: E731
    assert torch.autograd.grad(layer().sum(), x)[0].shape == x.shape
    layer().sum().backward(inputs=[x])
    assert x.grad is not None and w.grad is None
    for asks in (lambda y: torch.autograd.grad(y, (x, w)), lambda y: torch.autograd.grad(y, w), lambda y: y.backward(),
                 lambda y: y.backward(inputs=[w])):
        with pytest.raises(RuntimeError, match=REFUSED):
            asks(layer().sum())
    cast = w.float().to(torch.bfloat16)            # the same behind two casts
    assert torch.autograd.grad(qcp.int8_linear(x, cast).sum(), x)[0].shape == x.shape
    with pytest.raises(RuntimeError, match=REFUSED):
        torch.autograd.grad(qcp.int8_linear(x, cast).sum(), (x, w))
    del alive, cast                                # (a cast holds the node, too)
    torch.autograd.grad(layer().sum(), (x, w))


BETWEEN = {"own view and copy, and a cast": lambda t: t.to(torch.bfloat16).transpose(0, 1),
           "three": lambda t: (t * 2).float().to(torch.bfloat16),
           "seven": lambda t: ((((t + 1).float() * 2).exp() - 1).to(torch.float16)).to(torch.bfloat16),
           "a frozen layer": lambda t: qcp.int8_linear(t.to(torch.bfloat16), (torch.zeros(32, 128, dtype=torch.uint8), torch.ones(32)))}


@pytest.mark.parametrize("way", BETWEEN)
@pytest.mark.parametrize("of", ["x", "weight"])
def test_a_leaf_behind_other_operators_counts(stream, way, of):
    def layer(t):
        t = BETWEEN[way](t)
        return qcp.int8_linear(t, w) if of == "x" else qcp.int8_linear(x, t.flatten(0, -2))
    t, x, w = leaf(2, 3, 32, dtype=torch.float32), torch.ones(6, 32, dtype=torch.bfloat16), torch.ones(4, 32, dtype=torch.bfloat16)
    alive = layer(t)
    stream["is"] = 9
    y = layer(t)
    with pytest.raises(RuntimeError, match=REFUSED):
        y.sum().backward()
    del alive, y
    layer(t).sum().backward()


def test_all_that_lies_before_the_layer_in_the_captured_pass_is_looked_at(stream):
    """A noted leaf that the captured graph reaches by another way than the noted one."""
    t, u, w = leaf(6, 32), leaf(6, 32), torch.ones(32, 32, dtype=torch.bfloat16)
    alive = qcp.int8_linear(t, w)
    stream["is"] = 9
    y = qcp.int8_linear(qcp.int8_linear((u * t.cos() + 1) @ w, w).relu() + u, w)
    with pytest.raises(RuntimeError, match=REFUSED):
        torch.autograd.grad(y.sum(), (u, t))
    y = qcp.int8_linear(qcp.int8_linear((u * t.cos() + 1) @ w, w).relu() + u, w)
    torch.autograd.grad(y.sum(), u)
    del alive


@GPU
def test_captured_gradient_of_x_beside_a_living_graph_of_the_weight(gpu):  # noqa: F811
    """The weight's gradient is not asked for, so its node takes no part: captured, and replayed as
    the eager pass."""
    x, w = values(90, 300, "bf16", 1).requires_grad_(), values(140, 300, "bf16", 2).requires_grad_()
    dy = values(90, 140, "bf16", 3)
    want = torch.autograd.grad(qcp.int8_linear(x, w), x, dy)[0]
    alive = qcp.int8_linear(x.detach(), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(qcp.int8_linear(x, w), x, dy)[0]
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert alive.grad_fn is not None
