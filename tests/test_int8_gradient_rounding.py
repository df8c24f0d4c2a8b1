"""What the layer's backward products read: code * scale rounded to the gradient's type, where the forward
product takes code * scale as it is.  So a gradient is that of the forward product up to one rounding of each
value that it sums, also where the type's smallest and largest numbers come into it."""
import numpy as np
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests.test_int8 import DT, GPU, NAME, generator, gpu, wide  # noqa: F401
from tests import int8_reference as R


def check_sums(got, dy, payload, cols, dt):
    """dy times what a payload stands for, and times its own code * scale: K products exact in fp32, as many sums
    each off by 2^-23 of the sum of sizes, one rounding to got's type, and in the second case one rounding
    (half a step of dt, relative or its least) of each of the payload's values before."""
    kind = NAME[got.dtype]
    scaled = payload[0][:, :cols].astype(np.float64) * payload[1].astype(np.float64)[:, None]
    for values, off in ((R.read(payload[0][:, :cols], payload[1], dt), 0), (scaled, R.UNIT[dt] * 1.01 * np.abs(scaled) + R.LEAST[dt])):
        want, size = dy @ values, np.abs(dy) @ (np.abs(values) + off)
        before = np.abs(dy) @ (0 * values + off)
        bound = dy.shape[1] * 2.0 ** -23 * size + before
        bound = bound + R.UNIT[kind] * 1.01 * (np.abs(want) + bound) + R.LEAST[kind]
        assert (np.abs(wide(got) - want) <= bound).all()


@GPU
@pytest.mark.parametrize("kind", ["f32", "same"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gradients_are_those_of_the_forward_product_up_to_one_rounding(gpu, dt, kind):  # noqa: F811
    """Rows of x and of the weight from 2^-16 to 2^4: in fp16 the small codes of the smallest are subnormal."""
    T, I, O = 70, 130, 90
    g = generator(1)
    sizes = lambda n: torch.exp2(torch.randint(-16, 5, (n, 1), generator=g, device="cuda").float())  # noqa: E731
    x = (torch.randn(T, I, generator=g, device="cuda") * sizes(T)).to(DT[dt]).requires_grad_()
    w = (torch.randn(O, I, generator=g, device="cuda") * sizes(O)).to(torch.float32 if kind == "f32" else DT[dt]).requires_grad_()
    dy = torch.randn(T, O, generator=g, device="cuda").to(DT[dt])
    y = qcp.int8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    qx, qw = R.payload(wide(x)), R.payload(wide(w))
    assert (np.abs(wide(y) - R.product(qx, qw)) <= R.product_bound(R.product(qx, qw), dt)).all()
    check_sums(dx, wide(dy), qw, I, dt)
    check_sums(dw, wide(dy).T, qx, I, dt)


@GPU
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_weights_beyond_fp16_under_fp16_inputs(gpu, kind):  # noqa: F811
    """A weight above 65504 is an infinity in fp16, and so it is in x's gradient (0 * infinity, too, as in any product
    of fp16 matrices); y, which takes it as it is, stays finite, and so do the other columns and dw."""
    T, I, O = 20, 64, 40
    g = generator(2)
    x = (torch.randn(T, I, generator=g, device="cuda") * 1e-3).to(torch.float16).requires_grad_()
    w = torch.randn(O, I, generator=g, device="cuda")
    w[7, 5] = -2e5
    w = w.to(DT[kind]).requires_grad_()
    dy = torch.randn(T, O, generator=g, device="cuda").to(torch.float16)
    dy[3, 7] = 0
    y = qcp.int8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    qx, qw = R.payload(wide(x)), R.payload(wide(w))
    assert (np.abs(wide(y) - R.product(qx, qw)) <= R.product_bound(R.product(qx, qw), "f16")).all()
    others = torch.arange(I, device="cuda") != 5
    assert torch.isfinite(dx[:, others]).all() and torch.isfinite(dw).all()
    want = -torch.sign(dy[:, 7].float()) * float("inf")                  # NaN for 0
    assert torch.equal(torch.nan_to_num(dx[:, 5].float(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    z = x.detach().to(torch.bfloat16).requires_grad_()
    assert torch.isfinite(torch.autograd.grad(qcp.int8_linear(z, w), z, dy.to(torch.bfloat16))[0]).all()
