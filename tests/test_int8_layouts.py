"""The mixed product and the layer's backward pass on gradients whose rows lie very far apart, or are very
long: the kernels take rows up to 2^23 elements apart, the binding any."""
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from quantized_collective_payloads_amd import int8
from tests.test_int8 import GPU, check_mixed, generator, gpu, random_payload  # noqa: F401

FAR = (1 << 23) + 8


def layouts(device):
    """2-D views of one or two dimensions' worth of elements, by what is far apart or long in them."""
    big = torch.randint(-3, 4, (2, FAR), generator=torch.Generator(device).manual_seed(1), device=device, dtype=torch.int8)
    big = big.to(torch.bfloat16)
    return {"rows apart": big[:, :40], "columns apart": big[:, 3:43].t(), "long rows": big, "long columns": big.t(),
            "one long row": big[1:], "one long column": big[1:].t(), "long rows, every other": big[:, ::2][:, :41],
            "longest": big[:, 8:], "long rows within longer": big[:, :FAR - 3]}


NAMES = ["rows apart", "columns apart", "long rows", "long columns", "one long row", "one long column", "long rows, every other",
         "longest", "long rows within longer"]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_what_the_kernel_is_given_is_a_within_its_limits(monkeypatch, name, transpose):
    a = layouts("cpu")[name]
    M, K = (a.shape[1], a.shape[0]) if transpose else tuple(a.shape)
    asked = {}

    def scratch(_, like, m, n, k, flag, aligned):
        asked.update(sizes=(m, n, k), transpose=flag, aligned=aligned)
        return None, None, 0

    def launch(_, index, first, kind, lda, flag, codes, scales, m, n, k, c, *rest):
        rows, cols = (k, m) if flag else (m, k)
        assert flag == asked["transpose"] and (m, n, k) == asked["sizes"] == (M, 5, K)
        assert cols <= lda <= 1 << 23, lda
        # what lies there, read as the kernel does
        import ctypes
        size = (rows - 1) * lda + cols
        got = torch.frombuffer((ctypes.c_int16 * size).from_address(first), dtype=torch.bfloat16)
        got = torch.as_strided(got, (rows, cols), (lda, 1))
        assert torch.equal(got, a if flag == transpose else a.t())
        asked["launched"] = True
    monkeypatch.setattr(int8, "_scratch", scratch)
    monkeypatch.setattr(int8, "_enqueue", launch)
    int8._mixed(-1, a, 0, 0, M, 5, K, transpose, torch.empty(1, 5, dtype=torch.bfloat16))
    assert asked["launched"]


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_mixed_product_of_far_and_long_rows(gpu, name, transpose):  # noqa: F811
    """Small integers: of a long K one row in 101 counts, so no sum passes 3 * 2 * (2^23 + 8) / 101 < 2^19, and
    all are exact in fp32, whatever the order."""
    a = layouts("cuda")[name]
    M, K = (a.shape[1], a.shape[0]) if transpose else tuple(a.shape)
    codes = torch.zeros(K, 128, dtype=torch.int8, device="cuda")
    codes[::101 if K > 1000 else 1, :20] = torch.randint(-2, 3, (codes[::101 if K > 1000 else 1].shape[0], 20), generator=generator(2),
                                                         device="cuda").to(torch.int8)
    scales = torch.ones(K, device="cuda")
    c = qcp.int8_matmul_mixed(a, codes.view(torch.uint8), scales, 20, transpose=transpose, dtype=torch.float32)
    want = (a.double().t() if transpose else a.double()) @ codes[:, :20].double()
    assert torch.equal(c.double(), want)


@GPU
def test_backward_through_outputs_that_were_stacked(gpu):  # noqa: F811
    """A vocabulary's logits of 66 steps, stacked: each step's gradient is a view whose rows are
    66 * 128256 elements apart."""
    steps, O, I = 66, 128256, 64
    g = generator(3)
    x = torch.randn(steps, 2, I, generator=g, device="cuda").to(torch.bfloat16).requires_grad_()
    w = (torch.randn(O, I, generator=g, device="cuda") * 0.05).to(torch.bfloat16).requires_grad_()
    y = [qcp.int8_linear(x[t], w) for t in range(steps)]
    dy = torch.randn(2, steps, O, generator=g, device="cuda").to(torch.bfloat16)
    dx, dw = torch.autograd.grad(torch.stack(y, 1), (x, w), dy)
    payload = qcp.int8_quantize(w.detach())
    for t in (0, 7, steps - 1):
        assert torch.equal(dx[t], qcp.int8_matmul_mixed(dy[:, t].contiguous(), *payload, I))
    one = torch.autograd.grad(qcp.int8_linear(x[5], w), w, dy[:, 5])[0]
    assert torch.equal(one, qcp.int8_matmul_mixed(dy[:, 5].contiguous(), *qcp.int8_quantize(x[5].detach()), I, transpose=True))
    assert torch.isfinite(dw).all()


def test_scratch_memory_is_told_for_every_size_that_the_product_takes():
    """Its own bound on the tiles of C was the smaller one where N is a multiple of 256."""
    work = qcp.library().qcp_int8_mixed_work
    most = (2 ** 24 - 1) // 2                      # tiles of 256
    for N, rows in ((256, most), (255, most), (1, most), (512, most // 2), (1024, most // 4), (1 << 24, most // 65536)):
        assert work(256 * rows, N, 64, 0, 1) >= 0, N
        assert work(256 * rows + 1, N, 64, 0, 1) == -1, N
    assert work(0, 0, 64, 0, 1) == work(1 << 31, 0, 64, 1, 0) == 0
