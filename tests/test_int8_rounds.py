"""The mixed product where its work-groups walk over several tiles, in each type of results, and beside
memory that holds NaN."""
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests.test_int8 import DT, GPU, LARGER, generator, gpu, random_payload  # noqa: F401
from tests import int8_reference as R

# over two rounds of tiles of 128 (1014 on 512 work-groups) and of 256 (399 and 952 on 256), whose waits count the
# stores of the tile before by the type of the results, with more stages than are copied ahead; and
# an `a` that is copied to aligned rows beside slices of K
ROUNDS = [(4896, 3215, 520), (4896, 3215, 320), (5264, 4625, 456), (5264, 4625, 256), (14336, 4100, 456), (2047, 4095, 14335)]


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", LARGER + ROUNDS)
def test_every_type_of_results_is_the_exact_sum_rounded_once(gpu, M, N, K, dt, transpose):  # noqa: F811
    """|a| <= 3, |code| <= 9 and scales of 1/8 to 1: a sum is a multiple of 1/8 of at most 27 K < 2^19, so exact in
    fp32, whatever the order, and one rounding away from 16 bits."""
    g = generator(K + 1)
    a = torch.randint(-3, 4, (K, M) if transpose else (M, K), generator=g, device="cuda").to(DT[dt])
    codes = torch.randint(-9, 10, (K, R.padded(N)), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
    scales = torch.exp2(torch.randint(-3, 1, (K,), generator=g, device="cuda").float())
    x = codes.view(torch.int8)[:, :N].double() * scales.double()[:, None]
    want = ((a.double().t().contiguous() if transpose else a.double()) @ x).float()
    for out in (dt, "f32"):
        for _ in range(2):
            c = qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose, dtype=DT[out])
            assert torch.equal(c, want.to(DT[out])), out


# a whose rows are aligned, with a K that ends inside a stage: tiles of 128 and 256, one round and
# two, two slices; and one that is copied to aligned rows, without slices and with
BESIDE = [(2048, 2048, 1096, 8), (2304, 4096, 1096, 8), (4896, 3215, 328, 8), (5264, 4625, 456, 8), (520, 4099, 8200, 8),
          (1027, 4100, 4099, 7), (2047, 4095, 14335, 7)]


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,K,start", BESIDE)
def test_what_lies_beside_the_operands_is_not_summed(gpu, M, N, K, start, transpose):  # noqa: F811
    """NaN before, behind and between the rows of `a`, and behind the payload's scales; codes behind its rows."""
    shape = (K, M) if transpose else (M, K)
    a = torch.randn(*shape, generator=generator(1), device="cuda").to(torch.bfloat16)
    codes, scales = random_payload(K, N, 4)
    around = torch.full((shape[0] + 2, (shape[1] + 95) // 8 * 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = around[1:-1, start:start + shape[1]]
    view.copy_(a)
    more_codes = torch.full((K + 70, codes.shape[1]), 0x81, dtype=torch.uint8, device="cuda")
    more_scales = torch.full((K + 70,), float("nan"), device="cuda")
    more_codes[:K], more_scales[:K] = codes, scales
    want = qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose)
    assert torch.isfinite(want).all()
    assert torch.equal(qcp.int8_matmul_mixed(view, more_codes[:K], more_scales[:K], N, transpose=transpose), want)
    flat = a.float().t().contiguous() if transpose else a.float()
    x = codes.view(torch.int8)[:, :N].float() * scales[:, None]
    rows = torch.tensor([0, M // 2, M - 1], device="cuda")
    near = flat[rows].double() @ x.to(torch.bfloat16).double()
    size = flat[rows].double().abs() @ x.to(torch.bfloat16).double().abs()
    assert ((want[rows].double() - near).abs() <= K * 2.0 ** -23 * size + 2.0 ** -8 * 1.01 * near.abs()).all()
