"""int8 products whose rows begin anywhere in a 128-byte line: tiles of 128 channels, one to many stages of k with and
without a rest, ends of both matrices inside a tile, and operands that are aligned to 16 bytes alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def operands(m, n, k, at):
    """Codes that begin `at` bytes into an allocation, and scales."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    made = [torch.randint(-128, 128, (r * k + at,), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)[at:].view(r, k) for r in (m, n)]
    return made + [torch.exp(torch.randn(r, generator=g, device="cuda")) * 0.01 for r in (m, n)]


# 64 x 128 tiles (110 of them or more, few enough for one round) and 128 x 128 ones
@pytest.mark.parametrize("m,n", [(130, 5000), (200, 4990), (777, 4104), (900, 3200)])
@pytest.mark.parametrize("k", [144, 272, 400, 528, 560, 656, 784, 1168, 2064, 2176, 4112])
def test_products(gpu_lib, m, n, k):
    a, w, sa, sw = operands(m, n, k, 0)
    # sums below 2^31 are exact in fp64; the result is the documented one, bit by bit
    want = ((a.double() @ w.double().t()).float() * sa[:, None]) * sw
    assert torch.equal(gpu_lib.gemm_w8a8(a, sa, w, sw, out_dtype=torch.float32), want)
    assert torch.equal(gpu_lib.gemm_w8a8(a, sa, w, sw), want.to(torch.bfloat16))


@pytest.mark.parametrize("at", [16, 64, 112])
@pytest.mark.parametrize("m,n,k", [(200, 4990, 1168), (777, 4104, 2064), (777, 4104, 2048), (33, 700, 1168), (5, 300, 656)])
def test_operands_anywhere(gpu_lib, m, n, k, at):
    a, w, sa, sw = operands(m, n, k, at)
    assert a.data_ptr() % 128 == at
    want = ((a.double() @ w.double().t()).float() * sa[:, None]) * sw
    assert torch.equal(gpu_lib.gemm_w8a8(a, sa, w, sw, out_dtype=torch.float32), want)
    whole = [x.clone() for x in (a, w)]                     # one operand aligned, the other not
    assert torch.equal(gpu_lib.gemm_w8a8(whole[0], sa, w, sw, out_dtype=torch.float32), want)
    assert torch.equal(gpu_lib.gemm_w8a8(a, sa, whole[1], sw, out_dtype=torch.float32), want)
