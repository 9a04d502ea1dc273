"""int8 calls of more rows or channels than one launch's 2^32 threads would take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_quantize_more_rows_than_a_launch_takes(gpu_lib):
    rows = 2 ** 26 + 11
    x = torch.ones(rows, 16, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 2 ** 25, 2 ** 26 - 1, 2 ** 26, 2 ** 26 + 3, rows - 1]
    x[at] = (torch.arange(16 * len(at), device="cuda").view(-1, 16) - 50).to(torch.bfloat16)
    codes = torch.full((rows, 16), 7, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), 7.0, device="cuda")
    gpu_lib.int8_quantize(x, codes=codes, scales=scales)
    want, ws = gpu_lib.int8_quantize(x[at].contiguous())
    assert torch.equal(codes[at], want) and torch.equal(scales[at], ws)
    codes[at], scales[at] = 127, scales[2].item()
    assert (codes == 127).all() and (scales == scales[2]).all()


def test_product_of_more_channels_than_a_launch_takes(gpu_lib):
    n = 2 ** 28 + 37
    w = torch.ones(n, 16, dtype=torch.int8, device="cuda")
    at = [0, 15, 16, 2 ** 27, 2 ** 28 - 1, 2 ** 28, n - 1]
    w[at] = torch.arange(len(at) * 16, device="cuda").view(-1, 16).to(torch.int8)
    sw = torch.ones(n, device="cuda")
    x = (torch.arange(48, device="cuda").view(3, 16) - 20).to(torch.bfloat16)
    codes, scales = gpu_lib.int8_quantize(x)
    for got in (gpu_lib.int8_linear(x, w, sw), gpu_lib.gemm_w8a8(codes, scales, w, sw)):
        few = gpu_lib.gemm_w8a8(codes, scales, w[at].contiguous(), sw[:len(at)])
        assert torch.equal(got[:, at], few)
        one = gpu_lib.gemm_w8a8(codes, scales, torch.ones(16, 16, dtype=torch.int8, device="cuda"), sw[:16])[:, :1]
        got[:, at] = one
        assert (got == one).all()
