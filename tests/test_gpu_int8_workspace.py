"""One int8 workspace for every step of a serving loop, whatever it holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k", [(5120, 4096), (1069, 15744), (64, 16384)])
def test_one_workspace_serves_any_fewer_tokens(gpu_lib, n, k):
    g = torch.Generator(device="cuda").manual_seed(n)
    w, sw = gpu_lib.int8_quantize(torch.randn(n, k, generator=g, device="cuda").to(torch.bfloat16))
    ws = gpu_lib.gemm_w8a8_workspace(1000, n, k)
    assert ws.numel() > 0
    ws.fill_(0xff)
    for m in (1000, 1, 37, 300, 16, 64, 17, 100, 129, 33, 5):
        x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
        codes, scales = gpu_lib.int8_quantize(x)
        want = gpu_lib.gemm_w8a8(codes, scales, w, sw, out_dtype=torch.float32, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
        assert torch.equal(gpu_lib.gemm_w8a8(codes, scales, w, sw, out_dtype=torch.float32, workspace=ws), want)
        assert torch.equal(gpu_lib.int8_linear(x, w, sw, out_dtype=torch.float32, workspace=ws), want)
