"""int8 calls refuse what they write over anything else of the call: outputs over weights, scales or codes, codes and
scales over the activation or each other, workspaces over any of them.  What lies beside stays allowed."""
import pytest
import torch

from nvfp4_w4a4_gemm_quantize_amd.binding import NVFP4Error

pytestmark = pytest.mark.gpu
M, N, K = 37, 256, 4096        # k is split: with a workspace


def operands(m=M):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    return x, w, torch.rand(N, generator=g, device="cuda")


def floats(t, n, at=0):
    """n floats in a tensor's memory."""
    return t.view(-1).view(torch.uint8)[at:at + 4 * n].view(torch.float32)


def codes_in(t, m=M, at=0):
    return t.view(-1).view(torch.uint8)[at:at + m * K].view(torch.int8).view(m, K)


def refused(call):
    with pytest.raises(NVFP4Error, match="overlap"):
        call()


def bf16_out(t, m, at=0):
    return t.view(-1).view(torch.uint8)[at:at + 2 * m * N].view(torch.bfloat16).view(m, N)


@pytest.mark.parametrize("m", [1, 37, 300])
def test_outputs_over_operands(gpu_lib, m):
    x, w, sw = operands(m)
    keep = w.clone(), sw.clone()
    codes, scales = gpu_lib.int8_quantize(x)
    big_scales = torch.ones(max(N, m * N), device="cuda")
    refused(lambda: gpu_lib.gemm_w8a8(codes, scales, w, sw, out=bf16_out(w, m)))
    refused(lambda: gpu_lib.gemm_w8a8(codes, scales, w, sw, out=bf16_out(w, m, w.numel() - 2 * m * N)))
    refused(lambda: gpu_lib.gemm_w8a8(codes, scales, w, big_scales[:N], out=bf16_out(big_scales, m)))
    refused(lambda: gpu_lib.gemm_w8a8(codes, big_scales[:m], w, sw, out_dtype=torch.float32, out=big_scales[:m * N].view(m, N)))
    refused(lambda: gpu_lib.int8_linear(x, w, sw, out=bf16_out(w, m)))
    refused(lambda: gpu_lib.int8_linear(x, w, big_scales[:N], out=bf16_out(big_scales, m)))
    refused(lambda: gpu_lib.int8_linear(x, w, sw, codes=codes, scales=scales, out=bf16_out(codes, m)))
    refused(lambda: gpu_lib.int8_linear(x, w, sw, codes=codes, scales=big_scales[:m], out_dtype=torch.float32,
                                        out=big_scales[:m * N].view(m, N)))
    assert torch.equal(w, keep[0]) and torch.equal(sw, keep[1]) and (big_scales == 1).all()


@pytest.mark.parametrize("m", [1, 37, 300])
def test_codes_and_scales_over_the_activation_and_each_other(gpu_lib, m):
    x, w, sw = operands(m)
    before, weights = x.clone(), w.clone()
    codes, scales = torch.empty(m, K, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    for call in (lambda **kw: gpu_lib.int8_quantize(x, **kw), lambda **kw: gpu_lib.int8_linear(x, w, sw, **kw)):
        refused(lambda: call(codes=codes_in(x, m)))
        refused(lambda: call(codes=codes_in(x, m, m * K)))
        refused(lambda: call(scales=floats(x, m)))
        refused(lambda: call(codes=codes, scales=floats(codes, m, m * K - 4 * m)))
    if m <= N:
        refused(lambda: gpu_lib.int8_linear(x, w, sw, codes=codes_in(w, m)))
        refused(lambda: gpu_lib.int8_linear(x, w, sw, scales=floats(sw, m)))
    refused(lambda: gpu_lib.int8_linear(x, w, sw, scales=floats(w, m)))
    assert torch.equal(x, before) and torch.equal(w, weights)


def test_workspaces_over_the_rest(gpu_lib):
    x, w, sw = operands()
    codes, scales = gpu_lib.int8_quantize(x)
    need = gpu_lib.load().gemm_w8a8_workspace_bytes(M, N, K)
    assert need > 0
    both = torch.empty(need + M * K + 256, dtype=torch.uint8, device="cuda")
    ws, inside = both[:need], both[need - 256:][:M * K].view(torch.int8).view(M, K)
    inside.copy_(codes)
    refused(lambda: gpu_lib.gemm_w8a8(inside, scales, w, sw, workspace=ws))
    refused(lambda: gpu_lib.int8_linear(x, w, sw, codes=inside, scales=scales, workspace=ws))
    refused(lambda: gpu_lib.gemm_w8a8(codes, scales, w, sw, workspace=ws, out=both[:2 * M * N].view(torch.bfloat16).view(M, N)))
    refused(lambda: gpu_lib.gemm_w8a8(codes, scales, w, floats(both, N), workspace=ws))


@pytest.mark.parametrize("m", [1, 20, 37])
def test_what_lies_beside_is_allowed(gpu_lib, m):
    """All buffers in one allocation, end to end; codes in the gaps between the output's rows; a weight that is its own
    activation; scales that serve both sides."""
    x, w, sw = operands(m)
    want = gpu_lib.int8_linear(x, w, sw)
    wc, ws = gpu_lib.int8_quantize(x)
    need = max(gpu_lib.load().gemm_w8a8_workspace_bytes(m, N, K), 16)
    sizes = [m * K, (4 * m + 15) // 16 * 16, 2 * m * N, need]
    all_ = torch.empty(sum(sizes), dtype=torch.uint8, device="cuda")
    codes, scales, out, space = all_.split(sizes)
    codes, scales = codes.view(torch.int8).view(m, K), scales.view(torch.float32)[:m]
    out = out.view(torch.bfloat16).view(m, N)
    got = gpu_lib.int8_linear(x, w, sw, codes=codes, scales=scales, out=out, workspace=space)
    assert torch.equal(got, want) and torch.equal(codes, wc) and torch.equal(scales, ws)
    if m == 20:     # the scales between two rows of a strided output
        wide = torch.zeros(m, N + 64, dtype=torch.bfloat16, device="cuda")
        gap = wide.view(-1)[N:N + 64].view(torch.float32)[:m]
        gap.copy_(ws)
        assert torch.equal(gpu_lib.gemm_w8a8(wc, gap, w, sw, out=wide[:, :N]), want) and torch.equal(gap, ws)
    one = torch.ones(N, device="cuda")
    square = gpu_lib.gemm_w8a8(w, one, w, one, out_dtype=torch.float32)
    assert torch.equal(square, square.t().contiguous())
