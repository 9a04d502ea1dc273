"""int8_linear where k is split over the chip, in the form that makes its codes, scales and workspace itself: one
allocation, counters cleared in memory that held anything, a workspace a call."""
import pytest
import torch

pytestmark = pytest.mark.gpu
SIZES = [(37, 4104, 5120), (100, 4104, 5120), (20, 64, 16384), (100, 700, 8192), (33, 300, 2576)]


def case(lib, m, n, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(m + n + seed)
    x = torch.randn(m, k + 8, generator=g, device="cuda").to(torch.bfloat16)[:, :k]
    w, sw = lib.int8_quantize(torch.randn(n, k, generator=g, device="cuda").to(torch.bfloat16))
    assert lib.load().gemm_w8a8_workspace_bytes(m, n, k) > 0
    codes, scales = lib.int8_quantize(x)
    whole = torch.empty(0, dtype=torch.uint8, device="cuda")     # k in one part
    return x, w, sw, lib.gemm_w8a8(codes, scales, w, sw, out_dtype=torch.float32, workspace=whole)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_without_buffers(gpu_lib, m, n, k):
    x, w, sw, want = case(gpu_lib, m, n, k)
    for fill in (0xff, 0x01, 0x00):
        # the block that the call's allocation is likely to be given
        torch.full((m * k + 4 * m + 512 + gpu_lib.load().gemm_w8a8_workspace_bytes(m, n, k),), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(gpu_lib.int8_linear(x, w, sw, out_dtype=torch.float32), want)
    assert torch.equal(gpu_lib.int8_linear(x, w, sw), want.to(torch.bfloat16))


def test_two_streams_at_once(gpu_lib):
    cases = [case(gpu_lib, *size) for size in SIZES[:2]]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(10):
        for i, (x, w, sw, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(gpu_lib.int8_linear(x, w, sw, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for (_, _, _, want), all_ in zip(cases, got):
        for y in all_:
            assert torch.equal(y, want)


@pytest.mark.parametrize("m,n,k", SIZES[:3])
def test_two_captured_graphs_that_share_a_workspace(gpu_lib, m, n, k):
    """Replayed in turn, with eager calls on the same workspace between them."""
    ws = gpu_lib.gemm_w8a8_workspace(m, n, k)
    ws.fill_(0xff)
    made = []
    for seed in range(2):
        x, w, sw, _ = case(gpu_lib, m, n, k, seed)
        bufs = dict(codes=torch.empty(m, k, dtype=torch.int8, device="cuda"), scales=torch.empty(m, device="cuda"),
                    out=torch.empty(m, n, device="cuda"), out_dtype=torch.float32, workspace=ws)
        gpu_lib.int8_linear(x, w, sw, **bufs)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.int8_linear(x, w, sw, **bufs)
        made.append((graph, x, w, sw, bufs))
    for i in range(4):
        for graph, x, w, sw, bufs in made:
            x.mul_(-1.5 + 0.25 * i)
            graph.replay()
            got = bufs["out"].clone()
            assert torch.equal(got, gpu_lib.int8_linear(x, w, sw, out_dtype=torch.float32))
            assert torch.equal(got, gpu_lib.int8_linear(x, w, sw, out_dtype=torch.float32, workspace=ws))
