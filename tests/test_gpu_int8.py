"""GPU parity of the int8 linear layers against the oracle: codes, scales and outputs
equal bit by bit (the sum is exact, every other step one fp32 operation)."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8

pytestmark = pytest.mark.gpu


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def check_quantize(lib, x):
    codes, scales = lib.int8_quantize(x)
    want, ws = O8.int8_quantize(host(x))
    assert np.array_equal(host(codes), want) and np.array_equal(host(scales), ws, equal_nan=True)
    return codes, scales


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (5, 2048), (7, 5120), (2, 16384), (3, 16400), (2, 131056), (1024, 64), (1030, 4096),
                                       (1025, 4112), (300, 1040)])
@pytest.mark.parametrize("pad", [0, 24])
def test_quantize(gpu_lib, rows, cols, pad):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x[:, ::97] *= 30
    check_quantize(gpu_lib, x.to(torch.bfloat16)[:, :cols])


def test_quantize_edges(gpu_lib):
    """Rows of zeros, of one value, of subnormals, of the largest numbers, with infinities and NaN; exact halves."""
    x = torch.zeros(12, 64, device="cuda")
    x[1] = 3.0
    x[2, 5] = -2.0 ** -133
    x[3] = 2.0 ** -121
    x[4] = 2.0 ** -120
    x[4, 3] = -2.0 ** -126
    x[5, ::2], x[5, 1::2] = 3.38e38, -3.38e38
    x[6, 7] = float("inf")
    x[7, 9] = float("nan")
    x[8] = torch.arange(64, device="cuda") - 63.5
    x[8, 0] = 127.0
    x[9, :] = torch.arange(64, device="cuda") * 0.5
    x[9, 0] = -127.0
    x[10] = -0.0
    x[11, 0], x[11, 1] = float("-inf"), float("nan")
    codes, scales = check_quantize(gpu_lib, x.to(torch.bfloat16))
    assert scales[2] == 0 and scales[4] > 0 and torch.isnan(scales[[6, 7, 11]]).all() and (codes[[6, 7, 11]] == 0).all()


def product(lib, m, n, k, out_dtype=torch.bfloat16, ld=None, seed=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sa, sw = (torch.exp(torch.randn(x, generator=g, device="cuda")) * 0.01 for x in (m, n))
    out = None
    if ld is not None:
        wide = torch.full((m * ld + offset + 8,), 7.0, dtype=out_dtype, device="cuda")
        out = wide[offset:].as_strided((m, n), (ld, 1))
    ws = torch.randint(0, 256, (max(lib.load().gemm_w8a8_workspace_bytes(m, n, k), 1),), device="cuda", dtype=torch.int32).to(torch.uint8)
    got = lib.gemm_w8a8(a, sa, w, sw, out_dtype=out_dtype, out=out, workspace=ws)
    # exact sums: fp64 holds them, and the GPU's fp64 product is checked against integers below
    s = (a.double() @ w.double().t()).float()
    want = ((s * sa[:, None]) * sw).to(out_dtype)
    assert torch.equal(got, want), "%d of %d" % ((got != want).sum(), got.numel())
    got = got.cpu()
    if ld is not None:
        wide[offset:].as_strided((m, n), (ld, 1)).fill_(7.0)
        assert (wide == 7).all()
    if m * n * k <= 1 << 22:
        ref = torch.from_numpy(O8.gemm_w8a8(host(a), host(sa), host(w), host(sw)))
        assert torch.equal(got, ref.to(out_dtype))


SIZES_M = [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 257, 300]


@pytest.mark.parametrize("m", SIZES_M)
@pytest.mark.parametrize("n", [1, 17, 64, 130, 513])
@pytest.mark.parametrize("k", [16, 64, 80, 208, 1040])
def test_products(gpu_lib, m, n, k):
    product(gpu_lib, m, n, k, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 64), (4100, 4111, 144), (2000, 8200, 320), (1, 17408, 5120), (37, 5120, 17408), (64, 1024, 16384),
                                   (200, 1024, 8192), (129, 20000, 512), (1, 40, 131056), (70, 40, 131056), (5000, 300, 256), (1024, 1024, 4096)])
def test_large_products(gpu_lib, m, n, k):
    product(gpu_lib, m, n, k, seed=k)


@pytest.mark.parametrize("m", [3, 40, 200, 4097])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,ld,offset", [(264, 264, 0), (264, 272, 0), (264, 267, 0), (264, 264, 1), (260, 260, 4), (261, 261, 0)])
def test_out_strides_and_alignments(gpu_lib, m, out_dtype, n, ld, offset):
    product(gpu_lib, m, n if m < 4000 else n + 4000, 96, out_dtype, ld if m < 4000 else ld + 4000, offset=offset)


@pytest.mark.parametrize("m", [1, 64, 65, 300])
def test_largest_sums(gpu_lib, m):
    """Every product 2^14, at the largest k: the sum is 2^31 less 2^18."""
    k = 131056
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((20, k), -128, dtype=torch.int8, device="cuda")
    w[3] = 127
    one = torch.ones(max(m, 20), device="cuda")
    got = gpu_lib.gemm_w8a8(a, one[:m], w, one[:20], out_dtype=torch.float32)
    want = torch.full((m, 20), float(k * 16384), device="cuda")
    want[:, 3] = float(-k * 128 * 127)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 2, 5, 8, 9, 37, 100, 700])
@pytest.mark.parametrize("n,k", [(300, 512), (1000, 2064), (4104, 5120)])
def test_linear_is_quantise_and_product(gpu_lib, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k + 8, generator=g, device="cuda").to(torch.bfloat16)[:, :k]
    w, sw = gpu_lib.int8_quantize(torch.randn(n, k, generator=g, device="cuda").to(torch.bfloat16))
    codes, scales = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    got = gpu_lib.int8_linear(x, w, sw, codes=codes, scales=scales, out_dtype=torch.float32)
    c, s = check_quantize(gpu_lib, x)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    assert torch.equal(got, gpu_lib.gemm_w8a8(c, s, w, sw, out_dtype=torch.float32))
    # a row's result is its own, whatever stands beside it
    assert torch.equal(gpu_lib.int8_linear(x[:1], w, sw, out_dtype=torch.float32), got[:1])
    # quantisation's share of the error: half a step of each factor
    want = x.double() @ (w.double() * sw[:, None].double()).t().contiguous()
    bound = 0.5 * s.double()[:, None] * (w.double().abs().sum(1) * sw.double())[None] * (1 + 1e-5)
    assert ((got.double() - want).abs() <= bound + 1e-30).all()


def test_rows_that_are_not_finite_stay_alone(gpu_lib):
    for m in (3, 70):
        x = torch.randn(m, 256, device="cuda").to(torch.bfloat16)
        w, sw = gpu_lib.int8_quantize(torch.randn(50, 256, device="cuda").to(torch.bfloat16))
        clean = gpu_lib.int8_linear(x, w, sw)
        x[1, 7], x[2] = float("nan"), 0.0
        got = gpu_lib.int8_linear(x, w, sw)
        assert torch.isnan(got[1]).all() and (got[2] == 0).all() and torch.equal(got[0], clean[0]) and torch.equal(got[3:], clean[3:])


@pytest.mark.parametrize("m", [1, 20, 200])
def test_captured_and_replayed(gpu_lib, m):
    x = torch.randn(m, 512, device="cuda").to(torch.bfloat16)
    w, sw = gpu_lib.int8_quantize(torch.randn(700, 512, device="cuda").to(torch.bfloat16))
    bufs = dict(codes=torch.empty(m, 512, dtype=torch.int8, device="cuda"), scales=torch.empty(m, device="cuda"),
                out=torch.empty(m, 700, dtype=torch.bfloat16, device="cuda"))
    gpu_lib.int8_linear(x, w, sw, **bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.int8_linear(x, w, sw, **bufs)
    for _ in range(4):
        x.copy_(torch.randn(m, 512, device="cuda"))
        graph.replay()
        got = bufs["out"].clone()
        assert torch.equal(got, gpu_lib.int8_linear(x, w, sw))


def test_empty(gpu_lib):
    w, sw = gpu_lib.int8_quantize(torch.randn(50, 256, device="cuda").to(torch.bfloat16))
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.int8_linear(x, w, sw).shape == (0, 50)
    assert gpu_lib.int8_quantize(x)[0].shape == (0, 256)


def test_refusals(gpu_lib):
    E = gpu_lib.NVFP4Error
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros(8, 256, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    a = torch.zeros(4, 256, dtype=torch.int8, device="cuda")
    for call in (lambda: gpu_lib.int8_quantize(x[:, :250]), lambda: gpu_lib.int8_quantize(x.float()), lambda: gpu_lib.int8_quantize(x.t()),
                 lambda: gpu_lib.int8_quantize(torch.zeros(1, 131072, dtype=torch.bfloat16, device="cuda")),
                 lambda: gpu_lib.int8_linear(x, w[:, :128], s), lambda: gpu_lib.int8_linear(x, w.view(torch.uint8), s),
                 lambda: gpu_lib.int8_linear(x, w, s[:7]), lambda: gpu_lib.int8_linear(x, w, s.double()),
                 lambda: gpu_lib.int8_linear(x, w, s, out=torch.empty(4, 9, device="cuda", dtype=torch.bfloat16)),
                 lambda: gpu_lib.int8_linear(x, w, s, codes=a[:3]), lambda: gpu_lib.gemm_w8a8(a, s[:4], w.t(), s),
                 lambda: gpu_lib.gemm_w8a8(a, s[:3], w, s), lambda: gpu_lib.gemm_w8a8(a[:, :240], s[:4], w[:, :240], s),
                 lambda: gpu_lib.gemm_w8a8(a, s[:4], w, s, out=torch.empty(4, 8, device="cuda")),
                 lambda: gpu_lib.int8_linear(x.cpu(), w, s)):
        with pytest.raises(E):
            call()


@pytest.mark.parametrize("m,n,k", [(37, 5120, 4096), (100, 700, 8192), (20, 64, 4112)])
def test_split_sums(gpu_lib, m, n, k):
    """With and without parts of k, from any workspace: the same bits; one workspace serves a graph and the calls between."""
    g = torch.Generator(device="cuda").manual_seed(m)
    a = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sa, sw = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
    need = gpu_lib.load().gemm_w8a8_workspace_bytes(m, n, k)
    assert need > 0
    none = torch.empty(m, n, device="cuda")
    rc = gpu_lib.load().gemm_w8a8(a.data_ptr(), sa.data_ptr(), m, w.data_ptr(), sw.data_ptr(), n, k, none.data_ptr(), 0, n, None, 0,
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, device="cuda")
    f = lambda o: gpu_lib.gemm_w8a8(a, sa, w, sw, out_dtype=torch.float32, out=o, workspace=ws)  # noqa: E731
    assert torch.equal(f(out), none) and torch.equal(f(torch.empty_like(out)), none)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(out)
    for i in range(4):
        sa.mul_(-0.5)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, f(torch.empty_like(out)))
