"""gemm_w8a8's workspace: a size for the most tokens serves every smaller call (host only)."""
import os

import pytest
import torch

from nvfp4_w4a4_gemm_quantize_amd import binding

OK, EINVAL, ESHAPE, EUNSUPPORTED, EHIP, ESIZE = 0, -1, -2, -4, -5, -6
A16 = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libnvfp4.so is not built; run __graft_entry__.build() first")
    return binding.load()


SIZES = [(5120, 17408), (17408, 5120), (4104, 2064), (4104, 5120), (1024, 5120), (512, 4096), (64, 16384), (1, 131056), (130, 8192),
         (1069, 15744), (16384, 2560), (20000, 512), (8192, 4096), (40, 32)]


@pytest.mark.parametrize("n,k", SIZES)
def test_sizes_never_fall_as_tokens_rise(lib, n, k):
    at = list(range(0, 700)) + [b + d for b in range(704, 20000, 448) for d in (-1, 0, 1)] + [65536, 10 ** 6]
    got = [lib.gemm_w8a8_workspace_bytes(m, n, k) for m in at]
    falls = [(m, a, b) for m, a, b in zip(at[1:], got, got[1:]) if b < a]
    assert not falls, falls[:3]
    assert got[0] == 0 and got[-1] < 64 << 20


@pytest.mark.parametrize("n,k", SIZES)
def test_one_size_is_taken_by_every_smaller_call(lib, n, k):
    """Fake addresses: a call that passes the checks fails at its launch, without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("fake device pointers are for GPU-less hosts only")
    size = lib.gemm_w8a8_workspace_bytes(4096, n, k)
    for m in [1, 2, 8, 16, 17, 32, 33, 37, 64, 65, 100, 128, 129, 200, 256, 384, 385, 512, 1000, 2048, 4096]:
        assert lib.gemm_w8a8(A16, A16, m, A16, A16, n, k, A16, 1, n, A16, size, None) == EHIP, m
        assert lib.int8_linear(A16, m, k, k, A16, A16, A16, A16, n, A16, 1, n, A16, size, None) == EHIP, m


def test_sizes_of_no_product(lib):
    for m, n, k in ((-1, 512, 4096), (40, 0, 4096), (40, 512, 4095), (40, 512, 1 << 17), (1 << 31, 512, 4096)):
        assert lib.gemm_w8a8_workspace_bytes(m, n, k) == 0
        with pytest.raises(binding.NVFP4Error):
            binding.gemm_w8a8_workspace(m, n, k, device="cpu")
    ws = binding.gemm_w8a8_workspace(37, 5120, 17408, device="cpu")
    assert ws.dtype == torch.uint8 and ws.numel() == lib.gemm_w8a8_workspace_bytes(37, 5120, 17408) > 0
