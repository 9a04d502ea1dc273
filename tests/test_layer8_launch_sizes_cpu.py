"""Sizes of the 8-bit attention layer's calls whose threads one launch does not count are refused (host only)."""
import os

import pytest
import torch

from nvfp4_w4a4_gemm_quantize_amd import binding

EUNSUPPORTED, EHIP = -4, -5
A, B = 0x10000, 1 << 50


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("fake device pointers are for GPU-less hosts only")
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libnvfp4.so is not built; run __graft_entry__.build() first")
    return binding.load()


@pytest.mark.parametrize("dim", [128, 256, 1024])
def test_rotary(lib, dim):
    f = lambda T: lib.rotary(A, dim, T, 1, dim, A, A, 16, 0, 1.0, B, dim, None)  # noqa: E731
    most = 2 ** 36 // dim - 1
    assert f(min(most, 2 ** 31 - 1)) == EHIP and f(most + 1) == EUNSUPPORTED


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [0, 4])
def test_append(lib, kind, dim, heads):
    blocks = A if kind >= 2 else None
    f = lambda T: lib.paged_kv_append(A if heads else None, heads * dim, heads, B if heads else None, heads * dim, A, dim, A, dim, A, A,  # noqa: E731
                                      T, A, 16, 0, 1.0, A, A, kind, 1 << 20, 16, 1, dim, 16 * dim, 16 * dim, dim, None, None, blocks, blocks, None)
    most = 2 ** 34 // dim - 1
    assert f(most) == EHIP and f(most + 1) == EUNSUPPORTED
