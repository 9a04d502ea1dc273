"""Validation of attention calls without requests (host only): nothing is looked at unless padding is to be cleared."""
import os

import pytest
import torch

from nvfp4_w4a4_gemm_quantize_amd import binding

OK, EINVAL, ESHAPE, EALIGN, EHIP = 0, -1, -2, -3, -5
A, CLEAR = 0x10000, binding.OUT_CLEAR_PADDING


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("fake device pointers are for GPU-less hosts only")
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libnvfp4.so is not built; run __graft_entry__.build() first")
    return binding.load()


@pytest.mark.parametrize("blocks", [False, True])
def test_without_requests(lib, blocks):
    def f(T=4, out=A, od=1 | CLEAR, ldo=512, lse=None):
        cache = (A, A, 2 if blocks else 1, 4, 16, 2, 128, 4096, 2048, 128) + ((A, A) if blocks else ())
        scales = () if blocks else (None, None)
        fn = lib.paged_attention_blocks if blocks else lib.paged_attention
        return fn(None, 512, T, None, None, 0, 1, 50, 4, *cache, None, 0, 0, 0.1, 0, *scales, out, od, ldo, lse, None, 0, None)
    assert f() == EHIP and f(od=CLEAR) == EHIP and f(lse=A) == EHIP           # valid, but no GPU here
    assert f(od=1) == OK and f(T=0) == OK and f(od=1, out=None) == OK
    assert f(out=None) == EINVAL and f(od=3 | CLEAR) == EINVAL and f(ldo=511) == ESHAPE
    assert f(out=A + 8) == EALIGN and f(ldo=514) == EALIGN and f(lse=A + 2) == EALIGN
