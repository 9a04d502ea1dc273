"""A batch of padding alone (a replica without requests, in step with others): every row is cleared where padding is."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
T, HQ, HKV, PAGE = 5, 4, 2, 16


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_blocks", "int8_blocks"])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("max_new", [0, 1, 100])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_all_rows_are_padding(gpu_lib, kind, dim, max_new, out_dtype):
    dtype = {"bf16": torch.bfloat16, "int8_blocks": torch.int8}.get(kind, FP8)
    k, v = (torch.zeros(2, HKV, PAGE, dim, device="cuda").to(dtype) for _ in range(2))
    scales = [torch.full((2, HKV, 1), 127, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2)]
    q = torch.full((T, HQ * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    rest = (torch.empty(0, 3, **i32), torch.zeros(1, **i32), torch.empty(0, **i32), max_new, 50)

    def call(**kw):
        if kind.endswith("blocks"):
            return gpu_lib.paged_attention_blocks(q, k, v, *scales, *rest, out_dtype=out_dtype, return_lse=True, **kw)
        return gpu_lib.paged_attention(q, k, v, *rest, out_dtype=out_dtype, return_lse=True, **kw)

    out, lse = torch.full((T, HQ * dim + 8), 7.0, dtype=out_dtype, device="cuda"), torch.full((T, HQ), 7.0, device="cuda")
    call(out=out[:, :HQ * dim], lse=lse)
    assert (out == 7).all() and (lse == 7).all()             # left as they are
    call(out=out[:, :HQ * dim], lse=lse, clear_padding=True)
    assert (out[:, :HQ * dim] == 0).all() and (out[:, HQ * dim:] == 7).all() and torch.isneginf(lse).all()
    for _ in range(3):
        torch.full((T, HQ * dim), 7.0, dtype=out_dtype, device="cuda")
        got, lse = call()
        assert (got == 0).all() and torch.isneginf(lse).all()
