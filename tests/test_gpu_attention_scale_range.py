"""paged_attention_blocks over scale bytes near both ends of their range, keys and values apart: the bounds of
paged_attention, and what falls below the smallest normal bf16 number on its way into the matrix unit beside them.

The bound of the latter: INT8's weight times scale, or an element times its scale, below 2^-126 counts as rounded there
or as 0, which moves a product by less than 2^-126 x 127 (an element below it: by less than 2^-126 times a weight of up
to 2^8), so a row's sum over n keys by n 2^-118 at most; its weights sum to 1 or more."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8
from oracle import paged as OP
from tests.test_gpu_attention_blocks import E8M0, build, call, f64

pytestmark = pytest.mark.gpu


def shifted(kind, new, dim, by_k, by_v, seed):
    """A batch whose keys are 2^by_k as large, its queries as much smaller, and its values 2^by_v as large."""
    b = build([100, 33], [new, min(new, 5)], 4, 2, dim, 32, kind, seed=seed, poison=False)
    for name, by in (("k", by_k), ("v", by_v)):
        bytes_ = np.clip(b[name + "_scale"].view(torch.uint8).cpu().numpy().astype(int) + by, 1, O8.MOST_BYTE[kind]).astype(np.uint8)
        raw = b[name].view(torch.uint8).cpu().numpy()
        b[name + "_scale"] = torch.from_numpy(bytes_).to("cuda").view(E8M0)
        b[name + "_values"] = O8.block_values(O8.code_values(raw, kind), bytes_)
    b["q"] = (b["q"].float() * 2.0 ** -by_k).to(torch.bfloat16)
    return b


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 5, 70])           # the streaming kernel and the tiled one
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("by_k,by_v", [(0, -85), (0, -100), (0, -125), (0, 100), (100, 0), (-100, 0), (100, -85), (-100, 100)])
def test_both_ends(gpu_lib, kind, new, dim, by_k, by_v):
    b = shifted(kind, new, dim, by_k, by_v, seed=dim + new)
    out, lse = call(gpu_lib, b, out_dtype=torch.float32)
    want, wlse, tol, ltol = OP.attention(f64(b["q"]), b["k_values"], b["v_values"], b["table"], b["q_start"], b["lens"], b["page"],
                                         b["hq"], dim ** -0.5)
    tol = tol + max(b["lens"]) * 2.0 ** -118
    got = f64(out).reshape(want.shape)
    assert np.isfinite(got).all() and (np.abs(f64(lse) - wlse) <= ltol).all()
    assert (np.abs(got - want) <= tol).all(), "worst %.3g of its bound" % (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("byte", [0, 1, 2, 240, 246, 255])
def test_bytes_at_the_ends_stand_for_the_nearest_ones(gpu_lib, kind, new, byte):
    """Bytes outside the range are read as its ends, for keys and values."""
    b = build([40], [new], 4, 2, 64, 16, kind, seed=byte, poison=False)
    high = byte > 127
    b["q"] = (b["q"].float() * 2.0 ** (-100 if high else 100)).to(torch.bfloat16)
    made = []
    for at in (byte, min(max(byte, 1), O8.MOST_BYTE[kind])):
        for name in ("k_scale", "v_scale"):
            b[name].view(torch.uint8).fill_(at)
        made.append(call(gpu_lib, b))
    assert torch.equal(made[0][0].view(torch.int16), made[1][0].view(torch.int16)) and torch.equal(made[0][1].view(torch.int32), made[1][1].view(torch.int32))
