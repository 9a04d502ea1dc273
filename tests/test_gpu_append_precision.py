"""Keys rotated into block-scaled caches are the formula's, rounded once to fp32 and once to a code: rotated in fp64, they
leave the codes of the exact values only where those lie within the angle's own error of a tie.  (With fp32's
cosines, sines and products 2 to 5 codes of each case here would be others.)

The angle: position * step modulo a turn is exact but for its last 32 bits, 2^-32 of a turn or 1.47e-9 in radians; the
series are off by 1.2e-10 and fp64 by less than 1e-14.  So a rotated value is off by less than 1.6e-9 (|a| + |b|) times the
amplitude before it is rounded; both roundings are monotone, so its code lies between those of the two ends."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
T, HEADS, PAGE = 4096, 4, 64


def keys(dim, g, device):
    """Of nearly one size, so that most codes are large and fp32's last digit weighs most."""
    x = 1 + torch.rand(T, HEADS * dim, generator=g, device=device)
    return (x * (2 * torch.randint(0, 2, x.shape, generator=g, device=device) - 1)).to(torch.bfloat16)


def exact(k, positions, dim, layout, scaling, factor):
    """(rotated rows [T, heads, dim] in fp64, bound of the fp64 path's error)."""
    turn, amp = O8.turns(dim, scaling=scaling, factor=factor)
    x = k.float().cpu().numpy().astype(np.float64).reshape(T, HEADS, dim)
    rows, _ = O8.rotate(x, positions, turn, layout, amp)
    ia, ib = (slice(0, dim // 2), slice(dim // 2, dim)) if layout == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    err = np.zeros_like(x)
    err[..., ia] = err[..., ib] = 1.6e-9 * amp * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return rows, err


def outside(codes, bytes_, rows, err, kind, dim):
    """How many of the codes [T, heads, dim] and scale bytes [T / 16, heads] are none of the interval's."""
    f32 = lambda x: x.astype(np.float32).astype(np.float64)  # noqa: E731
    low, high = f32(rows - err), f32(rows + err)
    top = lambda x: np.abs(x).reshape(T // 16, 16, HEADS, dim).max((1, 3))  # noqa: E731
    least = np.maximum(np.minimum(np.abs(low), np.abs(high)) * (np.sign(low) == np.sign(high)), 0)
    byte = np.vectorize(lambda t: O8.scale_byte(t, kind))
    wrong = ((bytes_ < byte(top(least))) | (bytes_ > byte(top(np.maximum(np.abs(low), np.abs(high)))))).sum()
    by = np.exp2(127.0 - bytes_.astype(np.float64)).repeat(16, 0)[..., None]
    return wrong + ((codes < O8.round_codes(low * by, kind)) | (codes > O8.round_codes(high * by, kind))).sum()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,layout,scaling,factor", [(128, "interleaved", "yarn", 8.0), (256, "half", "linear", 4.0)])
def test_rotated_codes(gpu_lib, kind, dim, layout, scaling, factor):
    g = torch.Generator(device="cuda").manual_seed(dim)
    k = keys(dim, g, "cuda")
    positions = np.random.default_rng(dim).integers(0, 10 ** 6, T)
    pages = T // PAGE
    made = [torch.zeros(pages, HEADS, PAGE, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, HEADS, PAGE // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    dtype = FP8 if kind == "e4m3" else torch.int8
    gpu_lib.paged_kv_append(k, k, torch.tensor(positions, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda"),
                            *(c.view(dtype) for c in made), rotation=gpu_lib.rotary_table(dim, layout=layout, scaling=scaling, factor=factor),
                            k_scale=scales[0].view(E8M0), v_scale=scales[1].view(E8M0))
    raw = made[0].permute(0, 2, 1, 3).reshape(T, HEADS, dim).cpu().numpy()
    bytes_ = scales[0].permute(0, 2, 1).reshape(T // 16, HEADS).cpu().numpy()
    rows, err = exact(k, positions, dim, layout, scaling, factor)
    assert outside(O8.code_values(raw, kind), bytes_, rows, err, kind, dim) == 0
