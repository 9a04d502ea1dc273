"""GPU parity of rotary against the float64 oracle: every value within the bound of
one fp32 evaluation (oracle.layer8.rotate) and half a step of bf16."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8

pytestmark = pytest.mark.gpu
U_BF16 = 2.0 ** -8


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(lib, T, heads, dim, rot, layout="half", positions=None, pad=0, in_place=False, seed=0, **table):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn(T, heads * dim + pad, generator=g, device="cuda").to(torch.bfloat16)
    x = wide[:, :heads * dim]
    before = wide.clone()
    if positions is None:
        positions = torch.randint(0, 40000, (T,), generator=g, device="cuda", dtype=torch.int32).tolist()
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    r = lib.rotary_table(rot, layout=layout, **table)
    names = {"original_length": "original", "slow_turns": "slow", "fast_turns": "fast"}
    amplitude = table.pop("amplitude", None)
    turn, amp = O8.turns(rot, **{names.get(k, k): v for k, v in table.items()})
    amp = amp if amplitude is None else amplitude
    want, tol = O8.rotate(f64(x).reshape(T, heads, dim), positions, turn, layout, amp)
    if in_place:
        got = lib.rotary(x, pos, r, dim, out=x)
        assert got is x
        assert torch.equal(wide[:, heads * dim:], before[:, heads * dim:])
    else:
        got = lib.rotary(x, pos, r, dim)
        assert torch.equal(wide, before)
    off = np.abs(f64(got).reshape(want.shape) - want)
    tol = tol + U_BF16 * (np.abs(want) + tol)
    # what is not rotated is copied
    tol[..., rot:] = 0.0
    assert (off <= tol).all(), "%d of %d, worst %.3g of its bound" % ((off > tol).sum(), off.size, (off / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(16, 16), (48, 32), (64, 16), (64, 48), (64, 64), (80, 32), (96, 96), (128, 128), (256, 64),
                                     (256, 256), (1024, 1024)])
def test_head_layouts(gpu_lib, layout, dim, rot):
    check(gpu_lib, 5, 3, dim, rot, layout, seed=dim + rot)


@pytest.mark.parametrize("T", [1, 2, 31, 64, 257, 3000])
@pytest.mark.parametrize("heads", [1, 4, 5, 48])
def test_sizes(gpu_lib, T, heads):
    check(gpu_lib, T, heads, 64, 32, pad=8 * (T % 3), seed=T)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_beside_other_columns(gpu_lib, layout):
    check(gpu_lib, 40, 6, 128, 64, layout, pad=256, in_place=True)
    check(gpu_lib, 1, 6, 128, 64, layout, pad=8, in_place=True)


def test_far_positions_are_as_exact_as_near_ones(gpu_lib):
    at = [0, 1, 2, 1000, 131071, 1000003, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1]
    check(gpu_lib, len(at), 2, 128, 128, positions=at)


def test_quarters_of_a_turn(gpu_lib):
    """Angles around every border of the reduction: pair 0 turns by exactly one radian, pair_factors move it."""
    at = list(range(0, 700))
    check(gpu_lib, len(at), 1, 64, 16, positions=at, pair_factors=[2 / np.pi] * 8)   # pair 0: a quarter a position
    check(gpu_lib, len(at), 1, 64, 16, positions=at, pair_factors=[8 / np.pi * 1.0000001] * 8)


@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_negative_positions_are_copied(gpu_lib, in_place):
    check(gpu_lib, 6, 3, 64, 64, positions=[5, -1, 7, -5, -2 ** 31, 0], in_place=in_place, scaling="yarn", factor=4.0)


@pytest.mark.parametrize("table", [
    dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=16.0, original_length=4096),
    dict(scaling="yarn", factor=2.5, slow_turns=2.0, fast_turns=20.0), dict(scaling="wavelength", factor=8.0),
    dict(scaling="wavelength", factor=32.0, original_length=2048, slow_turns=0.5, fast_turns=9.0), dict(base=1e6),
    dict(pair_factors=[1.0 + 0.3 * i for i in range(32)]), dict(amplitude=1.7), dict(amplitude=-0.5),
    dict(scaling="linear", factor=1.0)])
def test_long_context_scalings(gpu_lib, table):
    check(gpu_lib, 9, 2, 64, 64, positions=[0, 1, 77, 4095, 4096, 32768, 100000, 500001, 2000000], **table)


def test_strides_past_32_bits_of_bytes(gpu_lib):
    """The last rows of a matrix that is longer than 2^32 bytes."""
    T, ld = 9, 2 ** 28 + 8
    big = torch.empty((T - 1) * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, 64), (ld, 1))
    x.copy_(torch.randn(T, 64, device="cuda"))
    r = gpu_lib.rotary_table(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = gpu_lib.rotary(x.contiguous(), pos, r, 64)
    assert torch.equal(gpu_lib.rotary(x, pos, r, 64), want)
    assert torch.equal(gpu_lib.rotary(x, pos, r, 64, out=x), want)


def test_empty(gpu_lib):
    r = gpu_lib.rotary_table(64)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.rotary(x, torch.empty(0, dtype=torch.int32, device="cuda"), r, 64).shape == (0, 128)


def test_captured_and_replayed_with_new_positions(gpu_lib):
    r = gpu_lib.rotary_table(64, layout="interleaved")
    x = torch.randn(7, 256, device="cuda").to(torch.bfloat16)
    pos = torch.arange(7, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    gpu_lib.rotary(x, pos, r, 64, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.rotary(x, pos, r, 64, out=out)
    for i in range(4):
        pos.add_(1000 * i + 1)
        x.mul_(-1.5)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, gpu_lib.rotary(x, pos, r, 64))


def test_refusals(gpu_lib):
    r = gpu_lib.rotary_table(64)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = gpu_lib.NVFP4Error
    for call in (lambda: gpu_lib.rotary(x.float(), pos, r, 64), lambda: gpu_lib.rotary(x, pos.long(), r, 64),
                 lambda: gpu_lib.rotary(x, pos[:3], r, 64), lambda: gpu_lib.rotary(x, pos, r, 60),
                 lambda: gpu_lib.rotary(x, pos, r, 0), lambda: gpu_lib.rotary(x, pos, r, 32),
                 lambda: gpu_lib.rotary(x, pos, None, 64), lambda: gpu_lib.rotary(x[:, 4:132], pos, r, 64),
                 lambda: gpu_lib.rotary(x, pos, r, 64, out=x[:, :128]), lambda: gpu_lib.rotary(x.t(), pos, r, 4),
                 lambda: gpu_lib.rotary(x[:, :128], pos, r, 64, out=x[:, 64:192]),
                 lambda: gpu_lib.rotary(x[:3, :128], pos[:3], r, 64, out=x[1:, :128]),
                 lambda: gpu_lib.rotary(x.cpu(), pos, r, 64)):
        with pytest.raises(E):
            call()
    gpu_lib.rotary(x[:, :128], pos, r, 64, out=x[:, 128:])    # slices that interleave share nothing
