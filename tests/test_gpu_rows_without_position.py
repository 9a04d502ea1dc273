"""Rows of a negative position (padding) leave rotary and paged_kv_append as they came, whatever they hold: infinities
beside numbers, NaN with their payloads, both zeros.  So does what no rotation touches."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
KINDS = ["bf16", "e4m3", "e4m3_blocks", "int8_blocks"]


def any_bits(*shape, seed=0):
    """bf16 of any bit pattern: infinities, NaN and both zeros often."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int32)
    odd = torch.tensor([0x7f80, 0xff80, 0x7fc0, 0x7f81, 0xffc1, 0x8000, 0x0000, 0x0001], device="cuda", dtype=torch.int32)
    pick = torch.randint(0, 32, shape, generator=g, device="cuda")
    bits = torch.where(pick < 8, odd[pick % 8], bits)
    return torch.where(bits >= 2 ** 15, bits - 2 ** 16, bits).to(torch.int16).view(torch.bfloat16)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rotary_copies_them(gpu_lib, layout, dim, rot, in_place):
    T, heads = 37, 5
    x = any_bits(T, heads * dim, seed=dim + rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[::2] = -1
    pos[4] = -2 ** 31
    table = gpu_lib.rotary_table(rot, layout=layout, scaling="yarn", factor=4.0)
    before = x.clone()
    got = gpu_lib.rotary(x, pos, table, dim, out=x if in_place else None)
    assert same(got[pos < 0], before[pos < 0])
    assert same(got.view(T, heads, dim)[:, :, rot:], before.view(T, heads, dim)[:, :, rot:])


def caches(kind, pages, heads, page, dim):
    dtype = {"bf16": torch.bfloat16, "int8_blocks": torch.int8}.get(kind, FP8)
    k, v = (torch.zeros(pages, heads, page, dim, device="cuda").to(dtype) for _ in range(2))
    if kind == "bf16":
        return k, v, None, None
    if kind == "e4m3":
        return k, v, torch.full((heads,), 0.5, device="cuda"), torch.full((heads,), 0.25, device="cuda")
    return (k, v) + tuple(torch.full((pages, heads, page // 16), 100, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))


def raw(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.uint8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 64), (256, 256)])
def test_append_takes_them_as_without_a_rotation(gpu_lib, kind, layout, dim, rot):
    T, heads, hq = 45, 2, 6
    x = any_bits(T, (hq + 2 * heads) * dim, seed=dim)
    q, k, v = x.split([hq * dim, heads * dim, heads * dim], 1)
    slots = torch.arange(T, device="cuda") + 3
    table = gpu_lib.rotary_table(rot, layout=layout, scaling="yarn", factor=4.0)
    made = []
    for rotation in (table, None):
        kc, vc, ks, vs = caches(kind, 4, heads, 16, dim)
        out = gpu_lib.paged_kv_append(k, v, torch.full((T,), -1, dtype=torch.int32, device="cuda"), slots, kc, vc, rotation=rotation,
                                      k_scale=ks, v_scale=vs, q=q)
        assert same(out, q)
        made.append([raw(t) for t in (kc, vc) + ((ks, vs) if kind.endswith("blocks") else ())])
        if kind == "bf16":
            for cache, rows in ((kc, k), (vc, v)):
                got = cache.permute(0, 2, 1, 3).reshape(64, heads * dim)[3:3 + T]
                assert same(got, rows)
    for a, b in zip(*made):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", KINDS)
def test_append_of_both_in_one_run(gpu_lib, kind):
    """Beside rotated rows of their block: q row by row, and infinities of k that stay alone in their rows."""
    T, heads, dim = 32, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, 8 * dim, generator=g, device="cuda").to(torch.bfloat16)
    x[::2, ::5] = float("inf")
    q, k, v = x.split([4 * dim, heads * dim, heads * dim], 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[::2] = -1
    kc, vc, ks, vs = caches(kind, 2, heads, 16, dim)
    out = gpu_lib.paged_kv_append(k, v, pos, torch.arange(T, device="cuda"), kc, vc, rotation=gpu_lib.rotary_table(dim), k_scale=ks,
                                  v_scale=vs, q=q)
    assert same(out[::2], q[::2])
    got = kc.float().permute(0, 2, 1, 3).reshape(T, heads * dim)
    most = {"bf16": float("inf"), "int8_blocks": 127.0}.get(kind, 448.0)
    assert torch.isfinite(x[1::2]).all() and torch.isfinite(got[1::2]).all()
    assert ((got[::2] == most) == torch.isinf(k[::2])).all() and not torch.isnan(got).any()
