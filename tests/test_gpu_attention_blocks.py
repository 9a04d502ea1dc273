"""GPU parity of paged_attention_blocks against the float64 oracle over the values that
the caches stand for, within paged_attention's own bounds: a scale that is a power of two
is applied exactly."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8
from oracle import paged as OP

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def codes_to(codes, kind):
    """Code values as a cache tensor."""
    t = torch.from_numpy(np.nan_to_num(codes, nan=0.0)).to("cuda")
    t = t.to(torch.int8) if kind == "int8" else t.to(torch.float32).to(FP8)
    if np.isnan(codes).any():
        t.view(torch.uint8)[torch.from_numpy(np.isnan(codes)).to("cuda")] = 0x7f
    return t


def build(ctx, new, hq, heads, dim, page, kind="e4m3", seed=0, poison=True, missing=(), extra_pages=3, spread=3.0):
    """A batch whose blocks have scales of their own; what no request holds is the largest code or NaN, and the scales of
    blocks without a key are those that a cache never has."""
    rng = np.random.default_rng(seed)
    lens = [c + n for c, n in zip(ctx, new)]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra_pages
    order = rng.permutation(pages)
    table = np.full((len(ctx), max(max(need), 1) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    free = np.ones((pages, page), bool)
    for r, n in enumerate(lens):
        for col in range(need[r]):
            free[table[r, col], :min(page, n - col * page)] = False
    b = dict(hq=hq, page=page, ctx=ctx, new=new, lens=lens, table=table, kind=kind)
    for name in "kv":
        x = rng.standard_normal((pages, heads, page, dim)) * np.exp2(rng.uniform(-spread, spread, (pages, heads, page // 16)).repeat(16, 2))[..., None]
        if name == "k":
            x = x / np.exp2(spread)
        codes, scales = O8.fill(x, kind)
        if poison:
            codes = np.where(free[:, None, :, None], 127.0 if kind == "int8" else np.nan, codes)
            empty = free.reshape(pages, page // 16, 16).all(2)[:, None, :].repeat(heads, 1)
            scales = np.where(empty, rng.choice([0, 255, 250], scales.shape), scales).astype(np.uint8)
        b[name], b[name + "_scale"] = codes_to(codes, kind), torch.from_numpy(scales).to("cuda").view(E8M0)
        b[name + "_values"] = O8.block_values(codes, np.clip(scales, 1, O8.MOST_BYTE[kind]))
    for r, col in missing:
        table[r, col] = -1 if (r + col) % 2 else pages + 5
    b["q"] = torch.from_numpy(rng.standard_normal((sum(new), hq * dim)) * 1.5).to("cuda").to(torch.bfloat16)
    b["q_start"] = np.concatenate([[0], np.cumsum(new)])
    return b


def call(lib, b, **kw):
    kw = {**dict(max_new=max(b["new"]), max_seq=max(b["lens"])), **kw}
    return lib.paged_attention_blocks(b["q"], b["k"], b["v"], b["k_scale"], b["v_scale"], i32(b["table"]), i32(b["q_start"]),
                                      i32(b["lens"]), return_lse=True, **kw)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(lib, b, scale=None, window=0, out_dtype=torch.bfloat16, **kw):
    out, lse = call(lib, b, scale=scale, window=window, out_dtype=out_dtype, **kw)
    dim = b["k"].shape[3]
    want, wlse, tol, ltol = OP.attention(f64(b["q"]), b["k_values"], b["v_values"], b["table"], b["q_start"], b["lens"], b["page"],
                                         b["hq"], dim ** -0.5 if scale is None else scale, window)
    got, glse = f64(out).reshape(want.shape), f64(lse)
    if out_dtype == torch.bfloat16:
        tol = tol + OP.U_BF16 * (np.abs(want) + tol)
    assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    assert (np.abs(glse - wlse)[fin] <= ltol[fin]).all()
    assert np.isfinite(got).all()
    off = np.abs(got - want) > tol
    assert not off.any(), "out: %d of %d off, worst %.3g" % (off.sum(), off.size, np.abs(got - want).max())
    again, lse2 = call(lib, b, scale=scale, window=window, out_dtype=out_dtype, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 30, 31, 32, 33, 127, 200])
def test_single_tokens(gpu_lib, dim, kind, ctx):
    group = 1 + ctx % 5
    check(gpu_lib, build([ctx, 3, ctx // 2], [1, 1, 1], 2 * group, 2, dim, 16, kind, seed=ctx))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,heads", [(1, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (40, 8), (12, 12), (7, 7)])
def test_head_layouts(gpu_lib, kind, hq, heads):
    check(gpu_lib, build([70, 5], [1, 1], hq, heads, 64, 32, kind, seed=hq))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [2, 5, 8, 9, 31, 32, 33, 64, 65, 100, 257])
def test_chunks(gpu_lib, dim, kind, new):
    check(gpu_lib, build([45, 0, 129], [new, 1, max(new // 2, 1)], 4, 1, dim, 16, kind, seed=new))


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_windows(gpu_lib, window, new):
    check(gpu_lib, build([150, 20], [new, new], 6, 2, 64, 16, "int8" if window % 2 else "e4m3", seed=window), window=window)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_page_sizes(gpu_lib, page, new, kind):
    check(gpu_lib, build([page + 3, 2 * page - 1], [new, new], 4, 2, 64, page, kind, seed=page))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_missing_pages_and_long_contexts(gpu_lib, dim, new, kind):
    """More than 64 tiles a wave's run, so that scales are fetched again; pages that are not there; rows that see nothing."""
    check(gpu_lib, build([5000, 40, 2500], [new, new, new], 4, 2, dim, 16, kind, seed=dim, missing=((0, 3), (1, 0), (2, 20), (0, 280))))
    b = build([20, 5], [new, new], 4, 2, dim, 16, kind, seed=1, missing=[(r, c) for r in range(2) for c in range(2 + new // 16 + 1)][:2])
    check(gpu_lib, b)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 80])
def test_wide_scales_fp32_out_and_negative_scale(gpu_lib, kind, new):
    check(gpu_lib, build([100, 33], [new, new], 4, 2, 128, 32, kind, seed=2, spread=12.0), out_dtype=torch.float32)
    check(gpu_lib, build([100, 33], [new, new], 4, 2, 128, 32, kind, seed=3), scale=-0.3)
    check(gpu_lib, build([100, 33], [new, new], 4, 2, 128, 32, kind, seed=3), scale=0.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 70])
def test_nan_values_reach_the_rows_that_see_them(gpu_lib, dim, new):
    b = build([40], [new], 4, 2, dim, 16, "e4m3", seed=5)
    clean = call(gpu_lib, b)[0].clone()
    key = 42
    b["v"].view(torch.uint8)[int(b["table"][0, key // 16]), 1, key % 16, 7] = 0x7f
    out = call(gpu_lib, b)[0].view(new, 4, dim)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[key - 40:, 2:, 7] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean.view(new, 4, dim)[~hit])


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_equals_paged_attention_where_one_scale_serves_all(gpu_lib, new, kind):
    """E4M3 codes with one power of two a head: paged_attention with that scale gives the same numbers."""
    b = build([300, 17], [new, new], 8, 2, 128, 16, kind, seed=9, poison=False)
    for n in "kv":
        b[n + "_scale"].view(torch.uint8).fill_(125)
    out, lse = call(gpu_lib, b)
    quarter = torch.full((2,), 0.25, device="cuda")
    if kind == "int8":
        ref, rl = gpu_lib.paged_attention(b["q"], b["k"].to(torch.bfloat16) * 0.25, b["v"].to(torch.bfloat16) * 0.25, i32(b["table"]),
                                          i32(b["q_start"]), i32(b["lens"]), new, 400, return_lse=True)
    else:
        ref, rl = gpu_lib.paged_attention(b["q"], b["k"], b["v"], i32(b["table"]), i32(b["q_start"]), i32(b["lens"]), new, 400,
                                          k_scale=quarter, v_scale=quarter, return_lse=True)
    # the same weights up to the order of fp32 sums, then bf16: a step at most
    assert (out.float() - ref.float()).abs().max() <= 2 * OP.U_BF16 * ref.float().abs().max()
    assert (lse - rl).abs().max() < 1e-5


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_padding_rows(gpu_lib, kind):
    b = build([30, 4], [1, 40], 4, 2, 64, 16, kind, seed=6)
    want = call(gpu_lib, b)[0]
    b["q"] = torch.cat([b["q"], torch.full_like(b["q"][:3], float("nan"))])
    out = torch.full((44, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    got, _ = call(gpu_lib, b, out=out)
    assert torch.equal(got[:41], want) and (got[41:] == 7).all()
    got, lse = call(gpu_lib, b)
    assert torch.equal(got[:41], want) and (got[41:] == 0).all() and torch.isneginf(lse[41:]).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_captured_and_replayed_and_a_shared_workspace(gpu_lib, kind):
    b = build([60, 300, 9], [1, 50, 3], 4, 2, 128, 16, kind, seed=7)
    ws = gpu_lib.paged_attention_workspace(64, 3, 4, 2, 128, 50, 400)
    out = torch.empty_like(b["q"])
    lens, start, table = i32(b["lens"]), i32(b["q_start"]), i32(b["table"])
    f = lambda o: gpu_lib.paged_attention_blocks(b["q"], b["k"], b["v"], b["k_scale"], b["v_scale"], table, start, lens, 50, 400,  # noqa: E731
                                                 out=o, workspace=ws)
    f(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(out)
    for i in range(4):
        b["q"].mul_(-0.9)
        lens.sub_(1)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, f(torch.empty_like(out)))


def test_pages_past_32_bits(gpu_lib):
    """Codes and scales of pages whose bytes lie past 2^32."""
    dim, page, heads = 256, 1024, 8
    pages = 2 ** 32 // (dim * page * heads) + 4
    k, v = (torch.zeros(pages, heads, page, dim, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, heads, page // 16), 100, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))
    b = build([1000], [40], 8, 8, dim, page, "int8", seed=4, poison=False, extra_pages=0)
    far = [pages - 1, pages - 3]
    for i, pg in enumerate(b["table"][0, :2].tolist()):
        k[far[i]], v[far[i]] = b["k"][pg], b["v"][pg]
        ks.view(torch.uint8)[far[i]], vs.view(torch.uint8)[far[i]] = b["k_scale"].view(torch.uint8)[pg], b["v_scale"].view(torch.uint8)[pg]
    for n in (40, 1):
        want = gpu_lib.paged_attention_blocks(b["q"][:n], b["k"], b["v"], b["k_scale"], b["v_scale"], i32(b["table"]), i32([0, n]), i32([1040]), n, 1040)
        got = gpu_lib.paged_attention_blocks(b["q"][:n], k, v, ks, vs, i32([far + [-1]]), i32([0, n]), i32([1040]), n, 1040)
        assert torch.equal(got, want)


def test_refusals(gpu_lib):
    b = build([20], [1], 4, 2, 64, 16, "int8")
    E = gpu_lib.NVFP4Error
    def bad(**kw):  # noqa: E306
        a = {**b, **kw}
        with pytest.raises(E):
            gpu_lib.paged_attention_blocks(a["q"], a["k"], a["v"], a["k_scale"], a["v_scale"], i32(b["table"]), i32([0, 1]), i32([21]), 1, 21,
                                           workspace=a.get("ws"))
    bad(k=b["k"].to(torch.bfloat16))
    bad(v=b["v"].view(FP8))
    bad(k_scale=b["k_scale"].view(torch.uint8))
    bad(k_scale=None)
    bad(v_scale=b["v_scale"][:, :1])
    bad(v_scale=b["v_scale"].view(torch.uint8).repeat_interleave(2, 2)[:, :, ::2].view(E8M0))
    bad(q=b["q"][:, :192])
    bad(q=b["q"].float())
    bad(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
