"""GPU parity of paged_attention against the float64 oracle, within the bound of
one fp32 pass with bf16 weights (oracle.paged.attention); the log-sum-exp is held
to its own, much tighter bound, which an absent or surplus key among thousands
exceeds."""
import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def build(ctx, new, hq, heads, dim, page, fp8=False, seed=0, layout="phtd", poison=True, missing=(), extra_pages=3):
    """A batch: every place of the caches that no request holds is NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, new)]
    need = [-(-n // page) for n in lens]
    cols = max(max(need), 1) + 1
    pages = sum(need) + extra_pages
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = np.full((len(ctx), cols), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        for col in range(n):
            table[r, col] = order[at]
            at += 1
    caches = []
    for _ in range(2):
        x = torch.randn(pages, heads, page, dim, generator=g, device="cuda")
        if poison:
            free = torch.ones(pages, page, dtype=torch.bool)
            for r, n in enumerate(lens):
                for col in range(need[r]):
                    free[table[r, col], :min(page, n - col * page)] = False
            x = x.masked_fill(free.cuda()[:, None, :, None], float("nan"))
        caches.append(x)
    for r, col in missing:
        table[r, col] = -1 if (r + col) % 2 else pages + 5
    b = dict(hq=hq, page=page, ctx=ctx, new=new, lens=lens, table=table, k_scale=None, v_scale=None)
    if fp8:
        b["k_scale"], b["v_scale"] = (0.01 + 0.02 * torch.rand(heads, generator=g, device="cuda") for _ in range(2))
        caches = [(x / s[:, None, None]).clamp(-448, 448).to(FP8) for x, s in zip(caches, (b["k_scale"], b["v_scale"]))]
    else:
        caches = [x.to(torch.bfloat16) for x in caches]
    if layout == "pthd":
        raw = torch.uint8 if fp8 else torch.bfloat16
        caches = [x.view(raw).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(x.dtype) for x in caches]
    b["k"], b["v"] = caches
    b["q"] = torch.randn(sum(new), hq * dim, generator=g, device="cuda").mul(1.5).to(torch.bfloat16)
    b["q_start"] = np.concatenate([[0], np.cumsum(new)])
    return b


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def call(lib, b, **kw):
    kw = {**dict(max_new=max(b["new"]), max_seq=max(b["lens"]), k_scale=b["k_scale"], v_scale=b["v_scale"]), **kw}
    return lib.paged_attention(b["q"], b["k"], b["v"], i32(b["table"]), i32(b["q_start"]), i32(b["lens"]), return_lse=True, **kw)


def check(lib, b, scale=None, window=0, out_dtype=torch.bfloat16, **kw):
    out, lse = call(lib, b, scale=scale, window=window, out_dtype=out_dtype, **kw)
    heads, dim = b["k"].shape[1], b["k"].shape[3]
    f = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    want, wlse, tol, ltol = OP.attention(f(b["q"]), f(b["k"]), f(b["v"]), b["table"], b["q_start"], b["lens"], b["page"], b["hq"],
                                         dim ** -0.5 if scale is None else scale, window,
                                         None if b["k_scale"] is None else f(b["k_scale"]),
                                         None if b["v_scale"] is None else f(b["v_scale"]))
    got, glse = f(out).reshape(want.shape), f(lse)
    if out_dtype == torch.bfloat16:
        tol = tol + OP.U_BF16 * (np.abs(want) + tol)
    assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    bad = np.abs(glse - wlse)[fin] > ltol[fin]
    assert not bad.any(), "lse: %d of %d, worst %.3g of its bound" % (bad.sum(), bad.size, (np.abs(glse - wlse)[fin] / ltol[fin]).max())
    assert np.isfinite(got).all()
    off = np.abs(got - want) > tol
    assert not off.any(), "out: %d of %d off, worst %.3g" % (off.sum(), off.size, np.abs(got - want).max())
    again, lse2 = call(lib, b, scale=scale, window=window, out_dtype=out_dtype, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 30, 31, 32, 33, 127, 200])
def test_single_tokens(gpu_lib, dim, fp8, ctx):
    """Decode: lengths around every tile and page border, groups of 1 to 5 heads, two requests of other lengths beside."""
    group = 1 + ctx % 5
    check(gpu_lib, build([ctx, 3, ctx // 2], [1, 1, 1], 2 * group, 2, dim, 16, fp8, seed=ctx))


@pytest.mark.parametrize("hq,heads", [(1, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (40, 8), (12, 12), (7, 7)])
def test_head_layouts(gpu_lib, hq, heads):
    check(gpu_lib, build([70, 5], [1, 1], hq, heads, 64, 32, seed=hq))


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)])
@pytest.mark.parametrize("new", [2, 5, 8, 9, 31, 32, 33, 64, 65, 100, 257])
def test_chunks(gpu_lib, dim, fp8, new):
    """From a few drafts to chunks over several row tiles, at group 4: both kernels, and both in one batch."""
    check(gpu_lib, build([45, 0, 129], [new, 1, max(new // 2, 1)], 4, 1, dim, 16, fp8, seed=new))


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_windows(gpu_lib, window, new):
    check(gpu_lib, build([150, 20], [new, new], 6, 2, 64, 16, seed=window), window=window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("new", [1, 70])
def test_page_sizes_and_layouts(gpu_lib, page, new):
    check(gpu_lib, build([page + 3, 2 * page - 1], [new, new], 4, 2, 64, page, fp8=page % 3 == 1, seed=page, layout="pthd"))


@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("dim,fp8", [(64, True), (128, False), (256, False)])
def test_missing_pages_and_empty_rows(gpu_lib, new, dim, fp8):
    """Pages that the table does not hold hide their keys; request 1 has none left, request 2 only its middle."""
    b = build([100, 10, 60], [new] * 3, 4, 2, dim, 16, fp8, seed=new,
              missing=[(0, 1), (0, 4)] + [(1, c) for c in range(5)] + [(2, 0), (2, 3), (2, 4), (2, 5), (2, 6), (2, 7)])
    check(gpu_lib, b)
    check(gpu_lib, b, window=20)


@pytest.mark.parametrize("new", [1, 40])
def test_sequence_shorter_than_its_chunk(gpu_lib, new):
    """Rows at negative positions see nothing."""
    b = build([6, 6], [new, new], 2, 1, 64, 16, seed=2)
    b["lens"] = [max(b["lens"][0] - 8, 0), b["lens"][1]]
    check(gpu_lib, b)


def test_requests_without_new_tokens_and_padding_rows(gpu_lib):
    for new in ([0, 1, 0, 3, 0], [0, 50, 0, 1, 0]):
        b = build([9, 8, 7, 40, 0], new, 4, 2, 64, 16, seed=4)
        check(gpu_lib, b)
        b["q"] = torch.cat([b["q"], torch.full_like(b["q"][:3], float("nan"))])
        T = b["q"].shape[0]
        out = torch.full((T, 4 * 64), 7.0, dtype=torch.float32, device="cuda")
        lse = torch.full((T, 4), 7.0, dtype=torch.float32, device="cuda")
        call(gpu_lib, b, out=out, lse=lse, out_dtype=torch.float32)
        assert out[-3:].eq(7).all() and lse[-3:].eq(7).all() and out[:-3].ne(7).all()


@pytest.mark.parametrize("new,hq,heads", [([0, 1, 0, 3, 0], 4, 2), ([0, 50, 0, 1, 0], 4, 2), ([60, 2, 0, 64, 40], 4, 2),
                                          ([0, 0, 0, 0, 0], 4, 2), ([0, 0, 0, 0, 0], 40, 1), ([1, 1, 0, 0, 1], 40, 1)])
def test_padding_rows_are_cleared(gpu_lib, new, hq, heads):
    """Outputs that the call allocates, and those it is asked to clear: 0 and -inf after the last request's rows, the
    others as without padding; columns beside a strided output stay."""
    b = build([9, 8, 7, 40, 0], new, hq, heads, 64, 16, seed=4)
    live, pad = b["q"].shape[0], 700
    b["q"] = torch.cat([b["q"], torch.full((pad, hq * 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    # the rows count in the rules that choose a kernel: the same call, told to leave them
    want, wlse = torch.zeros(live + pad, hq * 64, device="cuda"), torch.zeros(live + pad, hq, device="cuda")
    call(gpu_lib, b, out=want, lse=wlse, out_dtype=torch.float32, clear_padding=False)
    assert want[live:].eq(0).all() and wlse[live:].eq(0).all()
    want, wlse = want[:live], wlse[:live]
    stale = torch.full((live + pad, hq * 64), float("nan"), device="cuda")
    del stale                                      # what the allocator hands out next
    out, lse = call(gpu_lib, b, out_dtype=torch.float32)
    wide, lse2 = torch.full((live + pad, hq * 64 + 8), 7.0, device="cuda"), torch.full((live + pad, hq), 7.0, device="cuda")
    call(gpu_lib, b, out=wide[:, 4:-4], lse=lse2, out_dtype=torch.float32, clear_padding=True)
    half = torch.full((live + pad, hq * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    call(gpu_lib, b, out=half, clear_padding=True)
    for o, l in ((out, lse), (wide[:, 4:-4], lse2)):
        assert torch.equal(o[:live], want) and torch.equal(l[:live], wlse)
        assert o[live:].eq(0).all() and torch.isneginf(l[live:]).all()
    assert half[live:].eq(0).all() and torch.equal(half[:live], want.to(torch.bfloat16))
    assert wide[:, :4].eq(7).all() and wide[:, -4:].eq(7).all()


def test_a_padded_step_keeps_the_next_layers_scale(gpu_lib):
    """The dynamic global scale of a linear layer after a padded step is that of the live rows."""
    b = build([30, 70], [1, 4], 4, 2, 64, 16, seed=5)
    b["q"] = torch.cat([b["q"], torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")])
    for _ in range(3):
        stale = torch.full((8, 256), 3e38, dtype=torch.bfloat16, device="cuda")
        del stale
        out, _ = call(gpu_lib, b)
        codes, scales, g = gpu_lib.nvfp4_quantize(out)
        wcodes, wscales, wg = gpu_lib.nvfp4_quantize(out[:5].clone())
        assert float(g) == float(wg) and torch.equal(codes[:5], wcodes) and torch.equal(scales[:5], wscales)
        assert codes[5:].eq(0).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("new", [1, 50])
def test_scales(gpu_lib, scale, new):
    check(gpu_lib, build([77], [new], 4, 2, 128, 16, seed=1), scale=scale, out_dtype=torch.float32)


def test_negative_head_scale(gpu_lib):
    b = build([77, 12], [1, 60], 4, 2, 128, 16, fp8=True, seed=1)
    b["k_scale"][1] *= -1
    check(gpu_lib, b)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 60])
def test_a_nan_head_scale_reaches_its_heads_rows(gpu_lib, dim, new):
    """Rows of the head that see a key are NaN, rows that see none stay 0, and the other head is as ever."""
    b = build([77, 300, 6], [new] * 3, 4, 2, dim, 16, fp8=True, seed=1)
    b["lens"][2] = max(b["lens"][2] - 8, 0)        # the first rows of request 2 stand at negative positions
    want, wlse = call(gpu_lib, b)
    b["k_scale"] = torch.tensor([float(b["k_scale"][0]), float("nan")], device="cuda")
    out, lse = call(gpu_lib, b)
    out, want = out.reshape(-1, 2, 2, dim), want.reshape(-1, 2, 2, dim)
    lse, wlse = lse.reshape(-1, 2, 2), wlse.reshape(-1, 2, 2)
    assert torch.equal(out[:, 0], want[:, 0]) and torch.equal(lse[:, 0], wlse[:, 0])
    empty = torch.isneginf(wlse[:, 1])
    assert torch.isnan(out[:, 1][~empty]).all() and torch.isnan(lse[:, 1][~empty]).all()
    assert out[:, 1][empty].eq(0).all() and torch.isneginf(lse[:, 1][empty]).all()


@pytest.mark.parametrize("new,fp8", [(1, False), (1, True), (60, False), (60, True)])
def test_large_scores_and_rising_maximum(gpu_lib, new, fp8):
    """Keys that grow with their position: the running maximum rises in every tile, by hundreds."""
    b = build([500], [new], 2, 1, 128, 16, fp8=fp8, seed=3)
    ramp = torch.linspace(0.05, 3, 1000, device="cuda")
    k = b["k"].float()
    for col, p in enumerate(b["table"][0]):
        if p >= 0:
            k[p] *= ramp[col * 16:col * 16 + 16, None] / (3 if fp8 else 1)
    b["k"] = k.to(b["k"].dtype)
    check(gpu_lib, b, scale=1.0, out_dtype=torch.float32)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_rising_maximum_rounds_no_weight_again(gpu_lib, dim, fp8):
    """Keys 0 - 31 weigh 1 until the next tile's first key raises the maximum, by 2^0.96 for the rows looked at and by 2^20
    for their neighbours (whose rise scales them all).  The values are 1 at the former and 0 elsewhere, and a weight of 1
    needs no rounding: what is left is an exponent of 20 in fp32 (three roundings, 2.5e-6), the exponential's 2^-20 and a
    sum of 33 terms (2e-6), under 2^-17 in all; a weight rounded anew would be off by 2^-8.1."""
    tokens, rise, first = 64, 0.9609375, 32 if dim == 256 else 64
    b = build([128], [tokens], 1, 1, dim, 16, seed=1, poison=False)
    k, v = torch.zeros(192, dim, device="cuda"), torch.zeros(192, dim, device="cuda")
    k[32:, 0] = -448
    k[first, 0] = 1
    v[:32] = 1
    order = torch.tensor([int(p) for p in b["table"][0][:12]], device="cuda")
    for name, x in (("k", k), ("v", v)):
        b[name][order, 0] = x.view(12, 16, dim).to(torch.bfloat16)
        if fp8:
            b[name] = b[name].to(FP8)
    q = torch.zeros(tokens, dim, device="cuda")
    q[::2, 0], q[1::2, 0] = rise, 20
    b["q"] = q.to(torch.bfloat16)
    assert float(b["q"][0, 0]) == rise
    out, lse = call(gpu_lib, b, scale=float(np.log(2)), out_dtype=torch.float32)
    for x, got, glse in ((rise, out[::2], lse[::2]), (20, out[1::2], lse[1::2])):
        want = 32 / (32 + 2.0 ** x)
        assert (got.double() - want).abs().max() <= want * 2.0 ** -17, (got.double() / want - 1).abs().max()
        assert (glse.double() - np.log(32 + 2.0 ** x)).abs().max() <= 2.0 ** -17


@pytest.mark.parametrize("ctx,new,hq,heads,dim,fp8", [
    (20000, 1, 4, 2, 128, False), (9000, 5, 6, 1, 256, True), (9000, 40, 5, 1, 64, False), (6000, 300, 2, 1, 128, True),
])
def test_long_contexts_are_split_and_joined(gpu_lib, ctx, new, hq, heads, dim, fp8):
    check(gpu_lib, build([ctx], [new], hq, heads, dim, 64, fp8, seed=5))


def test_many_ragged_requests(gpu_lib):
    rng = np.random.default_rng(0)
    ctx, new = rng.integers(0, 130, 600).tolist(), rng.choice([0, 1, 1, 1, 2, 20], 600).tolist()
    check(gpu_lib, build(ctx, new, 3, 1, 64, 16, seed=6))


def test_far_pages(gpu_lib):
    """Pages whose byte offsets pass 2^32, in one batch with near ones; both kernels."""
    page, heads, dim, far = 64, 2, 128, 140000
    for new in (1, 60):
        b = build([100], [new], 4, heads, dim, page, seed=8, extra_pages=0)
        pages = b["k"].shape[0]
        want, wlse = call(gpu_lib, b, out_dtype=torch.float32)
        k, v = (torch.empty((far, heads, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k[far - pages:], v[far - pages:] = b["k"], b["v"]
        k[0], v[0] = b["k"][0], b["v"][0]
        t = np.where(b["table"] > 0, b["table"] + far - pages, b["table"])
        got, glse = call(gpu_lib, {**b, "k": k, "v": v, "table": t}, out_dtype=torch.float32)
        assert torch.equal(got, want) and torch.equal(glse, wlse)
        del k, v


def test_fused_projection_views_other_streams_and_graphs(gpu_lib):
    """q as columns of a wider buffer, a strided output, a side stream, and a captured step replayed on new lengths."""
    b = build([50, 90], [1, 40], 4, 2, 64, 16, seed=9)
    want, wlse = call(gpu_lib, b)
    T = b["q"].shape[0]
    wide = torch.randn(T, 4 * 64 * 2 + 8, device="cuda").to(torch.bfloat16)
    wide[:, 8:8 + 256] = b["q"]
    out = torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(gpu_lib, {**b, "q": wide[:, 8:8 + 256]}, out=out[:, 128:384])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 128:384], want) and out[:, :128].eq(0).all() and out[:, 384:].eq(0).all()

    table, start, lens = i32(b["table"]), i32(b["q_start"]), i32(b["lens"])
    ws = gpu_lib.paged_attention_workspace(T, 2, 4, 2, 64, 64, 256)
    res, lse = torch.empty_like(want), torch.empty_like(wlse)
    run = lambda: gpu_lib.paged_attention(b["q"], b["k"], b["v"], table, start, lens, 64, 256, out=res, lse=lse, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for cut in (0, 3, 11):
        lens.copy_(i32([b["lens"][0] - cut, b["lens"][1] - cut]))
        res.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = res.clone(), lse.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got[0], res) and torch.equal(got[1], lse)


def check_not_finite(gpu_lib, dim, fp8, new, window, **kw):
    b = build([700, 130], [new, new], 4, 2, dim, 32, fp8, seed=new + dim)
    kinds = [float("nan")] * 3 if fp8 else [float("nan"), float("inf"), float("-inf")]
    raw = torch.uint8 if fp8 else torch.bfloat16

    def put(cache, r, pos, d, x):
        x = torch.tensor([x], device="cuda").to(cache.dtype).view(raw)
        cache.view(raw)[int(b["table"][r, pos // 32]), 1, pos % 32, d] = x[0]
    for r, length in enumerate(b["lens"]):
        # new tokens, which only later ones see, and old ones, which a window hides from some
        for i, pos in enumerate({length - 1, length - 1 - new // 2, length - 2, length - new, length - 1 - max(window - 1, 0), length - 20 - window}):
            put(b["v"], r, pos, 5 + 7 * i, kinds[i % 3])
        put(b["k"], r, length - 1 - new // 4, 9, float("nan"))
    f = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    scales = [None if s is None else f(s) for s in (b["k_scale"], b["v_scale"])]
    want, wlse, tol, ltol = OP.attention(f(b["q"]), f(b["k"]), f(b["v"]), b["table"], b["q_start"], b["lens"], b["page"], 4,
                                         dim ** -0.5, window, *scales)
    # a row that sees such a value has it in its own column alone
    clean = f(b["v"])
    _, _, tol, _ = OP.attention(f(b["q"]), f(b["k"]), np.where(np.isfinite(clean), clean, 0.0), b["table"], b["q_start"], b["lens"],
                                b["page"], 4, dim ** -0.5, window, *scales)
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = call(gpu_lib, b, window=window, out_dtype=dtype, **kw)
        got, glse = f(out).reshape(want.shape), f(lse)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(glse), np.isnan(wlse))
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        fin, lfin = np.isfinite(want), np.isfinite(wlse)
        bound = tol + (OP.U_BF16 * (np.abs(want) + tol) if dtype == torch.bfloat16 else 0)
        assert (np.abs(got - want)[fin] <= bound[fin]).all() and (np.abs(glse - wlse)[lfin] <= ltol[lfin]).all()


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)])
@pytest.mark.parametrize("new,window", [(1, 0), (2, 0), (5, 40), (40, 0), (150, 0), (150, 90)])
def test_infinities_and_nan_reach_the_rows_that_see_them_and_no_others(gpu_lib, dim, fp8, new, window):
    check_not_finite(gpu_lib, dim, fp8, new, window)


# A bound far above the lengths makes the tiled kernel cut row tiles into shares.
LOOSE = 1 << 20


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)])
@pytest.mark.parametrize("new,window", [(40, 0), (150, 90)])
def test_infinities_and_nan_in_shares(gpu_lib, dim, fp8, new, window):
    check_not_finite(gpu_lib, dim, fp8, new, window, max_seq=LOOSE)


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)])
@pytest.mark.parametrize("ctx,new", [([0], [33]), ([3000, 0, 1], [100, 257, 1]), ([2000, 5000], [70, 40])])
def test_chunks_in_shares(gpu_lib, dim, fp8, ctx, new):
    check(gpu_lib, build(ctx, new, 4, 2, dim, 64, fp8, seed=len(ctx) + dim), max_seq=LOOSE)


@pytest.mark.parametrize("new", [(1, 33), (5, 40), (9, 9), (2, 100, 1, 1, 1, 1, 1, 1)])
def test_batches_that_one_kernel_takes_and_that_both_share(gpu_lib, new):
    """Requests of few rows among larger ones: with a bound on the new tokens that fits, and with one far above."""
    b = build([300 + 7 * i for i in range(len(new))], list(new), 4, 1, 128, 32, seed=len(new))
    check(gpu_lib, b)
    check(gpu_lib, b, max_new=512, max_seq=LOOSE)


def test_one_workspace_serves_calls_of_other_sizes(gpu_lib):
    """The counters that a call needs at zero are zero after every other one."""
    batches = [build(*a, seed=i) for i, a in enumerate([
        ([9000, 40, 3000], [1, 1, 1], 8, 2, 128, 64), ([300, 5000], [3, 200], 8, 2, 128, 64), ([4000], [900], 8, 2, 128, 64),
        ([20000], [1], 16, 1, 256, 64), ([100] * 40, [4] * 40, 4, 4, 64, 16)])]
    size = max(gpu_lib.paged_attention_workspace(b["q"].shape[0], len(b["ctx"]), b["hq"], b["k"].shape[1], b["k"].shape[3],
                                                 max(b["new"]), max(b["lens"])).numel() for b in batches)
    shared = torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda")
    shared[:2048] = 0
    want = [call(gpu_lib, b) for b in batches]
    for order in ([0, 1, 2, 3, 4], [4, 2, 0, 3, 1], [1, 1, 0, 0, 2]):
        for i in order:
            out, lse = call(gpu_lib, batches[i], workspace=shared)
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
            assert int(shared[:2048].count_nonzero()) == 0


def test_a_workspace_for_the_largest_step_serves_smaller_ones(gpu_lib):
    ws = gpu_lib.paged_attention_workspace(400, 4, 8, 2, 128, 100, 5000)
    for ctx, new in (([4900, 0, 3, 70], [100, 100, 100, 100]), ([3000, 9, 0, 70], [1, 1, 1, 1]), ([5], [40]), ([10, 4000], [1, 90])):
        b = build(ctx, new, 8, 2, 128, 64, seed=sum(new))
        out, lse = call(gpu_lib, b, max_new=100, max_seq=5000, workspace=ws)
        want, wlse = call(gpu_lib, b, max_new=100, max_seq=5000)
        assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_refusals(gpu_lib):
    E = gpu_lib.NVFP4Error
    b = build([20], [2], 4, 2, 64, 16)
    call(gpu_lib, b)
    half = torch.zeros(2, 256, dtype=torch.float16, device="cuda")
    for bad in (dict(q=half), dict(q=b["q"][:, :192]), dict(k=b["k"].float()), dict(v=b["v"][:, :1]), dict(q=b["q"].cpu()),
                dict(q_start=[0, 1, 2])):
        with pytest.raises(E):
            call(gpu_lib, {**b, **bad})
    for bad in (dict(window=-1), dict(scale=float("nan")), dict(max_new=-1), dict(k_scale=torch.ones(2, device="cuda")),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(out=torch.empty(2, 128, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(E):
            call(gpu_lib, b, **bad)


@pytest.mark.parametrize("shape", [(0, 1, 16, 64), (2, 0, 16, 64), (2, 1, 0, 64), (2, 1, 16, 0)])
def test_empty_caches_are_refused(gpu_lib, shape):
    b = build([20], [2], 1, 1, 64, 16)
    b["k"], b["v"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with pytest.raises(gpu_lib.NVFP4Error):
        call(gpu_lib, b)
    with pytest.raises(gpu_lib.NVFP4Error):
        gpu_lib.paged_kv_write(b["q"], b["q"], torch.arange(2, device="cuda"), b["k"], b["v"])


def test_strides_of_single_pages_and_heads_do_not_matter(gpu_lib):
    """K contiguous, V a view whose page and head strides say something else about the one page and the one head."""
    b = build([9], [2], 1, 1, 64, 16, extra_pages=0)
    want, _ = call(gpu_lib, b)
    assert b["k"].shape[0] == 1
    b["v"] = b["v"].as_strided(b["v"].shape, (8, 24, 64, 1))
    got, _ = call(gpu_lib, b)
    assert torch.equal(got, want)
    with pytest.raises(gpu_lib.NVFP4Error):
        call(gpu_lib, {**b, "v": torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device="cuda")[..., :64]})   # another token stride
    two = torch.zeros(2, 1, 32, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu_lib.NVFP4Error):
        call(gpu_lib, {**b, "k": torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda"), "v": two[:, :, :16]})
