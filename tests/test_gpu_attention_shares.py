"""Row tiles of the tiled attention kernel, cut into shares and whole: windows,
missing pages and non-finite values where a cut runs through a tile, and grids of
more whole tiles than the chip holds.  Which way a call went is read from its
workspace: shares leave their length there, whole tiles leave it untouched."""
import math

import pytest
import torch

from oracle import paged as OP
from tests.test_gpu_attention import FP8, LOOSE, build, call

pytestmark = pytest.mark.gpu
KINDS = [(64, False), (128, False), (256, False), (64, True), (128, True), (256, True)]


def reference(b, window, scale):
    """Float64 attention, its log-sum-exp and their bounds, with torch, a head at a time (as oracle.paged.attention)."""
    (heads, page, dim), hq = b["k"].shape[1:], b["hq"]
    T = b["q"].shape[0]
    out, tol = (torch.zeros(T, hq, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, ltol = (torch.zeros(T, hq, dtype=torch.float64, device="cuda") for _ in range(2))
    for r, L in enumerate(b["lens"]):
        t0, t1 = b["q_start"][r], b["q_start"][r + 1]
        if t0 == t1:
            continue
        table = torch.tensor(b["table"][r], device="cuda").long()
        j = torch.arange(L, device="cuda")
        pg = table[j // page]
        held = (pg >= 0) & (pg < b["k"].shape[0])
        pg = torch.where(held, pg, 0)
        pos = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        see = held[None] & (j[None] <= pos) & ((pos - j[None] < window) if window else True)
        for h in range(heads):
            K, V = (x.view(torch.uint8)[pg, h, j % page].view(FP8).double() if x.dtype == FP8 else x[pg, h, j % page].double()
                    for x in (b["k"], b["v"]))
            K, V = (torch.where(held[:, None], x, 0.0) for x in (K, V))
            c = scale * (1.0 if b["k_scale"] is None else float(b["k_scale"][h]))
            vs = 1.0 if b["v_scale"] is None else float(b["v_scale"][h])
            for hh in range(h * hq // heads, (h + 1) * hq // heads):
                q = b["q"][t0:t1, hh * dim:(hh + 1) * dim].double()
                s = (c * (q @ K.t().contiguous())).masked_fill(~see, -math.inf)
                size = (abs(c) * (q.abs() @ K.abs().t().contiguous())).masked_fill(~see, 0.0).amax(1)
                ds = size * dim * OP.U32 + 4 * OP.U32 * s.masked_fill(~see, 0.0).abs().amax(1)
                n = see.sum(1)
                lse[t0:t1, hh] = torch.logsumexp(s, 1)
                ltol[t0:t1, hh] = 2 * ds + n * OP.U32 + 2.0 ** -20 + 4 * OP.U32 * lse[t0:t1, hh].abs().nan_to_num(posinf=0)
                w = torch.softmax(s, 1).masked_fill(n[:, None] == 0, 0.0)
                finite = torch.isfinite(V)
                x = vs * (w @ torch.where(finite, V, 0.0))
                rel = OP.U_BF16 + 4 * ds + 2 * n * OP.U32 + 2.0 ** -19
                tol[t0:t1, hh] = rel[:, None] * abs(vs) * (w @ torch.where(finite, V, 0.0).abs())
                for i, d in (~finite).nonzero().tolist():      # 0 * inf is not 0: to the rows that see it alone
                    x[:, d] = torch.where(see[:, i], x[:, d] + V[i, d] * vs, x[:, d])
                out[t0:t1, hh] = x
    return out, lse, tol, ltol


def check(lib, b, cut, window=0, **kw):
    heads, _, dim = b["k"].shape[1:]
    scale, R, T = dim ** -0.5, len(b["lens"]), b["q"].shape[0]
    max_new, max_seq = max(b["new"]), kw.pop("max_seq", max(b["lens"]))
    group = b["hq"] // heads
    assert max_new * group > 32 and T * group >= 64 * R, "the streaming kernel would come first"
    want, wlse, tol, ltol = reference(b, window, scale)
    ws = lib.paged_attention_workspace(T, R, b["hq"], heads, dim, max_new, max_seq)
    ws[2048:] = 0x5a
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = call(lib, b, window=window, out_dtype=dtype, max_new=max_new, max_seq=max_seq, workspace=ws, **kw)
        share = int(ws[2048 + 8 * (R + 1):][:8].view(torch.int64))
        assert (share != 0x5a5a5a5a5a5a5a5a) == cut, "cut into shares: %s" % (not cut)
        got, glse = out.double().reshape(want.shape), lse.double()
        assert torch.equal(torch.isneginf(glse), torch.isneginf(wlse)) and not torch.isnan(glse).any()
        fin = torch.isfinite(wlse)
        assert ((glse - wlse).abs()[fin] <= ltol[fin]).all()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        inf = torch.isinf(want)
        assert torch.equal(got[inf], want[inf])
        fin = torch.isfinite(want)
        bound = tol + (OP.U_BF16 * (want.abs() + tol) if dtype == torch.bfloat16 else 0)
        off = (got - want).abs()[fin] > bound[fin]
        assert not off.any(), "%d of %d off" % (int(off.sum()), off.numel())


@pytest.mark.parametrize("dim,fp8", KINDS)
@pytest.mark.parametrize("ctx,new,window", [([4000, 0, 1800], [200, 300, 70], 1500), ([2500], [257], 1601),
                                            ([3000, 2990, 1, 5000], [64, 130, 150, 90], 2048)])
def test_windows_in_shares(gpu_lib, dim, fp8, ctx, new, window):
    check(gpu_lib, build(ctx, new, 4, 2, dim, 64, fp8, seed=window), True, window)
    check(gpu_lib, build(ctx, new, 3, 1, dim, 16, fp8, seed=window), True, window)


@pytest.mark.parametrize("dim,fp8", KINDS)
@pytest.mark.parametrize("window", [0, 1500])
def test_missing_pages_in_shares(gpu_lib, dim, fp8, window):
    """Holes of one and of many pages in tiles that are cut, a request without any, and one whose new tokens' are missing."""
    ctx, new = [3000, 1000, 2500, 2000], [150, 100, 80, 90]
    missing = [(0, c) for c in [0, 7, 8, 9, 30, 48, 49]] + [(1, c) for c in range(18)] + [(3, c) for c in (31, 32)] + [(0, c) for c in range(33, 43)]
    check(gpu_lib, build(ctx, new, 4, 2, dim, 64, fp8, seed=4, missing=missing), True, window, max_seq=3150 if window else LOOSE)


def put(b, r, pos, head, d, x):
    raw = torch.uint8 if b["v"].dtype == FP8 else torch.bfloat16
    page = b["v"].shape[2]
    b["v"].view(raw)[int(b["table"][r, pos // page]), head, pos % page, d] = torch.tensor([x], device="cuda").to(b["v"].dtype).view(raw)[0]


@pytest.mark.parametrize("dim,fp8", KINDS)
@pytest.mark.parametrize("window", [0, 1500])
def test_non_finite_values_in_shares(gpu_lib, dim, fp8, window):
    """At the window's edge, on the diagonal and between: in the tiles that not every row sees, of whichever part."""
    b = build([4000, 1800], [200, 150], 4, 2, dim, 64, fp8, seed=9)
    kinds = [float("nan")] * 3 if fp8 else [float("nan"), float("inf"), float("-inf")]
    for r, (c, n) in enumerate(zip(b["ctx"], b["new"])):
        edge = c - (window or c) + 1               # the first key that the first new token sees, if there is a window
        for i, pos in enumerate([edge + 3, edge + n // 2, edge + n - 2, max(edge - 1, 0), c, c + n // 3, c + n - 1]):
            put(b, r, pos, i % 2, 3 + 5 * i, kinds[i % 3])
    check(gpu_lib, b, True, window, max_seq=4200 if window else LOOSE)


@pytest.mark.parametrize("dim,fp8", KINDS)
@pytest.mark.parametrize("ctx,new,hq,heads,window", [([0], [2048], 32, 8, 0), ([100], [6000], 16, 16, 0), ([0, 500, 0], [1500, 1900, 2100], 32, 8, 0),
                                                     ([3000, 100], [2000, 1111], 16, 16, 777)])
def test_more_whole_tiles_than_workgroups_at_once(gpu_lib, dim, fp8, ctx, new, hq, heads, window):
    check(gpu_lib, build(ctx, new, hq, heads, dim, 64, fp8, seed=hq), False, window)
