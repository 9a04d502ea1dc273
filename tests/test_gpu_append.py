"""GPU parity of paged_kv_append against the oracle.  What no rotation touches is equal
bit by bit (codes, scale bytes, untouched places); rotated keys are within the bound of
one fp32 rotation and half a step of the cache's type."""
import numpy as np
import pytest
import torch

from oracle import layer8 as O8

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
KINDS = ["bf16", "e4m3", "e4m3_blocks", "int8_blocks"]
STEP = {"e4m3": 2.0 ** -4, "bf16": 2.0 ** -8}       # half a step, relative


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Cache:
    """A pair of caches of one kind, their bytes random (codes of a finite value) and their scales too."""

    def __init__(self, kind, pages, heads, page, dim, seed=0, layout="phtd"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.shape, self.short = kind, (pages, heads, page, dim), kind.split("_")[0]
        rnd = lambda lo, hi, shape, dt: torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32).to(dt)  # noqa: E731
        self.k_scale = self.v_scale = None
        made = []
        for _ in range(2):
            shape = (pages, heads, page, dim) if layout == "phtd" else (pages, page, heads, dim)
            if kind == "bf16":
                x = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
            elif kind == "int8_blocks":
                x = rnd(-127, 128, shape, torch.int8)
            else:
                x = rnd(0, 0x7f, shape, torch.uint8) | (rnd(0, 2, shape, torch.uint8) << 7)
                x = x.view(FP8)
            if layout != "phtd":
                raw = x.view(torch.uint8) if x.element_size() == 1 else x
                x = raw.permute(0, 2, 1, 3).view(x.dtype)
            made.append(x)
        self.k, self.v = made
        if kind == "e4m3":
            self.k_scale, self.v_scale = (0.005 + 0.01 * torch.rand(heads, generator=g, device="cuda") for _ in range(2))
        if kind.endswith("blocks"):
            self.k_scale, self.v_scale = (rnd(116, 124, (pages, heads, page // 16), torch.uint8).view(E8M0) for _ in range(2))

    def raw(self):
        return [x.view(torch.uint8).cpu().numpy().copy() if x.element_size() == 1 else x.view(torch.int16).cpu().numpy().copy()
                for x in (self.k, self.v)]

    def scales(self):
        return [x.view(torch.uint8).cpu().numpy().copy() for x in (self.k_scale, self.v_scale)]


def run(lib, kind, slots, heads, dim, page, pages, hq=0, rot=0, layout="half", positions=None, seed=0, values=None, cache_layout="phtd",
        cache=None, scaling="none", factor=1.0):
    T = len(slots)
    c = cache or Cache(kind, pages, heads, page, dim, seed, cache_layout)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    qkv = torch.randn(T, (hq + 2 * heads) * dim + 8, generator=g, device="cuda")
    qkv = (qkv * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    if values is not None:
        qkv[:, :] = values(qkv)
    q, k, v = qkv[:, :hq * dim], qkv[:, hq * dim:(hq + heads) * dim], qkv[:, (hq + heads) * dim:(hq + 2 * heads) * dim]
    if positions is None:
        positions = np.arange(T) * 3 + 7
    pos = torch.tensor(np.asarray(positions), dtype=torch.int32, device="cuda")
    table = lib.rotary_table(rot, layout=layout, scaling=scaling, factor=factor) if rot else None
    before, sb = c.raw(), c.scales() if kind.endswith("blocks") else None
    got_q = lib.paged_kv_append(k, v, pos, torch.tensor(slots, dtype=torch.int64, device="cuda"), c.k, c.v, rotation=table,
                                k_scale=c.k_scale, v_scale=c.v_scale, q=q if hq else None)
    turn, amp = O8.turns(rot, scaling=scaling, factor=factor) if rot else (np.zeros(0), 1.0)
    turned = lambda x, n: O8.rotate(f64(x).reshape(T, n, dim), positions, turn, layout, amp)  # noqa: E731
    if hq:
        want, tol = turned(q, hq)
        off = np.abs(f64(got_q).reshape(want.shape) - want)
        tol = tol + STEP["bf16"] * (np.abs(want) + tol)
        tol[..., rot:] = 0
        assert (off <= tol).all()
    kept = [t for t, s in enumerate(slots) if 0 <= s < pages * page]
    at = np.array([slots[t] for t in kept], np.int64)
    for i, (x, is_k) in enumerate(((k, True), (v, False))):
        rows, tol = turned(x, heads) if is_k and rot else (f64(x).reshape(T, heads, dim), np.zeros((T, heads, dim)))
        after = c.raw()[i]
        if kind.endswith("blocks"):
            check_blocks(c, i, rows, tol, slots, before[i], sb[i], exact=not (is_k and rot))
            continue
        want = before[i].copy()
        mask = np.zeros(after.shape[:1] + after.shape[2:3], bool)
        mask[at // page, at % page] = True
        stays = ~mask[:, None, :, None] & np.ones(after.shape, bool)
        assert np.array_equal(after[stays], want[stays])
        got = (f64(c.k if is_k else c.v))[at // page, :, at % page]
        ref = rows[kept]
        if kind == "e4m3":
            # x / scale in fp32, one rounding more
            ref = np.clip(ref / f64(c.k_scale if is_k else c.v_scale)[:, None], -448, 448)
            err = tol[kept] / f64(c.k_scale if is_k else c.v_scale)[:, None] + 2.0 ** -23 * np.abs(ref)
            bound = err + np.maximum(STEP["e4m3"] * (np.abs(ref) + err), 2.0 ** -10)
        else:
            bound = tol[kept] + STEP["bf16"] * (np.abs(ref) + tol[kept])
            if not (is_k and rot):
                bound = np.zeros_like(ref)
            else:
                bound[..., rot:] = 0
        assert (np.abs(got - ref) <= bound).all()
    return c


def check_blocks(c, i, rows, tol, slots, raw, scales, exact):
    kind = c.short
    want, ws = O8.append(rows, slots, O8.code_values(raw, kind), scales, kind)
    got, gs = O8.code_values(c.raw()[i], kind), c.scales()[i]
    if exact:
        assert np.array_equal(gs, ws), np.argwhere(gs != ws)[:4]
        assert np.array_equal(got, want, equal_nan=True), np.argwhere(got != want)[:4]
        return
    # a rotated maximum may fall on the other side of a power of two: only by its own error
    assert (np.abs(gs.astype(int) - ws) <= 1).all() and (gs != ws).mean() < 0.02
    for b in np.argwhere(gs != ws):
        run = [t for t, s in enumerate(slots) if s // 16 == (b[0] * c.shape[2] + 16 * b[2]) // 16]
        top = np.abs(rows[run, b[1]]).max()
        edge = O8.MOST[kind] * 2.0 ** (min(int(gs[tuple(b)]), int(ws[tuple(b)])) - 127)
        assert abs(top - edge) <= 2 * tol[run, b[1]].max()
    same = np.repeat(gs == ws, 16, 2)
    step = np.repeat(2.0 ** (gs.astype(float) - 127), 16, 2)[..., None]
    pages, heads, page, dim = got.shape
    err = np.zeros_like(got)
    half = np.zeros_like(got)
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            err[s // page, :, s % page] = tol[t]
            half[s // page, :, s % page] = np.maximum(np.abs(rows[t]) * 2.0 ** -4, 2.0 ** -10 * step[s // page, :, s % page]) if kind == "e4m3" \
                else 0.5 * step[s // page, :, s % page]
    written = half > 0
    keep = same[..., None] & ~written
    assert np.array_equal(got[keep], want[keep], equal_nan=True)
    value = got * step
    target = np.zeros_like(got)
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            target[s // page, :, s % page] = rows[t]
    off = np.abs(value - target)[written]
    most = (half + err * (1 + 2.0 ** -4))[written]
    assert (off <= most).all(), "worst %.3g" % (off / most).max()
    # and nearly everywhere the oracle's own code: only ties within the rotation's error differ
    assert (got != want)[same[..., None] & written].mean() < 1e-3


def sequence(*parts, pad=()):
    """Slots of requests laid end to end: (first slot, count) each; then padding."""
    return [s + i for s, n in parts for i in range(n)] + list(pad)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot,layout", [(0, "half"), (64, "half"), (64, "interleaved"), (48, "half"), (16, "interleaved")])
def test_kinds_and_rotations(gpu_lib, kind, dim, rot, layout):
    slots = sequence((0, 5), (37, 1), (64, 40), (127 + 16, 17), pad=(-1, -1))
    run(gpu_lib, kind, slots, 2, dim, 32, 8, hq=6, rot=rot, layout=layout, seed=dim + rot)


@pytest.mark.parametrize("kind", ["e4m3_blocks", "int8_blocks"])
@pytest.mark.parametrize("first", [0, 1, 7, 14, 15, 16, 17, 31])
@pytest.mark.parametrize("count", [1, 2, 15, 16, 17, 33, 50])
def test_runs_begin_and_end_anywhere(gpu_lib, kind, first, count):
    run(gpu_lib, kind, sequence((first, count), (200 + first, 1)), 1, 64, 64, 6, rot=32, seed=first * 100 + count)
    run(gpu_lib, kind, sequence((first, count)), 3, 128, 16, 6, seed=first + count)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_pages_and_cache_layouts(gpu_lib, kind, page):
    order = np.random.default_rng(page).permutation(4 * page // 16)[:9] * 16   # blocks anywhere
    slots = sequence(*((int(s), 16) for s in order[:5]), *((int(s) + 3, 2) for s in order[5:]))
    run(gpu_lib, kind, slots, 2, 64, page, 4, hq=2, rot=64, seed=page, cache_layout="pthd")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 64, 300, 1500])
def test_single_tokens_of_many_requests(gpu_lib, kind, T):
    """Every row a run of its own, at any place of its block, padding among them."""
    rng = np.random.default_rng(T)
    slots = [int(b) * 16 + int(rng.integers(0, 16)) for b in rng.permutation(T + 5)[:T]]
    for t in range(3, T, 7):
        slots[t] = -1
    run(gpu_lib, kind, slots, 2, 64, 32, (T + 6) // 2 + 1, hq=4, rot=64, seed=T)


@pytest.mark.parametrize("kind", KINDS)
def test_a_long_prompt(gpu_lib, kind):
    run(gpu_lib, kind, sequence((5, 1000), (1040, 777)), 1, 64, 16, 120, rot=16, seed=9)


@pytest.mark.parametrize("kind", ["e4m3_blocks", "int8_blocks"])
def test_scales_rise_and_never_fall_within_a_block(gpu_lib, kind):
    """Token by token: equal to the oracle's steps, and a new first token begins the block anew."""
    c = Cache(kind, 2, 2, 16, 64, seed=3)
    size = [1.0, 0.01, 3.0, 100.0, 1e-6, 7.0, 100.0, 3e4]
    for i, f in enumerate(size):
        run(gpu_lib, kind, [16 + i], 2, 64, 16, 2, seed=i, cache=c, values=lambda x: x * f)
    high = c.scales()[0][1].max()
    run(gpu_lib, kind, [16 + 3], 2, 64, 16, 2, seed=50, cache=c, values=lambda x: x * 1e-3)     # a refused draft's place
    assert c.scales()[0][1].max() == high
    run(gpu_lib, kind, [16], 2, 64, 16, 2, seed=51, cache=c, values=lambda x: x * 1e-3)
    assert c.scales()[0][1].max() < high and (c.raw()[0][1, :, 1:] == 0).all()


@pytest.mark.parametrize("kind", ["e4m3_blocks", "int8_blocks"])
def test_edge_values(gpu_lib, kind):
    """Powers of two and the codes' largest multiples exactly, zeros, subnormals, the largest finite values."""
    most = O8.MOST[kind.split("_")[0]]
    for f in (0.0, 1.0, most, most * 2.0 ** -100, most * 2.0 ** 90, 2.0 ** -126, 2.0 ** -133, 2.0 ** -119, 3.3e38, most * 2.0 ** -118):
        run(gpu_lib, kind, [0, 1, 18], 1, 64, 16, 2, seed=1, values=lambda x: (torch.sign(x) * f).to(torch.bfloat16))
    # just above the border: the next power
    run(gpu_lib, kind, [0, 1], 1, 64, 16, 1, seed=1, values=lambda x: torch.full_like(x, 452.0 if most > 200 else 128.0))


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan(gpu_lib, kind):
    def values(x):
        x[1, ::5], x[2, 1::7], x[0, 3::9] = float("inf"), float("-inf"), float("nan")
        return x
    c = Cache(kind, 1, 2, 16, 64, seed=8)
    x = values(torch.randn(4, 128, device="cuda").to(torch.bfloat16))
    s = torch.arange(4, device="cuda")
    gpu_lib.paged_kv_append(x, x, s.int(), s, c.k, c.v, k_scale=c.k_scale, v_scale=c.v_scale)
    got, ref = f64(c.k)[0, :, :4].transpose(1, 0, 2).reshape(4, 128), f64(x)
    if kind == "int8_blocks":
        assert (got[np.isnan(ref)] == 0).all() and (got[np.isposinf(ref)] == 127).all() and (got[np.isneginf(ref)] == -127).all()
    elif kind == "bf16":
        assert np.array_equal(got, ref, equal_nan=True)
    else:
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and (got[np.isposinf(ref)] == 448).all() and (got[np.isneginf(ref)] == -448).all()
    if kind.endswith("blocks"):
        top = np.abs(np.where(np.isfinite(ref), ref, 0)).reshape(4, 2, 64).max((0, 2))
        assert c.scales()[0][0, :, 0].tolist() == [O8.scale_byte(t, kind.split("_")[0]) for t in top]


@pytest.mark.parametrize("kind", KINDS)
def test_slots_outside_the_cache_are_skipped(gpu_lib, kind):
    run(gpu_lib, kind, [-1, 3, 4, 64, 2 ** 40, -2 ** 60, 20, 21, 63, 65], 2, 64, 16, 4, hq=2, rot=32,
        positions=[-1, 3, 4, 64, 7, -3, 20, 21, 63, 65], seed=4)


@pytest.mark.parametrize("kind", KINDS)
def test_yarn_amplitude(gpu_lib, kind):
    run(gpu_lib, kind, sequence((3, 30)), 2, 128, 16, 4, hq=2, rot=64, scaling="yarn", factor=8.0, positions=np.arange(30) + 99000)


def test_q_in_place_and_without_rotation(gpu_lib):
    c = Cache("int8_blocks", 2, 2, 16, 64)
    y = torch.randn(6, 64 * 8, device="cuda").to(torch.bfloat16)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    slots = torch.arange(6, device="cuda")
    r = gpu_lib.rotary_table(64)
    want = gpu_lib.rotary(y[:, :256], pos, r, 64)
    kv = y[:, 256:].clone()
    q = gpu_lib.paged_kv_append(y[:, 256:384], y[:, 384:], pos, slots, c.k, c.v, rotation=r, k_scale=c.k_scale, v_scale=c.v_scale,
                                q=y[:, :256], q_out=y[:, :256])
    assert torch.equal(q, want) and torch.equal(y[:, 256:], kv)
    plain = gpu_lib.paged_kv_append(y[:, 256:384], y[:, 384:], None, slots, c.k, c.v, k_scale=c.k_scale, v_scale=c.v_scale, q=y[:, :256])
    assert torch.equal(plain, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_without_rotation_it_is_paged_kv_write(gpu_lib, kind):
    a, b = Cache(kind, 4, 2, 16, 128, seed=2), Cache(kind, 4, 2, 16, 128, seed=2)
    x = torch.randn(30, 512, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(64, device="cuda")[:30]
    kw = dict(k_scale=a.k_scale, v_scale=a.v_scale)
    gpu_lib.paged_kv_write(x[:, :256], x[:, 256:], slots, a.k, a.v, **kw)
    gpu_lib.paged_kv_append(x[:, :256], x[:, 256:], None, slots, b.k, b.v, **kw)
    for p, q in zip(a.raw(), b.raw()):
        assert np.array_equal(p, q)


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed(gpu_lib, kind):
    c, d = Cache(kind, 8, 2, 16, 64, seed=5), Cache(kind, 8, 2, 16, 64, seed=5)
    r = gpu_lib.rotary_table(32)
    x = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
    pos, slots = torch.arange(20, dtype=torch.int32, device="cuda"), torch.arange(20, device="cuda")
    q_out = torch.empty(20, 256, dtype=torch.bfloat16, device="cuda")
    def call(cache, out):  # noqa: E306
        gpu_lib.paged_kv_append(x[:, 256:384], x[:, 384:], pos, slots, cache.k, cache.v, rotation=r, k_scale=cache.k_scale,
                                v_scale=cache.v_scale, q=x[:, :256], q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, q_out)
    for i in range(4):
        x.copy_(torch.randn(20, 512, device="cuda") * 2.0 ** i)
        pos.add_(20)
        slots.add_(21)
        graph.replay()
        got = q_out.clone()
        eager = torch.empty_like(q_out)
        call(d, eager)
        assert torch.equal(got, eager)
        for p, q in zip(c.raw() + (c.scales() if kind.endswith("blocks") else []), d.raw() + (d.scales() if kind.endswith("blocks") else [])):
            assert np.array_equal(p, q)


def test_refusals(gpu_lib):
    E = gpu_lib.NVFP4Error
    c, b = Cache("e4m3_blocks", 2, 2, 16, 64), Cache("bf16", 2, 2, 16, 64)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    pos, s = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.arange(4, device="cuda")
    r = gpu_lib.rotary_table(64)
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    f = gpu_lib.paged_kv_append
    for call in (lambda: f(x, x, pos, s, c.k, c.v, k_scale=c.k_scale), lambda: f(x, x, pos, s, b.k, b.v, **kw),
                 lambda: f(x, x, pos, s, c.k, c.v, k_scale=c.k_scale[:1], v_scale=c.v_scale),
                 lambda: f(x, x, pos, s, c.k.view(torch.uint8), c.v.view(torch.uint8), **kw),
                 lambda: f(x, x, pos, s.int(), c.k, c.v, **kw), lambda: f(x, x, None, s, c.k, c.v, rotation=r, **kw),
                 lambda: f(x, x, pos, s, c.k, c.v, rotation=gpu_lib.rotary_table(128), **kw),
                 lambda: f(x, x[:3], pos, s, c.k, c.v, **kw), lambda: f(x, x, pos, s, c.k, c.v, q_out=x, **kw),
                 lambda: f(x, x, pos, s, c.k, c.v, q=x[:, :72], **kw), lambda: f(x, x, pos, s, c.k, c.v, q=x.clone(), q_out=x, **kw),
                 lambda: f(x, x, pos, s, b.k.to(torch.int8), b.v.to(torch.int8)),
                 lambda: f(x, x, pos, s, c.k, b.v, **kw)):
        with pytest.raises(E):
            call()
