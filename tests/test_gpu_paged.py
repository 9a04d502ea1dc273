"""GPU parity of paged_plan and paged_kv_write against the oracle: whole numbers
equal, cache values equal bit by bit (a copy, or one rounding to E4M3)."""
import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def run_plan(lib, ctx, new, free, cursor, table, page, max_tokens):
    t = i32(table).reshape(len(ctx), -1) if len(ctx) else torch.empty((0, 4), dtype=torch.int32, device="cuda")
    p = lib.paged_plan(i32(ctx), i32(new), i32(free), t, page, max_tokens,
                       free_cursor=None if cursor is None else i32([cursor]))
    return [x.cpu().numpy() for x in (t, p.q_start, p.seq_lens, p.positions, p.slots, p.counts)]


def check_plan(lib, ctx, new, free, cursor, table, page, max_tokens):
    got = run_plan(lib, ctx, new, free, cursor, table, page, max_tokens)
    want = OP.plan(np.asarray(ctx, np.int64), np.asarray(new, np.int64), free, cursor or 0, table, page, max_tokens)
    for g, w, name in zip(got, want, ("block_table", "q_start", "seq_lens", "positions", "slots", "counts")):
        np.testing.assert_array_equal(g, w, err_msg=name)


def context_table(ctx, pages, page, rng):
    """Pages 1000.. for the contexts, -7 in the unset columns (they must stay)."""
    t = np.full((len(ctx), pages), -7, np.int32)
    at = 1000
    for r, c in enumerate(ctx):
        for col in range(min(-(-max(c, 0) // page), pages)):
            t[r, col] = at = at + 1
    return t


@pytest.mark.parametrize("ctx,new,page,pages,cursor,spare", [
    ([0], [1], 16, 4, 0, 10),
    ([16], [1], 16, 4, 0, 10),                     # a page ends with the context
    ([15], [1], 16, 4, 3, 10),                     # the last place of a page: no page needed
    ([5, 0, 33, 7], [1, 0, 17, 40], 16, 8, 2, 20),  # a request without new tokens among others
    ([0, 0, 0], [0, 0, 0], 32, 4, 0, 4),           # nothing at all
    ([100, 3], [200, 1], 64, 3, 0, 9),             # runs past the table: no page, no slot
    ([10, 20, 30], [30, 30, 30], 16, 8, 1, 3),     # the free list runs out
    ([1024, 4096], [1024, 1], 1024, 8, 0, 4),      # the largest pages
    ([-3, 5], [2, -1], 16, 4, 0, 4),               # negative lengths count as none
])
def test_plan_small(gpu_lib, ctx, new, page, pages, cursor, spare):
    rng = np.random.default_rng(1)
    table = context_table(ctx, pages, page, rng)
    free = rng.permutation(500)[:spare].astype(np.int32)
    check_plan(gpu_lib, ctx, new, free, cursor, table, page, max(sum(max(n, 0) for n in new), 1) + 5)


@pytest.mark.parametrize("requests", [1, 255, 256, 257, 1000, 5000])
def test_plan_many_requests(gpu_lib, requests):
    rng = np.random.default_rng(requests)
    ctx, new = rng.integers(0, 300, requests), rng.integers(0, 40, requests)
    new[rng.random(requests) < 0.3] = 0
    table = context_table(ctx, 24, 16, rng)
    free = rng.permutation(int(new.sum()) + requests).astype(np.int32)[:int(new.sum()) // 16 + requests]
    check_plan(gpu_lib, ctx, new, free, 3, table, 16, int(new.sum()) + 1)


def test_plan_step_larger_than_its_buffers(gpu_lib):
    table = context_table([0, 9], 8, 16, None)
    check_plan(gpu_lib, [0, 9], [20, 30], np.arange(40, dtype=np.int32), 0, table, 16, 37)


def test_plan_without_requests_and_without_free_pages(gpu_lib):
    got = run_plan(gpu_lib, [], [], [], None, [], 16, 3)
    assert got[1].tolist() == [0] and got[3].tolist() == [-1] * 3 and got[4].tolist() == [-1] * 3
    assert got[5].tolist() == [0, 0, 0, 0]
    check_plan(gpu_lib, [4], [30], np.zeros(0, np.int32), None, context_table([4], 4, 16, None), 16, 30)


def test_plan_slots_past_32_bits(gpu_lib):
    """Page numbers near 2^31 in pages of 1024 tokens: slots near 2^41."""
    big = np.array([2 ** 31 - 1, 2 ** 31 - 2], np.int64).astype(np.int32)
    check_plan(gpu_lib, [0], [1500], big, 0, np.full((1, 2), -7, np.int32), 1024, 1500)


def test_plan_reuses_its_tensors_and_strided_tables(gpu_lib):
    wide = torch.full((3, 16), -7, dtype=torch.int32, device="cuda")
    table, ctx, new = wide[:, :6], i32([0, 0, 0]), i32([20, 1, 33])
    free = i32(np.arange(10, 30))
    p = gpu_lib.paged_plan(ctx, new, free, table, 16, 60)
    again = gpu_lib.paged_plan(ctx, new, free, table, 16, 60, plan=p)
    assert again is p and p.counts.tolist() == [54, 6, 0, 6]
    assert wide[:, 6:].eq(-7).all()
    assert table.tolist() == [[10, 11, -7, -7, -7, -7], [12, -7, -7, -7, -7, -7], [13, 14, 15, -7, -7, -7]]


@pytest.mark.parametrize("requests,spare", [(1, 3), (7, 0), (300, 40), (1500, 1000)])
def test_plan_carries_lengths_and_cursor_in_place(gpu_lib, requests, spare):
    """Steps whose contexts are the plan's own seq_lens and whose cursor is its own last count, against the oracle's
    steps: one workgroup and many, and steps that run out of pages."""
    rng = np.random.default_rng(requests)
    page, cols = 16, 12
    ctx, cursor = rng.integers(0, 60, requests), 2
    free = rng.permutation(4000).astype(np.int32)[:requests * 4]
    table = context_table(ctx, cols, page, rng)
    steps = [rng.integers(0, 3, requests), rng.integers(0, 33, requests), np.ones(requests, np.int64), rng.integers(0, 40, requests)]
    most = max(int(n.sum()) for n in steps) + spare
    dev, free_dev = i32(table), i32(free)
    plan = gpu_lib.paged_plan(i32(ctx), i32(steps[0]), free_dev, dev, page, most, free_cursor=i32([cursor]))
    for s, new in enumerate(steps):
        if s:
            gpu_lib.paged_plan(plan.seq_lens, i32(new), free_dev, dev, page, most, free_cursor=plan.counts[3:], plan=plan)
        want = OP.plan(ctx, new, free, cursor, table, page, most)
        for g, w, name in zip((dev, *plan), want, ("block_table", "q_start", "seq_lens", "positions", "slots", "counts")):
            np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg="step %d: %s" % (s, name))
        table, ctx, cursor = want[0], want[2], int(want[5][3])


def test_plan_in_place_in_a_graph(gpu_lib):
    """A captured step that carries its own lengths: every replay is the next step."""
    free, table, new = i32(np.arange(100, 400)), torch.full((3, 16), -1, dtype=torch.int32, device="cuda"), i32([1, 0, 5])
    plan = gpu_lib.paged_plan(i32([14, 3, 0]), new, free, table, 16, 8)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.paged_plan(plan.seq_lens, new, free, table, 16, 8, free_cursor=plan.counts[3:], plan=plan)
    own, want = table.clone(), plan._make(x.clone() for x in plan)
    for _ in range(9):
        graph.replay()
        want = gpu_lib.paged_plan(want.seq_lens.clone(), new, free, own, 16, 8, free_cursor=want.counts[3:].clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((table, *plan), (own, *want)))


def test_plan_refuses_other_inputs_inside_its_outputs(gpu_lib):
    new, free, table = i32([1, 2, 3]), i32(np.arange(9)), i32(np.full((3, 4), -1))
    plan = gpu_lib.paged_plan(i32([0, 0, 0]), new, free, table, 16, 9)
    for bad in (dict(ctx_lens=plan.q_start[:3]), dict(ctx_lens=plan.positions[2:5]), dict(new_lens=plan.seq_lens),
                dict(free_pages=plan.positions), dict(free_cursor=plan.seq_lens[:1]), dict(free_cursor=plan.q_start[3:]),
                dict(ctx_lens=plan.slots.view(torch.int32)[1:4])):
        with pytest.raises(gpu_lib.NVFP4Error):
            gpu_lib.paged_plan(**{**dict(ctx_lens=plan.seq_lens, new_lens=new, free_pages=free, block_table=table, page_size=16,
                                         max_tokens=9, plan=plan), **bad})
    gpu_lib.paged_plan(plan.seq_lens, new, free, table, 16, 9, plan=plan, free_cursor=plan.counts[3:])
    assert plan.seq_lens.tolist() == [2, 4, 6] and plan.q_start.tolist() == [0, 1, 3, 6]


def test_plan_stays_in_range_whatever_shares_memory(gpu_lib):
    """The C entry takes the caller's word that nothing else overlaps.  Where it does, the plan is wrong and its accesses
    are not: the guards around every output stay."""
    R, T, cols, rng = 700, 900, 6, np.random.default_rng(1)
    lib, guard = gpu_lib.load(), 64
    lens = torch.full((R + 9 + 2 * guard,), -77, dtype=torch.int32, device="cuda")
    lens[guard:-guard] = i32(rng.integers(0, 90, R + 9))
    wide = torch.full((R + 2, cols + 8), -77, dtype=torch.int32, device="cuda")
    free, new = i32(np.arange(R * 4)), i32(rng.integers(0, 3, R))
    out = torch.full((R + 1 + T + 4 + 4 * guard,), -77, dtype=torch.int32, device="cuda")
    slots = torch.full((T + 2 * guard,), -77, dtype=torch.int64, device="cuda")
    q0, p0, c0 = guard, 2 * guard + R + 1, 3 * guard + R + 1 + T
    at = lambda x, i: x.data_ptr() + x.element_size() * i  # noqa: E731
    rc = lib.paged_plan(at(lens, guard), new.data_ptr(), R, 16, free.data_ptr(), R * 4, None, at(wide, cols + 8), cols, cols + 8, at(out, q0),
                        at(lens, guard + 9), at(out, p0), at(slots, guard), T, at(out, c0), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    keep = torch.ones_like(out, dtype=torch.bool)
    for begin, n in ((q0, R + 1), (p0, T), (c0, 4)):
        keep[begin:begin + n] = False
    assert out[keep].eq(-77).all() and slots[:guard].eq(-77).all() and slots[-guard:].eq(-77).all()
    assert lens[:guard].eq(-77).all() and lens[-guard:].eq(-77).all()
    assert wide[0].eq(-77).all() and wide[-1].eq(-77).all() and wide[:, cols:].eq(-77).all()


# --------------------------------------------------------------- K/V write --

FP8 = torch.float8_e4m3fn


def e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(FP8).float().numpy().astype(np.float64)


def to_e4m3(x):
    """Round to nearest even of clamped float64 values of float32 operands, by distance over the table of all values."""
    v = e4m3_values()
    order = np.argsort(v[:127])                    # 0 .. 448
    grid, codes = v[:127][order], np.arange(127)[order]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (codes[hi] % 2 == 0))
    c = np.where(up, codes[hi], codes[lo]).astype(np.uint8)
    return np.where(np.signbit(x), c | 0x80, c).astype(np.uint8)


@pytest.mark.parametrize("tokens,heads,dim,page,fp8,layout", [
    (1, 8, 128, 16, False, "phtd"), (1, 8, 128, 16, True, "phtd"), (37, 1, 64, 16, True, "pthd"),
    (130, 4, 256, 64, False, "pthd"), (65, 3, 64, 32, False, "phtd"), (300, 2, 256, 1024, True, "phtd"),
    (7, 40, 128, 128, True, "pthd"),
])
def test_kv_write(gpu_lib, tokens, heads, dim, page, fp8, layout):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    pages = -(-tokens // page) + 2
    qkv = torch.randn(tokens, heads * dim * 3 + 8, generator=g, device="cuda").mul(3).to(torch.bfloat16)
    k, v = qkv[:, 8:8 + heads * dim], qkv[:, 8 + heads * dim:8 + 2 * heads * dim]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    if tokens > 3:
        slots[1], slots[2], slots[3] = -1, pages * page, -2 ** 40      # padding, past the end, nonsense: skipped
    dtype = FP8 if fp8 else torch.bfloat16
    ks, vs = (0.5 + torch.rand(heads, generator=g, device="cuda") for _ in range(2)) if fp8 else (None, None)
    if fp8:
        ks[0] = 1e-3                               # exceeds the scale: saturates at 448
    raw = torch.uint8 if fp8 else torch.int16
    before = torch.randint(0, 100, (2, pages, heads, page, dim), generator=g, device="cuda").to(raw)
    if layout == "pthd":
        store = before.permute(0, 1, 3, 2, 4).contiguous()
        caches = store.permute(0, 1, 3, 2, 4)
    else:
        caches = before.clone()
    gpu_lib.paged_kv_write(k, v, slots, caches[0].view(dtype), caches[1].view(dtype), k_scale=ks, v_scale=vs)
    for x, cache, scale, old in ((k, caches[0], ks, before[0]), (v, caches[1], vs, before[1])):
        want = old.cpu().numpy().copy()
        xs = x.float().cpu().numpy()
        for t, slot in enumerate(slots.tolist()):
            if not 0 <= slot < pages * page:
                continue
            row = xs[t].reshape(heads, dim)
            if fp8:                                # one fp32 division, then one rounding
                row = to_e4m3(np.clip(row / scale.cpu().numpy()[:, None], np.float32(-448), np.float32(448)).astype(np.float64))
            else:
                row = x[t].view(torch.int16).cpu().numpy().reshape(heads, dim)
            want[slot // page, :, slot % page] = row
        np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_kv_write_rounds_every_step_to_nearest_even(gpu_lib):
    """Every midpoint between neighbouring E4M3 values, and both sides of it in bf16 steps."""
    v = np.sort(e4m3_values()[:127])
    mid = np.concatenate([v, (v[1:] + v[:-1]) / 2, [464.0, 1e4, 3e38]]).astype(np.float32)
    t = torch.tensor(np.concatenate([mid, -mid])).to(torch.bfloat16)
    bits = t.view(torch.int16).int()
    x = torch.cat([bits, (bits + 1).clamp(-32768, 32767), bits - 1]).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())]
    n = -(-x.numel() // 64)
    rows = torch.zeros(n * 64, dtype=torch.bfloat16)
    rows[:x.numel()] = x
    rows = rows.view(n, 64).cuda()
    cache = torch.zeros(2, -(-n // 16), 1, 16, 64, dtype=torch.uint8, device="cuda")
    gpu_lib.paged_kv_write(rows, rows, torch.arange(n, device="cuda"), cache[0].view(FP8), cache[1].view(FP8))
    want = to_e4m3(np.clip(rows.float().cpu().numpy().astype(np.float64), -448, 448))
    got = cache[0].reshape(-1, 64)[:n].cpu().numpy()
    np.testing.assert_array_equal(got, want)
    assert torch.equal(cache[0], cache[1])


def test_kv_write_infinities_and_nan(gpu_lib):
    """In E4M3 a NaN stays one, an infinity saturates (there is none), also where a scale of 0 or infinity makes them."""
    x = torch.tensor([float("nan"), float("-nan"), float("inf"), float("-inf"), 0.0, -0.0, 1.0, -3e38], dtype=torch.bfloat16)
    bits = x.view(torch.int16).clone()
    bits[1] = -1                                   # every bit set
    x = bits.view(torch.bfloat16).repeat(1, 32)    # one row of four heads of 64
    scales = torch.tensor([1.0, 0.0, float("inf"), -0.5], device="cuda")
    cache = torch.zeros(2, 1, 4, 16, 64, dtype=torch.uint8, device="cuda")
    gpu_lib.paged_kv_write(x.cuda(), x.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), cache[0].view(FP8), cache[1].view(FP8),
                           k_scale=scales, v_scale=scales)
    want = (x.float().view(4, 64) / scales.cpu()[:, None]).numpy()
    got = cache[0, 0, :, 0].cpu().view(FP8).float().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    keep = ~np.isnan(want)
    np.testing.assert_array_equal(cache[0, 0, :, 0].cpu().numpy()[keep], to_e4m3(np.clip(want[keep].astype(np.float64), -448, 448)))
    assert torch.equal(cache[0], cache[1])


def test_kv_write_far_pages(gpu_lib):
    """A cache of more than 2^32 bytes: the last page's offset passes 32 bits."""
    pages, heads, page, dim = 70000, 2, 128, 128
    store = torch.zeros(pages * heads * page * dim, dtype=torch.bfloat16, device="cuda")
    cache = store.view(pages, heads, page, dim)
    assert store.numel() * 2 > 2 ** 32
    x = torch.randn(3, heads * dim, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 0, (pages - 2) * page + 5], device="cuda")
    gpu_lib.paged_kv_write(x, x, slots, cache, cache)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(cache[s // page, :, s % page], x[t].view(heads, dim))
    assert int(store.ne(0).sum()) == int(x.ne(0).sum())


def test_plan_and_write_in_a_graph(gpu_lib):
    """A captured plan and write, replayed on new lengths with other work between, against the eager calls."""
    R, page, T = 3, 16, 40
    ctx, new, free = i32([5, 16, 0]), i32([1, 3, 20]), i32(np.arange(20)[::-1].copy())
    held = 20 + torch.arange(R * 6, dtype=torch.int32, device="cuda").reshape(R, 6)   # contexts' pages: no slot twice
    table = held.clone()
    k, v = (torch.randn(T, 2 * 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    caches = [torch.zeros(20 + R * 6, 2, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan = gpu_lib.paged_plan(ctx, new, free, table, page, T)

    def step():
        gpu_lib.paged_plan(ctx, new, free, table, page, T, plan=plan)
        gpu_lib.paged_kv_write(k, v, plan.slots, *caches)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c, n in (([0, 0, 0], [1, 1, 1]), ([40, 3, 31], [0, 30, 2]), ([16, 15, 17], [5, 1, 34])):
        ctx.copy_(i32(c)), new.copy_(i32(n))
        seen = []
        for call in (graph.replay, step):
            table.copy_(held)
            for x in (*plan, *caches):
                x.zero_()
            call()
            torch.cuda.synchronize()
            seen.append([x.clone() for x in (*plan, table, *caches)])
        assert all(torch.equal(a, b) for a, b in zip(*seen))


def test_refusals(gpu_lib):
    E = gpu_lib.NVFP4Error
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    k, slots = z(4, 256), z(4, dtype=torch.int64)
    good = z(2, 2, 16, 128)
    gpu_lib.paged_kv_write(k, k, slots[:4] + torch.arange(4, device="cuda"), good, good.clone())
    for bad in (z(2, 2, 24, 128), z(2, 2, 16, 96), z(2, 4, 16, 64).transpose(2, 3), z(2, 2, 16, 128, dtype=torch.float16)):
        with pytest.raises(E):
            gpu_lib.paged_kv_write(z(4, bad.shape[1] * bad.shape[3]), z(4, bad.shape[1] * bad.shape[3]), slots, bad, bad)
    with pytest.raises(E):
        gpu_lib.paged_kv_write(k.float(), k, slots, good, good)
    with pytest.raises(E):
        gpu_lib.paged_kv_write(k, k[:3], slots, good, good)
    with pytest.raises(E):
        gpu_lib.paged_kv_write(k, k, slots.int(), good, good)
    with pytest.raises(E):
        gpu_lib.paged_kv_write(k, k, slots, good, good, k_scale=z(2, dtype=torch.float32))   # a scale without an FP8 cache
    with pytest.raises(E):
        gpu_lib.paged_kv_write(k.cpu(), k, slots, good, good)
    with pytest.raises(E):
        gpu_lib.paged_kv_write(z(4, 260)[:, 4:], k, slots, good, good)                       # not 16-byte aligned
    lens, table = z(2, dtype=torch.int32), z(2, 4, dtype=torch.int32)
    for bad in (dict(page_size=24), dict(page_size=8), dict(page_size=2048), dict(max_tokens=-1)):
        with pytest.raises((E, RuntimeError)):
            gpu_lib.paged_plan(lens, lens, lens, table, **{**dict(page_size=16, max_tokens=4), **bad})
    with pytest.raises(E):
        gpu_lib.paged_plan(lens.long(), lens, lens, table, 16, 4)
    with pytest.raises(E):
        gpu_lib.paged_plan(lens, z(3, dtype=torch.int32), lens, table, 16, 4)
