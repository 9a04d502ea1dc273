"""The serving example with attention layers in 8 bits: the calls of a step together, each
against the float64 oracle on what the step itself handed it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layer8 as O8
from oracle import paged as OP

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")


@pytest.fixture(scope="module")
def serving(gpu_lib):
    spec = importlib.util.spec_from_file_location("paged_serving_layer8", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def small(serving, kind, **kw):
    return serving.Model(**{**dict(layers=2, hidden=256, hq=4, hkv=2, dim=64, ffn=256, vocab=512, pages=64, page=32, requests=3,
                                   max_seq=256, layer8=kind), **kw})


def f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def raw(x):
    return x.view(torch.uint8).cpu().numpy().copy()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_steps_agree_with_the_oracle_on_their_own_inputs(serving, kind):
    m = small(serving, kind)
    ctx, rng = [0, 0, 0], np.random.default_rng(0)
    turn, amp = O8.turns(32, scaling="yarn", factor=4.0, original=4096.0)
    for new in ([40, 1, 70], [1, 5, 1], [3, 0, 20], [1, 1, 1]):
        trace = []
        before = [{n: raw(b[n]) for n in ("k", "v", "k_scale", "v_scale")} for b in m.blocks]
        logits, plan = m.step(rng.integers(0, 512, sum(new)).tolist(), ctx, new, trace)
        table, slots, positions = m.table.cpu().numpy(), plan.slots.tolist(), plan.positions.tolist()
        assert plan.counts.tolist()[0] == sum(new) and plan.counts.tolist()[2] == 0
        for (q, k, v, a, turned), b, old in zip(trace, m.blocks, before):
            want, tol = O8.rotate(f64(q).reshape(-1, 4, 64), positions, turn, "half", amp)
            tol = tol + OP.U_BF16 * (np.abs(want) + tol)
            assert (np.abs(f64(turned).reshape(want.shape) - want) <= tol).all()
            # v's codes and scales are the oracle's; a key's code is next to the oracle's own at most, and nearly always it
            codes, scales = O8.append(f64(v).reshape(-1, 2, 64), slots, O8.code_values(old["v"], kind), old["v_scale"], kind)
            assert np.array_equal(raw(b["v_scale"]), scales) and np.array_equal(O8.code_values(raw(b["v"]), kind), codes)
            turned_k, ktol = O8.rotate(f64(k).reshape(-1, 2, 64), positions, turn, "half", amp)
            codes, scales = O8.append(turned_k, slots, O8.code_values(old["k"], kind), old["k_scale"], kind)
            got = O8.code_values(raw(b["k"]), kind)
            assert np.array_equal(raw(b["k_scale"]), scales)
            assert (got != codes).mean() < 1e-3
            step = np.maximum(np.abs(codes) * 2.0 ** -3, 2.0 ** -9) if kind == "e4m3" else 1.0
            assert (np.abs(got - codes) <= step).all()
            values = [O8.block_values(O8.code_values(raw(b[n]), kind), np.clip(raw(b[n + "_scale"]), 1, O8.MOST_BYTE[kind])) for n in "kv"]
            out, _, tol, _ = OP.attention(f64(turned), *values, table, plan.q_start.tolist(), plan.seq_lens.tolist(), 32, 4, 64 ** -0.5)
            tol = tol + OP.U_BF16 * (np.abs(out) + tol)
            assert (np.abs(f64(a).reshape(out.shape) - out) <= tol).all()
        assert torch.isfinite(logits.float()).all()
        m.take_pages(ctx, new, new)
        ctx = [c + n for c, n in zip(ctx, new)]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_padded_steps_agree_with_steps_of_their_own_size(serving, kind):
    """A row of a linear layer in int8 has its own scale, so padding changes nothing in it; NVFP4's share one."""
    rng = np.random.default_rng(3)
    models, ctx = [small(serving, kind), small(serving, kind)], [0, 0, 0]
    for new in ([40, 1, 70], [1, 5, 1], [2, 0, 1]):
        tokens, trace, plain = rng.integers(0, 512, sum(new)).tolist(), [], []
        want, plan = models[0].step(tokens, ctx, new, plain)
        got, padded = models[1].step(tokens, ctx, new, trace, rows=128)
        assert torch.equal(padded.slots[:sum(new)], plan.slots) and padded.slots[sum(new):].eq(-1).all()
        for q, k, v, a, turned in trace:
            assert all(x[sum(new):].eq(0).all() for x in (q, k, v, a, turned))
        for x, y in zip(trace[0], plain[0]):         # the first layer, before any NVFP4 one
            assert torch.equal(x[:sum(new)], y)
        off = (got[:sum(new)].float() - want.float()).norm() / want.float().norm()
        assert off < 0.05, off
        for m in models:
            m.take_pages(ctx, new, new)
        ctx = [c + n for c, n in zip(ctx, new)]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_generation_keeps_its_books(serving, kind):
    prompts = [[1, 2, 3, 4, 5] * 8, [7], [9, 8] * 5]
    runs = []
    for _ in range(2):
        m, log = small(serving, kind), []
        texts = serving.generate(m, prompts, 12, 3, 0.7, seed=5, log=log)
        assert all(len(t) == len(p) + 13 + sum(k[r] for k in log) for r, (t, p) in enumerate(zip(texts, prompts)))
        held = [pg for r, t in enumerate(texts) for pg in m.table[r, :-(-(len(t) - 1) // 32)].tolist()]
        assert sorted(held + m.free) == list(range(64))
        runs.append((texts, log))
    assert runs[0] == runs[1]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_layer_captured_and_replayed(serving, gpu_lib, kind):
    """The chain of one layer for a decode step, in a graph, over growing lengths: each replay equals the eager calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    R, hq, hkv, dim, page, hidden = 5, 4, 2, 64, 16, 256
    qkv = serving.Int8Linear((hq + 2 * hkv) * dim, hidden, g)
    o = serving.Int8Linear(hidden, hq * dim, g)
    rot = gpu_lib.rotary_table(dim, layout="interleaved")
    def cache():  # noqa: E306
        c = [torch.zeros(40, hkv, page, dim, device="cuda").to(torch.int8 if kind == "int8" else torch.float8_e4m3fn) for _ in range(2)]
        return c + [torch.zeros(40, hkv, page // 16, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2)]
    first, second = cache(), cache()
    table = torch.randperm(40, generator=g, device="cuda")[:R * 4].to(torch.int32).view(R, 4)
    x = torch.empty(R, hidden, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([0, 3, 15, 16, 30], dtype=torch.int32, device="cuda")
    slots, lens = torch.empty(R, dtype=torch.int64, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    start = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    ws = gpu_lib.paged_attention_workspace(R, R, hq, hkv, dim, 1, 64)

    def layer(c):
        y = qkv(x)
        q = gpu_lib.paged_kv_append(y[:, hq * dim:(hq + hkv) * dim], y[:, (hq + hkv) * dim:], pos, slots, *c[:2], rotation=rot,
                                    k_scale=c[2], v_scale=c[3], q=y[:, :hq * dim])
        return o(gpu_lib.paged_attention_blocks(q, *c, table, start, lens, 1, 64, workspace=ws))

    def inputs():
        x.copy_(torch.randn(R, hidden, generator=g, device="cuda"))
        slots.copy_(table.long().gather(1, (pos.long() // page)[:, None])[:, 0] * page + pos % page)
        lens.copy_(pos + 1)

    inputs()
    layer(first)
    layer(second)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(first)
    for _ in range(6):
        pos.add_(1)
        inputs()
        graph.replay()
        got = out.clone()
        want = layer(second)
        assert torch.equal(got, want)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, second))
