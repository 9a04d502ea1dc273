"""The serving example: the calls of a step together, each against the float64
oracle on what the step itself handed it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")


@pytest.fixture(scope="module")
def serving(gpu_lib):
    spec = importlib.util.spec_from_file_location("paged_serving", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def small(serving, **kw):
    return serving.Model(**{**dict(layers=2, hidden=256, hq=4, hkv=2, dim=64, ffn=256, vocab=512, pages=64, page=16, requests=3,
                                   max_seq=256), **kw})


def f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def test_steps_agree_with_the_oracle_on_their_own_inputs(serving):
    m = small(serving)
    ctx, rng = [0, 0, 0], np.random.default_rng(0)
    for new in ([40, 1, 70], [1, 5, 1], [3, 0, 20]):
        trace = []
        logits, plan = m.step(rng.integers(0, 512, sum(new)).tolist(), ctx, new, trace)
        table = m.table.cpu().numpy()
        assert plan.counts.tolist()[0] == sum(new) and plan.counts.tolist()[2] == 0
        assert plan.seq_lens.tolist() == [c + n for c, n in zip(ctx, new)]
        at = [(table[r, p // 16], p % 16) for r in range(3) for p in range(ctx[r], ctx[r] + new[r])]
        assert plan.slots[:sum(new)].tolist() == [pg * 16 + i for pg, i in at]
        for (q, k, v, a), b in zip(trace, m.blocks):
            for rows, cache, scale in ((k, b["k"], b["k_scale"]), (v, b["v"], b["v_scale"])):
                want = (rows.float().reshape(-1, 2, 64) / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                got = torch.stack([cache.view(torch.uint8)[int(pg), :, int(i)] for pg, i in at])
                assert torch.equal(got, want.view(torch.uint8))
            out, _, tol, _ = OP.attention(f64(q), f64(b["k"]), f64(b["v"]), table, plan.q_start.tolist(), plan.seq_lens.tolist(), 16, 4,
                                          64 ** -0.5, 0, f64(b["k_scale"]), f64(b["v_scale"]))
            tol = tol + OP.U_BF16 * (np.abs(out) + tol)
            assert (np.abs(f64(a).reshape(out.shape) - out) <= tol).all()
        assert torch.isfinite(logits.float()).all()
        m.take_pages(ctx, new, new)
        ctx = [c + n for c, n in zip(ctx, new)]


def test_padded_steps_agree_with_steps_of_their_own_size(serving):
    """Padding rows stay zero through every layer, and the live rows' logits are those of a step without padding: within the
    differences of kernels for other row counts, which bf16 roundings of the layers between pass on."""
    rng = np.random.default_rng(3)
    models, ctx = [small(serving), small(serving)], [0, 0, 0]
    for new in ([40, 1, 70], [1, 5, 1], [2, 0, 1]):
        tokens, trace = rng.integers(0, 512, sum(new)).tolist(), []
        want, plan = models[0].step(tokens, ctx, new)
        for _ in range(3):
            stale = torch.full((128, 4 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
            del stale
        got, padded = models[1].step(tokens, ctx, new, trace, rows=128)
        assert padded.counts.tolist() == plan.counts.tolist() and padded.slots[sum(new):].eq(-1).all()
        assert torch.equal(padded.slots[:sum(new)], plan.slots)
        for q, k, v, a in trace:
            assert all(x[sum(new):].eq(0).all() for x in (q, k, v, a))
        assert got[sum(new):].eq(0).all() and torch.isfinite(got.float()).all()
        off = (got[:sum(new)].float() - want.float()).norm() / want.float().norm()
        assert off < 0.05, off
        for m in models:
            m.take_pages(ctx, new, new)
        ctx = [c + n for c, n in zip(ctx, new)]


@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_generation_keeps_its_books(serving, temperature):
    """Pages are neither lost nor given twice, every step says at least one token a request, and a rerun says the same."""
    prompts = [[1, 2, 3, 4, 5] * 8, [7], [9, 8] * 5]
    runs = []
    for _ in range(2):
        m, log = small(serving), []
        texts = serving.generate(m, prompts, 12, 3, temperature, seed=5, log=log)
        assert all(len(t) == len(p) + 13 + sum(k[r] for k in log) for r, (t, p) in enumerate(zip(texts, prompts)))
        assert all(0 <= x < 512 for t in texts for x in t)
        held = [pg for r, t in enumerate(texts) for pg in m.table[r, :-(-(len(t) - 1) // 16)].tolist()]
        assert sorted(held + m.free) == list(range(64))
        runs.append((texts, log))
    assert runs[0] == runs[1]


def test_varied_steps_need_no_more_memory(serving):
    """Workspaces are the model's, whatever the sizes of its steps."""
    m, ctx, held = small(serving), [0, 0, 0], []
    for new in ([5, 1, 9], [40, 1, 1], [1, 1, 1], [2, 9, 17], [3, 0, 33]):
        m.step([1] * sum(new), ctx, new)
        m.take_pages(ctx, new, new)
        ctx = [c + n for c, n in zip(ctx, new)]
        torch.cuda.synchronize()
        held.append(torch.cuda.memory_allocated())
    assert held == held[:1] * len(held), held
