"""GPU parity of verify_drafts against the float64 oracle: tokens and counts
equal, log-probabilities within fp32 error; and the distribution of what it
emits."""
import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu


def build(R, K, V, drafts, f32, probs, temps, seed=0, pad=0):
    rng = np.random.default_rng(seed)
    n = np.asarray(drafts)
    rows = np.maximum(n, 0) + 1
    start = np.cumsum(rows) - rows
    N = int(rows.sum())
    logits = torch.tensor(rng.standard_normal((N, V + pad)) * 2.5, dtype=torch.float32 if f32 else torch.bfloat16)[:, :V]
    x = logits.float().numpy().astype(np.float64)
    q = np.zeros((R, K, V), np.float32)
    d = np.zeros((R, K), np.int64)
    for r in range(R):
        for i in range(K):
            z = x[min(start[r] + i, N - 1)] + rng.standard_normal(V) * 0.7
            e = np.exp(z - z.max())
            q[r, i] = e / e.sum()
            d[r, i] = rng.choice(V, p=q[r, i].astype(np.float64) / q[r, i].sum(dtype=np.float64)) if probs else z.argmax()
    return dict(logits=logits, row_start=start, num_drafts=n, draft_tokens=d, uniform=rng.random((R, K)).astype(np.float32),
                noise=rng.standard_exponential((R, V)).astype(np.float32) + np.float32(1e-30),
                draft_probs=q if probs else None, temperature=None if temps is None else np.asarray(temps, np.float32))


def run(lib, b):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda x: None if x is None else torch.tensor(x, device="cuda")  # noqa: E731
    base = b["logits"]
    dev = torch.empty_strided(base.shape, base.stride(), dtype=base.dtype, device="cuda")
    dev.copy_(base)
    out = lib.verify_drafts(dev, i32(b["row_start"]), i32(b["num_drafts"]), i32(b["draft_tokens"]).reshape(len(b["num_drafts"]), -1),
                            f32(b["uniform"]), f32(b["noise"]), draft_probs=f32(b["draft_probs"]), temperature=f32(b["temperature"]))
    return [x.cpu().numpy() for x in out]


def check(lib, b):
    got = run(lib, b)
    want = OP.verify(b["logits"].float().numpy(), b["row_start"], b["num_drafts"], b["draft_tokens"], b["uniform"], b["noise"],
                     b["draft_probs"], b["temperature"])
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    # x / T, its difference to the maximum and the logarithm: a few fp32 roundings of values up to 64, and the
    # sum's relative error (the exponential's argument up to 64 in fp32, and V terms in any order)
    V = b["logits"].shape[1]
    tol = 64 * 8 * OP.U32 + min(V, 4096) * OP.U32 + 1e-6 * np.abs(want[2])
    assert np.all(np.abs(got[2] - want[2]) <= tol), np.abs(got[2] - want[2]).max()
    for a, c in zip(got, run(lib, b)):
        np.testing.assert_array_equal(a, c)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 2047, 2048, 2049, 8191, 8192, 8193, 20001, 70003])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("probs", [False, True])
def test_vocabularies(gpu_lib, V, f32, probs):
    check(gpu_lib, build(4, 3, V, [3, 0, 2, 3], f32, probs, [1.0, 0.6, 1.7, 0.0], seed=V))


@pytest.mark.parametrize("K", [0, 1, 2, 8, 33, 255])
def test_draft_counts(gpu_lib, K):
    check(gpu_lib, build(3, K, 301, [K, K // 2, 0], True, K > 0, None, seed=K))


def test_many_requests(gpu_lib):
    rng = np.random.default_rng(3)
    check(gpu_lib, build(300, 4, 1003, rng.integers(-1, 5, 300), False, True, rng.choice([0.0, 0.7, 1.0, 1.3], 300), seed=3))


def test_strided_logits(gpu_lib):
    check(gpu_lib, build(3, 2, 999, [2, 1, 2], False, True, None, seed=5, pad=7))
    check(gpu_lib, build(3, 2, 999, [2, 1, 2], True, False, [0.0, 1.0, 0.5], seed=5, pad=2))


def test_masked_vocabulary(gpu_lib):
    """Words of probability 0, a single word left, none left, NaN logits, and the type's lowest value."""
    b = build(6, 2, 500, [2] * 6, True, True, [1.0, 0.0, 1.0, 0.0, 1.0, 0.8], seed=7)
    x = b["logits"]
    x[0:3, 100:] = -np.inf
    x[3:6, :] = -np.inf
    x[3:6, 77] = 3.0
    x[6:9, :] = -np.inf                            # nothing can be drawn
    x[9:12, :] = -np.inf
    x[12:15, 5:495] = np.nan
    x[15:18, 3:] = float(np.finfo(np.float32).min)
    check(gpu_lib, b)
    got = run(gpu_lib, b)
    assert got[0][2, 0] == -1 and got[0][3, 0] == -1 and got[1][2] == 0


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("probs", [False, True])
def test_extreme_temperatures(gpu_lib, f32, probs):
    """Down to the smallest positive number the largest logit has all the probability; up to the largest, every word has the same."""
    temps = [1e-30, 1.2e-38, 4.3e-39, 4e-39, 1e-39, 1e-44, 1e30, 3e38]
    b = build(8, 2, 777, [2] * 8, f32, probs, temps, seed=21)
    for r in range(8):
        b["draft_tokens"][r, 0] = int(b["logits"][b["row_start"][r]].float().argmax())   # kept where all is on the largest
    check(gpu_lib, b)


def test_a_nan_temperature_samples_nothing(gpu_lib):
    b = build(2, 1, 300, [1, 1], True, True, [float("nan"), 1.0], seed=22)
    tokens, kept, logprobs = run(gpu_lib, b)
    assert tokens[0].tolist() == [-1, -1] and kept[0] == 0 and logprobs[0].tolist() == [0, 0]
    assert tokens[1, 0] >= 0


def test_equal_maxima_and_equal_scores(gpu_lib):
    """Greedy ties and race ties go to the lowest index, also across lanes, waves and slices."""
    V = 40000
    b = build(4, 1, V, [0, 0, 1, 1], True, False, [0.0, 1.0, 0.0, 1.0], seed=9)
    b["logits"][:] = -3.0
    for row, words in ((0, (39999, 8192, 8191)), (2, (20000, 16))):
        for w in words:
            b["logits"][row, w] = 2.0
    b["noise"][1] = 1.0                            # all scores equal: word 0
    b["noise"][3] = 1.0
    b["draft_tokens"][2, 0], b["draft_tokens"][3, 0] = 16, 0
    b["uniform"][3, 0] = 0.9                       # refuses word 0: the next lowest
    check(gpu_lib, b)
    got = run(gpu_lib, b)[0]
    assert got[0, 0] == 8191 and got[1, 0] == 0 and got[2, 0] == 16 and got[3, 0] == 1


def test_draft_equal_to_target_and_bad_drafts(gpu_lib):
    """p == q: accepted whatever u is; a refused draft with p == q everywhere falls back to p; tokens outside are refused."""
    b = build(3, 2, 64, [2, 2, 2], True, True, None, seed=11)
    b["logits"][:] = 0.0
    b["draft_probs"][:] = np.float32(1 / 64)
    b["uniform"][:] = np.float32(1 - 2.0 ** -24)
    b["draft_tokens"][1, 0], b["draft_tokens"][2, 1] = 64, -5
    check(gpu_lib, b)
    assert run(gpu_lib, b)[1].tolist() == [2, 0, 1]


def test_rows_outside_the_logits_are_not_sampled(gpu_lib):
    b = build(3, 2, 100, [2, 2, 2], True, False, None, seed=12)
    b["row_start"] = np.array([-1, 3, 7])          # the last would need rows 7, 8, 9 of 9
    check(gpu_lib, b)
    assert run(gpu_lib, b)[0][2].tolist() == [-1, -1, -1]


def test_emitted_tokens_follow_the_target(gpu_lib):
    """The first token's frequencies over many requests are the target's, whatever the drafter proposes (chi-square)."""
    V, R = 12, 60000
    rng = np.random.default_rng(0)
    x = rng.standard_normal(V).astype(np.float32) * 1.5
    p = np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum()
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    b = dict(logits=torch.tensor(x).repeat(2 * R, 1), row_start=2 * np.arange(R), num_drafts=np.ones(R, int),
             draft_tokens=rng.choice(V, (R, 1), p=q.astype(np.float64) / q.sum(dtype=np.float64)),
             uniform=rng.random((R, 1)).astype(np.float32), noise=rng.standard_exponential((R, V)).astype(np.float32) + np.float32(1e-30),
             draft_probs=np.broadcast_to(q, (R, 1, V)).copy(), temperature=None)
    tokens = run(gpu_lib, b)[0][:, 0]
    count = np.bincount(tokens, minlength=V)
    chi2 = ((count - R * p) ** 2 / (R * p)).sum()
    assert chi2 < 40, chi2                         # 11 degrees of freedom: P(> 40) = 4e-5


def on_device(b):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda x: None if x is None else torch.tensor(x, device="cuda")  # noqa: E731
    return dict(logits=b["logits"].cuda(), row_start=i32(b["row_start"]), num_drafts=i32(b["num_drafts"]),
                draft_tokens=i32(b["draft_tokens"]), uniform=f32(b["uniform"]), noise=f32(b["noise"]),
                draft_probs=f32(b["draft_probs"]), temperature=f32(b["temperature"]))


def test_one_workspace_serves_calls_of_other_sizes(gpu_lib):
    """The counters that a call needs at zero are zero after every other one."""
    batches = [build(1, 0, 70003, [0], False, False, None), build(5, 3, 20001, [3, 0, 2, 1, 3], True, True, None, seed=1),
               build(40, 2, 900, [2, -1] * 20, False, True, [0.0, 0.8] * 20, seed=2), build(2, 8, 33000, [8, 5], False, False, [0.5, 0.0], seed=3)]
    sizes = [(*b["draft_tokens"].shape, b["logits"].shape[1]) for b in batches]
    shared = torch.full((max(gpu_lib.verify_drafts_workspace(*s).numel() for s in sizes),), 0x5a, dtype=torch.uint8, device="cuda")
    shared[:1 << 18] = 0
    want = [run(gpu_lib, b) for b in batches]
    dev = [on_device(b) for b in batches]
    for order in ([0, 1, 2, 3], [3, 1, 0, 2], [2, 2, 1, 1]):
        for i in order:
            for got, w in zip(gpu_lib.verify_drafts(workspace=shared, **dev[i]), want[i]):
                np.testing.assert_array_equal(got.cpu().numpy(), w)
            assert int(shared[:1 << 18].count_nonzero()) == 0


def test_other_streams_and_graphs(gpu_lib):
    """A call on a side stream, and a captured one replayed on new inputs with other work between."""
    b = build(3, 4, 20001, [4, 2, 0], False, True, [1.0, 0.0, 0.6], seed=4)
    want, d = run(gpu_lib, b), on_device(b)
    ws = gpu_lib.verify_drafts_workspace(3, 4, 20001)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu_lib.verify_drafts(workspace=ws, **d)
    torch.cuda.current_stream().wait_stream(side)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gpu_lib.verify_drafts(workspace=ws, **d)
    for drafts in ([0, 4, 1], [4, 4, -1], [1, 0, 3]):
        d["num_drafts"].copy_(torch.tensor(drafts, dtype=torch.int32))
        d["uniform"].mul_(0.7)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        for g, w in zip(got, gpu_lib.verify_drafts(**d)):
            assert torch.equal(g, w)
        torch.cuda.synchronize()


def test_refusals(gpu_lib):
    E = gpu_lib.NVFP4Error
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    ok = dict(logits=z(4, 32), row_start=i(2), num_drafts=i(2), draft_tokens=i(2, 1), uniform=z(2, 1), noise=z(2, 32) + 1)
    gpu_lib.verify_drafts(**ok)
    for bad in (dict(logits=z(4, 32, dtype=torch.float16)), dict(logits=z(32, 4).t()), dict(row_start=i(3)),
                dict(num_drafts=z(2, dtype=torch.int64)), dict(uniform=z(2, 2)), dict(noise=z(2, 31)), dict(draft_probs=z(2, 2, 32)),
                dict(temperature=z(3)), dict(workspace=z(4, dtype=torch.uint8)), dict(draft_tokens=i(2, 300), uniform=z(2, 300)),
                dict(logits=z(4, 32).cpu())):
        with pytest.raises(E):
            gpu_lib.verify_drafts(**{**ok, **bad})


def test_rows_further_on_go_by_row_start(gpu_lib):
    """A slice that does not begin 16-byte aligned is refused, and says so; the same rows by their numbers are not."""
    b = build(2, 2, 301, [2, 1], False, True, None, seed=8)
    d = on_device(b)
    want = gpu_lib.verify_drafts(**d)
    more = torch.zeros(d["logits"].shape[0] + 1, 301, dtype=torch.bfloat16, device="cuda")
    more[1:] = d["logits"]
    with pytest.raises(gpu_lib.NVFP4Error, match="align"):
        gpu_lib.verify_drafts(**{**d, "logits": more[1:]})
    for g, w in zip(gpu_lib.verify_drafts(**{**d, "logits": more, "row_start": d["row_start"] + 1}), want):
        assert torch.equal(g, w)
