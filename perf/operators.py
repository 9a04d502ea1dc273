"""The paged serving step's operators as measured cases: paged_plan, paged_kv_write, paged_attention and verify_drafts.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) where ``own`` is false, and calls
the library where it is true.  Lengths of ragged batches follow from the case alone, values from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
GOLDEN = 0.6180339887498949
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases ----

def listed():
    plan = dict(op="plan", page=16)
    write = dict(op="write")
    attn = dict(op="attention", ragged=False, window=0, fp8=False)
    ver = dict(op="verify", probs=True, f32=False, greedy=False)
    return [
        # a decode step of a few requests: one token each, a page now and then; latency
        dict(plan, name="plan_decode_8", requests=8, new=1, context=5000, max_pages=512),
        # a step of a loaded server: many requests, prompt chunks among single tokens
        dict(plan, name="plan_mixed_1024", requests=1024, new=64, context=30000, max_pages=2048),
        # the new K/V rows of a decode batch, 8 KV heads of 128
        dict(write, name="write_decode_64_bf16", tokens=64, hkv=8, dim=128, page=16, fp8=False),
        # a prompt chunk into an FP8 cache with calibrated scales
        dict(write, name="write_prompt_16k_fp8", tokens=16384, hkv=8, dim=128, page=64, fp8=True),
        # one request being generated: 5120 hidden columns as 40 heads of 128, groups of 5; latency
        dict(attn, name="attn_decode_one", requests=1, new=1, context=1000, hq=40, hkv=8, dim=128, page=16),
        # a full decode batch of ragged lengths: the HBM-bound heart of serving
        dict(attn, name="attn_decode_64", requests=64, new=1, context=16384, ragged=True, hq=40, hkv=8, dim=128, page=16),
        # four drafts and the last token of 32 requests over an FP8 cache, heads of 256
        dict(attn, name="attn_drafts_32_fp8", requests=32, new=5, context=8192, hq=24, hkv=4, dim=256, page=64, fp8=True),
        # prompt chunks of ragged lengths over ragged contexts, a sliding window, heads of 64 without groups
        dict(attn, name="attn_chunks_8_window", requests=8, new=777, context=6000, ragged=True, hq=16, hkv=16, dim=64,
             page=32, window=2000),
        # a long prompt's second half: matrix-bound
        dict(attn, name="attn_prompt_8k", requests=1, new=8192, context=8192, hq=40, hkv=8, dim=128, page=64),
        # one request, three drafts, a small vocabulary; latency
        dict(ver, name="verify_one", requests=1, drafts=3, vocab=32768),
        # a decode batch with four drafts each and the drafter's probabilities
        dict(ver, name="verify_64", requests=64, drafts=4, vocab=131072),
        # greedy requests among sampled ones, a drafter without probabilities, fp32 logits, an odd vocabulary
        dict(ver, name="verify_7_odd", requests=7, drafts=7, vocab=100003, probs=False, f32=True, greedy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "write", "attention", "attention", "verify"))
    if op == "plan":
        page = rng.choice((16, 32, 64, 128))
        context = _log(rng, 1, 30000)
        new = _log(rng, 1, 64)
        return dict(op=op, requests=_log(rng, 1, 1024), new=new, context=context, page=page,
                    max_pages=-(-(context + new) // page) + rng.randrange(8))
    if op == "write":
        hkv, dim = rng.choice(((8, 128), (4, 256), (16, 64), (1, 128), (2, 256)))
        return dict(op=op, tokens=_log(rng, 1, 16384 * 1024 // (hkv * dim)), hkv=hkv, dim=dim,
                    page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
    if op == "attention":
        hkv, group, dim = rng.choice(((8, 5, 128), (4, 6, 256), (16, 1, 64), (1, 16, 128), (2, 7, 128), (3, 8, 64)))
        new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 9, 2048)))
        context = _log(rng, 1, 16384)
        keys = 64 * 8192 * 8 * 128                  # the decode batch's K elements, about
        pairs = 40 * 8192 * 8192                    # half of the long prompt's padded scores
        most = min(keys // ((context + new) * hkv * dim), pairs // (hkv * group * new * (context + new)), 64)
        return dict(op=op, requests=_log(rng, 1, max(1, most)), new=new, context=context, ragged=rng.random() < 0.5,
                    hq=hkv * group, hkv=hkv, dim=dim, page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5,
                    window=rng.choice((0, 0, _log(rng, 1, 4096))))
    vocab, drafts = _log(rng, 1000, 131072), rng.randint(1, 8)
    return dict(op=op, requests=_log(rng, 1, max(1, min(64, 64 * 5 * 131072 // ((drafts + 1) * vocab)))), drafts=drafts,
                vocab=vocab, probs=rng.random() < 0.5, f32=rng.random() < 0.3, greedy=rng.random() < 0.5)


def _spread(most, count, step):
    """`count` lengths in 1 .. most, evenly spread in a fixed order; the first is `most`."""
    return [most if r == 0 else 1 + int(most * ((r * step) % 1.0)) for r in range(count)]


def _lens(c):
    """(context, new) of every request."""
    R = c["requests"]
    if c["op"] == "plan":
        ctx = [n - 1 for n in _spread(c["context"], R, GOLDEN)]
        # every eighth request is in its prompt and brings a chunk, the others bring one token
        return ctx, [n if r % 8 == 0 else 1 for r, n in enumerate(_spread(c["new"], R, math.sqrt(2)))]
    if not c["ragged"]:
        return [c["context"]] * R, [c["new"]] * R
    return [n - 1 for n in _spread(c["context"], R, GOLDEN)], _spread(c["new"], R, math.sqrt(2))


def _drafts(c):
    """Drafts of every request: mostly the full count, every third fewer, one in nine none."""
    return [0 if r % 9 == 4 else c["drafts"] - (c["drafts"] // 2 if r % 3 == 2 else 0) for r in range(c["requests"])]


def _pairs(ctx, new, window):
    """Visible (row, key) pairs of one head."""
    total = 0
    for c, n in zip(ctx, new):
        full = n * c + n * (n + 1) // 2
        if window:
            over = max(0, c + n - window)           # rows whose window leaves keys out: they leave over, over - 1, ...
            rows = min(n, over)
            full -= rows * over - rows * (rows - 1) // 2
        total += full
    return total


def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new = _lens(c)
        pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(ctx, new))
        touched = sum(-(-(a + b) // c["page"]) - a // c["page"] for a, b in zip(ctx, new))
        return {"bytes": 16 * len(ctx) + 12 * sum(new) + 8 * pages + 4 * touched, "flops": 0}
    if c["op"] == "write":
        return {"bytes": c["tokens"] * (2 * c["hkv"] * c["dim"] * (2 + (1 if c["fp8"] else 2)) + 8), "flops": 0}
    if c["op"] == "attention":
        ctx, new = _lens(c)
        seen = sum(min(a + b, c["window"] + b - 1) if c["window"] else a + b for a, b in zip(ctx, new))
        cache = 2 * seen * c["hkv"] * c["dim"] * (1 if c["fp8"] else 2)
        return {"bytes": cache + sum(new) * c["hq"] * (4 * c["dim"] + 4),
                "flops": 4 * c["dim"] * c["hq"] * _pairs(ctx, new, c["window"])}
    rows = sum(_drafts(c)) + c["requests"]
    return {"bytes": rows * c["vocab"] * (4 if c["f32"] else 2) + c["requests"] * c["vocab"] * (8 if c["probs"] else 4),
            "flops": 4 * rows * c["vocab"]}


# ----------------------------------------------------------------- inputs ----

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    if c["op"] == "plan":
        ctx, new = _lens(c)
        R, P, MP = c["requests"], c["page"], c["max_pages"]
        pool = torch.randperm(R * MP + 64, generator=g, device=DEV, dtype=torch.int32)
        s["ctx"], s["new"] = _ints(ctx), _ints(new)
        held = (s["ctx"][:, None] + P - 1) // P > torch.arange(MP, device=DEV)[None]
        s["table"] = torch.where(held, pool[:R * MP].view(R, MP), -1)       # the contexts' pages; the rest unset
        s["free"] = torch.cat([pool[R * MP:], pool[:R * MP].view(R, MP)[~held]])[:sum(new) + R].contiguous()
        s["cursor"] = _ints([0])
        s["max_tokens"] = sum(new) + 3                                      # a fixed-size step's padding
    elif c["op"] == "write":
        T, H, D, P = c["tokens"], c["hkv"], c["dim"], c["page"]
        qkv = randn(T, 4 * H * D)                                           # the fused projection's output: q (2 H D) | k | v
        s["k"], s["v"] = qkv[:, 2 * H * D:3 * H * D], qkv[:, 3 * H * D:]
        pages = -(-T // P) + 8
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        s["slots"] = order[t // P] * P + t % P
        s["slots"][T // 2] = -1                                             # a padding token
        dtype = FP8 if c["fp8"] else torch.bfloat16
        s["k_cache"] = torch.zeros(pages, H, P, D, device=DEV, dtype=torch.bfloat16).to(dtype)
        s["v_cache"] = s["k_cache"].clone()
        s["k_scale"] = (0.01 + 0.01 * rand(H)) if c["fp8"] else None
        s["v_scale"] = (0.01 + 0.01 * rand(H)) if c["fp8"] else None
    elif c["op"] == "attention":
        ctx, new = _lens(c)
        R, H, D, P = c["requests"], c["hkv"], c["dim"], c["page"]
        T = sum(new)
        lens = [a + b for a, b in zip(ctx, new)]
        need = [-(-n // P) for n in lens]
        pages = sum(need) + 8
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
        MP = max(need)
        first = [sum(need[:r]) for r in range(R)]
        col = torch.arange(MP, device=DEV)[None]
        held = col < _ints(need)[:, None]
        s["table"] = torch.where(held, order[(_ints(first)[:, None] + col).clamp(max=pages - 1)], -1).to(torch.int32)
        s["q"] = randn(T, c["hq"] * D)
        k, v = randn(pages, H, P, D), randn(pages, H, P, D)
        if c["fp8"]:                                                        # values over the whole E4M3 range, as calibrated
            s["k_scale"], s["v_scale"] = 0.01 + 0.01 * rand(H), 0.01 + 0.01 * rand(H)
            k = (k.float() / s["k_scale"][:, None, None]).clamp(-448, 448).to(FP8)
            v = (v.float() / s["v_scale"][:, None, None]).clamp(-448, 448).to(FP8)
        else:
            s["k_scale"] = s["v_scale"] = None
        s["k_cache"], s["v_cache"] = k, v
        s["q_start"] = _ints([sum(new[:r]) for r in range(R + 1)])
        s["seq_lens"] = _ints(lens)
        s["scale"] = 1.5 / math.sqrt(D)
    else:
        R, K, V = c["requests"], c["drafts"], c["vocab"]
        drafts = _drafts(c)
        N = sum(drafts) + R
        s["row_start"] = _ints([sum(drafts[:r]) + r for r in range(R)])
        s["num_drafts"] = _ints(drafts)
        logits = 2.5 * randn(N, V, dtype=torch.float32)
        # one row's draft distribution is a disturbed copy of the target's
        at = (s["row_start"][:, None] + torch.arange(K, device=DEV)[None]).clamp(max=N - 1)
        near = logits[at] + 0.7 * randn(R, K, V, dtype=torch.float32)
        probs = torch.softmax(near, -1)
        race = probs / -torch.log(rand(R, K, V).clamp(1e-7, 1 - 1e-7))
        s["draft_tokens"] = (race if c["probs"] else near).argmax(-1).to(torch.int32)
        s["draft_probs"] = probs if c["probs"] else None
        s["logits"] = logits if c["f32"] else logits.to(torch.bfloat16)
        s["temperature"] = torch.where(torch.arange(R, device=DEV) % 2 == (0 if c["greedy"] else 2), 0.0, 0.7 + 0.6 * rand(R))
        s["uniform"] = rand(R, K)
        s["noise"] = -torch.log(1 - rand(R, V).clamp(max=1 - 2 ** -24)).clamp(min=1e-30)
    return s


# -------------------------------------------------------------- operators ----

def _plain_plan(s):
    P, MP, T = s["case"]["page"], s["case"]["max_pages"], s["max_tokens"]
    ctx, new, free, F = s["ctx"].clamp(min=0), s["new"].clamp(min=0), s["free"], s["free"].numel()
    end = torch.cumsum(new, 0, dtype=torch.int32)
    q_start = torch.cat([torch.zeros_like(end[:1]), end])
    seq = ctx + new
    before, after = ((ctx + P - 1) // P).clamp(max=MP), ((seq + P - 1) // P).clamp(max=MP)
    need = after - before
    off = torch.cumsum(need, 0, dtype=torch.int32) - need + s["cursor"]
    col = torch.arange(MP, device=DEV, dtype=torch.int32)[None]
    at = off[:, None] + col - before[:, None]
    page = torch.where(at < F, free[at.clamp(0, F - 1)], -1)
    s["table"].copy_(torch.where((col >= before[:, None]) & (col < after[:, None]), page, s["table"]))
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    r = torch.searchsorted(end, t, right=True, out_int32=True).clamp(max=end.numel() - 1)
    live = t < end[-1]
    pos = torch.where(live, ctx[r] + t - q_start[r], -1)
    c = pos.clamp(min=0) // P
    page = torch.where(live & (c < MP), s["table"][r, c.clamp(max=MP - 1)], -1).to(torch.int64)
    slots = torch.where(page >= 0, page * P + pos % P, -1)
    total = need.sum(dtype=torch.int32)
    taken = torch.minimum(total, (F - s["cursor"][0]).clamp(min=0))
    counts = torch.stack([end[-1], taken, total - taken, s["cursor"][0] + taken]).to(torch.int32)
    return s["table"], q_start, seq, pos, slots, counts


def _plain_write(s):
    H, D, P = (s["case"][n] for n in ("hkv", "dim", "page"))
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        rows = x.reshape(-1, H, D)[keep]
        if scale is not None:
            rows = (rows.float() / scale[:, None]).clamp(-448, 448).to(FP8)
        raw = torch.uint8 if scale is not None else torch.bfloat16          # indexing has no FP8 form
        cache.view(raw)[slots // P, :, slots % P] = rows.view(raw)
    return s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    R, HQ, H, D, P, W = (c[n] for n in ("requests", "hq", "hkv", "dim", "page", "window"))
    G, T, N, L = HQ // H, s["q"].shape[0], c["new"], s["table"].shape[1] * P
    start, lens = s["q_start"].to(torch.int64), s["seq_lens"].to(torch.int64)
    new = start[1:] - start[:-1]

    def keys(cache, scale):                        # [R, H, L, D]
        raw = cache.view(torch.uint8) if c["fp8"] else cache
        x = raw[s["table"].clamp(min=0).long()]    # [R, pages, H, P, D]
        x = (x.view(FP8) if c["fp8"] else x).float()
        x = x.permute(0, 2, 1, 3, 4).reshape(R, H, L, D)
        return x if scale is None else x * scale[:, None, None]

    i = torch.arange(N, device=DEV)
    row = (start[:-1, None] + i).clamp(max=T - 1)                           # [R, N]
    q = s["q"].float().view(T, H, G, D)[row].permute(0, 2, 1, 3, 4).reshape(R, H, N * G, D)
    x = torch.matmul(q * s["scale"], keys(s["k_cache"], s["k_scale"]).transpose(-1, -2).contiguous()).view(R, H, N, G, L)
    pos = (lens - new)[:, None] + i                                         # [R, N]
    j = torch.arange(L, device=DEV)
    seen = j <= pos[:, :, None]
    if W:
        seen = seen & (j > pos[:, :, None] - W)
    x = x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(R, H, N * G, L), keys(s["v_cache"], s["v_scale"])).view(R, H, N, G, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 2, 1, 3, 4).reshape(R, N, HQ * D)
    lse = (m + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(R, N, HQ)
    live = i < new[:, None]
    return o[live].to(torch.bfloat16), lse[live]


def _plain_verify(s):
    K, V = s["case"]["drafts"], s["case"]["vocab"]
    N = s["logits"].shape[0]
    n, d = s["num_drafts"][:, None], s["draft_tokens"].long()               # [R, 1], [R, K]
    k = torch.arange(K + 1, device=DEV)[None]
    x = s["logits"][(s["row_start"][:, None] + k).clamp(max=N - 1)].float()  # [R, K + 1, V]
    t = s["temperature"][:, None, None]
    greedy = t == 0
    x = x / torch.where(greedy, 1.0, t)
    m = x.amax(-1, keepdim=True)
    word = torch.arange(V, device=DEV)
    best = torch.where(x == m, word, V).amin(-1)                            # the lowest of equal maxima
    e = torch.exp(x - m)
    p = e / e.sum(-1, keepdim=True)
    logp = x - m - torch.log(e.sum(-1, keepdim=True))
    pd = p[:, :K].gather(-1, d[..., None])[..., 0]
    qd = 1.0 if s["draft_probs"] is None else s["draft_probs"].gather(-1, d[..., None])[..., 0]
    ok = torch.where(greedy[..., 0], d == best[:, :K], s["uniform"] * qd < pd) & (k[:, :K] < n)
    a = torch.cumprod(ok.int(), 1).sum(1, keepdim=True)                     # [R, 1]
    pa = p.gather(1, a[..., None].expand(-1, 1, V))[:, 0]                   # [R, V]
    at = a.clamp(max=K - 1)
    if s["draft_probs"] is None:
        q = (word == d.gather(1, at)).float()
    else:
        q = s["draft_probs"].gather(1, at[..., None].expand(-1, 1, V))[:, 0]
    left = torch.where(a < n, (pa - q).clamp(min=0), pa)
    left = torch.where((left > 0).any(-1, keepdim=True), left, pa)
    race = torch.where(left > 0, left / s["noise"], -1.0)
    top = race.amax(-1, keepdim=True)
    drawn = torch.where(race == top, word, V).amin(-1, keepdim=True)
    nxt = torch.where(greedy[..., 0], best.gather(1, a), drawn)             # [R, 1]
    tokens = torch.where(k < a, torch.cat([d, d[:, :1]], 1), torch.where(k == a, nxt, -1))
    logprobs = torch.where(k <= a, logp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0], 0.0)
    return tokens.to(torch.int32), a[:, 0].to(torch.int32), logprobs


def _own(s):
    from nvfp4_w4a4_gemm_quantize_amd import binding as B
    c = s["case"]
    if c["op"] == "plan":
        p = B.paged_plan(s["ctx"], s["new"], s["free"], s["table"], c["page"], s["max_tokens"], free_cursor=s["cursor"])
        return s["table"], p.q_start, p.seq_lens, p.positions, p.slots, p.counts
    if c["op"] == "write":
        B.paged_kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"]
    if c["op"] == "attention":
        most = c["context"] + c["new"]
        if "workspace" not in s:
            s["workspace"] = B.paged_attention_workspace(s["q"].shape[0], c["requests"], c["hq"], c["hkv"], c["dim"], c["new"],
                                                         most)
        return B.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["seq_lens"], c["new"], most,
                                 scale=s["scale"], window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 workspace=s["workspace"], return_lse=True)
    if "workspace" not in s:
        s["workspace"] = B.verify_drafts_workspace(c["requests"], c["drafts"], c["vocab"])
    return B.verify_drafts(s["logits"], s["row_start"], s["num_drafts"], s["draft_tokens"], s["uniform"], s["noise"],
                           draft_probs=s["draft_probs"], temperature=s["temperature"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "write": _plain_write, "attention": _plain_attention,
            "verify": _plain_verify}[state["case"]["op"]](state)


# ------------------------------------------------------------- definition ----

def exact(case, seed):
    """The outputs from the definitions in 64 bits, request by request."""
    c = case
    if c["op"] == "attention":
        return _exact_attention(c, prepare(case, seed))
    if c["op"] == "verify":
        return None, None, _exact_logprobs(c, prepare(case, seed))
    if c["op"] == "write":
        return _exact_write(c, prepare(case, seed))
    return None                                     # plan: whole numbers


def _exact_write(c, s):
    """The caches' values before their rounding to the cache's type."""
    caches = s["k_cache"].double(), s["v_cache"].double()
    at = [(t, slot // c["page"], slot % c["page"]) for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    t, page, place = (torch.tensor(x, device=DEV) for x in zip(*at))
    for h in range(c["hkv"]):
        for name, cache in zip("kv", caches):
            x = s[name][t, h * c["dim"]:(h + 1) * c["dim"]].double()
            cache[page, h, place] = (x / s[name + "_scale"][h].double()).clamp(-448, 448) if c["fp8"] else x
    return caches


def _exact_attention(c, s):
    H, D, P = c["hkv"], c["dim"], c["page"]
    G = c["hq"] // H
    start, lens, table = s["q_start"].tolist(), s["seq_lens"].tolist(), s["table"].long()
    T = s["q"].shape[0]
    out = torch.zeros(T, c["hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, c["hq"], dtype=torch.float64, device=DEV)
    for r, n in enumerate(lens):
        if start[r + 1] == start[r]:
            continue
        pages = table[r, :-(-n // P)]
        pos = torch.arange(n - (start[r + 1] - start[r]), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hidden = (j > pos) | ((pos - j >= c["window"]) if c["window"] else False)
        for h in range(H):
            k, v = ((x.view(torch.uint8)[pages, h].view(FP8) if c["fp8"] else x[pages, h]).double().reshape(-1, D)[:n]
                    for x in (s["k_cache"], s["v_cache"]))
            if c["fp8"]:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for head in range(h * G, h * G + G):
                q = s["q"][start[r]:start[r + 1], head * D:(head + 1) * D].double()
                z = (q @ k.t().contiguous()) * s["scale"]
                z[hidden] = -math.inf
                lse[start[r]:start[r + 1], head] = torch.logsumexp(z, 1)
                out[start[r]:start[r + 1], head] = torch.softmax(z, 1) @ v
    return out.reshape(T, -1), lse


def _exact_logprobs(c, s):
    """log p of the tokens that the definition emits."""
    out = torch.zeros(c["requests"], c["drafts"] + 1, dtype=torch.float64, device=DEV)
    for r, n in enumerate(_drafts(c)):
        temp = float(s["temperature"][r])
        row = int(s["row_start"][r])
        for i in range(n + 1):
            x = s["logits"][row + i].double()
            lp = torch.log_softmax(x / temp if temp else x, 0)
            d = int(s["draft_tokens"][r, i]) if i < n else -1
            q = torch.zeros_like(lp)
            if i < n:
                q = s["draft_probs"][r, i].double() if c["probs"] else q.index_fill(0, torch.tensor([d], device=DEV), 1.0)
            if temp == 0:
                token = int((x == x.max()).nonzero()[0])
                accepted = token == d
            elif i < n and float(s["uniform"][r, i]) * float(q[d]) < math.exp(float(lp[d])):
                token, accepted = d, True
            else:
                w = (lp.exp() - q).clamp(min=0) if i < n else lp.exp()
                token, accepted = int((w / s["noise"][r].double()).argmax()), False
            out[r, i] = lp[token]
            if not accepted:
                break
    return out
