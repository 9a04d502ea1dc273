"""The softmax-attention layer in 8 bits as measured cases: rotary, paged_kv_append, paged_attention_blocks, int8_linear.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) where ``own`` is
false, and calls the library where it is true.  Lengths of ragged batches follow from the case alone, values from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
GOLDEN = 0.6180339887498949
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BLOCK = 16                                          # tokens that share a scale (per head)
MOST = {"e4m3_blocks": 448.0, "int8_blocks": 127.0}


# ------------------------------------------------------------------ cases ----

def listed():
    rot = dict(op="rotary", scaling="none", factor=1.0, original=8192)
    app = dict(op="append", page=64, scaling="none", factor=1.0, original=8192)
    attn = dict(op="attention", ragged=False, window=0)
    lin = dict(op="int8")
    return [
        # q and k of a small decode batch side by side, a quarter of heads of 256 rotated; latency
        dict(rot, name="rotary_decode_8", tokens=8, heads=28, dim=256, rot=64, layout="half", start=30000),
        # q and k of a long prompt behind a longer one, whole heads of 128, frequencies stretched for long contexts
        dict(rot, name="rotary_prompt_16k", tokens=16384, heads=48, dim=128, rot=128, layout="interleaved", start=100000,
             scaling="yarn", factor=16.0),
        # a decode batch's q, k and v into a block-scaled E4M3 cache, in the middle of blocks; latency
        dict(app, name="append_decode_64_e4m3", requests=64, new=1, context=500, ragged=True, hq=40, hkv=8, dim=128, rot=128,
             layout="half", kind="e4m3_blocks"),
        # a prompt into a block-scaled E4M3 cache
        dict(app, name="append_prompt_16k_e4m3", requests=1, new=16384, context=0, ragged=False, hq=40, hkv=8, dim=128, rot=128,
             layout="half", kind="e4m3_blocks"),
        # ragged prompt chunks into a bf16 cache, three quarters of heads of 64 rotated
        dict(app, name="append_chunks_8_bf16", requests=8, new=777, context=1000, ragged=True, hq=16, hkv=16, dim=64, rot=48,
             layout="interleaved", kind="bf16", page=32, scaling="wavelength", factor=8.0),
        # a full decode batch of ragged lengths over a block-scaled E4M3 cache: the HBM-bound heart of serving
        dict(attn, name="attn_decode_64_e4m3", requests=64, new=1, context=16384, ragged=True, hq=40, hkv=8, dim=128, page=16,
             kind="e4m3_blocks"),
        # four drafts and the last token of 32 requests over an INT8 cache, heads of 256
        dict(attn, name="attn_drafts_32_int8", requests=32, new=5, context=8192, hq=24, hkv=4, dim=256, page=64,
             kind="int8_blocks"),
        # a long prompt's second half over an INT8 cache: matrix-bound
        dict(attn, name="attn_prompt_4k_int8", requests=1, new=4096, context=4096, hq=40, hkv=8, dim=128, page=64,
             kind="int8_blocks"),
        # one token through a wide projection: the weights' bytes
        dict(lin, name="int8_decode_one", m=1, n=17408, k=5120),
        # a decode batch through the way back
        dict(lin, name="int8_decode_37", m=37, n=5120, k=17408),
        # a ragged chunk, odd sizes
        dict(lin, name="int8_chunk_777", m=777, n=4104, k=2064),
        # a prompt through a wide projection: matrix-bound
        dict(lin, name="int8_prompt_4096", m=4096, n=17408, k=5120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _draw_rotation(rng, dim):
    scaling = rng.choice(("none", "linear", "ntk", "yarn", "wavelength"))
    return dict(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= dim]), layout=rng.choice(("half", "interleaved")),
                scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0, 32.0)), original=8192)


def draw(rng):
    op = rng.choice(("rotary", "append", "append", "attention", "attention", "int8", "int8"))
    if op == "rotary":
        dim = rng.choice((64, 128, 256))
        heads = rng.randint(1, 48)
        return dict(op=op, tokens=_log(rng, 1, 16384 * 48 * 128 // (heads * dim)), heads=heads, dim=dim,
                    start=_log(rng, 1, 1000000), **_draw_rotation(rng, dim))
    if op == "append":
        hkv, group, dim = rng.choice(((8, 5, 128), (4, 6, 256), (16, 1, 64), (1, 16, 128), (3, 8, 64), (2, 7, 128)))
        requests, new = _log(rng, 1, 64), rng.choice((1, 1, rng.randint(2, 40), _log(rng, 40, 2048)))
        new = max(1, min(new, 16384 * 48 * 128 // (requests * hkv * (group + 1) * dim)))
        return dict(op=op, requests=requests, new=new, context=_log(rng, 1, 1500), ragged=rng.random() < 0.7, hq=hkv * group,
                    hkv=hkv, dim=dim, page=rng.choice((16, 32, 64, 128)),
                    kind=rng.choice(("bf16", "e4m3", "e4m3_blocks", "int8_blocks")), **_draw_rotation(rng, dim))
    if op == "attention":
        hkv, group, dim = rng.choice(((8, 5, 128), (4, 6, 256), (16, 1, 64), (1, 16, 128), (2, 7, 128), (3, 8, 64)))
        new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 9, 2048)))
        context = _log(rng, 1, 16384)
        keys, pairs = 64 * 8192 * 8 * 128, 40 * 4096 * 6144
        most = min(keys // ((context + new) * hkv * dim), pairs // (hkv * group * new * (context + new)), 64)
        return dict(op=op, requests=_log(rng, 1, max(1, most)), new=new, context=context, ragged=rng.random() < 0.5,
                    hq=hkv * group, hkv=hkv, dim=dim, page=rng.choice((16, 32, 64, 128)),
                    kind=rng.choice(("e4m3_blocks", "int8_blocks")), window=rng.choice((0, 0, _log(rng, 1, 4096))))
    n, k = _log(rng, 64, 17408), 16 * _log(rng, 4, 1088)
    return dict(op=op, m=_log(rng, 1, max(1, min(4096, 4096 * 17408 * 5120 // (n * k)))), n=n, k=k)


def _spread(most, count, step):
    """`count` lengths in 1 .. most, evenly spread in a fixed order; the first is `most`."""
    return [most if r == 0 else 1 + int(most * ((r * step) % 1.0)) for r in range(count)]


def _lens(c):
    """(context, new) of every request."""
    R = c["requests"]
    if not c["ragged"]:
        return [c["context"]] * R, [c["new"]] * R
    return [n - 1 for n in _spread(c["context"], R, GOLDEN)], _spread(c["new"], R, math.sqrt(2))


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


def _code_bytes(kind):
    return 2 if kind == "bf16" else 1


def work(case):
    c = case
    if c["op"] == "rotary":
        return {"bytes": c["tokens"] * (4 * c["heads"] * c["dim"] + 4), "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        ctx, new = _lens(c)
        T = sum(new)
        blocks = sum(-(-(a + b) // BLOCK) - a // BLOCK for a, b in zip(ctx, new))
        row = 4 * c["hq"] * c["dim"] + 2 * c["hkv"] * c["dim"] * (2 + _code_bytes(c["kind"])) + 12
        return {"bytes": T * row + (2 * blocks * c["hkv"] * 2 if c["kind"] in MOST else 0),
                "flops": 3 * T * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "attention":
        ctx, new = _lens(c)
        seen = sum(min(a + b, c["window"] + b - 1) if c["window"] else a + b for a, b in zip(ctx, new))
        cache = 2 * seen * c["hkv"] * c["dim"] + 2 * seen * c["hkv"] // BLOCK
        return {"bytes": cache + sum(new) * c["hq"] * (4 * c["dim"] + 4),
                "flops": 4 * c["dim"] * c["hq"] * _pairs(ctx, new, c["window"])}
    return {"bytes": 2 * c["m"] * c["k"] + c["n"] * c["k"] + 4 * c["n"] + 2 * c["m"] * c["n"],
            "flops": 2 * c["m"] * c["n"] * c["k"]}


# ----------------------------------------------------------------- inputs ----

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _inverse_frequencies(c):
    """(radians a position of every pair in 64 bits, the factor on cosine and sine)."""
    rot, base, f, L = c["rot"], 10000.0, c["factor"], float(c["original"])
    if c["scaling"] == "ntk":
        base *= f ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if c["scaling"] == "linear":
        inv = [w / f for w in inv]
    if c["scaling"] == "wavelength":                # pairs that turn seldom within the original length are stretched
        low, high, slow = 1.0, 4.0, []
        for w in inv:
            turns = L * w / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            slow.append(w * keep + w / f * (1 - keep))
        inv = slow
    if c["scaling"] == "yarn":
        at = [rot * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = [min(max((i - first) / max(last - first, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        inv = [w / f * r + w * (1 - r) for w, r in zip(inv, ramp)]
    return torch.tensor(inv, dtype=torch.float64, device=DEV), 0.1 * math.log(f) + 1.0 if c["scaling"] == "yarn" else 1.0


def _needed(top, most):
    """E8M0 byte of the smallest power of two s with top <= most * s."""
    m, e = torch.frexp(top / most)
    return torch.where(top > 0, (127 + e - (m == 0.5).int()).clamp(1, 254), 1)


def _power(e):
    """2^e in 32 bits for whole e in -127 .. 127."""
    return torch.exp2(e.double()).float()


def _codes(x, kind):
    """Codes of values that have been divided by their scales."""
    return x.clamp(-448, 448).to(FP8) if kind != "int8_blocks" else x.round().clamp(-127, 127).to(torch.int8)


def _to_blocks(x, kind):
    """x [pages, heads, page, dim] fp32 as (codes, scales [pages, heads, page / 16])."""
    pages, heads, page, dim = x.shape
    b = x.view(pages, heads, page // BLOCK, BLOCK, dim)
    e = _needed(b.abs().amax((-1, -2)), MOST[kind])
    return _codes(b * _power(127 - e)[..., None, None], kind).view(x.shape), e.to(torch.uint8).view(E8M0)


def _pages(c, s, g, extra):
    """Block tables of the requests' pages in a random order; returns the number of pages of the cache."""
    ctx, new = _lens(c)
    need = [-(-(a + b) // c["page"]) for a, b in zip(ctx, new)]
    pages, MP = sum(need) + extra, max(need)
    order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
    first = [sum(need[:r]) for r in range(len(need))]
    col = torch.arange(MP, device=DEV)[None]
    at = (_ints(first)[:, None] + col).clamp(max=pages - 1)
    s["table"] = torch.where(col < _ints(need)[:, None], order[at], -1).to(torch.int32)
    return pages


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def cache(pages):
        """Codes and scales of a filled cache: tokens of different sizes, a block's scale their largest one's."""
        x = randn(pages, c["hkv"], c["page"], c["dim"], dtype=torch.float32)
        x.mul_(torch.exp(0.5 * randn(pages, c["hkv"], c["page"], 1, dtype=torch.float32)))
        return _to_blocks(x, c["kind"])

    if c["op"] in ("rotary", "append"):
        s["inv"], s["amplitude"] = _inverse_frequencies(c)
    if c["op"] == "rotary":
        T = c["tokens"]
        s["x"] = randn(T, c["heads"] * c["dim"] + 2 * c["dim"])[:, :c["heads"] * c["dim"]]    # in front of v in the projection's output
        s["positions"] = c["start"] + torch.arange(T, device=DEV, dtype=torch.int32)
        if T < 1000:                                # requests of their own lengths
            s["positions"] = (s["positions"] * rand(T)).to(torch.int32)
    elif c["op"] == "append":
        ctx, new = _lens(c)
        T, hq, H, D, P = sum(new), c["hq"], c["hkv"], c["dim"], c["page"]
        pages = _pages(c, s, g, 4)
        qkv = randn(T, (hq + 2 * H) * D) * torch.exp(0.5 * randn(T, 1))
        s["q"], s["k"], s["v"] = qkv[:, :hq * D], qkv[:, hq * D:(hq + H) * D], qkv[:, (hq + H) * D:]
        s["positions"] = torch.cat([torch.arange(a, a + b, device=DEV, dtype=torch.int32) for a, b in zip(ctx, new)])
        r = torch.repeat_interleave(torch.arange(len(new), device=DEV), _ints(new), output_size=T)
        at = s["positions"].long()
        s["slots"] = s["table"][r, at // P].long() * P + at % P
        s["k_scale"] = s["v_scale"] = None
        if c["kind"] in MOST:
            (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = cache(pages), cache(pages)
        else:
            dtype = FP8 if c["kind"] == "e4m3" else torch.bfloat16
            s["k_cache"] = torch.zeros(pages, H, P, D, device=DEV, dtype=torch.bfloat16).to(dtype)
            s["v_cache"] = s["k_cache"].clone()
            if c["kind"] == "e4m3":
                s["k_scale"], s["v_scale"] = 0.01 + 0.01 * rand(H), 0.01 + 0.01 * rand(H)
    elif c["op"] == "attention":
        ctx, new = _lens(c)
        pages = _pages(c, s, g, 8)
        s["q"] = randn(sum(new), c["hq"] * c["dim"])
        (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = cache(pages), cache(pages)
        s["q_start"] = _ints([sum(new[:r]) for r in range(len(new) + 1)])
        s["seq_lens"] = _ints([a + b for a, b in zip(ctx, new)])
        s["scale"] = 1.0 / math.sqrt(c["dim"])
    else:
        M, N, K = c["m"], c["n"], c["k"]
        s["x"] = randn(M, K) * torch.where(rand(K) < 0.001, 20.0, 1.0).to(torch.bfloat16)   # a few channels stand out
        w = randn(N, K, dtype=torch.float32) * K ** -0.5
        s["w_scale"] = w.abs().amax(1) / 127
        s["w"] = (w / s["w_scale"][:, None]).round().to(torch.int8)
    return s


# -------------------------------------------------------------- operators ----

def _values(codes, scales):
    """What a block-scaled cache stands for: exact in bf16."""
    pages, heads, page, dim = codes.shape
    x = codes.to(torch.bfloat16).view(pages, heads, page // BLOCK, BLOCK, dim)
    return (x * scales.to(torch.bfloat16)[..., None, None]).view(codes.shape)


def _caches(s):
    """The caches as they are compared: whole codes as the values that they stand for."""
    if s["case"]["kind"] == "int8_blocks":
        return _values(s["k_cache"], s["k_scale"]), _values(s["v_cache"], s["v_scale"]), s["k_scale"], s["v_scale"]
    if s["case"]["kind"] == "e4m3_blocks":
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return s["k_cache"], s["v_cache"]


def _rotate(x, heads, s):
    """x [T, heads * dim] rotated, fp32 [T, heads, dim]."""
    c = s["case"]
    rot, n = c["rot"], c["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv"]
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.reshape(x.shape[0], heads, c["dim"]).float()
    if c["layout"] == "half":
        a, b = y[..., :n], y[..., n:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_rotary(s):
    return _rotate(s["x"], s["case"]["heads"], s).to(torch.bfloat16).flatten(1)


def _store(s, rows, cache, scale):
    """rows [T, heads, dim] fp32 into the cache, by its kind."""
    kind, P, slots = s["case"]["kind"], s["case"]["page"], s["slots"]
    if kind not in MOST:
        raw = torch.uint8 if kind == "e4m3" else torch.bfloat16             # indexing has no FP8 form
        rows = _codes(rows / scale[:, None], kind) if kind == "e4m3" else rows.to(torch.bfloat16)
        cache.view(raw)[slots // P, :, slots % P] = rows.view(raw)
        return
    pages, H, _, D = cache.shape
    blocks, at = torch.unique(slots // BLOCK, return_inverse=True)
    page, col, n = blocks // (P // BLOCK), blocks % (P // BLOCK), blocks.numel()
    top = torch.zeros(n, H, device=DEV).index_reduce_(0, at, rows.abs().amax(-1), "amax")
    fresh = torch.zeros(n, device=DEV).index_reduce_(0, at, (slots % BLOCK == 0).float(), "amax")[:, None] > 0
    bytes_ = scale.view(torch.uint8)
    old = torch.where(fresh, 1, bytes_[page, :, col].int())
    new = torch.maximum(_needed(top, MOST[kind]), old)
    raw = cache.view(torch.uint8).view(pages, H, P // BLOCK, BLOCK, D)
    held = raw[page, :, col].view(cache.dtype).float() * _power((old - new).clamp(min=-127))[..., None, None]
    codes = _codes(torch.where(fresh[..., None, None], 0.0, held), kind).view(torch.uint8)
    codes[at, :, slots % BLOCK] = _codes(rows * _power(127 - new)[at][..., None], kind).view(torch.uint8)
    raw[page, :, col] = codes
    bytes_[page, :, col] = new.to(torch.uint8)


def _plain_append(s):
    c = s["case"]
    q = _rotate(s["q"], c["hq"], s).to(torch.bfloat16).flatten(1)
    _store(s, _rotate(s["k"], c["hkv"], s), s["k_cache"], s["k_scale"])
    _store(s, s["v"].reshape(-1, c["hkv"], c["dim"]).float(), s["v_cache"], s["v_scale"])
    return (q,) + _caches(s)


def _plain_attention(s):
    c = s["case"]
    R, HQ, H, D, P, W = (c[n] for n in ("requests", "hq", "hkv", "dim", "page", "window"))
    G, T, N, L = HQ // H, s["q"].shape[0], c["new"], s["table"].shape[1] * P
    start, lens = s["q_start"].to(torch.int64), s["seq_lens"].to(torch.int64)
    new = start[1:] - start[:-1]
    pages = s["table"].clamp(min=0).long()

    def keys(cache, scale):                         # [R, H, L, D]
        x = cache.view(torch.uint8)[pages].view(cache.dtype).float()        # [R, pages, H, P, D]
        x = x.view(*x.shape[:3], P // BLOCK, BLOCK, D)
        x = x * scale.view(torch.uint8)[pages].view(E8M0).float()[..., None, None]
        return x.flatten(3, 4).permute(0, 2, 1, 3, 4).reshape(R, H, L, D)

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


def _plain_int8(s):
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    codes = (x * (127 / top)).round()
    return (torch.matmul(codes, s["w"].float().t()) * (top / 127) * s["w_scale"]).to(torch.bfloat16)


def _own(s):
    from nvfp4_w4a4_gemm_quantize_amd import binding as B
    c = s["case"]
    if c["op"] == "int8":
        return B.int8_linear(s["x"], s["w"], s["w_scale"])
    if c["op"] == "attention":
        most = c["context"] + c["new"]
        if "workspace" not in s:
            s["workspace"] = B.paged_attention_workspace(s["q"].shape[0], c["requests"], c["hq"], c["hkv"], c["dim"], c["new"],
                                                         most)
        return B.paged_attention_blocks(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["q_start"],
                                        s["seq_lens"], c["new"], most, scale=s["scale"], window=c["window"],
                                        workspace=s["workspace"], return_lse=True)
    if "rotation" not in s:
        s["rotation"] = B.rotary_table(c["rot"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                       original_length=c["original"])
    if c["op"] == "rotary":
        return B.rotary(s["x"], s["positions"], s["rotation"], c["dim"])
    q = B.paged_kv_append(s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], rotation=s["rotation"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"], q=s["q"])
    return (q,) + _caches(s)


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "append": _plain_append, "attention": _plain_attention,
            "int8": _plain_int8}[state["case"]["op"]](state)


# ------------------------------------------------------------- definition ----

def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"rotary": lambda: _exact_turn(s, s["x"], case["heads"]).flatten(1), "append": lambda: _exact_append(case, s),
            "attention": lambda: _exact_attention(case, s), "int8": lambda: _exact_int8(s)}[case["op"]]()


def _exact_turn(s, x, heads):
    """Pairs as complex numbers, times amplitude * e^(i angle)."""
    c, n = s["case"], s["case"]["rot"] // 2
    y = x.reshape(x.shape[0], heads, c["dim"]).double().clone()
    re, im = (slice(0, n), slice(n, 2 * n)) if c["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    turn = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=DEV), s["positions"].double()[:, None] * s["inv"])
    z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn[:, None]
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_append(c, s):
    """q before its rounding; the caches' codes (INT8: values) with every rounding that the definition has."""
    q = _exact_turn(s, s["q"], c["hq"]).flatten(1)
    k, v = _exact_turn(s, s["k"], c["hkv"]), s["v"].reshape(-1, c["hkv"], c["dim"]).double()
    P, slots, outs, scales = c["page"], s["slots"], [], []
    for rows, name in ((k, "k"), (v, "v")):
        cache = s[name + "_cache"].double()
        if c["kind"] in MOST:
            most, grid = MOST[c["kind"]], (torch.round if c["kind"] == "int8_blocks" else lambda x: x.to(FP8).double())
            e = s[name + "_scale"].view(torch.uint8).double() - 127
            order = slots.tolist()
            groups = {}
            for t, slot in enumerate(order):
                groups.setdefault(slot // BLOCK, []).append((t, slot % BLOCK))
            width = max(len(x) for x in groups.values())
            pad = [x + [x[0]] * (width - len(x)) for x in groups.values()]              # a token twice changes nothing
            at = torch.tensor(list(groups), device=DEV)
            t, place = (torch.tensor([[y[i] for y in x] for x in pad], device=DEV) for i in (0, 1))
            page, col = at // (P // BLOCK), at % (P // BLOCK)
            fresh = (place == 0).any(1)
            new = rows[t]                                                               # [blocks, width, heads, dim]
            want = torch.ceil(torch.log2(new.abs().amax((1, 3)).clamp(min=2.0 ** -126) / most)).clamp(-126, 127)
            have = torch.where(fresh[:, None], torch.full_like(want, -126), e[page, :, col])
            now = torch.maximum(want, have)
            view = cache.view(cache.shape[0], c["hkv"], P // BLOCK, BLOCK, c["dim"])
            held = grid(view[page, :, col] * torch.exp2(have - now)[..., None, None])
            held[fresh] = 0.0
            held[torch.arange(len(groups), device=DEV)[:, None], :, place] = grid(new * torch.exp2(-now)[:, None, :, None])
            view[page, :, col] = held
            e[page, :, col] = now
            if c["kind"] == "int8_blocks":
                view *= torch.exp2(e)[..., None, None]
            scales.append(torch.exp2(e))
        else:
            x = (rows / s[name + "_scale"].double()[:, None]).clamp(-448, 448) if c["kind"] == "e4m3" else rows
            cache[slots // P, :, slots % P] = x
        outs.append(cache)
    return (q, *outs, *scales)


def _exact_attention(c, s):
    H, D, P = c["hkv"], c["dim"], c["page"]
    G = c["hq"] // H
    start, lens, table = s["q_start"].tolist(), s["seq_lens"].tolist(), s["table"].long()
    T = s["q"].shape[0]
    out = torch.zeros(T, c["hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, c["hq"], dtype=torch.float64, device=DEV)
    for r, n in enumerate(lens):
        pages = table[r, :-(-n // P)]
        pos = torch.arange(n - (start[r + 1] - start[r]), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)
        hidden = (j > pos) | ((pos - j >= c["window"]) if c["window"] else False)
        for h in range(H):
            kv = []
            for name in ("k", "v"):
                code = s[name + "_cache"].view(torch.uint8)[pages, h].view(s[name + "_cache"].dtype).double().reshape(-1, D)[:n]
                e = s[name + "_scale"].view(torch.uint8)[pages, h].double().reshape(-1)
                kv.append(code * torch.exp2(e - 127)[j // BLOCK][:, None])
            for head in range(h * G, h * G + G):
                q = s["q"][start[r]:start[r + 1], head * D:(head + 1) * D].double()
                z = (q @ kv[0].t().contiguous()) * s["scale"]
                z[hidden] = -math.inf
                lse[start[r]:start[r + 1], head] = torch.logsumexp(z, 1)
                out[start[r]:start[r + 1], head] = torch.softmax(z, 1) @ kv[1]
    return out.reshape(T, -1), lse


def _exact_int8(s):
    x = s["x"].double()
    step = x.abs().amax(1, keepdim=True) / 127
    return (torch.round(x / step) @ s["w"].double().t().contiguous()) * step * s["w_scale"].double()
