"""Text generation with drafted tokens on one MI355X: the paged serving step
of softmax-attention layers between NVFP4 W4A4 linear layers.

Every step is the same chain of calls, whether it brings prompts, single tokens
or tokens with drafts:

    paged_plan -> per layer [nvfp4_linear (q, k, v) -> paged_kv_write -> paged_attention -> nvfp4_linear (o) -> MLP]
               -> nvfp4_linear (logits) -> verify_drafts

The drafts are looked up in the request's own text (what followed the last two
tokens before), so they cost nothing; verification keeps what the target would
have said.  Weights are random: the text means nothing, the steps are real.

    python examples/paged_serving.py [--steps N] [--drafts K] [--temperature T]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_w4a4_gemm_quantize_amd import binding as B  # noqa: E402


class Linear:
    """A W4A4 linear layer, with random weights if none are given."""

    def __init__(self, n, k, gen, w=None):
        if w is None:
            w = (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(torch.bfloat16)
        self.packed, self.scale = B.nvfp4_pack_weights(w)
        self.n = n

    def __call__(self, x, **kw):
        return B.nvfp4_linear(x, self.packed, self.scale[:1], self.n, **kw)[0]


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Model:
    """A decoder of softmax-attention layers with an E4M3 cache."""

    def __init__(self, layers=2, hidden=1024, hq=8, hkv=2, dim=128, ffn=2048, vocab=4096, pages=256, page=64, requests=4,
                 max_seq=2048, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.dim, self.page, self.vocab, self.max_seq = hq, hkv, dim, page, vocab, max_seq
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").to(torch.bfloat16)
        self.blocks = [dict(qkv=Linear((hq + 2 * hkv) * dim, hidden, gen), o=Linear(hidden, hq * dim, gen),
                            gate_up=Linear(2 * ffn, hidden, gen), down=Linear(hidden, ffn, gen),
                            k=torch.zeros(pages, hkv, page, dim, device="cuda").to(torch.float8_e4m3fn),
                            v=torch.zeros(pages, hkv, page, dim, device="cuda").to(torch.float8_e4m3fn),
                            # |k| and |v| stay below 448 of these steps; a real model has them calibrated
                            k_scale=torch.full((hkv,), 0.02, device="cuda"), v_scale=torch.full((hkv,), 0.02, device="cuda"))
                       for _ in range(layers)]
        # the embedding again, so that the model says what it has heard and drafts are worth their verification
        self.head = Linear(vocab, hidden, gen, self.embed * hidden ** -0.5)
        self.table = torch.full((requests, max_seq // page), -1, dtype=torch.int32, device="cuda")
        self.free = list(range(pages))
        # One workspace serves every step that is no larger.  An attention step's depends on its requests, and on whether
        # one of them may bring more than 32 rows a KV head, as a prompt does.
        self.attention_ws = B.paged_attention_workspace(requests * max_seq, requests, hq, hkv, dim, max_seq, max_seq)

    def step(self, tokens, ctx, new, trace=None, rows=None):
        """Logits of the step's tokens (all requests' new ones end to end), and its plan.  `rows` above the number of
        tokens makes a step of that size, as one that is captured has: the last rows are padding, zero from layer to
        layer, so that they change no linear layer's global scale."""
        i32 = dict(dtype=torch.int32, device="cuda")
        T, R = len(tokens) if rows is None else rows, len(new)
        plan = B.paged_plan(torch.tensor(ctx, **i32), torch.tensor(new, **i32), torch.tensor(self.free, **i32), self.table,
                            self.page, T)
        x = self.embed.new_zeros(T, self.embed.shape[1])
        x[:len(tokens)] = self.embed[torch.tensor(tokens, device="cuda")]
        nq, nk = self.hq * self.dim, self.hkv * self.dim
        for b in self.blocks:
            y = b["qkv"](norm(x))
            q, k, v = y[:, :nq], y[:, nq:nq + nk], y[:, nq + nk:]    # views: no copies
            B.paged_kv_write(k, v, plan.slots, b["k"], b["v"], b["k_scale"], b["v_scale"])
            a = B.paged_attention(q, b["k"], b["v"], self.table, plan.q_start, plan.seq_lens, max(new), self.max_seq,
                                  k_scale=b["k_scale"], v_scale=b["v_scale"], workspace=self.attention_ws)
            if trace is not None:
                trace.append((q, k, v, a))
            x = x + b["o"](a)
            x = x + b["down"](b["gate_up"](norm(x), epilogue="silu_mul"))
        return self.head(norm(x)), plan

    def take_pages(self, ctx, new, kept):
        """The host's list of free pages after a step: without the pages that it took, with those that only refused drafts
        reached (the next step gives their columns new ones)."""
        cols = lambda n: -(-n // self.page)  # noqa: E731
        del self.free[:sum(cols(c + n) - cols(c) for c, n in zip(ctx, new))]
        for r, (c, n) in enumerate(zip(ctx, new)):
            self.free += self.table[r, cols(c + kept[r]):cols(c + n)].tolist()


def look_up(text, count):
    """What followed the last earlier place of the text's last two tokens, over and over."""
    for period in range(1, len(text) - 1):
        if text[-2 - period:-period] == text[-2:]:
            return [text[len(text) - period + i % period] for i in range(count)]
    return []


def generate(model, prompts, steps, drafts, temperature=0.0, seed=0, log=None):
    """Texts of all requests after a prompt step and `steps` verified ones; log gets each step's accepted counts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, V = len(prompts), model.vocab
    texts, ctx, guesses = [list(p) for p in prompts], [0] * R, [[] for _ in prompts]
    temps = torch.full((R,), temperature, device="cuda")
    verify_ws = B.verify_drafts_workspace(R, drafts, V)
    for s in range(steps + 1):
        new = [len(t) - c + len(g) for t, c, g in zip(texts, ctx, guesses)]
        logits, plan = model.step([x for t, c, g in zip(texts, ctx, guesses) for x in t[c:] + g], ctx, new)
        # the last row before the drafts of each request, then one row a draft
        first = torch.tensor([n - len(g) - 1 for n, g in zip(new, guesses)], dtype=torch.int32, device="cuda")
        padded = torch.tensor([g + [0] * (drafts - len(g)) for g in guesses], dtype=torch.int32, device="cuda").reshape(R, drafts)
        u = torch.rand(R, drafts, generator=gen, device="cuda")
        noise = torch.empty(R, V, device="cuda").exponential_(generator=gen)
        out, kept, _ = B.verify_drafts(logits, plan.q_start[:R] + first,
                                       torch.tensor([len(g) for g in guesses], dtype=torch.int32, device="cuda"), padded, u, noise,
                                       temperature=temps, workspace=verify_ws)
        assert int(plan.counts[2]) == 0, "out of pages"
        kept = kept.tolist()
        if log is not None:
            log.append(kept)
        valid = [n - len(g) + k for n, g, k in zip(new, guesses, kept)]   # tokens of the chunk that stay
        model.take_pages(ctx, new, valid)
        for r, row in enumerate(out.tolist()):
            texts[r] += row[:kept[r] + 1]
            ctx[r] += valid[r]
        guesses = [look_up(t, drafts) for t in texts]
    return texts


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.0)
    args = ap.parse_args()
    model = Model()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=gen).tolist() for n in (200, 17, 90, 1)]
    # prompts that repeat themselves give the look-up something to find
    prompts = [p + p[:len(p) // 2] for p in prompts]
    torch.cuda.synchronize()
    t, log = time.perf_counter(), []
    texts = generate(model, prompts, args.steps, args.drafts, args.temperature, log=log)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) * 1e3
    said = sum(len(a) - len(p) for a, p in zip(texts, prompts))
    print("%d requests, %d steps: %d tokens, %d of them drafts kept, %.2f ms a step (host loop included)" %
          (len(prompts), args.steps + 1, said, sum(map(sum, log)), ms / (args.steps + 1)))


if __name__ == "__main__":
    main()
