"""The paged serving step's operators from their definitions, in numpy and in
float64, request by request: the plan (block tables and slot maps), the K/V
write, attention over the paged cache with an error bound, and the verification
of drafted tokens."""
import numpy as np

U32 = 2.0 ** -24       # unit roundoff of fp32
U_BF16 = 2.0 ** -8     # unit roundoff of bf16 (8 significant bits)


def plan(ctx, new, free, cursor, table, page, max_tokens):
    """Returns (table, q_start, seq_lens, positions, slots, counts) as paged_plan leaves them."""
    table = np.array(table)
    R, MP = table.shape
    c, n = np.maximum(ctx, 0).astype(np.int64), np.maximum(new, 0).astype(np.int64)
    q_start = np.concatenate([[0], np.cumsum(n)])
    taken = missing = 0
    positions, slots = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    for r in range(R):
        before, after = min(-(-c[r] // page), MP), min(-(-(c[r] + n[r]) // page), MP)
        for col in range(before, after):
            at = cursor + taken + missing
            if at < len(free):
                table[r, col] = free[at]
                taken += 1
            else:
                table[r, col] = -1
                missing += 1
        for i in range(n[r]):
            t, pos = q_start[r] + i, c[r] + i
            if t >= max_tokens:
                break
            positions[t] = pos
            if pos // page < MP and table[r, pos // page] >= 0:
                slots[t] = table[r, pos // page].astype(np.int64) * page + pos % page
    return (table, np.minimum(q_start, max_tokens), c + n, positions, slots,
            np.array([q_start[-1], taken, missing, cursor + taken]))


def kv_write(x, slots, cache, scale=None):
    """cache [pages, heads, page, dim] (float64 values) after the rows x [T, heads * dim] went in, before rounding."""
    pages, heads, page, dim = cache.shape
    out = cache.copy()
    for t, slot in enumerate(slots):
        if 0 <= slot < pages * page:
            row = x[t].reshape(heads, dim)
            out[slot // page, :, slot % page] = row if scale is None else np.clip(row / scale[:, None], -448, 448)
    return out


def attention(q, k_cache, v_cache, table, q_start, seq_lens, page, hq, scale, window=0, k_scale=None, v_scale=None):
    """float64 attention.  q [T, hq * dim]; caches [pages, heads, page, dim]; rows of no request stay NaN.

    Returns (out [T, hq, dim], lse [T, hq], tol [T, hq, dim], lse_tol [T, hq]).  The bounds are those of one pass in
    fp32 with the weights rounded to bf16 (2^-8): a score's error is at most dim u sum|q k| |scale| for any order of
    its fp32 sum plus 4 u of its size for the scaling and the exponent's argument; a weight's relative error is twice
    that (its own maximum's too) plus 2^-8 plus 2^-20 for the hardware exponential; sums over n keys add n u; the
    output carries the weights' relative errors times sum w |v| / sum w, twice for numerator and denominator's share."""
    T = q.shape[0]
    pages, heads, _, dim = k_cache.shape
    G = hq // heads
    out, lse = np.full((T, hq, dim), np.nan), np.full((T, hq), np.nan)
    tol, lse_tol = np.zeros((T, hq, dim)), np.zeros((T, hq))
    for r, L in enumerate(seq_lens):
        t0, t1 = q_start[r], q_start[r + 1]
        L_held = min(max(L, 0), table.shape[1] * page)
        j = np.arange(L_held)
        pg = table[r, j // page]
        held = (pg >= 0) & (pg < pages)
        pg = np.where(held, pg, 0)
        for h in range(heads):
            K = np.where(held[:, None], k_cache[pg, h, j % page], 0.0)
            V = np.where(held[:, None], v_cache[pg, h, j % page], 0.0)
            c = scale * (1.0 if k_scale is None else float(k_scale[h]))
            vs = 1.0 if v_scale is None else float(v_scale[h])
            for t in range(t0, t1):
                p = L - (t1 - t0) + (t - t0)
                see = held & (j <= p) & ((j > p - window) if window else True)
                for hh in range(h * G, h * G + G):
                    qq = q[t, hh * dim:(hh + 1) * dim]
                    if not see.any():
                        out[t, hh], lse[t, hh] = 0.0, -np.inf
                        continue
                    s = c * (K[see] @ qq)
                    ds = abs(c) * np.max(np.abs(K[see]) @ np.abs(qq)) * dim * U32 + 4 * U32 * np.max(np.abs(s))
                    m = s.max()
                    w = np.exp(s - m)
                    den = w.sum()
                    n = see.sum()
                    lse[t, hh] = m + np.log(den)
                    lse_tol[t, hh] = 2 * ds + n * U32 + 2.0 ** -20 + 4 * U32 * abs(lse[t, hh])
                    out[t, hh] = vs * (w @ V[see]) / den
                    rel = U_BF16 + 4 * ds + 2 * n * U32 + 2.0 ** -19
                    tol[t, hh] = rel * abs(vs) * (w @ np.abs(V[see])) / den
    return out, lse, tol, lse_tol


def verify(logits, row_start, num_drafts, draft_tokens, uniform, noise, draft_probs=None, temperature=None):
    """(tokens [R, K + 1], accepted [R], logprobs [R, K + 1]) in float64 (sums in any order are exact enough that only
    comparisons within about 1e-12 of equality could differ)."""
    R, K = draft_tokens.shape
    N, V = logits.shape
    tokens, accepted, logprobs = np.full((R, K + 1), -1), np.zeros(R, int), np.zeros((R, K + 1))
    for r in range(R):
        n = min(num_drafts[r], K)
        if n < 0 or row_start[r] < 0 or row_start[r] + n >= N:
            continue
        T = 1.0 if temperature is None else float(temperature[r])
        for i in range(n + 1):
            x = logits[row_start[r] + i].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x) / (T if T else 1.0)
            top = x.max()
            e = np.exp(x - top) if top > -np.inf else np.zeros(V)
            p = e / e.sum() if top > -np.inf else e
            d = draft_tokens[r, i] if i < n else -1
            inside = 0 <= d < V
            q = np.zeros(V)
            if i < n:
                if draft_probs is not None:
                    q = draft_probs[r, i].astype(np.float64)
                elif inside:
                    q[d] = 1.0
            best = int(np.argmax(x)) if top > -np.inf else -1
            kept = i < n and inside and (d == best if T == 0 else float(uniform[r, i]) * q[d] < p[d])
            if kept:
                token = d
            elif T == 0:
                token = best
            else:
                w = np.maximum(p - q, 0.0) if i < n else p
                w = w if (w > 0).any() else p
                score = np.where(w > 0, w / noise[r].astype(np.float64), -1.0)
                token = int(np.argmax(score)) if (w > 0).any() else -1
            tokens[r, i] = token
            if token >= 0:
                logprobs[r, i] = x[token] - top - np.log(e.sum())
            if not kept:
                break
            accepted[r] += 1
    return tokens, accepted, logprobs
