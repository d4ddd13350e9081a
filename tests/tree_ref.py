"""Attention of drafted trees over the quantized cache, and keeping tokens, in plain 64-bit torch and
Python on the CPU, from their definitions in include/hqq.h."""
import math

import torch

import cache_ref as R


def random_masks(counts, gen, words):
    """Masks [rows, words] of random trees: a token's parent is an earlier one or none."""
    rows = []
    for n in counts:
        seen = []
        for j in range(n):
            parent = int(torch.randint(-1, j, (1,), generator=gen)) if j else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        rows += seen
    return to_words(rows, words)


def to_words(masks, words):
    """Whole numbers as rows of 64-bit words (int64)."""
    out = [[m >> 64 * w & (1 << 64) - 1 for w in range(words)] for m in masks]
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in out], dtype=torch.int64).reshape(len(masks), words)


def attention(held, table, lens, cu, q, scale, tree):
    """(out, lse, bound, bound of lse) as cache_ref.attention gives them, whose bound is derived there;
    only what a row sees is another."""
    c = held.c
    heads, dim = c["n_heads"], c["head_dim"]
    n, hq, _ = q.shape
    per = hq // heads
    words = tree.cpu().tolist()
    out = torch.full((n, hq, dim), math.nan, dtype=torch.float64)
    lse = torch.full((n, hq), math.nan, dtype=torch.float64)
    bound, blse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (lo, hi) in enumerate(R.rows_of(cu, n, len(lens))):
        if hi == lo:
            continue
        t, ln = hi - lo, min(max(lens[b], 0), len(table[b]) * c["page_size"])
        k, ka, ok = held.tokens("k", table[b], ln)
        v, va, _ = held.tokens("v", table[b], ln)
        seen = torch.ones(t, ln, dtype=torch.bool)
        for i in range(t):
            for p in range(max(ln - t, 0), ln):
                j = p - (ln - t)
                seen[i, p] = j // 64 < tree.shape[1] and words[lo + i][j // 64] >> j % 64 & 1
        seen = (seen & ok[None])[None, None]
        x = q[lo:hi].cpu().double().reshape(t, heads, per, dim).permute(1, 2, 0, 3)
        s = torch.matmul(x, k.transpose(1, 2)[:, None]) * scale
        mag = torch.matmul(x.abs(), ka.transpose(1, 2)[:, None]) * abs(scale)
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True) if ln else torch.full((*s.shape[:-1], 1), -math.inf, dtype=torch.float64)
        w = torch.exp(s - m.clamp(min=-1e300))
        tot = w.sum(-1, keepdim=True)
        p = w / tot.clamp(min=1e-300)
        a2 = torch.matmul(p, (held.steps(table[b], ln) * 2.0 ** (c["nbits"] - 1))[:, None]) * 2.0 ** -11
        if ln:
            a2 = a2 + ln * 2.0 ** -26 * held.steps(table[b], ln).amax() * 2.0 ** c["nbits"]
        ds = torch.where(p > 1e-12, mag, 0.0).amax(-1, keepdim=True) * (dim + 8) * 2.0 ** -24 if ln else torch.zeros_like(m)
        rel = 4 * ds + 2.0 ** -17 + ln * 2.0 ** -24
        put = lambda y: y.permute(2, 0, 1, *range(3, y.dim())).reshape(t, hq, *y.shape[3:])
        out[lo:hi] = put(torch.matmul(p, v[:, None]))
        bound[lo:hi] = put(torch.matmul(p, va[:, None]) * rel + a2)
        lse[lo:hi] = put((m + torch.log(tot)).squeeze(-1))
        blse[lo:hi] = put((2 * ds + 2.0 ** -18 + ln * 2.0 ** -24 + m.abs().nan_to_num(0, 0, 0) * 2.0 ** -22).squeeze(-1))
    return out, lse, bound, blse


def kept_of(row, n):
    """The entries of a list that count."""
    out = []
    for j in row:
        if j < 0 or j >= n or (out and j <= out[-1]):
            break
        out.append(j)
    return out


def keep(cache, table, lens, cu, n_tokens, kept):
    """What a cache's buffers hold after the call, and the new lengths."""
    c, page = cache, cache["page_size"]
    args = (page, c["head_dim"], c["nbits"], c["group_size"])
    n_pages = c["k_codes"].shape[0]
    codes = {w: R.pages_to_codes(c[w + "_codes"], *args, w) for w in "kv"}
    meta = {w: c[w + "_meta"].cpu().clone() for w in "kv"}
    new = []
    for b, (lo, hi) in enumerate(R.rows_of(cu, n_tokens, len(lens))):
        ln = min(max(lens[b], 0), len(table[b]) * page)
        first = ln - (hi - lo)

        def place(pos):
            p = table[b][pos // page] if 0 <= pos < len(table[b]) * page else -1
            return (p, pos % page) if 0 <= p < n_pages else None
        entries = kept_of(kept[b], hi - lo)
        for i, j in enumerate(entries):
            src, dst = place(first + j), place(first + i)
            if src and dst:
                for w in "kv":
                    codes[w][dst[0], :, dst[1]] = codes[w][src[0], :, src[1]]
                    meta[w][dst[0], :, dst[1]] = meta[w][src[0], :, src[1]]
        new.append(max(first + len(entries), 0))
    out = {w + "_codes": R.codes_to_pages(codes[w], c["nbits"], c["group_size"], w) for w in "kv"}
    return {**out, "k_meta": meta["k"], "v_meta": meta["v"]}, new
