"""Attention over the quantized cache in plain 64-bit torch on the CPU, with a bound of its own for
every row, head and dimension: only what the row sees counts, each token by its weight."""
import math

import torch

import cache_ref as R

LOG2E = 1 / math.log(2)


def attention(held, table, lens, cu, q, scale, prefix_pages=(), prefix_len=0, whole=False):
    """(out, lse, bound, blse) in float64, as cache_ref.attention lays them out; rows of no sequence
    are NaN. `bound` is what a binary32 evaluation may be off before the output's own rounding.
    With u = 2^-24, G groups and scores in base 2 (S = scale log2(e) <q, k>, M the largest |S| seen):

    A score: the sum over a group of query times code has at most g roundings of u of its
    magnitude, and none where queries are whole numbers and it stays below 2^24 (`whole`); step and
    base take scale in (a rounding each, and scale log2(e)'s own), 2 G + 1 sums of at most the
    magnitudes and M follow, and bases that go in as three bfloat16 parts leave out 2 u of theirs:
    (g + 2 G + 8) u (mag + M), with 0 for g where it is exact. The maximum that scores are taken
    from moves at most once for every 32 tokens, by a sum off by u M. exp2 is off by 2 u, and 4 u more
    where parts of the row are joined. So a weight is off by r_t = ln 2 (that sum) + 2^-20, relative;
    the sum that divides by R = sum p_t r_t + n u; weights below 2^-119 of the largest may be lost.

    Values: the weight times V's step is rounded to binary16 after a multiplication by a power of
    two that brings the step to 1 or more (so that the weight of the largest score, 1 at least, and
    those below it keep 11 bits, 2^-11 of the product, down to 2^-25 of the largest weight; a
    rounding moves nothing by more than itself), and meets a code less the middle one, at most
    2^(nbits - 1). The sums of n such products and of weights times middles add (n + 4) u."""
    c = held.c
    heads, dim, g = c["n_heads"], c["head_dim"], c["group_size"]
    u = 2.0 ** -24
    n, hq, _ = q.shape
    per, groups = hq // heads, dim // g
    out = torch.full((n, hq, dim), math.nan, dtype=torch.float64)
    lse = torch.full((n, hq), math.nan, dtype=torch.float64)
    bound, blse = torch.zeros_like(out), torch.zeros_like(lse)

    def grids(which, pages, m):
        """Values, base and step (by dimension) of the first m tokens: [heads, m, dim] each."""
        size, n_pages = c["page_size"], c["k_codes"].shape[0]
        pages = list(pages)[:-(-m // size)]
        ok = torch.tensor([0 <= p < n_pages for p in pages], dtype=torch.bool).repeat_interleave(size)[:m]
        idx = torch.tensor([p if 0 <= p < n_pages else 0 for p in pages], dtype=torch.long)
        meta = c[which + "_meta"].cpu()[idx].double()
        parts = [held.part[which][0][idx]] + [meta[..., e].repeat_interleave(g, -1) for e in (1, 0)]
        parts = [x.transpose(0, 1).reshape(heads, -1, dim)[:, :m] for x in parts]
        return [torch.where(ok[None, :, None], x, torch.zeros_like(x)) for x in parts] + [ok]

    pre = {w: grids(w, prefix_pages, prefix_len) for w in "kv"}
    for b, (lo, hi) in enumerate(R.rows_of(cu, n, len(lens))):
        if hi == lo:
            continue
        ln = min(max(lens[b], 0), len(table[b]) * c["page_size"])
        own = {w: grids(w, table[b], ln) for w in "kv"}
        (k, kb, ks), (v, vb, vs) = ([torch.cat((pre[w][e], own[w][e]), 1) for e in range(3)] for w in "kv")
        tokens = prefix_len + ln
        x = q[lo:hi].cpu().double().reshape(hi - lo, heads, per, dim).permute(1, 2, 0, 3)
        pos = ln - (hi - lo) + torch.arange(hi - lo)
        seen = torch.cat((pre["k"][3][None].expand(hi - lo, -1),
                          own["k"][3][None] & (torch.arange(ln)[None] <= pos[:, None])), 1)[None, None]
        s = torch.matmul(x, k.transpose(1, 2)[:, None]) * (scale * LOG2E)
        if whole:
            mag = torch.zeros_like(s)
            for a in range(0, dim, g):
                y = x[..., a:a + g]
                kq = torch.where(ks[..., a:a + g] > 0, k[..., a:a + g] - kb[..., a:a + g], 0.0)
                mag += torch.matmul(y, kq.transpose(1, 2)[:, None]).abs()
                mag += y.sum(-1, keepdim=True).abs() * kb[:, None, None, :, a].abs()
        else:
            mag = torch.matmul(x.abs(), (kb.abs() + (k - kb).abs()).transpose(1, 2)[:, None])
        mag = (mag * abs(scale) * LOG2E).masked_fill(~seen, 0.0)
        big = s.abs().masked_fill(~seen, 0.0).amax(-1, keepdim=True) if tokens else torch.zeros(*s.shape[:-1], 1, dtype=s.dtype)
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True) if tokens else torch.full((*s.shape[:-1], 1), -math.inf, dtype=s.dtype)
        w = torch.exp2(s - m.clamp(min=-1e300))
        tot = w.sum(-1, keepdim=True)
        p = w / tot.clamp(min=1e-300)
        top = 1 / tot.clamp(min=1.0)            # the largest weight
        r = math.log(2) * ((0 if whole else g) + 2 * groups + 8) * u * (mag + big) + \
            math.log(2) * (tokens / 32 + 2) * u * big + 2.0 ** -20
        lost = torch.minimum(p, 2.0 ** -119 * top)
        total = (p * r + lost).sum(-1, keepdim=True) + tokens * u
        half, top_code = 2.0 ** (c["nbits"] - 1), 2.0 ** c["nbits"] - 1

        def weigh(y, z):
            return torch.matmul(y, z[:, None])
        size = vb.abs() + (v - vb).abs()
        e = weigh(p * (r + total) + lost, torch.maximum(size, vs * top_code + vb.abs()))
        e = e + weigh(2.0 ** -11 * p + torch.minimum(p, 2.0 ** -25 * top), vs * half)
        e = e + (tokens + 4) * u * weigh(p, vs * half + (vb + vs * half).abs())
        put = lambda y: y.permute(2, 0, 1, *range(3, y.dim())).reshape(hi - lo, hq, *y.shape[3:])
        out[lo:hi], bound[lo:hi] = put(weigh(p, v)), put(e)
        lse[lo:hi] = put((m + torch.log2(tot)).squeeze(-1)) / LOG2E
        worst = r.masked_fill(~seen, 0.0).amax(-1) if tokens else torch.zeros(s.shape[:-1], dtype=s.dtype)
        blse[lo:hi] = put(worst + total.squeeze(-1) + m.squeeze(-1).abs().nan_to_num(0, 0, 0) * 2.0 ** -22 + 2.0 ** -20)
    return out, lse, bound, blse


# half of the spacing of the smallest numbers; what sums may lose, below a step of bfloat16's grids
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -100}


def check(got, got_lse, ref, mine):
    """Compares a call's outputs with attention()'s; rows where `mine` is False are skipped."""
    out, lse, bound, blse = ref
    x, y, e = got.cpu().double()[mine], out[mine], bound[mine]
    tol = e + R.HALF_STEP[got.dtype] * (y.abs() + e) + SMALLEST[got.dtype]
    assert torch.isfinite(x).all(), "outputs are not finite"
    bad = (x - y).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off, worst {float(((x - y).abs() / tol).max()):.3g} of the tolerance"
    if got_lse is not None:
        a, b = got_lse.cpu().double()[mine], lse[mine]
        none = torch.isinf(b)
        assert torch.equal(torch.isinf(a) & (a < 0), none), "rows that see nothing"
        d = (a - b).abs()[~none]
        assert (d <= blse[mine][~none]).all(), f"lse off by {float(d.max()):.3g}"
