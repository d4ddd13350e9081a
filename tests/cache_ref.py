"""The quantized key/value cache in plain 64-bit torch on the CPU, from its definition in
include/hqq.h: the grid, the layout of the pages, and attention over what they hold."""
import math

import torch

TOP = {4: 15, 8: 255}
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # a rounding's, relative


def grid(x, nbits, group):
    """Codes (int64) and step, base (float64) of values x [..., dim] of a 16-bit type."""
    top, dtype = TOP[nbits], x.dtype
    v = x.double().reshape(*x.shape[:-1], -1, group)
    base, span = v.amin(-1), v.amax(-1) - v.amin(-1)
    # the smallest number of the type with step * top >= span, among neighbours of span / top
    near = (span / top).to(dtype)
    bits = near.view(torch.int16)
    below = torch.where(bits > 0, bits - 1, bits).view(dtype).double()
    above = (bits + 1).view(dtype).double()
    step = torch.where(below * top >= span, below, torch.where(near.double() * top >= span, near.double(), above))
    if dtype == torch.bfloat16:
        step = torch.where(span > 0, step.clamp(min=2.0 ** -100), step)
    last = torch.full_like(step, top)
    if dtype == torch.float16:
        last = torch.where(base + top * step >= 65520.0, last - 1, last)
    q = ((v - base[..., None]) / torch.where(step > 0, step, torch.ones_like(step))[..., None]).round()
    q = torch.minimum(q, last[..., None]).to(torch.int64)
    return q.reshape(x.shape), step, base


def value(q, step, base):
    """base + q * step in float64, q [..., dim]."""
    g = q.shape[-1] // step.shape[-1]
    return (q.double().reshape(*step.shape, g) * step[..., None] + base[..., None]).reshape(q.shape)


def key_byte(t, d, dim, nbits):
    """Byte of the page and half of it that hold dimension d of token t's key."""
    a, m, e = d // 8 % 4, d // 32, d % 8
    unit = t * (dim * nbits // 8) + (a * (dim // 32) + m) * nbits
    return (unit + e % 4, e // 4) if nbits == 4 else (unit + e, 0)


def value_byte(t, d, dim, nbits, g):
    r, i = d % g // (g // 16), d // g * (g // 16) + d % (g // 16)
    row = (t // 4 * 16 + r) * 4 + t % 4
    width = dim // 16
    return (row * (width // 2) + i // 2, i % 2) if nbits == 4 else (row * width + i, 0)


def _places(page, dim, nbits, g, which):
    f = (lambda t, d: key_byte(t, d, dim, nbits)) if which == "k" else (lambda t, d: value_byte(t, d, dim, nbits, g))
    at = [[f(t, d) for d in range(dim)] for t in range(page)]
    return torch.tensor([[x[0] for x in row] for row in at]), torch.tensor([[x[1] for x in row] for row in at])


def pages_to_codes(buf, page, dim, nbits, g, which):
    """uint8 [n_pages, heads, bytes] -> int64 codes [n_pages, heads, page, dim]."""
    byte, half = _places(page, dim, nbits, g, which)
    x = buf.cpu().to(torch.int64)[:, :, byte]
    return x if nbits == 8 else (x >> (4 * half)) & 15


def codes_to_pages(q, nbits, g, which):
    n, h, page, dim = q.shape
    byte, half = _places(page, dim, nbits, g, which)
    out = torch.zeros(n, h, page * dim * nbits // 8, dtype=torch.int64)
    flat = (q << (4 * half)).reshape(n, h, -1)
    out.scatter_add_(2, byte.reshape(-1).expand(n, h, -1), flat)     # halves of a byte add up
    return out.to(torch.uint8)


def rows_of(cu, n_tokens, n_seqs):
    if cu is None:
        each = n_tokens // n_seqs
        return [(b * each, b * each + each) for b in range(n_seqs)]
    out = []
    for b in range(n_seqs):
        lo = min(max(cu[b], 0), n_tokens)
        out.append((lo, min(max(cu[b + 1], lo), n_tokens)))
    return out


def where(table, lens, cu, n_tokens, page, n_pages):
    """For every row of a call: None (of no sequence) or (sequence, position, page or -1)."""
    at = [None] * n_tokens
    for b, (lo, hi) in enumerate(rows_of(cu, n_tokens, len(lens))):
        ln = min(max(lens[b], 0), len(table[b]) * page)
        for i in range(lo, hi):
            pos = ln - (hi - i)
            p = table[b][pos // page] if 0 <= pos < len(table[b]) * page else -1
            at[i] = (b, pos, p if 0 <= p < n_pages else -1)
    return at


class Held:
    """What a cache's buffers hold, on the CPU in 64 bits."""

    def __init__(self, cache):
        self.c = cache
        args = (cache["page_size"], cache["head_dim"], cache["nbits"], cache["group_size"])
        self.part = {}
        for w in "kv":
            q = pages_to_codes(cache[w + "_codes"], *args, w).double()
            m = cache[w + "_meta"].cpu().double()
            g = cache["group_size"]
            step = m[..., 0].repeat_interleave(g, -1)
            base = m[..., 1].repeat_interleave(g, -1)
            self.part[w] = (base + q * step, base.abs() + q * step)

    def steps(self, pages, n):
        """V's steps by dimension of the first n tokens of `pages`, [heads, n, dim]; 0 where not
        in the cache."""
        c, size = self.c, self.c["page_size"]
        pages = list(pages)[:-(-n // size)]
        n_pages = c["k_codes"].shape[0]
        ok = torch.tensor([0 <= p < n_pages for p in pages], dtype=torch.bool).repeat_interleave(size)[:n]
        idx = torch.tensor([p if 0 <= p < n_pages else 0 for p in pages], dtype=torch.long)
        step = c["v_meta"].cpu().double()[..., 0].repeat_interleave(c["group_size"], -1)
        y = step[idx].transpose(0, 1).reshape(c["n_heads"], -1, c["head_dim"])[:, :n]
        return torch.where(ok[None, :, None], y, torch.zeros_like(y))

    def tokens(self, which, pages, n):
        """Values and their parts' magnitudes of the first n tokens of `pages`: [heads, n, dim],
        and which of them are in the cache."""
        c, size = self.c, self.c["page_size"]
        n_pages = c["k_codes"].shape[0]
        pages = list(pages)[:-(-n // size)]
        ok = torch.tensor([0 <= p < n_pages for p in pages], dtype=torch.bool).repeat_interleave(size)[:n]
        idx = torch.tensor([p if 0 <= p < n_pages else 0 for p in pages], dtype=torch.long)
        out = []
        for x in self.part[which]:
            y = x[idx].transpose(0, 1).reshape(c["n_heads"], -1, c["head_dim"])[:, :n]
            out.append(torch.where(ok[None, :, None], y, torch.zeros_like(y)))
        return out[0], out[1], ok


def attention(held, table, lens, cu, q, scale, prefix_pages=(), prefix_len=0):
    """(out, lse, bound) in float64 for q [n, heads, dim]; rows of no sequence are NaN. `bound`
    is how far a binary32 evaluation with V's weights rounded to binary16 may be off, before the
    output's own rounding:

    A score is a sum of dim exact products of a 16-bit number and a code, scaled: its error is
    at most (dim + 8) 2^-24 of the sum of magnitudes S (2 of the 8 for bases that enter as
    products of bfloat16 parts, which leave out 2^-23 of theirs), so a weight's relative error is twice
    scale*S*(dim + 8)*2^-24, once more for the sum that divides, plus 2^-18 for exp2 (its
    argument below 2^6 in magnitude where it matters, and a unit in the last place). Sums over
    n tokens add n 2^-24 at most. All of it weighs on A = sum of p (|base| + q step).
    Weight times step is rounded to binary16's 11 bits, by at most half a step of them, and
    meets a code less the middle one: 2^-11 of sum p step 2^(nbits - 1), and where it is below
    binary16's normal numbers n 2^-26 of the largest step (steps are scaled to 2^8, the
    largest weight is at least 1, and a subnormal number is off by 2^-25 at most)."""
    c = held.c
    heads, dim = c["n_heads"], c["head_dim"]
    n, hq, _ = q.shape
    per = hq // heads
    out = torch.full((n, hq, dim), math.nan, dtype=torch.float64)
    lse = torch.full((n, hq), math.nan, dtype=torch.float64)
    bound = torch.zeros((n, hq, dim), dtype=torch.float64)
    blse = torch.zeros((n, hq), dtype=torch.float64)
    pk, pka, pok = held.tokens("k", prefix_pages, prefix_len)
    pv, pva, _ = held.tokens("v", prefix_pages, prefix_len)
    for b, (lo, hi) in enumerate(rows_of(cu, n, len(lens))):
        if hi == lo:
            continue
        ln = min(max(lens[b], 0), len(table[b]) * c["page_size"])
        k, ka, ok = held.tokens("k", table[b], ln)
        v, va, _ = held.tokens("v", table[b], ln)
        k, ka, v, va = (torch.cat(x, 1) for x in ((pk, k), (pka, ka), (pv, v), (pva, va)))
        x = q[lo:hi].cpu().double().reshape(hi - lo, heads, per, dim).permute(1, 2, 0, 3)
        s = torch.einsum("hptd,hsd->hpts", x, k) * scale
        mag = torch.einsum("hptd,hsd->hpts", x.abs(), ka) * abs(scale)
        pos = ln - (hi - lo) + torch.arange(hi - lo)
        seen = torch.cat((pok[None].expand(hi - lo, -1), ok[None] & (torch.arange(ln)[None] <= pos[:, None])), 1)
        s = s.masked_fill(~seen[None, None], -math.inf)
        m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full((*s.shape[:-1], 1), -math.inf, dtype=torch.float64)
        w = torch.exp(s - m.clamp(min=-1e300))
        tot = w.sum(-1, keepdim=True)
        p = w / tot.clamp(min=1e-300)
        o = torch.einsum("hpts,hsd->hptd", p, v)
        a = torch.einsum("hpts,hsd->hptd", p, va)
        vs = torch.cat((held.steps(prefix_pages, prefix_len), held.steps(table[b], ln)), 1) * 2.0 ** (c["nbits"] - 1)
        a2 = torch.einsum("hpts,hsd->hptd", p, vs) * 2.0 ** -11
        if vs.shape[1]:
            a2 = a2 + s.shape[-1] * 2.0 ** -26 * vs.amax((0, 1, 2)) * 2
        ds = torch.where(p > 1e-12, mag, torch.zeros_like(mag)).amax(-1, keepdim=True) * (dim + 8) * 2.0 ** -24 \
            if s.shape[-1] else torch.zeros_like(m)
        rel = 4 * ds + 2.0 ** -17 + s.shape[-1] * 2.0 ** -24
        out[lo:hi] = o.permute(2, 0, 1, 3).reshape(hi - lo, hq, dim)
        bound[lo:hi] = (a * rel + a2).permute(2, 0, 1, 3).reshape(hi - lo, hq, dim)
        lse[lo:hi] = (m + torch.log(tot)).squeeze(-1).permute(2, 0, 1).reshape(hi - lo, hq)
        blse[lo:hi] = (2 * ds + 2.0 ** -18 + s.shape[-1] * 2.0 ** -24 + m.abs().nan_to_num(0, 0, 0) * 2.0 ** -22) \
            .squeeze(-1).permute(2, 0, 1).reshape(hi - lo, hq)
    return out, lse, bound, blse


def check_attention(got, got_lse, ref, mine):
    """Compares a call's outputs with attention()'s; rows where `mine` is False are skipped."""
    out, lse, bound, blse = ref
    dtype = got.dtype
    x, y = got.cpu().double()[mine], out[mine]
    tol = bound[mine] + HALF_STEP[dtype] * (y.abs() + bound[mine]) + 2.0 ** -25
    bad = (x - y).abs() > tol
    assert torch.isfinite(x).all(), "outputs are not finite"
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off, worst {float(((x - y).abs() / tol).max()):.3g} of the tolerance"
    if got_lse is not None:
        a, b = got_lse.cpu().double()[mine], lse[mine]
        none = torch.isinf(b)
        assert torch.equal(torch.isinf(a) & (a < 0), none), "rows that see nothing"
        e = (a - b).abs()[~none]
        assert (e <= blse[mine][~none]).all(), f"lse off by {float(e.max()):.3g}"
