"""The quantized key/value cache: writing and reading it back, and attention over it.

The cases, inputs and plain forms of four operators that work on one paged cache of one layer:

* writing tokens' keys and values into the cache as 8- or 4-bit codes, and reading them back;
* reading whole sequences back;
* attention of new tokens over the cache (one token per sequence, a few, or a prompt's chunk);
* the same for a batch whose sequences share a long prefix that the cache holds once.

The cache. A head's vector of one token (``head_dim`` values) is cut into groups of
``group_size``. A group's values v become codes q on a min-max grid, both in the type of the
values (binary16 or bfloat16):

    base = min(v)
    step = the smallest number of the type with step >= (max(v) - min(v)) / (2^nbits - 1);
           0 when the range is 0, at least 2^-100 otherwise
    q    = min(round to nearest, ties to even, of the exact (v - base) / step, top)
    top  = 2^nbits - 1, or one less when base + (2^nbits - 1) * step would not be finite in
           the type

and stand for base + q * step. Codes lie in pages, uint8 ``[n_pages, heads, page bytes]``:

* keys: per token of the page, code e of unit (a, m) is dimension 32 m + 8 a + e; the units
  are in order (a, m), a < 4, m < head_dim / 32. A unit of 4-bit codes is 4 bytes, byte i
  with code i in its low half and code i + 4 in its high half; of 8-bit codes, 8 bytes.
* values: per four tokens, 16 rows r; in a row the four tokens in turn, each with the codes of
  the dimensions group * G + r * (G / 16) + j (G = group_size) in order (group, j); 4-bit
  codes go two to a byte, the first in the low half.

``k_meta`` and ``v_meta`` hold {step, base}: ``[n_pages, heads, page_size, groups, 2]``.
``table[b]`` lists the pages of sequence b in order, -1 behind the last; ``lens[b]`` is its
length with the call's own tokens, which are its last ones. Tokens of a call lie one sequence
after another: sequence b has rows ``cu[b]`` to ``cu[b + 1]``.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------------------------
def _case(kind, dtype, nbits, group, dim, kv_heads, per_head, page, seqs, lo, hi, new, prefix=0):
    """lo..hi: lengths over the batch; new: tokens of the call for each sequence (0: all)."""
    return {"kind": kind, "dtype": dtype, "nbits": nbits, "group": group, "dim": dim,
            "kv_heads": kv_heads, "per_head": per_head, "page": page, "seqs": seqs, "lo": lo,
            "hi": hi, "new": new, "prefix": prefix}


def listed():
    c = _case
    rows = {
        # one token of one sequence enters the cache: a decode step's smallest call
        "write 1 token": c("write", "fp16", 4, 64, 128, 8, 1, 64, 1, 700, 700, 1),
        # a decode step of a large batch, one token for each sequence
        "write 256 x 1 token": c("write", "bf16", 8, 128, 128, 8, 1, 32, 256, 1, 600, 1),
        # prompts of odd lengths enter the cache whole, a layer with as many key heads as query heads
        "write 8 prompts": c("write", "fp16", 4, 64, 128, 32, 1, 64, 8, 515, 4001, 0),
        # short sequences read back, small heads and groups, pages of 16
        "read 16 short": c("read", "bf16", 4, 32, 64, 8, 1, 16, 16, 1, 1999, 0),
        # one long context read back for a layer that wants it in full
        "read 1 long": c("read", "fp16", 8, 128, 128, 8, 1, 128, 1, 65521, 65521, 0),
        # the first tokens of one answer: one sequence, a short context, 32 heads
        "attend 1 x 300": c("attend", "fp16", 4, 64, 128, 32, 1, 64, 1, 300, 300, 1),
        # a decode step of a served batch, eight query heads to a key head
        "attend 64 x 8190": c("attend", "bf16", 4, 64, 128, 8, 8, 64, 64, 4100, 8190, 1),
        # one token over a very long context
        "attend 1 x 131071": c("attend", "fp16", 8, 128, 128, 8, 8, 128, 1, 131071, 131071, 1),
        # five tokens a sequence, drafted and to be checked at once, wide heads
        "attend 16 x 2900, 5 new": c("attend", "bf16", 8, 64, 256, 4, 4, 32, 16, 800, 2900, 5),
        # a chunk of two prompts over what came before it
        "attend 2 x 4000, 500 new": c("attend", "fp16", 4, 64, 128, 40, 1, 64, 2, 3500, 4000, 500),
        # a few questions to one instruction of a page or two
        "prefix 1000, 8 x 60": c("prefix", "fp16", 4, 64, 128, 40, 1, 16, 8, 1, 60, 1, 1000),
        # many questions to one long document
        "prefix 16390, 64 x 1000": c("prefix", "bf16", 4, 64, 128, 8, 8, 64, 64, 1, 1000, 1, 16390),
    }
    return [dict(v, name=k) for k, v in rows.items()]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [work(c) for c in listed()]
    by, fl = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        kind = rng.choice(["write", "read", "attend", "attend", "prefix"])
        dim = rng.choice([64, 128, 128, 256])
        group = rng.choice([g for g in (32, 64, 128) if g <= dim])
        kv, per = rng.choice([(8, 8), (8, 4), (32, 1), (40, 1), (4, 4), (2, 7), (1, 16), (5, 3)])
        seqs, hi = _log(rng, 1, 256), _log(rng, 1, 131071)
        lo = rng.choice([1, (hi + 1) // 2, hi])
        new = prefix = 0
        if kind == "prefix":
            seqs, hi, prefix = min(seqs, 96), min(hi, 2000), _log(rng, 1, 32000)
            lo = min(lo, hi)
        if kind == "write":
            new = rng.choice([0, 1, 1, _log(rng, 1, hi)])
        elif kind in ("attend", "prefix"):
            new = rng.choice([1, 1, 1, _log(rng, 2, 9), _log(rng, 1, 600)])
        if kind == "write" or kind == "read":
            per = 1
        new = min(new, hi)
        c = _case(kind, rng.choice(["fp16", "bf16"]), rng.choice([4, 8]), group, dim, kv, per,
                  rng.choice([16, 32, 64, 128, 256]), seqs, lo, hi, new, prefix)
        w, tokens = work(c), seqs * hi + prefix
        rows = sum(_new(c)) * kv * per
        # within the listed cases' work, and with room for the plain form's 32-bit scores
        if w["bytes"] <= by and w["flops"] <= fl and tokens * kv * dim <= 1 << 29 and \
                (kind in ("write", "read") or rows * (hi + prefix) <= 1 << 29):
            return c


def _lens(c):
    """Lengths of the sequences, the call's tokens included: lo to hi in mixed order."""
    n, span = c["seqs"], c["hi"] - c["lo"]
    return [c["hi"] - (span * ((i * 37) % n)) // max(n - 1, 1) for i in range(n)]


def _new(c):
    """Tokens of the call for each sequence; where several are, every third has one less."""
    lens = _lens(c)
    if c["new"] == 0:
        return lens
    return [min(ln, c["new"] - (1 if c["new"] > 1 and i % 3 == 2 else 0)) for i, ln in enumerate(lens)]


def work(c):
    lens, new, groups = _lens(c), _new(c), c["dim"] // c["group"]
    row = c["kv_heads"] * 2 * (c["dim"] * c["nbits"] // 8 + groups * 4)  # a token in the cache
    n = sum(new)
    full = n * c["kv_heads"] * c["dim"] * 2 * 2                           # its plain k and v
    if c["kind"] == "write":
        return {"bytes": 2 * full + 2 * n * row, "flops": 8 * n * c["kv_heads"] * c["dim"]}
    if c["kind"] == "read":
        return {"bytes": full + n * row, "flops": 4 * n * c["kv_heads"] * c["dim"]}
    heads = c["kv_heads"] * c["per_head"]
    # a token sees its sequence up to itself, and the whole prefix
    seen = sum(t * ln - t * (t - 1) // 2 for t, ln in zip(new, lens)) + n * c["prefix"]
    return {"bytes": (sum(lens) + c["prefix"]) * row + 2 * n * heads * c["dim"] * 2,
            "flops": 4 * seen * heads * c["dim"]}


# ---- inputs ----------------------------------------------------------------------------------
def _values(n, heads, dim, dtype, gen, channels):
    """Keys or values of n tokens: normal, with a mean and a width of its own per channel
    (a few channels of keys stand out by far in trained models)."""
    mean, width = channels
    x = torch.randn(n, heads, dim, generator=gen, device="cuda")
    return (x * width + mean).to(dtype)


def _channels(heads, dim, gen, spread):
    r = torch.rand(heads, dim, generator=gen, device="cuda")
    mean = torch.randn(heads, dim, generator=gen, device="cuda") * (0.2 + spread * (r > 0.97))
    return mean, 0.6 + 0.8 * r


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, heads, dim, page = TYPES[c["dtype"]], c["kv_heads"], c["dim"], c["page"]
    lens, new = _lens(c), _new(c)
    per_seq = [-(-ln // page) for ln in lens]
    pre_pages = -(-c["prefix"] // page)
    used = sum(per_seq) + pre_pages
    n_pages = used + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda")[:used].to(torch.int32)
    table = torch.full((c["seqs"], max(per_seq)), -1, dtype=torch.int32)
    pages = order.cpu()
    at = pre_pages
    for b, n in enumerate(per_seq):
        table[b, :n] = pages[at:at + n]
        at += n
    groups = dim // c["group"]
    cache = {"k_codes": torch.zeros(n_pages, heads, page * dim * c["nbits"] // 8, dtype=torch.uint8, device="cuda"),
             "v_codes": torch.zeros(n_pages, heads, page * dim * c["nbits"] // 8, dtype=torch.uint8, device="cuda"),
             "k_meta": torch.zeros(n_pages, heads, page, groups, 2, dtype=dtype, device="cuda"),
             "v_meta": torch.zeros(n_pages, heads, page, groups, 2, dtype=dtype, device="cuda"),
             "page_size": page, "n_heads": heads, "head_dim": dim, "nbits": c["nbits"],
             "group_size": c["group"]}
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    n = cu[-1]
    kc, vc = _channels(heads, dim, gen, 4.0), _channels(heads, dim, gen, 0.0)
    s = {"case": c, "cache": cache, "table": table.cuda(), "prefix_pages": order[:pre_pages].contiguous(),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "n": n,
         # which sequence and which place of the call's tokens a row is
         "seq_of": torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(new)).cuda(),
         "most_new": max(new)}
    s["place"] = torch.arange(n, device="cuda") - s["cu"].long()[s["seq_of"]]
    s["pos"] = s["lens"].long()[s["seq_of"]] - torch.tensor(new, device="cuda")[s["seq_of"]] + s["place"]
    if c["kind"] == "write":
        s["k"] = _values(n, heads, dim, dtype, gen, kc)
        s["v"] = _values(n, heads, dim, dtype, gen, vc)
        return s
    # a full cache: every page holds tokens, a few pages at a time
    chunk = max(1, (1 << 25) // (page * heads * dim))
    for a in range(0, n_pages, chunk):
        m = min(chunk, n_pages - a)
        for codes, meta, units, ch in (("k_codes", "k_meta", _k_units, kc), ("v_codes", "v_meta", _v_units, vc)):
            q, mt = _quantize(_values(m * page, heads, dim, dtype, gen, ch), c["nbits"], c["group"])
            cache[codes][a:a + m] = units(q.view(m, page, heads, dim).transpose(1, 2), c["nbits"], c["group"])
            cache[meta][a:a + m] = mt.view(m, page, heads, groups, 2).transpose(1, 2)
    if c["kind"] != "read":
        s["q"] = torch.randn(n, heads * c["per_head"], dim, generator=gen, device="cuda").to(dtype)
    return s


# ---- plain forms -----------------------------------------------------------------------------
def _quantize(x, nbits, group):
    """Codes (uint8, x's shape) and {step, base} of values x [..., dim]."""
    top, dtype = 2 ** nbits - 1, x.dtype
    v = x.reshape(*x.shape[:-1], -1, group)
    base = v.amin(-1)
    span = v.amax(-1).double() - base.double()
    near = (span / top).to(dtype)
    up = (near.view(torch.int16) + 1).view(dtype)  # the next number of the type
    step = torch.where(near.double() * top < span, up, near)
    if dtype == torch.bfloat16:
        step = torch.where(span > 0, step.clamp(min=2.0 ** -100), step)
    last = base.float() + top * step.float()
    cap = torch.where(last >= 65520.0, top - 1, top) if dtype == torch.float16 else torch.full_like(last, top)
    # in 64 bits: a quotient next to a half goes the way of its exact value
    safe = torch.where(step > 0, step, torch.ones_like(step)).double()
    q = ((v.double() - base.double()[..., None]) / safe[..., None]).round()
    q = torch.minimum(q, cap.double()[..., None]).to(torch.uint8)
    return q.view(x.shape), torch.stack((step, base), -1)


def _k_units(q, nbits, group):
    """Codes [pages, heads, tokens, dim] as pages of keys."""
    u = q.reshape(*q.shape[:-1], -1, 4, 8).transpose(-3, -2)
    if nbits == 4:
        u = u[..., :4] | (u[..., 4:] << 4)
    return u.reshape(*q.shape[:2], -1)


def _v_units(q, nbits, group):
    """Codes [pages, heads, tokens, dim] as pages of values."""
    p, h, t, d = q.shape
    u = q.reshape(p, h, t // 4, 4, d // group, 16, group // 16).permute(0, 1, 2, 5, 3, 4, 6).reshape(p, h, -1)
    if nbits == 4:
        u = u[..., 0::2] | (u[..., 1::2] << 4)
    return u


def _keys(cache, pages):
    """What the cache holds of the keys of `pages` [..., n]: float32 [..., heads, tokens, dim]."""
    return _stands_for(cache, pages, "k", False)


def _stands_for(cache, pages, which, of_values):
    nbits, group, dim = cache["nbits"], cache["group_size"], cache["head_dim"]
    at = pages.clamp(min=0).long().reshape(-1)
    c, m = cache[which + "_codes"][at], cache[which + "_meta"][at].float()
    n, h, _ = c.shape
    if of_values:
        if nbits == 4:
            c = torch.stack((c & 15, c >> 4), -1)
        c = c.reshape(n, h, -1, 16, 4, dim // group, group // 16).permute(0, 1, 2, 4, 5, 3, 6)
    else:
        c = c.reshape(n, h, -1, 4, dim // 32, nbits)
        if nbits == 4:
            c = torch.cat((c & 15, c >> 4), -1)
        c = c.transpose(-3, -2)
    x = c.reshape(n, h, -1, dim // group, group).float() * m[..., 0:1] + m[..., 1:2]
    x = x.reshape(*pages.shape, h, -1, dim)
    return x.transpose(-4, -3).reshape(*pages.shape[:-1], h, -1, dim)


def _values_of(cache, pages):
    return _stands_for(cache, pages, "v", True)


def _plain_write(s):
    cache = s["cache"]
    nbits, group, dim, page, heads = (cache[k] for k in ("nbits", "group_size", "head_dim", "page_size", "n_heads"))
    at = s["table"].long()[s["seq_of"], s["pos"] // page]
    t = s["pos"] % page
    q, meta = _quantize(s["k"], nbits, group)
    cache["k_meta"][at, :, t] = meta
    cache["k_codes"].view(-1, heads, page, dim * nbits // 8)[at, :, t] = _k_units(q[:, :, None], nbits, group)
    q, meta = _quantize(s["v"], nbits, group)
    cache["v_meta"][at, :, t] = meta
    # a token's codes lie 16 rows apart, in its quarter of each
    u = q.reshape(s["n"], heads, dim // group, 16, group // 16).transpose(2, 3).reshape(s["n"], heads, 16, -1)
    if nbits == 4:
        u = u[..., 0::2] | (u[..., 1::2] << 4)
    cache["v_codes"].view(-1, heads, page // 4, 16, 4, dim * nbits // 128)[at, :, t // 4, :, t % 4] = u


def _plain_read(s):
    cache = s["cache"]
    page = cache["page_size"]
    at = s["table"].long()[s["seq_of"], s["pos"] // page]
    row = at * page + s["pos"] % page
    pages, back = torch.unique(at, return_inverse=True)
    row = back * page + s["pos"] % page
    dtype = cache["k_meta"].dtype
    return {"k": _keys(cache, pages)[:, row].transpose(0, 1).to(dtype).contiguous(),
            "v": _values_of(cache, pages)[:, row].transpose(0, 1).to(dtype).contiguous()}


def _plain_attend(s):
    c, cache, q = s["case"], s["cache"], s["q"]
    heads, per, dim, n = c["kv_heads"], c["per_head"], c["dim"], s["n"]
    t = s["most_new"]
    # queries by sequence, [seqs, heads, per * t, dim], rows beyond a sequence's own are zero
    x = torch.zeros(c["seqs"], t, heads, per, dim, device="cuda")
    x[s["seq_of"], s["place"]] = q.float().view(n, heads, per, dim)
    pos = torch.full((c["seqs"], t), -1, device="cuda")
    pos[s["seq_of"], s["place"]] = s["pos"]
    x = x.permute(0, 2, 3, 1, 4).reshape(c["seqs"], heads, per * t, dim) / math.sqrt(dim)
    k = _keys(cache, s["table"])
    score = torch.matmul(x, k.transpose(-1, -2).contiguous())
    del k
    seen = torch.arange(score.shape[-1], device="cuda") <= pos[:, :, None]
    score = score.view(c["seqs"], heads, per, t, -1).masked_fill_(~seen[:, None, None], -math.inf)
    if c["prefix"]:
        pk = _keys(cache, s["prefix_pages"])[:, :c["prefix"]]
        y = x.transpose(0, 1).reshape(heads, -1, dim)
        first = torch.matmul(y, pk.transpose(-1, -2).contiguous())
        first = first.view(heads, c["seqs"], per, t, -1).transpose(0, 1)
        score = torch.cat((first, score), -1)
    score = score - score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-38)
    own_part = p[..., c["prefix"]:].reshape(c["seqs"], heads, per * t, -1)
    out = torch.matmul(own_part, _values_of(cache, s["table"])).view(c["seqs"], heads, per, t, dim)
    if c["prefix"]:
        pv = _values_of(cache, s["prefix_pages"])[:, :c["prefix"]].contiguous()
        w = p[..., :c["prefix"]].transpose(0, 1).reshape(heads, -1, c["prefix"])
        out = out + torch.matmul(w, pv).view(heads, c["seqs"], per, t, dim).transpose(0, 1)
    out = out.permute(0, 3, 1, 2, 4)[s["seq_of"], s["place"]]
    return out.reshape(n, heads * per, dim).to(q.dtype)


def run(s):
    kind = s["case"]["kind"]
    if own:
        from calibration_free_weight_amd import hqq
        cache, table, lens, cu = s["cache"], s["table"], s["lens"], s["cu"]
        if kind == "write":
            hqq.hqq_cache_write(cache, table, lens, s["k"], s["v"], cu_tokens=cu)
        if kind in ("write", "read"):
            k, v = hqq.cache_read(cache, table, lens, s["n"], cu_tokens=cu)
            return {"k": k, "v": v}
        if kind == "prefix":
            return hqq.cache_attention_prefix(cache, table, lens, s["prefix_pages"], s["case"]["prefix"],
                                              s["q"], cu_tokens=cu)
        return hqq.cache_attention(cache, table, lens, s["q"], cu_tokens=cu)
    if kind == "write":
        _plain_write(s)
    return _plain_read(s) if kind in ("write", "read") else _plain_attend(s)


# ---- the definition in 64 bits ---------------------------------------------------------------
def _code_at(codes, nbits, byte, high):
    b = codes[..., byte].to(torch.int64)
    return b if nbits == 8 else torch.where(high, b >> 4, b & 15)


def _token_values(s, which, pages):
    """The values of the tokens of `pages` [n], by each dimension's own byte: [heads, tokens, dim]."""
    cache, c = s["cache"], s["case"]
    nbits, g, dim, page = c["nbits"], c["group"], c["dim"], c["page"]
    d = torch.arange(dim, device="cuda")
    t = torch.arange(page, device="cuda")[:, None]
    if which == "k":
        unit = (d // 8 % 4) * (dim // 32) + d // 32
        byte = t * (dim * nbits // 8) + unit * nbits + (d % 8 if nbits == 8 else d % 4)
        high = d % 8 >= 4
    else:
        r, i = d % g // (g // 16), d // g * (g // 16) + d % (g // 16)
        byte = ((t // 4 * 16 + r) * 4 + t % 4) * (dim * nbits // 128) + (i if nbits == 8 else i // 2)
        high = i % 2 == 1
    q = _code_at(cache[which + "_codes"][pages], nbits, byte, high.expand(page, dim)).double()
    m = cache[which + "_meta"][pages].double()[:, :, :, d // g]
    return (q * m[..., 0] + m[..., 1]).transpose(0, 1).reshape(c["kv_heads"], -1, dim)


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e11:
        return None
    s = prepare(case, seed)
    lens, new = _lens(case), _new(case)
    if case["kind"] == "write":
        out = {}
        for name in ("k", "v"):
            x = s[name].double().reshape(s["n"], case["kv_heads"], -1, case["group"])
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            top, bits = 2 ** case["nbits"] - 1, 10 if case["dtype"] == "fp16" else 7
            want = (hi - lo) / top
            # the type's grid around `want`: bits + 1 significant bits
            want = want.clamp(min=2.0 ** (-14 if bits == 10 else -100))
            unit = want / torch.frexp(want).mantissa * 2.0 ** (-1 - bits)
            step = torch.ceil((hi - lo) / (top * unit)) * unit
            q = torch.round((x - lo) / step.clamp(min=1e-300)).clamp(max=top)
            out[name] = (lo + q * step).reshape(s[name].shape)
        return out
    parts = {"k": [], "v": []} if case["kind"] == "read" else []
    pre = s["prefix_pages"].long()
    at = 0
    for b, (ln, t) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-ln // case["page"])].long()
        k, v = (_token_values(s, x, pages)[:, :ln] for x in ("k", "v"))
        if case["kind"] == "read":
            parts["k"].append(k[:, ln - t:].transpose(0, 1))
            parts["v"].append(v[:, ln - t:].transpose(0, 1))
            continue
        if case["prefix"]:
            if b == 0:
                pk, pv = (_token_values(s, x, pre)[:, :case["prefix"]] for x in ("k", "v"))
            k, v = torch.cat((pk, k), 1), torch.cat((pv, v), 1)
        q = s["q"][at:at + t].double().view(t, case["kv_heads"], case["per_head"], -1).permute(1, 2, 0, 3)
        sc = torch.matmul(q.reshape(case["kv_heads"], -1, case["dim"]), k.transpose(1, 2)) / math.sqrt(case["dim"])
        sc = sc.view(case["kv_heads"], case["per_head"], t, -1)
        last = case["prefix"] + ln - t + torch.arange(t, device="cuda")
        sc.masked_fill_(torch.arange(sc.shape[-1], device="cuda") > last[:, None], -math.inf)
        p = torch.softmax(sc, -1).view(case["kv_heads"], -1, sc.shape[-1])
        o = torch.matmul(p, v).view(case["kv_heads"], case["per_head"], t, -1)
        parts.append(o.permute(2, 0, 1, 3).reshape(t, -1, case["dim"]))
        at += t
    if case["kind"] == "read":
        return {k: torch.cat(v) for k, v in parts.items()}
    return torch.cat(parts)
