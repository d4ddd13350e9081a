"""The quantized key/value cache on the GPU: written, read back and attended to, against its
definition in 64 bits (tests/cache_ref.py)."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


def poison(cache):
    """Every byte 0xff: codes at their top, grids NaN in either type."""
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
        cache[x].view(torch.uint8).fill_(255)
    return cache


def layout(lens, page, gen, spare=3, extra=1):
    """A table of shuffled pages (-1 behind each sequence's last) and the number of pages."""
    need = [-(-max(x, 0) // page) for x in lens]
    n = sum(need) + spare
    order = torch.randperm(n, generator=gen).tolist()
    width = max(need, default=0) + extra
    table, at = [], 0
    for k in need:
        table.append(order[at:at + k] + [-1] * (width - k))
        at += k
    return table, n, order[at:]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def values(n, heads, dim, dtype, gen, scale=1.0):
    x = torch.randn(n, heads, dim, generator=gen) * scale + torch.randn(heads, dim, generator=gen)
    return x.to(dtype).cuda()


def cumulated(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def expect_written(before, k, v, at):
    """The buffers a write leaves, from those before it: {name: tensor}, on the CPU."""
    c = before
    page, dim, nbits, g = c["page_size"], c["head_dim"], c["nbits"], c["group_size"]
    out = {}
    for w, x in (("k", k), ("v", v)):
        codes = R.pages_to_codes(c[w + "_codes"], page, dim, nbits, g, w)
        meta = c[w + "_meta"].cpu().clone()
        q, step, base = R.grid(x.cpu(), nbits, g)
        for i, a in enumerate(at):
            if a is None or a[2] < 0:
                continue
            codes[a[2], :, a[1] % page] = q[i]
            meta[a[2], :, a[1] % page] = torch.stack((step[i], base[i]), -1).to(meta.dtype)
        out[w + "_codes"] = R.codes_to_pages(codes, nbits, g, w)
        out[w + "_meta"] = meta
    return out


def same_bits(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


WRITES = [
    # dtype, nbits, dim, group, page, heads, lens, new (None: as long as the sequence)
    (F, 4, 128, 64, 64, 8, [1], [1]),
    (B, 4, 128, 64, 16, 3, [40, 1, 0, 17], None),
    (F, 8, 128, 128, 32, 8, [33, 64, 31], [1, 1, 1]),
    (B, 8, 64, 32, 16, 5, [90, 16, 15], [7, 16, 2]),
    (F, 4, 64, 64, 128, 1, [200], [200]),
    (B, 4, 256, 128, 16, 2, [19, 5], None),
    (F, 8, 256, 32, 64, 4, [70, 3], [66, 3]),
    (F, 4, 128, 32, 16, 2, [5] * 70, [1, 2, 0, 3, 1] * 14),
    (B, 4, 64, 32, 4096, 2, [4097], [130]),
]


@pytest.mark.parametrize("dtype,nbits,dim,group,page,heads,lens,new", WRITES)
def test_write_and_read(H, dtype, nbits, dim, group, page, heads, lens, new):
    gen = torch.Generator().manual_seed(dim + nbits + heads)
    new = lens if new is None else new
    table, n_pages, _ = layout(lens, page, gen)
    cu = cumulated(new)
    n = cu[-1]
    cache = poison(H.alloc_cache(n_pages, page, heads, dim, nbits, group, dtype))
    # rows of a wider tensor: strides beyond the heads, and three rows of no sequence
    wide = torch.full((n + 3, 2 * heads + 2, dim), 7.0, dtype=dtype, device="cuda")
    wide[:n, :heads] = values(n, heads, dim, dtype, gen)
    wide[:n, heads + 1:2 * heads + 1] = values(n, heads, dim, dtype, gen, 0.3)
    k, v = wide[:, :heads], wide[:, heads + 1:2 * heads + 1]
    at = R.where(table, lens, cu, n, page, n_pages) + [None] * 3
    want = expect_written(cache, k, v, at)
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v, cu_tokens=i32(cu))
    for name, x in want.items():
        assert same_bits(cache[name], x), name
    back = torch.full((n + 3, 2, heads + 1, dim), 9.0, dtype=dtype, device="cuda")
    H.hqq_cache_read(cache, i32(table), i32(lens), back[:, 0, :heads], back[:, 1, :heads], cu_tokens=i32(cu))
    for j, x in enumerate((k, v)):
        ref = R.value(*R.grid(x[:n].cpu(), nbits, group)).to(dtype)
        assert same_bits(back[:n, j, :heads], ref)
    assert (back[n:] == 9).all() and (back[:, :, heads] == 9).all()      # rows of no sequence, and beside
    # the documented bound: half a step, and the rounding of the result
    _, step, _ = R.grid(k[:n].cpu(), nbits, group)
    err = (back[:n, 0, :heads].cpu().double() - k[:n].cpu().double()).abs()
    lim = step.repeat_interleave(group, -1) / 2 + R.HALF_STEP[dtype] * (k[:n].cpu().double().abs() + step.repeat_interleave(group, -1))
    assert (err <= lim).all()


def edge_rows(dtype, dim):
    """Rows where the grid can go wrong, [n, dim] float64 numbers of the type."""
    r = torch.linspace(-1, 1, dim, dtype=torch.float64)
    i = torch.arange(dim, dtype=torch.float64)
    rows = [torch.zeros(dim), torch.full((dim,), -0.0), torch.full((dim,), 3.25), r,
            i % 16, i % 16 + 0.5, (i * 37) % 256 / 2,                  # on the grid, and on its ties
            torch.where(i == 3, 1.0, 0.0), torch.where(i == 3, -1.0, 1000.0), 1000 + r, r * 2.0 ** -20]
    if dtype == F:
        rows += [r * 65504, torch.where(i % 2 == 0, 65504.0, -65504.0), torch.where(i == 0, 65504.0, 65472.0),
                 r * 2.0 ** -24, (i % 3) * 2.0 ** -24, torch.where(i == 1, -100.0, 2.0 ** -24 * (i + 1))]
    else:
        rows += [r * 2.0 ** 119, r * 2.0 ** -110, torch.where(i == 1, 2.0 ** 100, r), r * 2.0 ** -126, 2.0 ** -133 * (i % 5)]
    return torch.stack([x.double() for x in rows]).to(dtype)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("nbits,dim,group", [(4, 128, 64), (8, 128, 128), (4, 64, 32), (8, 256, 64)])
def test_grid_edges(H, dtype, nbits, dim, group):
    x = edge_rows(dtype, dim)
    n = x.shape[0]
    k = x[:, None].contiguous().cuda()
    v = x.flip(0)[:, None].contiguous().cuda()
    cache = poison(H.alloc_cache(3, 16, 1, dim, nbits, group, dtype))
    table, lens = [[2, 0]], [n]
    want = expect_written(cache, k, v, R.where(table, lens, None, n, 16, 3))
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v)
    for name, y in want.items():
        assert same_bits(cache[name], y), name
    bk, bv = H.cache_read(cache, i32(table), i32(lens), n)
    assert torch.isfinite(bk).all() and torch.isfinite(bv).all()
    assert same_bits(bk, R.value(*R.grid(k.cpu(), nbits, group)).to(dtype))


@pytest.mark.parametrize("dtype,nbits", [(F, 4), (B, 4), (F, 8), (B, 8)])
def test_values_that_are_not_finite_stay_in_their_group(H, dtype, nbits):
    gen = torch.Generator().manual_seed(5)
    k = values(16, 2, 128, dtype, gen)
    clean = k.clone()
    k[3, 1, 70], k[5, 0, 2], k[6, 1, 127] = math.nan, math.inf, -math.inf
    cache = poison(H.alloc_cache(1, 16, 2, 128, nbits, 64, dtype))
    H.hqq_cache_write(cache, i32([[0]]), i32([16]), k, k.flip(0).contiguous())
    bk, bv = H.cache_read(cache, i32([[0]]), i32([16]), 16)
    ref = R.value(*R.grid(clean.cpu(), nbits, 64)).to(dtype)
    keep = torch.ones_like(ref, dtype=torch.bool)
    keep[3, 1, 64:], keep[5, 0, :64], keep[6, 1, 64:] = False, False, False
    assert torch.equal(bk.cpu()[keep], ref[keep]) and torch.equal(bv.cpu()[keep.flip(0)], ref.flip(0)[keep.flip(0)])
    assert torch.isnan(bk.cpu()[~keep]).all() and torch.isnan(bv.cpu()[~keep.flip(0)]).all()


def test_pages_and_positions_that_are_not_there(H):
    """Bad table entries, lengths beyond the table, more rows than the sequence has, row offsets
    out of range: writes drop such tokens, reads give zeros, attention does not see them."""
    gen = torch.Generator().manual_seed(6)
    page, n_pages, dim = 16, 5, 64
    table = [[3, -1, 99], [-7, 2, 1], [4, 0, -2147483648], [2147483647, 5, -1]]
    lens, cu = [40, 1000000, 3, -5], [0, 20, 40, 46, 50]
    cache = poison(H.alloc_cache(n_pages, page, 2, dim, 4, 32, F))
    k, v = values(50, 2, dim, F, gen), values(50, 2, dim, F, gen)
    at = R.where(table, lens, cu, 50, page, n_pages)
    assert sum(a[2] >= 0 for a in at) > 10 and sum(a[2] < 0 for a in at) > 10
    want = expect_written(cache, k, v, at)
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v, cu_tokens=i32(cu))
    for name, y in want.items():
        assert same_bits(cache[name], y), name
    bk, _ = H.cache_read(cache, i32(table), i32(lens), 50, cu_tokens=i32(cu))
    ref = R.value(*R.grid(k.cpu(), 4, 32)).to(F)
    there = torch.tensor([a[2] >= 0 for a in at])
    assert torch.equal(bk.cpu()[there], ref[there]) and (bk.cpu()[~there] == 0).all()
    q = values(50, 4, dim, F, gen)
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):        # every page holds numbers
        fill = torch.randint(0, 255, cache[x].shape, generator=gen) if "codes" in x else torch.rand(cache[x].shape, generator=gen)
        cache[x].copy_(fill)
    lse = torch.empty(50, 4, dtype=torch.float32, device="cuda")
    out = H.cache_attention(cache, i32(table), i32(lens), q, cu_tokens=i32(cu), lse=lse)
    ref = R.attention(R.Held(cache), table, lens, cu, q, dim ** -0.5)
    R.check_attention(out, lse, ref, torch.ones(50, dtype=torch.bool))
    # offsets that leave the tensors: those rows do not exist
    for bad in ([-9, 20, 20, 46, 99], [0, 0, 0, 0, 0], [7, 20, 30, 30, 45]):
        o = torch.full_like(q, 5.0)
        H.hqq_cache_attention(cache, i32(table), i32(lens), q, o, cu_tokens=i32(bad))
        mine = torch.tensor([a is not None for a in R.where(table, lens, bad, 50, page, n_pages)])
        R.check_attention(o, None, R.attention(R.Held(cache), table, lens, bad, q, dim ** -0.5), mine)
        assert (o.cpu()[~mine] == 5).all()


# dtype, nbits, dim, group, page, kv heads, per, lens, new
ATTEND = [
    (F, 4, 128, 64, 64, 2, 1, [1], [1]),
    (F, 4, 128, 64, 16, 1, 1, [300], [1]),
    (B, 4, 128, 64, 64, 2, 8, [511, 0, 1, 129, 1000], [1, 1, 1, 1, 1]),
    (F, 8, 128, 128, 32, 2, 8, [700, 2049], [1, 1]),
    (B, 8, 256, 64, 32, 2, 4, [200, 77, 5], [5, 4, 5]),
    (F, 4, 256, 128, 16, 1, 3, [260], [2]),
    (B, 4, 64, 32, 16, 3, 5, [99, 100, 101], [1, 7, 3]),
    (F, 8, 64, 64, 128, 2, 16, [400, 30], [1, 2]),
    (F, 4, 128, 32, 64, 2, 1, [333, 150], [133, 150]),
    (B, 4, 128, 128, 256, 1, 7, [513], [40]),
    (F, 8, 256, 32, 64, 1, 2, [140], [60]),
    (B, 8, 128, 64, 16, 2, 2, [3, 5], [6, 5]),                 # more rows than tokens: they see nothing
    (F, 4, 128, 64, 64, 1, 1, [130, 64], [0, 64]),
    (B, 8, 64, 32, 16, 2, 40, [65], [1]),                      # more query heads than a tile holds
    (B, 4, 128, 64, 16, 2, 8, [700, 33, 90, 5], [6, 7, 5, 5]),
    (F, 8, 128, 64, 64, 1, 5, [1000, 64], [9, 10]),
    (F, 4, 64, 32, 32, 2, 2, [900, 129], [300, 129]),
    (B, 8, 64, 64, 16, 1, 1, [777, 100, 0, 65], [500, 100, 0, 64]),
    (B, 4, 256, 128, 64, 1, 4, [600, 61], [30, 61]),
    (F, 8, 256, 64, 16, 1, 16, [130, 400], [2, 1]),
    (F, 4, 128, 128, 128, 2, 1, [1500, 20], [129, 20]),
]


def filled(H, dtype, nbits, dim, group, page, kv, lens, gen, scale=1.0, extra_pages=0):
    """A poisoned cache with the sequences' tokens written into it."""
    table, n_pages, free = layout(lens, page, gen, spare=3 + extra_pages)
    cache = poison(H.alloc_cache(n_pages, page, kv, dim, nbits, group, dtype))
    cu = cumulated([max(x, 0) for x in lens])
    if cu[-1]:
        H.hqq_cache_write(cache, i32(table), i32(lens), values(cu[-1], kv, dim, dtype, gen, scale),
                          values(cu[-1], kv, dim, dtype, gen), cu_tokens=i32(cu))
    return cache, table, free


@pytest.mark.parametrize("dtype,nbits,dim,group,page,kv,per,lens,new", ATTEND)
def test_attention(H, dtype, nbits, dim, group, page, kv, per, lens, new):
    gen = torch.Generator().manual_seed(dim + nbits + sum(lens))
    cache, table, _ = filled(H, dtype, nbits, dim, group, page, kv, lens, gen)
    cu = cumulated(new)
    n = cu[-1]
    buf = torch.randn(n + 2, kv * per + 1, dim, generator=gen).to(dtype).cuda()
    q = buf[:, :kv * per]
    obuf = torch.full((n + 2, kv * per + 2, dim), 11.0, dtype=dtype, device="cuda")
    out = obuf[:, 1:kv * per + 1]
    lse = torch.full((n + 2, kv * per), 13.0, dtype=torch.float32, device="cuda")
    H.hqq_cache_attention(cache, i32(table), i32(lens), q, out, lse=lse, cu_tokens=i32(cu))
    mine = torch.tensor([True] * n + [False] * 2)
    ref = R.attention(R.Held(cache), table, lens, cu, q, dim ** -0.5)
    R.check_attention(out, lse, ref, mine)
    assert (obuf[n:] == 11).all() and (obuf[:, 0] == 11).all() and (obuf[:, -1] == 11).all() and (lse[n:] == 13).all()
    if len(set(new)) == 1 and new[0] > 0:       # the same without row offsets
        again = H.cache_attention(cache, i32(table), i32(lens), q[:n])
        R.check_attention(again, None, tuple(x[:n] for x in ref), mine[:n])


@pytest.mark.parametrize("dtype,nbits,dim,group,page,kv,per,lens,new,prefix", [
    (F, 4, 128, 64, 16, 2, 1, [60, 1, 33], [1, 1, 1], 100),
    (B, 4, 128, 64, 64, 2, 8, [100, 0, 7, 200], [1, 1, 1, 1], 1000),
    (F, 8, 64, 32, 32, 1, 4, [9, 40], [9, 3], 1),
    (B, 8, 256, 128, 16, 2, 2, [20] * 9, [5] * 9, 333),
    (F, 4, 128, 128, 128, 1, 8, [30] * 20, [1] * 20, 2500),
    (F, 4, 128, 64, 64, 2, 2, [0, 0], [1, 1], 64),
    (B, 4, 64, 64, 16, 2, 3, [5, 6], [1, 2], 0),
])
def test_attention_with_a_shared_prefix(H, dtype, nbits, dim, group, page, kv, per, lens, new, prefix):
    gen = torch.Generator().manual_seed(dim + nbits + prefix)
    pre_pages = -(-prefix // page)
    cache, table, free = filled(H, dtype, nbits, dim, group, page, kv, lens, gen, extra_pages=pre_pages)
    pages = free[:pre_pages]
    if prefix:
        H.hqq_cache_write(cache, i32([pages]), i32([prefix]), values(prefix, kv, dim, dtype, gen),
                          values(prefix, kv, dim, dtype, gen))
    cu = cumulated(new)
    q = torch.randn(cu[-1], kv * per, dim, generator=gen).to(dtype).cuda()
    lse = torch.empty(cu[-1], kv * per, dtype=torch.float32, device="cuda")
    out = H.cache_attention_prefix(cache, i32(table), i32(lens), i32(pages), prefix, q, cu_tokens=i32(cu), lse=lse)
    ref = R.attention(R.Held(cache), table, lens, cu, q, dim ** -0.5, pages, prefix)
    R.check_attention(out, lse, ref, torch.ones(cu[-1], dtype=torch.bool))
    # the same as one table for each sequence, where the prefix ends with a page
    if prefix % page == 0:
        joined = [pages + t for t in table]
        whole = H.cache_attention(cache, i32(joined), i32([x + prefix for x in lens]), q, cu_tokens=i32(cu))
        R.check_attention(whole, None, ref, torch.ones(cu[-1], dtype=torch.bool))


@pytest.mark.parametrize("dtype", [F, B])
def test_scores_far_apart(H, dtype):
    """Large scores that grow and shrink along the sequence, one that outweighs all others, a
    negative and a zero scale."""
    gen = torch.Generator().manual_seed(11)
    cache, table, _ = filled(H, dtype, 8, 128, 64, 16, 2, [700], gen, scale=6.0)
    q = (torch.randn(1, 8, 128, generator=gen) * 8).to(dtype).cuda()
    for scale in (1.0, 128 ** -0.5, -0.3, 0.0):
        lse = torch.empty(1, 8, dtype=torch.float32, device="cuda")
        out = H.cache_attention(cache, i32(table), i32([700]), q, scale=scale, lse=lse)
        R.check_attention(out, lse, R.attention(R.Held(cache), table, [700], None, q, scale), torch.ones(1, dtype=torch.bool))


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("size", [2.0 ** -18, 2000.0])
def test_values_of_any_size(H, dtype, size):
    """Values far below and above one, whose steps reach the ends of binary16."""
    gen = torch.Generator().manual_seed(12)
    cache = poison(H.alloc_cache(20, 16, 1, 64, 4, 32, dtype))
    table, n = [list(range(19, -1, -1))], 310
    k, v = values(n, 1, 64, dtype, gen), (torch.randn(n, 1, 64, generator=gen) * size).to(dtype).cuda()
    H.hqq_cache_write(cache, i32(table), i32([n]), k, v)
    q = values(1, 4, 64, dtype, gen)
    out = H.cache_attention(cache, i32(table), i32([n]), q)
    R.check_attention(out, None, R.attention(R.Held(cache), table, [n], None, q, 0.125), torch.ones(1, dtype=torch.bool))


def test_same_bits_whatever_the_workspace_held(H):
    gen = torch.Generator().manual_seed(13)
    lens = [900, 3, 260, 0]
    cache, table, free = filled(H, F, 4, 128, 64, 32, 2, lens, gen, extra_pages=8)
    H.hqq_cache_write(cache, i32([free[:8]]), i32([250]), values(250, 2, 128, F, gen), values(250, 2, 128, F, gen))
    q = torch.randn(4, 8, 128, generator=gen).half().cuda()
    t, ln, pp = i32(table), i32(lens), i32(free[:8])
    for prefix in (0, 250):
        need = H.hqq_cache_attention_workspace(cache, t, ln, 4, 8, prefix)
        outs = []
        for fill in (0, 255, 127):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            o = torch.empty_like(q)
            H.hqq_cache_attention_prefix(cache, t, ln, pp, prefix, q, o, workspace=ws)
            outs.append(o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        with pytest.raises(H.HQQError) as e:
            H.hqq_cache_attention_prefix(cache, t, ln, pp, prefix, q, outs[0], workspace=ws[:need - 1])
        assert e.value.status == H.HQQ_ERR_WORKSPACE
    # sequences that one block takes whole need none
    short = t[:, :512 // 32].contiguous()
    assert H.hqq_cache_attention_workspace(cache, short, ln, 4, 8) == 0


def test_wrong_tensors_are_refused(H):
    cache = H.alloc_cache(4, 16, 2, 64, 4, 32, F)
    t, ln = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), i32([5])
    q = torch.zeros(1, 4, 64, dtype=F, device="cuda")
    k = torch.zeros(1, 2, 64, dtype=F, device="cuda")

    def refused(f, *a, **kw):
        with pytest.raises(H.HQQError) as e:
            f(*a, **kw)
        assert e.value.status == H.HQQ_ERR_ARG
    for bad in (dict(k_codes=cache["k_codes"][:, :1]), dict(v_codes=cache["v_codes"][:3]), dict(k_meta=cache["k_meta"].float()),
                dict(v_meta=cache["v_meta"].to(B)), dict(page_size=32), dict(n_heads=4), dict(group_size=64), dict(nbits=8),
                dict(k_meta=cache["k_meta"].cpu()), dict(v_codes=cache["v_codes"].transpose(0, 1))):
        refused(H.cache_attention, {**cache, **bad}, t, ln, q)
    for bt, bl in ((t.long(), ln), (t[0], ln), (t.cpu(), ln), (t, ln.long()), (t, i32([5, 5])), (t, ln.cpu()),
                   (torch.zeros(1, 4, dtype=torch.int32, device="cuda")[:, ::2], i32([5]).expand(2)[:1].float())):
        refused(H.cache_attention, cache, bt, bl, q)
        refused(H.hqq_cache_write, cache, bt, bl, k, k)
    refused(H.cache_attention, cache, t, ln, q, cu_tokens=i32([0]))
    refused(H.cache_attention, cache, t, ln, q, cu_tokens=torch.tensor([0, 1], device="cuda"))
    for bq in (q.to(B), q[:, :3], q[..., :32], q.cpu(), q[0], torch.zeros(1, 4, 128, dtype=F, device="cuda")[..., ::2],
               torch.zeros(2, 4 * 65, dtype=F, device="cuda")[:, 1:].as_strided((2, 4, 64), (260, 64, 1))):
        refused(H.cache_attention, cache, t, ln, bq)
    refused(H.hqq_cache_attention, cache, t, ln, q, torch.zeros(1, 2, 64, dtype=F, device="cuda"))
    refused(H.cache_attention, cache, t, ln, q, lse=torch.zeros(1, 4, dtype=F, device="cuda"))
    refused(H.cache_attention_prefix, cache, t, ln, t, 5, q)
    refused(H.cache_attention_prefix, cache, t, ln, t[0], 33, q)
    refused(H.hqq_cache_write, cache, t, ln, k, k[:, :1])
    refused(H.hqq_cache_read, cache, t, ln, k.expand(3, 2, 64)[:, :, :32], k)


def test_answering_step_by_step(H):
    """Prompts enter the cache, then every step writes one token for each sequence and attends;
    the same as attention over everything written so far, and as one call with all tokens."""
    gen = torch.Generator().manual_seed(14)
    page, kv, per, dim, steps, starts = 16, 2, 4, 128, 5, [37, 1, 64]
    ends = [x + steps for x in starts]
    table, n_pages, _ = layout(ends, page, gen)
    cache = poison(H.alloc_cache(n_pages, page, kv, dim, 4, 64, B))
    t = i32(table)
    pk, pv = values(sum(starts), kv, dim, B, gen), values(sum(starts), kv, dim, B, gen)
    H.hqq_cache_write(cache, t, i32(starts), pk, pv, cu_tokens=i32(cumulated(starts)))
    lens = i32(starts)
    rows, queries = [], []
    for s in range(steps):
        lens += 1
        k, v, q = values(3, kv, dim, B, gen), values(3, kv, dim, B, gen), values(3, kv * per, dim, B, gen)
        H.hqq_cache_write(cache, t, lens, k, v)
        out = H.cache_attention(cache, t, lens, q)
        ref = R.attention(R.Held(cache), table, [x + s + 1 for x in starts], None, q, dim ** -0.5)
        R.check_attention(out, None, ref, torch.ones(3, dtype=torch.bool))
        rows.append(out)
        queries.append(q)
    q = torch.stack(queries, 1).reshape(-1, kv * per, dim)
    out = H.cache_attention(cache, t, lens, q)
    ref = R.attention(R.Held(cache), table, ends, None, q, dim ** -0.5)
    R.check_attention(out, None, ref, torch.ones(3 * steps, dtype=torch.bool))
    both = torch.stack(rows, 1).reshape(-1, kv * per, dim)
    assert (out.double() - both.double()).abs().max() <= 2 ** -7 * both.double().abs().max()


def test_captured_steps(H):
    """A step captured into a graph and replayed, with eager work between: lengths, tokens and
    pages change under it; two graphs with a workspace each replayed in turn."""
    gen = torch.Generator().manual_seed(15)
    page, kv, dim, cap = 16, 2, 64, 120
    table, n_pages, _ = layout([cap, cap], page, gen)
    t = i32(table)

    def make():
        cache = poison(H.alloc_cache(n_pages, page, kv, dim, 8, 32, F))
        start = [50, 3]
        H.hqq_cache_write(cache, t, i32(start), values(53, kv, dim, F, gen), values(53, kv, dim, F, gen),
                          cu_tokens=i32([0, 50, 53]))
        s = dict(cache=cache, lens=i32(start), k=values(2, kv, dim, F, gen), v=values(2, kv, dim, F, gen),
                 q=values(2, 8, dim, F, gen), out=torch.empty(2, 8, dim, dtype=F, device="cuda"))
        need = H.hqq_cache_attention_workspace(cache, t, s["lens"], 2, 8)
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")

        def step():
            s["lens"].add_(1)
            H.hqq_cache_write(s["cache"], t, s["lens"], s["k"], s["v"])
            H.hqq_cache_attention(s["cache"], t, s["lens"], s["q"], s["out"], workspace=s["ws"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        s["g"], s["at"] = g, [51, 4]
        return s
    states = [make(), make()]
    for _ in range(4):
        for s in states:
            for x in ("k", "v", "q"):
                s[x].copy_(values(*s[x].shape, F, gen))
            s["out"].fill_(7)
            s["g"].replay()
            s["at"] = [x + 1 for x in s["at"]]
        torch.cuda.synchronize()
        for s in states:
            assert s["lens"].tolist() == s["at"]
            ref = R.attention(R.Held(s["cache"]), table, s["at"], None, s["q"], dim ** -0.5)
            R.check_attention(s["out"], None, ref, torch.ones(2, dtype=torch.bool))
            eager = H.cache_attention(s["cache"], t, s["lens"], s["q"])
            assert torch.equal(eager, s["out"])


def test_two_streams(H):
    gen = torch.Generator().manual_seed(16)
    jobs = []
    for lens in ([2000, 700], [1500, 5]):
        cache, table, _ = filled(H, F, 4, 128, 64, 64, 4, lens, gen)
        q = values(2, 16, 128, F, gen)
        jobs.append((cache, i32(table), i32(lens), q, H.cache_attention(cache, i32(table), i32(lens), q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for k, (cache, t, ln, q, _) in enumerate(jobs):
            with torch.cuda.stream(streams[k]):
                outs[k].append(H.cache_attention(cache, t, ln, q))
    # a stream named in the call, with no context of its own
    o = torch.empty_like(jobs[0][3])
    H.hqq_cache_attention(*jobs[0][:4], o, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o, jobs[0][4])
    for k in range(2):
        assert all(torch.equal(x, jobs[k][4]) for x in outs[k])


def test_offsets_beyond_32_bits(H):
    """Pages at the end of a cache of more than 2^32 bytes of keys."""
    gen = torch.Generator().manual_seed(17)
    page, kv, dim = 64, 8, 128
    n_pages = (1 << 32) // (page * kv * dim) + 40
    cache = H.alloc_cache(n_pages, page, kv, dim, 8, 128, B)
    assert cache["k_codes"].numel() > 1 << 32
    table = [[n_pages - 1, n_pages - 7, 0], [n_pages - 3, 1, n_pages - 2]]
    lens = [150, 190]
    k, v = values(340, kv, dim, B, gen), values(340, kv, dim, B, gen)
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v, cu_tokens=i32([0, 150, 340]))
    bk, bv = H.cache_read(cache, i32(table), i32(lens), 340, cu_tokens=i32([0, 150, 340]))
    assert torch.equal(bk.cpu(), R.value(*R.grid(k.cpu(), 8, 128)).to(B))
    assert torch.equal(bv.cpu(), R.value(*R.grid(v.cpu(), 8, 128)).to(B))
    q = values(2, kv, dim, B, gen)
    out = H.cache_attention(cache, i32(table), i32(lens), q)
    used = sorted({p for row in table for p in row})
    small = {x: cache[x][torch.tensor(used, device="cuda")] for x in ("k_codes", "v_codes", "k_meta", "v_meta")}
    small = {**cache, **small}
    ref = R.attention(R.Held(small), [[used.index(p) for p in row] for row in table], lens, None, q, dim ** -0.5)
    R.check_attention(out, None, ref, torch.ones(2, dtype=torch.bool))


def test_many_sequences(H):
    """The most sequences a call takes, most of them short or empty."""
    gen = torch.Generator().manual_seed(18)
    n, page, dim = 4096, 16, 64
    lens = [(i * 7) % 20 if i % 5 else 0 for i in range(n)]
    cache, table, _ = filled(H, F, 4, dim, 64, page, 1, lens, gen)
    q = values(n, 2, dim, F, gen)
    lse = torch.empty(n, 2, dtype=torch.float32, device="cuda")
    out = H.cache_attention(cache, i32(table), i32(lens), q, lse=lse)
    R.check_attention(out, lse, R.attention(R.Held(cache), table, lens, None, q, dim ** -0.5), torch.ones(n, dtype=torch.bool))


def test_empty_calls(H):
    gen = torch.Generator().manual_seed(19)
    cache, table, _ = filled(H, F, 4, 64, 32, 16, 2, [20], gen)
    q = torch.empty(0, 4, 64, dtype=F, device="cuda")
    assert H.cache_attention(cache, i32(table), i32([20]), q).shape == (0, 4, 64)
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    out = torch.full((3, 4, 64), 5.0, dtype=F, device="cuda")
    H.hqq_cache_attention(cache, none, i32([]), torch.zeros_like(out), out)     # rows of no sequence
    assert (out == 5).all()
    k, v = H.cache_read(cache, i32(table), i32([20]), 0)
    assert k.shape == (0, 2, 64)
    # a table without pages: nothing is in the cache
    bare = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    lse = torch.empty(3, 4, dtype=torch.float32, device="cuda")
    out = H.cache_attention(cache, bare, i32([20]), torch.ones(3, 4, 64, dtype=F, device="cuda"), lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()


# dtype, nbits, dim, group, page, kv heads, per, lens, new: many rows, more than 64 sequences, pieces
MANY = [
    (F, 4, 256, 32, 16, 1, 8, [300, 70], [40, 33]),
    (B, 4, 256, 32, 32, 1, 16, [90], [50]),
    (F, 8, 128, 32, 16, 2, 4, [700, 64, 1], [40, 40, 1]),
    (F, 4, 64, 64, 16, 1, 8, [800, 33] + [20] * 70, [60, 9] + [9] * 70),
    (B, 8, 128, 128, 64, 1, 1, [5] * 80 + [1200], [1] * 81),
    (F, 4, 128, 64, 4096, 1, 2, [4099, 9], [130, 9]),
    (B, 4, 128, 64, 16, 4, 4, [1300, 1000, 600], [1, 1, 1]),
    # enough heads that tiles of 128 rows are taken
    (F, 4, 128, 64, 16, 128, 1, [1500, 300, 2000], [130, 100, 140]),
    (B, 4, 64, 32, 32, 256, 2, [1300, 1200], [60, 60]),
    (B, 8, 128, 32, 16, 128, 1, [900, 700, 900, 500], [120, 140, 97, 120]),
    (F, 8, 64, 64, 16, 256, 1, [1000, 240], [200, 40]),
    (F, 4, 128, 128, 64, 128, 1, [2000, 1990], [110, 128]),
    (F, 8, 128, 32, 16, 32, 10, [990] * 5, [50] * 5),
    # and for heads of 256, of 64 and 32
    (F, 4, 256, 64, 16, 256, 1, [600, 560, 300], [100, 60, 130]),
    (B, 8, 256, 128, 32, 256, 1, [700, 600], [20, 30]),
    (F, 8, 256, 32, 16, 256, 2, [600, 580], [15, 12]),
]


@pytest.mark.parametrize("dtype,nbits,dim,group,page,kv,per,lens,new", MANY)
def test_many_rows_bad_pages_and_far_bases(H, dtype, nbits, dim, group, page, kv, per, lens, new):
    """Keys far from zero (their scores are mostly the bases' part), pages that are not there in
    the middle of sequences, NaN in all that is not written; with a prefix of such pages too."""
    gen = torch.Generator().manual_seed(dim + nbits + len(lens))
    table, n_pages, free = layout(lens, page, gen, spare=8 if kv < 128 else 100)
    cache = poison(H.alloc_cache(n_pages, page, kv, dim, nbits, group, dtype))
    cu = cumulated(lens)
    far = values(cu[-1], kv, dim, dtype, gen) + 30 * torch.randn(kv, dim, generator=gen).to(dtype).cuda()
    H.hqq_cache_write(cache, i32(table), i32(lens), far, values(cu[-1], kv, dim, dtype, gen), cu_tokens=i32(cu))
    prefix = 600 if page > 1000 else 3 * page + 5 if kv < 128 else 1500
    pages = free[:-(-prefix // page)]
    H.hqq_cache_write(cache, i32([pages]), i32([prefix]), values(prefix, kv, dim, dtype, gen), values(prefix, kv, dim, dtype, gen))
    for b in range(0, len(lens), 2):
        for x in range(1, -(-lens[b] // page), 3):
            table[b][x] = [-1, n_pages, 1 << 30][x % 3]
    cu = cumulated(new)
    q = (torch.rand(cu[-1], kv * per, dim, generator=gen) - 0.3).to(dtype).cuda()
    every = torch.ones(cu[-1], dtype=torch.bool)
    lse = torch.empty(cu[-1], kv * per, dtype=torch.float32, device="cuda")
    held, scale = R.Held(cache), 0.25 / dim
    out = H.cache_attention(cache, i32(table), i32(lens), q, cu_tokens=i32(cu), scale=scale, lse=lse)
    R.check_attention(out, lse, R.attention(held, table, lens, cu, q, scale), every)
    if len(pages) > 2:
        pages[1] = -5
    out = H.cache_attention_prefix(cache, i32(table), i32(lens), i32(pages), prefix, q, cu_tokens=i32(cu), scale=scale, lse=lse)
    R.check_attention(out, lse, R.attention(held, table, lens, cu, q, scale, pages, prefix), every)


@pytest.mark.parametrize("dtype,nbits,dim,group,heads,per,new,n", [
    (F, 4, 128, 64, 1, 1, 7, 250), (B, 8, 128, 32, 1, 4, 8, 250), (F, 8, 128, 128, 1, 4, 30, 250), (B, 4, 64, 32, 1, 2, 60, 250),
    (F, 4, 256, 32, 1, 1, 9, 250), (B, 8, 256, 64, 1, 8, 12, 250), (F, 4, 64, 32, 1024, 1, 128, 500),
    (B, 8, 128, 64, 1024, 1, 128, 500), (F, 4, 256, 64, 1024, 1, 60, 1000)])
def test_values_that_are_not_finite_are_not_seen_before_they_come(H, dtype, nbits, dim, group, heads, per, new, n):
    """Rows before a token with NaN or an infinity in its key or value give what they give
    without it; rows from it on see NaN in the value's group at most, or in all with the key's."""
    gen = torch.Generator().manual_seed(dim + new)
    table, n_pages, _ = layout([n], 16, gen)
    k, v = values(n, heads, dim, dtype, gen), values(n, heads, dim, dtype, gen)
    q = torch.randn(new, heads * per, dim, generator=gen).to(dtype).cuda()
    clean = poison(H.alloc_cache(n_pages, 16, heads, dim, nbits, group, dtype))
    H.hqq_cache_write(clean, i32(table), i32([n]), k, v)
    ref = R.attention(R.Held(clean), table, [n], None, q, dim ** -0.5)
    at = n - 3                          # the last three rows see it
    for bad in (math.nan, math.inf, -math.inf):
        for which in (0, 1):
            kv = [k.clone(), v.clone()]
            kv[which][at, :, 3] = bad
            cache = poison(H.alloc_cache(n_pages, 16, heads, dim, nbits, group, dtype))
            H.hqq_cache_write(cache, i32(table), i32([n]), *kv)
            out = H.cache_attention(cache, i32(table), i32([n]), q)
            before = torch.arange(new) < new - 3
            R.check_attention(out, None, ref, before)
            if which:                   # the value's other groups
                R.check_attention(out[..., group:], None, tuple(x[..., group:] if x.dim() == 3 else x for x in ref), ~before)


@pytest.mark.parametrize("n_seqs,per,new", [(3, 1, 1), (70, 1, 1), (3, 8, 40), (70, 8, 20)])
def test_row_offsets_that_fall(H, n_seqs, per, new):
    """Attention leaves all rows as they were."""
    gen = torch.Generator().manual_seed(n_seqs)
    lens = [600] + [40] * (n_seqs - 1)
    cache, table, free = filled(H, F, 4, 64, 32, 16, 2, lens, gen, extra_pages=2)
    cu = cumulated([new] * n_seqs)
    q = torch.randn(cu[-1], 2 * per, 64, generator=gen).half().cuda()
    cu[n_seqs // 2] = cu[-1]
    for prefix in (0, 20):
        out = torch.full_like(q, 5.0)
        H.hqq_cache_attention_prefix(cache, i32(table), i32(lens), i32(free[:2]), prefix, q, out, cu_tokens=i32(cu))
        assert (out == 5).all()


def test_captured_prefix_steps(H):
    """Many rows and a prefix in a graph, lengths and row offsets changing between replays."""
    gen = torch.Generator().manual_seed(21)
    page, dim, kv, per, cap, n = 16, 128, 2, 4, [200, 900, 30], 90
    cache, table, free = filled(H, B, 4, dim, 64, page, kv, cap, gen, extra_pages=20)
    pages, prefix = free[:20], 315
    H.hqq_cache_write(cache, i32([pages]), i32([prefix]), values(prefix, kv, dim, B, gen), values(prefix, kv, dim, B, gen))
    t, pp, lens, cu = i32(table), i32(pages), i32([200, 900, 30]), i32([0, 30, 60, 90])
    q = values(n, kv * per, dim, B, gen)
    out, lse = torch.empty_like(q), torch.empty(n, kv * per, dtype=torch.float32, device="cuda")
    ws = torch.empty(H.hqq_cache_attention_workspace(cache, t, lens, n, kv * per, prefix), dtype=torch.uint8, device="cuda")

    def step():
        H.hqq_cache_attention_prefix(cache, t, lens, pp, prefix, q, out, lse=lse, cu_tokens=cu, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    held = R.Held(cache)
    for ln, rows in (([200, 900, 30], [0, 30, 60, 90]), ([1, 33, 0], [0, 1, 89, 90]), ([150, 899, 30], [0, 0, 90, 90]),
                     ([200, 640, 7], [5, 20, 20, 80])):
        lens.copy_(i32(ln))
        cu.copy_(i32(rows))
        q.copy_(values(*q.shape, B, gen))
        out.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        mine = torch.tensor([rows[0] <= i < rows[-1] for i in range(n)])
        R.check_attention(out, lse, R.attention(held, table, ln, rows, q, dim ** -0.5, pages, prefix), mine)
        assert (out.cpu()[~mine] == 3).all()
        eager = torch.full_like(q, 3.0)
        H.hqq_cache_attention_prefix(cache, t, lens, pp, prefix, q, eager, cu_tokens=cu)
        assert torch.equal(eager, out)


def test_rows_of_any_stride(H):
    """One query row for all tokens (stride 0), heads before tokens, and a workspace elsewhere."""
    gen = torch.Generator().manual_seed(22)
    lens = [700, 130]
    cache, table, _ = filled(H, F, 8, 64, 64, 32, 2, lens, gen)
    t, ln = i32(table), i32(lens)
    one = torch.randn(1, 6, 64, generator=gen).half().cuda()
    q = one.expand(40, 6, 64)
    out = torch.empty(6, 40, 64, dtype=F, device="cuda").transpose(0, 1)
    H.hqq_cache_attention(cache, t, ln, q, out)
    R.check_attention(out, None, R.attention(R.Held(cache), table, lens, None, q, 0.125), torch.ones(40, dtype=torch.bool))
    need = H.hqq_cache_attention_workspace(cache, t, ln, 40, 6)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(H.HQQError):
            H.hqq_cache_attention(cache, t, ln, q, out, workspace=ws)
