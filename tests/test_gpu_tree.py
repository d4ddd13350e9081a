"""Attention of drafted trees over the quantized cache, and keeping the accepted tokens, on the GPU."""
import math

import pytest
import torch

import cache_ref as R
import tree_ref as T
from test_gpu_cache import cumulated, filled, i32, layout, poison, same_bits, values

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


# dtype, nbits, dim, group, page, kv heads, per, lens, new, words
TREES = [
    (F, 4, 128, 64, 64, 2, 1, [1], [1], 1),
    (F, 4, 128, 64, 16, 2, 1, [300], [26], 1),
    (B, 4, 128, 64, 64, 2, 8, [511, 0, 7, 129, 1000], [7, 0, 7, 6, 5], 1),
    (F, 8, 128, 128, 32, 2, 8, [700, 2049], [64, 63], 1),
    (B, 8, 256, 64, 32, 2, 4, [200, 77, 65], [5, 65, 65], 2),
    (F, 4, 256, 128, 16, 1, 3, [260], [100], 2),
    (B, 4, 64, 32, 16, 3, 5, [99, 100, 101], [1, 7, 3], 3),
    (F, 8, 64, 64, 128, 2, 16, [400, 30], [9, 2], 1),
    (B, 4, 128, 128, 256, 1, 7, [513], [130], 3),
    (F, 4, 128, 32, 64, 1, 2, [900, 450], [300, 200], 5),
    (B, 8, 128, 64, 16, 2, 2, [3, 5], [6, 5], 1),              # more rows than tokens
    (F, 8, 128, 64, 64, 2, 1, [333], [200], 2),                 # tokens behind the words are not seen
    (B, 4, 64, 64, 16, 1, 4, [40] * 70, [3] * 70, 1),           # more sequences than a wave has lanes
    (F, 8, 256, 32, 64, 1, 16, [130, 400], [33, 64], 1),
    (B, 4, 128, 64, 64, 8, 8, [800, 750], [100, 128], 2),
    # tiles of 128 rows, and of 64 and 32 with heads of 256
    (B, 4, 128, 64, 64, 40, 1, [4000, 3900, 4000, 100], [100, 100, 97, 100], 2),
    (F, 8, 64, 32, 32, 64, 1, [3000, 2900, 3000], [100, 101, 99], 2),
    (F, 8, 256, 128, 64, 16, 1, [4600, 4600, 4500, 4600], [100, 99, 100, 100], 2),
    (B, 4, 256, 64, 32, 16, 1, [2000] * 8, [25] * 8, 1),
]


@pytest.mark.parametrize("dtype,nbits,dim,group,page,kv,per,lens,new,words", TREES)
def test_tree_attention(H, dtype, nbits, dim, group, page, kv, per, lens, new, words):
    gen = torch.Generator().manual_seed(dim + nbits + sum(lens))
    cache, table, _ = filled(H, dtype, nbits, dim, group, page, kv, lens, gen)
    cu = cumulated(new)
    n = cu[-1]
    masks = T.random_masks(new, gen, words)
    buf = torch.randn(n + 2, kv * per + 1, dim, generator=gen).to(dtype).cuda()
    q = buf[:, :kv * per]
    obuf = torch.full((n + 2, kv * per + 2, dim), 11.0, dtype=dtype, device="cuda")
    out = obuf[:, 1:kv * per + 1]
    lse = torch.full((n + 2, kv * per), 13.0, dtype=torch.float32, device="cuda")
    tree = torch.cat((masks, torch.full((2, words), -1, dtype=torch.int64))).cuda()
    H.hqq_cache_attention_tree(cache, i32(table), i32(lens), tree, q, out, lse=lse, cu_tokens=i32(cu))
    mine = torch.tensor([True] * n + [False] * 2)
    ref = T.attention(R.Held(cache), table, lens, cu, q, dim ** -0.5, torch.cat((masks, masks[:1], masks[:1])))
    R.check_attention(out, lse, ref, mine)
    assert (obuf[n:] == 11).all() and (obuf[:, 0] == 11).all() and (obuf[:, -1] == 11).all() and (lse[n:] == 13).all()
    if len(set(new)) == 1 and new[0] > 0:       # the same without row offsets
        again = H.cache_attention_tree(cache, i32(table), i32(lens), tree[:n], q[:n])
        R.check_attention(again, None, tuple(x[:n] for x in ref), mine[:n])


@pytest.mark.parametrize("dtype,nbits,kv,per,lens,new", [(F, 4, 2, 4, [900, 33, 64], [5, 7, 64]), (B, 8, 1, 8, [300, 140], [60, 128])])
def test_masks_of_chains_are_attention(H, dtype, nbits, kv, per, lens, new):
    """A chain's masks give what cache_attention gives, to the bit."""
    gen = torch.Generator().manual_seed(3)
    cache, table, _ = filled(H, dtype, nbits, 128, 64, 16, kv, lens, gen)
    cu = cumulated(new)
    words = (max(new) + 63) // 64
    masks = T.to_words([(1 << (j + 1)) - 1 for n in new for j in range(n)], words).cuda()
    q = torch.randn(cu[-1], kv * per, 128, generator=gen).to(dtype).cuda()
    args = (cache, i32(table), i32(lens))
    assert torch.equal(H.cache_attention_tree(*args, masks, q, cu_tokens=i32(cu)), H.cache_attention(*args, q, cu_tokens=i32(cu)))


@pytest.mark.parametrize("dtype,nbits,dim,kv,per,lens,new", [(B, 4, 128, 2, 8, [700, 90], [7, 9]), (F, 8, 64, 1, 4, [500], [80]),
                                                             (B, 8, 128, 40, 1, [3000, 3100, 3000, 3000], [120] * 4)])
def test_chains_over_values_of_very_different_size(H, dtype, nbits, dim, kv, per, lens, new):
    """Tokens whose values lie far apart in size come behind the others in an item: with masks too."""
    gen = torch.Generator().manual_seed(9)
    table, n_pages, _ = layout(lens, 64, gen)
    cache = H.alloc_cache(n_pages, 64, kv, dim, nbits, 32, dtype)
    n = sum(lens)
    k = values(n, kv, dim, dtype, gen)
    size = 2.0 ** torch.randint(-18, 8, (n, 1, 1), generator=gen)
    v = (torch.randn(n, kv, dim, generator=gen) * size).to(dtype).cuda()
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v, cu_tokens=i32(cumulated(lens)))
    cu, words = cumulated(new), (max(new) + 63) // 64
    masks = T.to_words([(1 << (j + 1)) - 1 for m in new for j in range(m)], words).cuda()
    q = torch.randn(cu[-1], kv * per, dim, generator=gen).to(dtype).cuda()
    args = (cache, i32(table), i32(lens))
    got = H.cache_attention_tree(*args, masks, q, cu_tokens=i32(cu))
    assert torch.isfinite(got).all() and torch.equal(got, H.cache_attention(*args, q, cu_tokens=i32(cu)))


def test_masks_of_any_bits(H):
    """Random bits, all of them and none: rows that see nothing, themselves not, or what comes after."""
    gen = torch.Generator().manual_seed(4)
    lens, new = [70, 100, 12, 90], [70, 40, 12, 64]
    cache, table, _ = filled(H, F, 4, 64, 32, 16, 2, lens, gen)
    cu = cumulated(new)
    for fill in ("random", 0, -1):
        masks = torch.randint(-2 ** 63, 2 ** 63 - 1, (cu[-1], 2), generator=gen) if fill == "random" else torch.full((cu[-1], 2), fill)
        q = torch.randn(cu[-1], 6, 64, generator=gen).half().cuda()
        lse = torch.empty(cu[-1], 6, dtype=torch.float32, device="cuda")
        out = H.cache_attention_tree(cache, i32(table), i32(lens), masks.cuda(), q, cu_tokens=i32(cu), lse=lse)
        R.check_attention(out, lse, T.attention(R.Held(cache), table, lens, cu, q, 0.125, masks), torch.ones(cu[-1], dtype=torch.bool))
        if fill == 0:
            assert (out[:70] == 0).all() and (lse[:70] == -math.inf).all()


def test_what_a_row_does_not_see_does_not_change_it(H):
    """NaN among the drafted tokens, and in the pages behind them, stays out of rows without them."""
    gen = torch.Generator().manual_seed(5)
    lens, new, dim = [80], [20], 128
    table, n_pages, _ = layout(lens, 16, gen)
    cache = poison(H.alloc_cache(n_pages, 16, 2, dim, 8, 64, B))
    k, v = values(80, 2, dim, B, gen), values(80, 2, dim, B, gen)
    k[70, 0, 5], v[66, 1, 100], v[79, 0, 3] = math.nan, math.inf, math.nan
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v)
    bad = {6, 10, 19}                               # numbers among the drafted
    masks = [sum(1 << j for j in range(i + 1) if j not in bad) for i in range(20)]
    q = torch.randn(20, 8, dim, generator=gen).to(B).cuda()
    out = H.cache_attention_tree(cache, i32(table), i32(lens), T.to_words(masks, 1).cuda(), q)
    k[70, 0, 5], v[66, 1, 100], v[79, 0, 3] = 0, 0, 0
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v)
    ref = T.attention(R.Held(cache), table, lens, None, q, dim ** -0.5, T.to_words(masks, 1))
    R.check_attention(out, None, ref, torch.ones(20, dtype=torch.bool))


def test_bad_tables_and_offsets(H):
    gen = torch.Generator().manual_seed(6)
    table = [[3, -1, 99], [-7, 2, 1], [4, 0, -2147483648], [2147483647, 5, -1]]
    lens, cu = [40, 1000000, 3, -5], [0, 20, 40, 46, 50]
    cache = poison(H.alloc_cache(5, 16, 2, 64, 4, 32, F))
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
        cache[x].copy_(torch.randint(0, 255, cache[x].shape, generator=gen) if "codes" in x else torch.rand(cache[x].shape, generator=gen))
    masks = torch.randint(-2 ** 63, 2 ** 63 - 1, (50, 1), generator=gen)
    q = torch.randn(50, 4, 64, generator=gen).half().cuda()
    lse = torch.empty(50, 4, dtype=torch.float32, device="cuda")
    out = H.cache_attention_tree(cache, i32(table), i32(lens), masks.cuda(), q, cu_tokens=i32(cu), lse=lse)
    R.check_attention(out, lse, T.attention(R.Held(cache), table, lens, cu, q, 0.125, masks), torch.ones(50, dtype=torch.bool))
    for bad in ([-9, 20, 20, 46, 99], [0, 0, 0, 0, 0], [7, 20, 30, 30, 45]):
        o = torch.full_like(q, 5.0)
        H.hqq_cache_attention_tree(cache, i32(table), i32(lens), masks.cuda(), q, o, cu_tokens=i32(bad))
        mine = torch.tensor([a is not None for a in R.where(table, lens, bad, 50, 16, 5)])
        R.check_attention(o, None, T.attention(R.Held(cache), table, lens, bad, q, 0.125, masks), mine)
        assert (o.cpu()[~mine] == 5).all()
    o = torch.full_like(q, 5.0)                     # offsets that fall: nothing is done
    H.hqq_cache_attention_tree(cache, i32(table), i32(lens), masks.cuda(), q, o, cu_tokens=i32([0, 30, 10, 40, 50]))
    assert (o == 5).all()


def test_the_binding_refuses(H):
    gen = torch.Generator().manual_seed(7)
    cache, table, _ = filled(H, F, 4, 64, 32, 16, 2, [40], gen)
    q, good = torch.zeros(3, 4, 64, dtype=F, device="cuda"), torch.zeros(3, 1, dtype=torch.int64, device="cuda")
    for bad in (None, good.cpu(), good[:2], good.int(), good[:, 0], torch.zeros(3, 2, dtype=torch.int64, device="cuda")[:, ::2],
                torch.zeros(3, 0, dtype=torch.int64, device="cuda"), torch.zeros(3, 257, dtype=torch.int64, device="cuda")):
        with pytest.raises(H.HQQError):
            H.cache_attention_tree(cache, i32(table), i32([40]), bad, q)
        with pytest.raises(H.HQQError):
            H.hqq_cache_attention_tree(cache, i32(table), i32([40]), bad, q, torch.empty_like(q))


# ---- accepted tokens -------------------------------------------------------------------------
def some(H, layers, dtype, nbits, dim, group, page, kv, n_pages, gen):
    """Caches that hold numbers everywhere."""
    out = []
    for _ in range(layers):
        c = H.alloc_cache(n_pages, page, kv, dim, nbits, group, dtype)
        for x in ("k_codes", "v_codes"):
            c[x].copy_(torch.randint(0, 256, c[x].shape, generator=gen))
        for x in ("k_meta", "v_meta"):
            c[x].copy_(torch.randn(c[x].shape, generator=gen))
        out.append(c)
    return out


def check_kept(H, caches, table, lens, cu, n, kept, lens_out=True):
    want = [T.keep(c, table, lens, cu, n, kept) for c in caches]
    args = (i32(table), i32(lens), i32(kept).reshape(len(lens), -1), n)
    kw = {} if cu is None else dict(cu_tokens=i32(cu))
    if lens_out:
        assert H.cache_keep(caches, *args, **kw).tolist() == want[0][1]
    else:
        H.hqq_cache_keep(caches, *args, **kw)
    for c, (bufs, _) in zip(caches, want):
        for name, x in bufs.items():
            assert same_bits(c[name], x), name


KEEPS = [
    # dtype, nbits, dim, group, page, kv heads, layers, lens, new, max_kept
    (F, 4, 64, 32, 16, 2, 1, [30], [9], 5),
    (B, 4, 128, 64, 16, 8, 3, [33, 64, 31, 5], [20, 17, 1, 5], 7),
    (F, 8, 128, 128, 32, 3, 2, [100, 40], [33, 40], 33),
    (B, 4, 256, 64, 64, 2, 2, [70, 0, 66], [66, 0, 2], 6),
    (F, 8, 256, 32, 16, 1, 1, [200], [180], 150),
    (B, 8, 64, 64, 128, 5, 65, [90, 16, 15], [7, 16, 2], 4),
    (F, 4, 128, 32, 16, 2, 2, [25] * 70, [12] * 70, 12),
]


@pytest.mark.parametrize("dtype,nbits,dim,group,page,kv,layers,lens,new,most", KEEPS)
def test_keep(H, dtype, nbits, dim, group, page, kv, layers, lens, new, most):
    gen = torch.Generator().manual_seed(dim + nbits + kv)
    table, n_pages, _ = layout(lens, page, gen)
    caches = some(H, layers, dtype, nbits, dim, group, page, kv, n_pages, gen)
    kept = []
    for n in new:
        m = int(torch.randint(0, min(n, most) + 1, (1,), generator=gen))
        row = sorted(torch.randperm(n, generator=gen)[:m].tolist())
        kept.append(row + [-1] * (most - m))
    cu = cumulated(new)
    check_kept(H, caches, table, lens, cu, cu[-1] + 3, kept)
    if len(set(new)) == 1:
        check_kept(H, caches, table, lens, None, cu[-1], kept, lens_out=False)


def test_lists_that_end_early_and_places_that_are_not_there(H):
    gen = torch.Generator().manual_seed(8)
    table = [[3, -1, 9], [0, 2, 1], [4, 99, 5], [6, 7, 8], [10, 11, 12], [13, 14, 15], [16, 17, 18]]
    lens = [40, 45, 40, 1000000, 3, -5, 48]
    new = [20, 30, 30, 30, 9, 4, 48]
    kept = [[2, 4, 9, 15, 19, -1], [5, 5, 6, 7, 8, 9], [0, 3, 12, 20, 28, 29], [1, 29, 30, 31, 32, 33], [6, 7, 8, -1, 3, 4],
            [0, 1, 2, 3, 4, 5], [7, 6, 9, 10, 11, 12]]
    caches = some(H, 2, F, 4, 128, 64, 16, 2, 19, gen)
    check_kept(H, caches, table, lens, cumulated(new), sum(new), kept)
    for bad in ([-5, 20, 50, 80, 300, 300, 300, 400], [0] * 8, [9, 9, 40, 60, 60, 60, 60, 60]):
        check_kept(H, caches, table, lens, bad, sum(new), kept)
    wide = [[-1] * 6] * 6 + [list(range(1, 48)) + [3] * 100]
    check_kept(H, caches, table, lens, cumulated(new), sum(new), [r + [-1] * (147 - len(r)) for r in wide])
    check_kept(H, caches, table, lens, cumulated(new), sum(new), [[]] * 7)


def test_keep_refuses_in_the_binding(H):
    gen = torch.Generator().manual_seed(9)
    a, b = some(H, 2, F, 4, 64, 32, 16, 1, 3, gen)
    t, ln, good = i32([[0, 1]]), i32([20]), i32([[0, 2]])
    odd = some(H, 1, B, 4, 64, 32, 16, 1, 3, gen)[0]
    for caches, kept, kw in (([], good, {}), ([a, a], good, {}), ([a, odd], good, {}), (a, good[0], {}), (a, good.long(), {}),
                             (a, good.cpu(), {}), (a, i32([[0], [1]]), {}), (a, i32([[0, 1, 2, 3]])[:, ::2], {}),
                             (a, good, dict(lens_out=ln)), (a, good, dict(lens_out=i32([1, 2]))), (a, good, dict(lens_out=ln.long())),
                             (a, good, dict(cu_tokens=i32([0])))):
        with pytest.raises(H.HQQError):
            H.hqq_cache_keep(caches, t, ln, kept, 4, **kw)
    assert H.cache_keep([a, b], t[:0].contiguous(), ln[:0], good[:0], 0).shape == (0,)
