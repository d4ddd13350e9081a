"""Attention over values of very different size: a token that a row does not see, or hardly weighs,
leaves it alone, whatever its size; groups of a head, and tokens one after another, have sizes of their
own. Against the 64-bit definition, with a bound that counts only what a row sees (cache_bound.py)."""
import pytest
import torch

import cache_bound as CB
import cache_ref as R

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def held_cache(H, dtype, nbits, group, page, width, k, v, gen):
    """A cache of one sequence k, v [n, heads, dim] under a table `width` tokens wide."""
    n, heads, dim = k.shape
    need = -(-n // page)
    order = torch.randperm(need + 2, generator=gen).tolist()
    table = [order[:need] + [-1] * (-(-width // page) - need)]
    cache = H.alloc_cache(need + 2, page, heads, dim, nbits, group, dtype)
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
        cache[x].view(torch.uint8).fill_(255)
    H.hqq_cache_write(cache, i32(table), i32([n]), k.to(dtype).cuda(), v.to(dtype).cuda())
    return cache, table


# dtype, nbits, dim, group, heads, query heads to each, tokens, new ones, width of the table: tiles of
# 16 rows; of 32; of 128, or of 32 and 64 for heads of 256, which take many heads and wide tables
FORMS = [
    (B, 4, 128, 64, 2, 1, 250, 7, 256), (B, 8, 64, 32, 2, 2, 250, 8, 256), (B, 4, 256, 32, 1, 1, 250, 9, 256),
    (B, 8, 128, 128, 1, 8, 700, 1, 704), (F, 4, 128, 64, 2, 1, 250, 7, 256),
    (B, 4, 128, 32, 256, 1, 200, 100, 1024), (B, 8, 64, 64, 256, 1, 200, 100, 1024), (F, 8, 64, 32, 256, 1, 200, 100, 1024),
    (B, 4, 128, 64, 256, 1, 200, 128, 2048), (B, 8, 64, 32, 256, 1, 200, 128, 2048), (F, 8, 128, 128, 256, 1, 200, 128, 2048),
    (B, 8, 256, 128, 256, 1, 100, 30, 1024), (B, 4, 256, 64, 256, 1, 100, 60, 2048),
]


def sizes(scene, dtype, n, dim, group):
    """What values are multiplied by, [n, dim]; small is where the others go in binary16, whose
    numbers end at 65504."""
    x = torch.ones(n, dim, dtype=torch.float64)
    t = torch.arange(n)
    half = dtype == F
    if scene == "one behind":               # a token that only the last row sees
        x *= 2.0 ** -10 if half else 1.0
        x[-1] = 7000.0 if half else 2.0 ** 40
    elif scene == "one far behind":
        x *= 2.0 ** -13 if half else 2.0 ** -60
        x[-1] = 7000.0 if half else 2.0 ** 90
    elif scene == "ends of the range":
        x *= 2.0 ** -14 if half else 2.0 ** -84
        x[-1] = 7000.0 if half else 2.0 ** 112
    elif scene == "a step far larger":      # all tokens of some steps, which the first of many rows do not see
        x *= 2.0 ** -14 if half else 2.0 ** -84
        x[-40:] = 7000.0 if half else 2.0 ** 100
    elif scene == "groups apart":
        x[:, :group] = 2.0 ** 10 if half else 2.0 ** 50
        x[:, group:] = 2.0 ** -11 if half else 2.0 ** -30
    elif scene == "rising and falling":     # up to the middle and down again
        e = (1 - (2 * t / n - 1).abs()).double()
        x *= torch.exp2((22 * e - 10) if half else (160 * e - 80))[:, None]
    elif scene == "mixed":
        x *= torch.tensor([1.0, 2.0 ** -12, 2.0 ** 11] if half else [1.0, 2.0 ** -30, 2.0 ** 35], dtype=torch.float64)[t * 7 % 3][:, None]
    elif scene == "hardly weighed":         # in front; the test makes its score low
        x *= 2.0 ** -10 if half else 1.0
        x[5] = 7000.0 if half else 2.0 ** 40
    return x


@pytest.mark.parametrize("scene", ["one behind", "one far behind", "ends of the range", "a step far larger", "groups apart", "rising and falling", "mixed", "hardly weighed"])
@pytest.mark.parametrize("dtype,nbits,dim,group,heads,per,n,new,width", FORMS)
def test_values_of_very_different_size(H, scene, dtype, nbits, dim, group, heads, per, n, new, width):
    gen = torch.Generator().manual_seed(dim + nbits + len(scene))
    k = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * 0.5
    v = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) + torch.randn(heads, dim, generator=gen)
    v *= sizes(scene, dtype, n, dim, group)[:, None]
    q = torch.randn(new, heads * per, dim, generator=gen) * 0.5
    scale = dim ** -0.5
    if scene == "hardly weighed":           # 60 lower than the others: 2^-86 of their weight
        q[..., 0], k[5, :, 0] = 4.0, -15.0 / scale
    cache, table = held_cache(H, dtype, nbits, group, 16, width, k, v, gen)
    q = q.to(dtype).cuda()
    lse = torch.empty(new, heads * per, dtype=torch.float32, device="cuda")
    out = H.cache_attention(cache, i32(table), i32([n]), q, lse=lse)
    ref = CB.attention(R.Held(cache), table, [n], None, q, scale)
    # the bound is a small part of what it bounds: of the row's group, in which sizes are alike
    size = ref[0].reshape(new, heads * per, -1, group)
    part = ref[2].reshape(size.shape).amax(-1) / size.square().mean(-1).sqrt()
    assert part.median() < 0.03 and part.max() < 0.2, (float(part.median()), float(part.max()))
    CB.check(out, lse, ref, torch.ones(new, dtype=torch.bool))


@pytest.mark.parametrize("new,heads,width", [(5, 2, 704), (100, 256, 1024), (128, 256, 2048)])
def test_sizes_that_change_between_prefix_and_sequences(H, new, heads, width):
    """A prefix of far larger values than the sequences', and the other way round."""
    gen = torch.Generator().manual_seed(new)
    dim, page, n, prefix = 64, 16, 130, 170
    for big, small in ((2.0 ** 40, 2.0 ** -20), (2.0 ** -20, 2.0 ** 40)):
        k = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * 0.5
        v = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * small
        cache, table = held_cache(H, B, 4, 32, page, width, k, v, gen)
        more = H.alloc_cache(cache["k_codes"].shape[0] + 11, page, heads, dim, 4, 32, B)
        first = cache["k_codes"].shape[0]
        for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
            more[x].view(torch.uint8).fill_(255)
            more[x][:first] = cache[x]
        pages = list(range(first, first + 11))
        H.hqq_cache_write(more, i32([pages]), i32([prefix]),
                          (torch.randn(prefix, heads, dim, generator=gen) * 0.5).to(B).cuda(),
                          (torch.randn(prefix, heads, dim, generator=gen) * big).to(B).cuda())
        q = (torch.randn(new, heads, dim, generator=gen) * 0.5).to(B).cuda()
        lse = torch.empty(new, heads, dtype=torch.float32, device="cuda")
        out = H.cache_attention_prefix(more, i32(table), i32([n]), i32(pages), prefix, q, lse=lse)
        ref = CB.attention(R.Held(more), table, [n], None, q, 0.125, pages, prefix)
        CB.check(out, lse, ref, torch.ones(new, dtype=torch.bool))


@pytest.mark.parametrize("dtype,nbits,heads,per,n_seqs,longest,new", [
    (B, 4, 2, 1, 70, 150, 1), (B, 8, 3, 4, 5, 900, 3), (F, 4, 2, 2, 70, 40, 2), (B, 4, 128, 1, 12, 600, 40)])
def test_sequences_of_very_different_size(H, dtype, nbits, heads, per, n_seqs, longest, new):
    """Several sequences to a block, each of a size of its own, some with a token far above or below."""
    gen = torch.Generator().manual_seed(n_seqs + heads)
    dim, group, page = 128, 64, 16
    lens = [1 + (i * 37) % longest for i in range(n_seqs)]
    new = [min(new, x) for x in lens]
    order = torch.randperm(sum(-(-x // page) for x in lens), generator=gen).tolist()
    table, width = [], -(-longest // page)
    for x in lens:
        own, order = order[:-(-x // page)], order[-(-x // page):]
        table.append(own + [-1] * (width - len(own)))
    n_pages = 1 + max(max(t) for t in table)
    cache = H.alloc_cache(n_pages, page, heads, dim, nbits, group, dtype)
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
        cache[x].view(torch.uint8).fill_(255)
    span = (-9, 9) if dtype == F else (-70, 70)
    k, v = [], []
    for i, x in enumerate(lens):
        y = torch.randn(x, heads, dim, generator=gen, dtype=torch.float64) * 2.0 ** (span[0] + (span[1] - span[0]) * (i % 7) / 6)
        if i % 3 == 0:
            y[(i * 5) % x] = torch.randn(heads, dim, generator=gen, dtype=torch.float64) * 2.0 ** (span[1] + 3)
        if i % 4 == 1:
            y[(i * 11) % x, :, :group] *= 2.0 ** (-11 if dtype == F else -40)
        v.append(y.to(dtype))
        k.append((torch.randn(x, heads, dim, generator=gen) * 0.5).to(dtype))
    cu = lambda c: i32([sum(c[:i]) for i in range(len(c) + 1)])
    H.hqq_cache_write(cache, i32(table), i32(lens), torch.cat(k).cuda(), torch.cat(v).cuda(), cu_tokens=cu(lens))
    q = (torch.randn(sum(new), heads * per, dim, generator=gen) * 0.5).to(dtype).cuda()
    lse = torch.empty(sum(new), heads * per, dtype=torch.float32, device="cuda")
    out = H.cache_attention(cache, i32(table), i32(lens), q, cu_tokens=cu(new), lse=lse)
    ref = CB.attention(R.Held(cache), table, lens, cu(new).tolist(), q, dim ** -0.5)
    CB.check(out, lse, ref, torch.ones(sum(new), dtype=torch.bool))


@pytest.mark.parametrize("scene", ["usual", "hardly weighed", "mixed"])
@pytest.mark.parametrize("heads,new,width", [(2, 7, 256), (256, 100, 1024), (256, 128, 2048)])
def test_queries_that_are_not_finite_leave_other_rows_alone(H, scene, heads, new, width):
    gen = torch.Generator().manual_seed(new + len(scene))
    dim, n = 64, 200
    k = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * 0.5
    v = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * sizes(scene, B, n, dim, 32)[:, None]
    q = torch.randn(new, heads, dim, generator=gen) * 0.5
    if scene == "hardly weighed":
        q[..., 0], k[5, :, 0] = 4.0, -120.0
    cache, table = held_cache(H, B, 4, 32, 16, width, k, v, gen)
    bad = {0: float("nan"), 3: float("inf"), 5: float("-inf")}
    ref = CB.attention(R.Held(cache), table, [n], None, q.to(B), 0.125)
    for i, x in bad.items():
        q[i, :, 7] = x
    out = H.cache_attention(cache, i32(table), i32([n]), q.to(B).cuda())
    CB.check(out, None, ref, torch.tensor([i not in bad for i in range(new)]))


@pytest.mark.parametrize("heads,new,width", [(2, 7, 704), (256, 128, 2048)])
def test_captured_calls_on_values_that_change_their_size(H, heads, new, width):
    """A graph replayed over values of usual and of very different sizes in turn."""
    gen = torch.Generator().manual_seed(new)
    dim, n = 64, 200
    made = []
    for scene in ("usual", "mixed", "usual", "one behind"):
        k = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * 0.5
        v = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) * sizes(scene, B, n, dim, 32)[:, None]
        made.append(held_cache(H, B, 8, 32, 16, width, k, v, torch.Generator().manual_seed(1)))
    cache, table = {**made[0][0]}, made[0][1]
    for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
        cache[x] = cache[x].clone()
    t, lens = i32(table), i32([n])
    q = (torch.randn(new, heads, dim, generator=gen) * 0.5).to(B).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(H.hqq_cache_attention_workspace(cache, t, lens, new, heads), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        H.hqq_cache_attention(cache, t, lens, q, out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hqq_cache_attention(cache, t, lens, q, out, workspace=ws)
    for other, same_table in made + made[:2]:
        assert same_table == table
        for x in ("k_codes", "v_codes", "k_meta", "v_meta"):
            cache[x].copy_(other[x])
        out.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        ref = CB.attention(R.Held(cache), table, [n], None, q, dim ** -0.5)
        CB.check(out, None, ref, torch.ones(new, dtype=torch.bool))
        assert torch.equal(H.cache_attention(cache, t, lens, q), out)
