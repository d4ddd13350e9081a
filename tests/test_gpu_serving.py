"""Rotary positions, prompt attention, the cache, tree attention and keeping accepted tokens as a program
calls them: one after another, on other streams, and captured."""
import math

import pytest
import torch

import cache_ref as R
import tree_ref as T
from test_gpu_cache import i32, same_bits
from test_gpu_prompt import check as check_prompt, reference as prompt_reference
from test_gpu_rotary import check as check_rotary, reference as rotary_reference

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


@pytest.mark.parametrize("dtype,nbits,dim,hq,hk", [(F, 4, 128, 8, 2), (B, 8, 64, 6, 3)])
def test_a_prompt_a_draft_and_what_is_accepted(H, dtype, nbits, dim, hq, hk):
    """Two layers of a batch: prompts are turned, attended to and written; drafted trees are turned by
    their depth, written behind them and attend by their masks; the accepted path is kept, and the next
    token's attention is what it is over a cache that was written without the others."""
    gen = torch.Generator().manual_seed(dim)
    page, lens, drafted, layers = 16, [70, 1, 33], [9, 5, 7], 2
    depth = [[0, 0, 1, 1, 1, 2, 2, 3, 0], [0, 0, 1, 1, 2], [0, 1, 2, 0, 1, 2, 3]]
    parent = [[-1, -1, 0, 0, 1, 2, 4, 6, -1], [-1, -1, 1, 0, 2], [-1, 0, 1, -1, 3, 4, 5]]
    path = [[1, 4, 6, 7], [1, 2, 4], [0]]                        # each the parent of the next
    for p, q in zip(parent, path):
        assert all(p[b] == a for a, b in zip(q, q[1:]))
    freqs = H.rotary_frequencies(dim // 2, theta=10000.0, factor=2.0, original_len=64)
    width = -(-(max(lens) + max(drafted)) // page) + 1
    table = torch.randperm(3 * width, generator=gen).view(3, width).tolist()
    cu = [0, 70, 71, 104]
    caches, plain = ([H.alloc_cache(3 * width, page, hk, dim, nbits, 32, dtype) for _ in range(layers)] for _ in range(2))
    full = [n + d for n, d in zip(lens, drafted)]
    cu_d = [0, 9, 14, 21]
    masks = []
    for p in parent:
        seen = []
        for j, a in enumerate(p):
            seen.append((seen[a] if a >= 0 else 0) | 1 << j)
        masks += seen
    tree = T.to_words(masks, 1).cuda()
    kept = i32([q + [-1] * (4 - len(q)) for q in path])
    prompts = [torch.randn(104, hq + 2 * hk, dim, generator=gen).to(dtype).cuda() for _ in range(layers)]
    drafts = [torch.randn(21, hq + 2 * hk, dim, generator=gen).to(dtype).cuda() for _ in range(layers)]
    at = [i for n in lens for i in range(n)]
    at_d = [n + x for n, d in zip(lens, depth) for x in d]
    for layer in range(layers):
        x = prompts[layer]
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        ref = rotary_reference(freqs.tolist(), at, k, False, 1.0)
        H.hqq_rotary(freqs, i32(at), q, k)                      # in place, in the projection's output
        check_rotary(k, ref)
        out = H.prompt_attention(q, k, v, cu_tokens=i32(cu))
        check_prompt(out, None, prompt_reference(q, k, v, list(zip(cu, cu[1:])), dim ** -0.5))
        for c in (caches, plain):
            H.hqq_cache_write(c[layer], i32(table), i32(lens), k, v, cu_tokens=i32(cu))
        x = drafts[layer]
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        H.hqq_rotary(freqs, i32(at_d), q, k)
        H.hqq_cache_write(caches[layer], i32(table), i32(full), k, v, cu_tokens=i32(cu_d))
        out = H.cache_attention_tree(caches[layer], i32(table), i32(full), tree, q, cu_tokens=i32(cu_d))
        R.check_attention(out, None, T.attention(R.Held(caches[layer]), table, full, cu_d, q, dim ** -0.5, tree),
                          torch.ones(21, dtype=torch.bool))
        # a path's rows see what a chain of its tokens sees
        rows = [c + j for c, p in zip(cu_d, path) for j in p]
        cu_p = [0, 4, 7, 8]
        H.hqq_cache_write(plain[layer], i32(table), i32([n + len(p) for n, p in zip(lens, path)]), k[rows], v[rows], cu_tokens=i32(cu_p))
    new = H.cache_keep(caches, i32(table), i32(full), kept, 21, cu_tokens=i32(cu_d))
    assert new.tolist() == [n + len(p) for n, p in zip(lens, path)]
    q = torch.randn(3, hq, dim, generator=gen).to(dtype).cuda()
    for layer in range(layers):
        n = int(new.sum())
        for a, b in zip(H.cache_read(caches[layer], i32(table), new, n, cu_tokens=i32([0] + torch.cumsum(new.cpu(), 0).tolist())),
                        H.cache_read(plain[layer], i32(table), new, n, cu_tokens=i32([0] + torch.cumsum(new.cpu(), 0).tolist()))):
            assert torch.equal(a, b)
        assert torch.equal(H.cache_attention(caches[layer], i32(table), new, q), H.cache_attention(plain[layer], i32(table), new, q))


def case(H):
    gen = torch.Generator().manual_seed(1)
    s = {"lens": i32([200, 90]), "cu": i32([0, 12, 20]), "table": torch.arange(28, dtype=torch.int32, device="cuda").view(2, 14)}
    s["caches"] = [H.alloc_cache(28, 16, 2, 64, 4, 32) for _ in range(3)]
    for c in s["caches"]:
        k, v = (torch.randn(290, 2, 64, generator=gen).half().cuda() for _ in range(2))
        H.hqq_cache_write(c, s["table"], s["lens"], k, v, cu_tokens=i32([0, 200, 290]))
    s["q"], s["k"], s["v"] = (torch.randn(20, h, 64, generator=gen).half().cuda() for h in (8, 2, 2))
    s["tree"] = T.random_masks([12, 8], gen, 1).cuda()
    s["pos"], s["freqs"] = torch.arange(20, dtype=torch.int32, device="cuda"), H.rotary_frequencies(64)
    s["kept"] = i32([[0, 5, 7, -1], [2, 3, 4, 6]])
    return s


def run(H, s, call, **kw):
    if call == "rotary":
        return list(H.rotary(s["freqs"], s["pos"], s["q"], s["k"], **kw))
    if call == "prompt":
        return [H.prompt_attention(s["q"], s["k"], s["v"], cu_tokens=s["cu"], **kw)]
    if call == "tree":
        return [H.cache_attention_tree(s["caches"][0], s["table"], s["lens"], s["tree"], s["q"], cu_tokens=s["cu"], **kw)]
    return [H.cache_keep(s["caches"], s["table"], s["lens"], s["kept"], 20, cu_tokens=s["cu"], **kw)]


@pytest.mark.parametrize("call", ["rotary", "prompt", "tree", "keep"])
def test_what_a_call_allocates_belongs_to_its_stream(H, call):
    """Memory that the current stream has yet to write is not what a call on another stream fills."""
    s = case(H)
    want = run(H, s, call)
    slow = torch.empty(1 << 31, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    left = [torch.empty_like(x) for x in want]
    for _ in range(30):
        slow.fill_(1)
    for x in left:
        x.fill_(7)              # still to come when the call on the other stream is done
    del left, x
    got = run(H, s, call, stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed(H):
    """All four in one graph, on values, lengths, masks and lists that change between the replays."""
    s = case(H)
    q_out, k_out, out, tree_out, lens_out = (torch.empty_like(x) for x in (s["q"], s["k"], s["q"], s["q"], s["lens"]))

    def calls():
        H.hqq_rotary(s["freqs"], s["pos"], s["q"], s["k"], q_out, k_out)
        H.hqq_prompt_attention(q_out, k_out, s["v"], out, cu_tokens=s["cu"])
        H.hqq_cache_write(s["caches"][0], s["table"], s["lens"], k_out, s["v"], cu_tokens=s["cu"])
        H.hqq_cache_attention_tree(s["caches"][0], s["table"], s["lens"], s["tree"], q_out, tree_out, cu_tokens=s["cu"])
        H.hqq_cache_keep(s["caches"], s["table"], s["lens"], s["kept"], 20, lens_out, cu_tokens=s["cu"])
    held = [{x: c[x].clone() for x in ("k_codes", "v_codes", "k_meta", "v_meta")} for c in s["caches"]]

    def restore():
        for c, h in zip(s["caches"], held):
            for x, y in h.items():
                c[x].copy_(y)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    gen = torch.Generator().manual_seed(2)
    for i in range(4):
        s["q"].copy_(torch.randn(20, 8, 64, generator=gen).half())
        s["k"].copy_(torch.randn(20, 2, 64, generator=gen).half())
        s["pos"].add_(1000 * i)
        s["lens"].copy_(i32([200 - 31 * i, 90 + i]))
        s["cu"].copy_(i32([0, 12 - i, 20 - 2 * i]))
        s["tree"].copy_(T.random_masks([20], gen, 1))
        s["kept"].copy_(i32([[i, 5, 7, -1], [2, 3, 4 + i // 2, 6]]))
        results = []
        for go in (calls, graph.replay):
            restore()
            for x in (out, tree_out):
                x.fill_(3)
            go()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (q_out, k_out, out, tree_out, lens_out)] +
                           [c[x].clone() for c in s["caches"] for x in held[0]])
        # by their bits: what was never written may be NaN
        assert all(same_bits(a, b) for a, b in zip(*results)), i


def test_two_streams_at_once(H):
    """Calls that run at the same time, on outputs of their own."""
    gen = torch.Generator().manual_seed(3)
    streams = [torch.cuda.Stream() for _ in range(2)]
    x = [torch.randn(700, 12, 128, generator=gen).half().cuda() for _ in range(2)]
    s = case(H)
    want = [H.prompt_attention(y[:, :8], y[:, 8:10], y[:, 10:]) for y in x] + run(H, s, "tree")
    torch.cuda.synchronize()
    got = [None] * 3
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = H.prompt_attention(x[i][:, :8], x[i][:, 8:10], x[i][:, 10:])
                if i:
                    got[2] = run(H, s, "tree")[0]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tree_of_a_padded_batch(H):
    """Rows behind the last sequence's, lists behind the last entry and sequences of no tokens."""
    gen = torch.Generator().manual_seed(4)
    s = case(H)
    q = torch.randn(64, 8, 64, generator=gen).half().cuda()
    tree = T.random_masks([64], gen, 1).cuda()
    cu = i32([0, 30, 30])
    out = torch.full_like(q, 2.0)
    H.hqq_cache_attention_tree(s["caches"][0], s["table"], s["lens"], tree, q, out, cu_tokens=cu)
    ref = T.attention(R.Held(s["caches"][0]), s["table"].tolist(), [200, 90], [0, 30, 30], q, 0.125, tree)
    R.check_attention(out, None, ref, torch.tensor([True] * 30 + [False] * 34))
    assert (out[30:] == 2).all()
    lens = H.cache_keep(s["caches"], s["table"], s["lens"], i32([[0, 3, -1], [0, 1, 2]]), 64, cu_tokens=cu)
    assert lens.tolist() == [172, 90]


def test_a_prompt_beyond_2_31_bytes(H):
    """Keys whose last rows lie 2^32 bytes behind the first: strides of a wide projection."""
    n, wide = 300, 1 << 23
    buf = torch.empty(n * wide // 2 + 4096, dtype=F, device="cuda")
    x = torch.as_strided(buf, (n, 3, 64), (wide // 2, 64, 1))
    x.copy_(torch.randn(n, 3, 64, generator=torch.Generator().manual_seed(5)).half())
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    check_prompt(H.prompt_attention(q, k, v), None, prompt_reference(q, k, v, [(0, n)], 0.125))
    freqs, p = H.rotary_frequencies(64), torch.arange(n, dtype=torch.int32, device="cuda")
    check_rotary(H.rotary(freqs, p, q), rotary_reference(freqs.tolist(), p.tolist(), q, False, 1.0))
    assert math.isfinite(float(x.float().sum()))
