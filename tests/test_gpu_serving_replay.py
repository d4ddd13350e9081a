"""The calls around a served model's cache in one captured graph, each of whose outputs is filled with
another value before every pass: what a pass does not write shows."""
import pytest
import torch

import tree_ref as T
from test_gpu_cache import i32, same_bits
from test_gpu_serving import H, case       # noqa: F401 (H is a fixture)

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.mark.parametrize("in_place", [False, True])
def test_each_pass_writes_all_outputs(H, in_place):     # noqa: F811
    s = case(H)
    q_out, k_out, out, tree_out, lens_out = (torch.empty_like(x) for x in (s["q"], s["k"], s["q"], s["q"], s["lens"]))
    q, k = (torch.empty_like(x) for x in (s["q"], s["k"]))

    def calls():
        if in_place:                    # queries in place, keys not
            H.hqq_rotary(s["freqs"], s["pos"], q, k, k_out=k_out)
        else:
            H.hqq_rotary(s["freqs"], s["pos"], q, k, q_out, k_out)
        turned = q if in_place else q_out
        H.hqq_prompt_attention(turned, k_out, s["v"], out, cu_tokens=s["cu"])
        H.hqq_cache_write(s["caches"][0], s["table"], s["lens"], k_out, s["v"], cu_tokens=s["cu"])
        H.hqq_cache_attention_tree(s["caches"][0], s["table"], s["lens"], s["tree"], turned, tree_out, cu_tokens=s["cu"])
        H.hqq_cache_keep(s["caches"], s["table"], s["lens"], s["kept"], 20, lens_out, cu_tokens=s["cu"])
    parts = ("k_codes", "v_codes", "k_meta", "v_meta")
    held = [{x: c[x].clone() for x in parts} for c in s["caches"]]
    outputs = (k_out, out, tree_out) if in_place else (q_out, k_out, out, tree_out)

    def begin(fill):
        for c, h in zip(s["caches"], held):
            for x, y in h.items():
                c[x].copy_(y)
        q.copy_(s["q"])
        k.copy_(s["k"])
        for x in outputs:
            x.fill_(fill)
        lens_out.fill_(-77)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        begin(0)
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    gen = torch.Generator().manual_seed(2)
    last = None
    for i in range(4):
        s["q"].copy_(torch.randn(20, 8, 64, generator=gen).half())
        s["k"].copy_(torch.randn(20, 2, 64, generator=gen).half())
        s["pos"].add_(1000 * i)
        s["lens"].copy_(i32([200 - 31 * i, 90 + i]))
        rows = 20 - 2 * i
        s["cu"].copy_(i32([0, 12 - i, rows]))
        s["tree"].copy_(T.random_masks([20], gen, 1))
        kept = [[i, 5, 7, -1], [2, 3, 4 + i // 2, 6]]
        s["kept"].copy_(i32(kept))
        lens = [a - n + len(T.kept_of(row, n)) for a, n, row in zip((200 - 31 * i, 90 + i), (12 - i, 8 - i), kept)]
        results = []
        for go, fill in ((calls, 3.0), (graph.replay, 5.0)):
            begin(fill)
            go()
            torch.cuda.synchronize()
            # rotary turns all rows; the others leave those behind the last sequence as they were
            for x in outputs[:-2]:
                assert (x != fill).all(), i
            for x in (out, tree_out):
                assert (x[:rows] != fill).any(-1).all() and (x[rows:] == fill).all(), i
            assert lens_out.tolist() == lens, i
            results.append([x.clone() for x in (q, *outputs[:-2], out[:rows], tree_out[:rows], lens_out)] +
                           [c[x].clone() for c in s["caches"] for x in parts])
        assert all(same_bits(a, b) for a, b in zip(*results)), i
        assert last is None or not torch.equal(last[-1], results[0][1])
        last = [results[0][1]]
