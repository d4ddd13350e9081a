"""The cache's calls as a program makes them: on a stream of its own, with queries of any layout, on a
GPU that other work shares."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


def small(H, n=200, heads=2, dim=64):
    gen = torch.Generator().manual_seed(n)
    cache = H.alloc_cache(-(-n // 16), 16, heads, dim, 4, 32)
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, heads, dim, generator=gen).half().cuda() for _ in range(2))
    H.hqq_cache_write(cache, table, lens, k, v)
    return cache, table, lens, torch.randn(n, 2 * heads, dim, generator=gen).half().cuda()


@pytest.mark.parametrize("call", ["read", "attention", "prefix"])
def test_what_a_call_allocates_belongs_to_its_stream(H, call):
    """Memory that the current stream has yet to write is not what a call on another stream fills."""
    cache, table, lens, q = small(H)

    def run(**kw):
        if call == "read":
            return torch.stack(H.cache_read(cache, table, lens, 200, **kw))
        if call == "attention":
            return H.cache_attention(cache, table, lens, q, **kw)
        return H.cache_attention_prefix(cache, table, lens, table[0], 30, q, **kw)
    want = run()
    slow = torch.empty(1 << 31, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    shape = (2, 200, 2, 64) if call == "read" else q.shape
    left = torch.empty(shape, dtype=torch.float16, device="cuda")
    for _ in range(30):
        slow.fill_(1)
    left.fill_(7)               # still to come when the call on the other stream is done
    del left
    if call == "read":
        got = H.cache_read(cache, table, lens, 200, stream=side.cuda_stream)
    else:
        got = run(stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(torch.stack(got) if call == "read" else got, want)


def test_outputs_are_contiguous_whatever_the_queries(H):
    cache, table, lens, q = small(H)
    want = H.cache_attention(cache, table, lens, q)
    wide = torch.zeros(q.shape[0], q.shape[1] + 3, q.shape[2], dtype=q.dtype, device="cuda")
    wide[:, 1:-2] = q
    for x in (q.transpose(0, 1).contiguous().transpose(0, 1), wide[:, 1:-2]):       # heads first; a part of more
        out = H.cache_attention(cache, table, lens, x)
        assert out.is_contiguous() and torch.equal(out.view(q.shape[0], -1), want.view(q.shape[0], -1))
        out = H.cache_attention_prefix(cache, table, lens, table[0], 0, x)
        assert out.is_contiguous() and torch.equal(out, want)
