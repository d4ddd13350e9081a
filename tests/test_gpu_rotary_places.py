"""Rotary calls of one tensor in place and another not, and of rows that share what is not turned."""
import pytest
import torch

from test_gpu_rotary import check, i32, reference

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


@pytest.mark.parametrize("dtype,dim,rot,interleaved,hq,hk,n", [
    (F, 128, 64, False, 32, 8, 1), (B, 64, 32, True, 5, 5, 70), (F, 80, 26, True, 3, 2, 9), (B, 128, 74, False, 5, 3, 3),
    (F, 128, 128, False, 4, 1, 5), (B, 65, 64, False, 2, 1, 4), (F, 1024, 2, True, 1, 2, 3), (F, 128, 64, False, 300, 7, 2)])
@pytest.mark.parametrize("place", ["q", "k"])
def test_one_in_place_the_other_not(H, dtype, dim, rot, interleaved, hq, hk, n, place):
    gen = torch.Generator().manual_seed(dim + rot + n)
    freqs, positions = H.rotary_frequencies(rot), [7 * i + 3 for i in range(n)]
    wide = torch.randn(n, hq + hk + 1, dim, generator=gen).to(dtype).cuda()
    before = wide.clone()
    q, k = wide[:, :hq], wide[:, hq:hq + hk]
    refs = [reference(freqs.tolist(), positions, x, interleaved, 1.0) for x in (q, k)]
    moved = k if place == "q" else q
    other = torch.full((moved.shape[1] + 1, n + 1, dim), 5.0, dtype=dtype, device="cuda").transpose(0, 1)
    H.hqq_rotary(freqs, i32(positions), q, k, interleaved=interleaved, **{("k" if place == "q" else "q") + "_out": other[:n, :-1]})
    here, there = (refs[0], refs[1]) if place == "q" else (refs[1], refs[0])
    check(q if place == "q" else k, here)
    check(other[:n, :-1], there)
    assert (other[n:] == 5).all() and (other[:, -1] == 5).all()
    left = slice(hq, None) if place == "q" else slice(0, hq)
    assert torch.equal(wide[:, left], before[:, left]) and torch.equal(wide[..., rot:], before[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_whose_other_dimensions_are_the_next_rows(H, interleaved):
    """In place, the dimensions behind those that are turned are not touched: they may be another row's,
    which turns them, also beside a tensor that goes to another place."""
    n, heads, rot, dim = 50, 6, 32, 64
    gen = torch.Generator().manual_seed(1)
    freqs, p = H.rotary_frequencies(rot), i32(list(range(3, 3 + n)))
    flat = torch.randn(n * heads * rot + dim - rot, generator=gen).half().cuda()
    before = flat.clone()
    x = torch.as_strided(flat, (n, heads, dim), (heads * rot, rot, 1))
    alone = flat[:n * heads * rot].view(n, heads, rot)
    ref = reference(freqs.tolist(), p.tolist(), alone.clone(), interleaved, 1.0)
    k = torch.randn(n, 3, dim, generator=gen).half().cuda()
    k_out = torch.empty_like(k)
    H.hqq_rotary(freqs, p, x, k, k_out=k_out, interleaved=interleaved)
    check(alone, ref)
    check(k_out, reference(freqs.tolist(), p.tolist(), k, interleaved, 1.0))
    assert torch.equal(flat[n * heads * rot:], before[n * heads * rot:])


def test_expanded_outputs_are_refused(H):
    """Rows that lie on each other would be turned once or several times."""
    freqs, p = H.rotary_frequencies(64), i32([1, 2, 3])
    q, k = torch.ones(3, 4, 64, dtype=F, device="cuda"), torch.ones(3, 2, 64, dtype=F, device="cuda")
    one, other = k[:, :1].expand(3, 2, 64), torch.ones(3, 1, 64, dtype=F, device="cuda").expand(3, 2, 64)
    for args, kw in (((q, one), {}), ((one,), {}), ((k[:1].expand(3, 2, 64),), {}), ((k,), dict(q_out=other)), ((q, k), dict(k_out=other)),
                     ((q, q), {})):
        with pytest.raises(H.HQQError, match="overlap"):
            H.hqq_rotary(freqs, p, *args, **kw)
    assert (q == 1).all() and (k == 1).all()
    # inputs may be, and what has one token or head may have any strides
    want = H.rotary(freqs, p, k)
    assert torch.equal(H.rotary(freqs, p, one), want)
    assert torch.equal(H.rotary(freqs, p[:1], one[:1, :1]), want[:1, :1])
    x = k[:, :1].clone()
    H.hqq_rotary(freqs, p, torch.as_strided(x, (3, 1, 64), (64, 0, 1)))
    assert torch.equal(x, want[:, :1])
