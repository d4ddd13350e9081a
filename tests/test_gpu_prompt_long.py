"""Attention of long prompts on the GPU, some of whose rows are held against 64 bits."""
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


def check_row(out, lse, q, k, v, i, begin, scale):
    """Row i (of the call) and its query heads against the definition. The bound is that of
    test_gpu_prompt.reference, a binary32 evaluation whose weights are rounded to the type where they meet
    the values: half a step, and with binary16 2^-32 of the row's largest at least."""
    n, (hq, dim), hk = i + 1 - begin, q.shape[1:], k.shape[1]
    half = R.HALF_STEP[q.dtype]
    x = q[i].double().view(hk, hq // hk, dim)
    y, z = (a[begin:i + 1].double().transpose(0, 1).contiguous() for a in (k, v))
    yt = y.transpose(1, 2).contiguous()
    s = torch.matmul(x, yt) * scale
    mag = torch.matmul(x.abs(), yt.abs()) * abs(scale)
    m = s.amax(-1, keepdim=True)
    w = torch.exp(s - m)
    tot = w.sum(-1, keepdim=True)
    p = w / tot
    r = 2 * (mag * (dim + 4) * 2.0 ** -24 + s.abs().amax(-1, keepdim=True) * 2.0 ** -23) + 2.0 ** -21
    total = (p * r).sum(-1, keepdim=True) + n * 2.0 ** -23
    rounded = p * half if q.dtype == B else torch.maximum(p * half, 2.0 ** -32 / tot)
    want = torch.matmul(p, z)
    e = torch.matmul(p * (r + total + n * 2.0 ** -23) + rounded, z.abs())
    got = out[i].double().view_as(want)
    tol = e + half * (want.abs() + e) + (2.0 ** -25 if q.dtype == F else 2.0 ** -130)
    d = (got - want).abs()
    assert (d <= tol).all(), f"row {i}: worst {float((d / tol).max()):.3g} of the tolerance, {float(d.max()):.3g}"
    d = (lse[i].double().view(hk, -1) - (m + torch.log(tot)).squeeze(-1)).abs()
    assert (d <= r.amax(-1) + total.squeeze(-1) + m.squeeze(-1).abs() * 2.0 ** -22).all(), f"row {i}: lse off by {float(d.max()):.3g}"


@pytest.mark.parametrize("dtype,dim,hk,per", [(F, 64, 1, 1), (F, 128, 1, 4), (F, 128, 1, 1), (F, 256, 1, 1), (B, 128, 1, 1)])
def test_many_small_weights_beside_a_large_one(H, dtype, dim, hk, per):
    """One key lies about 25.6 powers of two above all others, whose weights together are 2^-8.6 of its
    own: where its value is 0, they are the output."""
    n = 131072
    gen = torch.Generator().manual_seed(dim + per)
    q = torch.zeros(n, hk * per, dim)
    q[..., 0] = 1
    k = torch.randn(n, hk, dim, generator=gen) * 0.5
    k[0, :, 0] += 17.75
    v = torch.rand(n, hk, dim, generator=gen) + 0.5
    v[0] = 0
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    lse = torch.empty(n, hk * per, dtype=torch.float32, device="cuda")
    out = H.prompt_attention(q, k, v, scale=1.0, lse=lse)
    for i in (n - 1, 100003, 65535, 40000, 300):
        check_row(out, lse, q, k, v, i, 0, 1.0)


@pytest.mark.parametrize("dtype,dim,hk,per,n", [(F, 64, 2, 4, 30011), (B, 128, 2, 8, 20001), (F, 256, 1, 5, 16500)])
def test_long_prompts(H, dtype, dim, hk, per, n):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(n, hk * (per + 2), dim, generator=gen) + torch.randn(hk * (per + 2), dim, generator=gen) * 0.5
    x = x.to(dtype).cuda()
    q, k, v = x[:, :hk * per], x[:, hk * per:hk * (per + 1)], x[:, hk * (per + 1):]
    lse = torch.empty(n, hk * per, dtype=torch.float32, device="cuda")
    out = H.prompt_attention(q, k, v, lse=lse)
    for i in (n - 1, n // 2, 8191, 4097, 1000, 31, 0):
        check_row(out, lse, q, k, v, i, 0, dim ** -0.5)
    assert math.isfinite(float(out.float().sum()))


@pytest.mark.parametrize("dtype,dim,per,mean", [(F, 128, 4, 2100), (B, 128, 5, 2300), (B, 256, 1, 4200)])
def test_blocks_of_256_rows_and_many_sequences(H, dtype, dim, per, mean):
    """More sequences than a wave has lanes, some empty and one six times the mean: in blocks of 256
    rows, like the two halves of the batch by themselves, whose sequences fit a wave."""
    gen = torch.Generator().manual_seed(dim + per)
    lens = [0, 1, 6 * mean, 255, 256, 257] + [mean + 7 * (i % 9 - 4) for i in range(64)] + [2 * mean, 0]
    assert len(lens) == 72
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    n = cu[-1]
    x = torch.randn(n + 3, per + 2, dim, generator=gen, dtype=torch.float32).to(dtype).cuda()
    q, k, v = x[:, :per], x[:, per:per + 1], x[:, per + 1:]
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    out = torch.full((n + 3, per, dim), 11.0, dtype=dtype, device="cuda")
    lse = torch.full((n + 3, per), 13.0, dtype=torch.float32, device="cuda")
    H.hqq_prompt_attention(q, k, v, out, cu_tokens=i32(cu), lse=lse)
    assert (out[n:] == 11).all() and (lse[n:] == 13).all()
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        for row in {hi - 1, (lo + hi) // 2, lo} if i % 5 < 2 and hi > lo else ():
            check_row(out, lse, q, k, v, row, lo, dim ** -0.5)
    for lo, hi in ((0, 36), (36, 72)):          # the same bits: a step has as many keys
        part = slice(cu[lo], cu[hi])
        assert sum(lens[lo:hi]) // 36 >= (2048 if dim == 128 else 4096)
        got = H.prompt_attention(q[part], k[part], v[part], cu_tokens=i32([c - cu[lo] for c in cu[lo:hi + 1]]))
        assert torch.equal(got, out[part])


@pytest.mark.parametrize("dtype,dim,hk,per,lens", [(F, 128, 32, 1, [520] * 24 + [900, 1, 0, 1300] * 8), (B, 256, 16, 2, [640, 515] * 16),
                                                   (B, 128, 16, 4, [600] * 80)])
def test_keys_and_values_beyond_the_caches(H, dtype, dim, hk, per, lens):
    """Medium sequences whose keys and values are more than 256 MB: some rows of some heads."""
    gen = torch.Generator().manual_seed(dim + hk)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    n = cu[-1]
    assert n * hk * dim * 4 >= 1 << 28 and n // len(lens) >= 512
    x = torch.randn(n, hk * (per + 2), dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    q, k, v = x[:, :hk * per], x[:, hk * per:hk * (per + 1)], x[:, hk * (per + 1):]
    lse = torch.empty(n, hk * per, dtype=torch.float32, device="cuda")
    out = H.prompt_attention(q, k, v, cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"), lse=lse)
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        for row in {hi - 1, (lo + hi) // 2, lo} if hi > lo else ():
            h = int(torch.randint(0, hk, (1,), generator=gen))
            mine = slice(h * per, h * per + per)
            check_row(out[:, mine], lse[:, mine], q[:, mine], k[:, h:h + 1], v[:, h:h + 1], row, lo, dim ** -0.5)
    assert torch.isfinite(out).all()
