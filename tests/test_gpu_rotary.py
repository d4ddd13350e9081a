"""Rotary positions on the GPU against the formula, with angles from whole numbers."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


def reference(freqs, positions, x, interleaved, scale):
    """(turned x, |a| + |b| by dimension) in float64: angles exact to 2^-53 of a turn."""
    turns = torch.tensor([[(p * (f % (1 << 64)) % (1 << 64)) / 2.0 ** 64 for f in freqs] for p in positions], dtype=torch.float64)
    turns = turns.reshape(len(positions), len(freqs))
    cos, sin = (f(2 * math.pi * turns)[:, None] * scale for f in (torch.cos, torch.sin))
    y, n = x.cpu().double(), 2 * len(freqs)
    i = torch.arange(n // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, n // 2 + i)
    a, b = y[..., one], y[..., two]
    out, size = y.clone(), torch.zeros_like(y)
    out[..., one], out[..., two] = a * cos - b * sin, b * cos + a * sin
    size[..., one] = size[..., two] = (a.abs() + b.abs()) * abs(scale)
    return out, size


def check(got, ref):
    """Cosine and sine, as the documentation says, are off by 2^-23, the product with scale and those
    with a and b round by 2^-24 of 1 and of the magnitudes, their sum once more: 2^-21 of |a| + |b|
    holds all of it. Then the type's rounding, half of its smallest number at least."""
    want, size = ref
    half, least = (2.0 ** -11, 2.0 ** -25) if got.dtype == F else (2.0 ** -8, 2.0 ** -134)
    e = 2.0 ** -21 * size
    bad = (got.cpu().double() - want).abs() > e + half * (want.abs() + e) + torch.where(size > 0, least, 0.0)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"
    same = size == 0
    assert torch.equal(got.cpu().double()[same], want[same])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


CASES = [
    # dtype, dim, rotary_dim, interleaved, heads, kv heads, positions
    (F, 128, 128, False, 32, 8, [700]),
    (B, 128, 128, False, 8, 1, list(range(70))),
    (F, 64, 32, True, 5, 5, [0, 1, -1, 130000, 2 ** 31 - 1, -2 ** 31]),
    (B, 256, 256, True, 3, 2, [5, 1048575, 77]),
    (F, 64, 16, False, 1, 1, [3] * 300),
    (B, 96, 48, False, 2, 1, [9, 10]),
    (F, 128, 2, False, 4, 2, [1, 2, 3]),
    (B, 64, 2, True, 1, 1, list(range(2100))),
    (F, 80, 26, True, 3, 2, [1000001, 5]),
    (B, 34, 34, False, 2, 3, [7, 8, 9]),
    (F, 1024, 1024, False, 2, 1, [123456]),
    (B, 65, 64, False, 2, 1, [4, 5]),
    (F, 128, 64, False, 300, 7, [11, 12, 13]),
    (B, 128, 74, False, 5, 3, [1, 70000, 3]),
    (F, 256, 254, True, 3, 1, [5, 6]),
    (B, 31, 30, False, 3, 2, [17]),
]


@pytest.mark.parametrize("dtype,dim,rot,interleaved,hq,hk,positions", CASES)
def test_rotary(H, dtype, dim, rot, interleaved, hq, hk, positions):
    gen = torch.Generator().manual_seed(dim + rot)
    n = len(positions)
    freqs = H.rotary_frequencies(rot, theta=10000.0, factor=4.0, original_len=512)
    wide = (torch.randn(n, hq + hk + 1, dim, generator=gen) * 3).to(dtype).cuda()
    before = wide.clone()
    q, k = wide[:, :hq], wide[:, hq:hq + hk]
    for scale in (1.0, -0.75):
        q_out, k_out = H.rotary(freqs, i32(positions), q, k, interleaved=interleaved, scale=scale)
        for got, x in ((q_out, q), (k_out, k)):
            assert got.is_contiguous()
            check(got, reference(freqs.tolist(), positions, x, interleaved, scale))
    assert torch.equal(wide, before)
    # the same bits in place, and where only one is turned, and into rows of another layout
    q_out, k_out = H.rotary(freqs, i32(positions), q, k, interleaved=interleaved)
    assert torch.equal(H.rotary(freqs, i32(positions), k, interleaved=interleaved), k_out)
    other = torch.full((hq + 1, n + 1, dim), 5.0, dtype=dtype, device="cuda").transpose(0, 1)
    H.hqq_rotary(freqs, i32(positions), q, q_out=other[:n, :hq], interleaved=interleaved)
    assert torch.equal(other[:n, :hq], q_out) and (other[n:] == 5).all() and (other[:, hq:] == 5).all()
    H.hqq_rotary(freqs, i32(positions), q, k, interleaved=interleaved)
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(wide[:, hq + hk:], before[:, hq + hk:])


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_of_any_alignment(H, dtype, shift):
    gen = torch.Generator().manual_seed(shift)
    freqs, positions = H.rotary_frequencies(32), [5, 900, 3]
    flat = torch.randn(3 * 4 * 67 + shift, generator=gen).to(dtype).cuda()
    x = flat[shift:shift + 3 * 4 * 67].view(3, 4, 67)[..., :64]
    check(H.rotary(freqs, i32(positions), x), reference(freqs.tolist(), positions, x, False, 1.0))


def test_every_quarter_turn_and_far_positions(H):
    """One pair with frequencies of a power of two of a turn: cosine and sine of known angles."""
    for p, f, cs in ((1, 1 << 62, (0, 1)), (2, 1 << 62, (-1, 0)), (3, 1 << 62, (0, -1)), (4, 1 << 62, (1, 0)),
                     (2 ** 30, 1 << 33, (-1, 0)), (-1, 1 << 62, (0, -1)), (2 ** 31 - 1, 1 << 63, (-1, 0)),
                     (1, 1 << 61, (2 ** -0.5, 2 ** -0.5)), (3, 1 << 61, (-2 ** -0.5, 2 ** -0.5))):
        freqs = torch.tensor([f - (1 << 64) if f >> 63 else f], dtype=torch.int64, device="cuda")
        x = torch.tensor([[[1.0, 0.0]]], dtype=F, device="cuda")
        got = H.rotary(freqs, i32([p]), x).cpu().double()[0, 0]
        want = torch.tensor(cs, dtype=torch.float64)
        assert ((got - want).abs() <= 2.0 ** -22 + 2.0 ** -11 * want.abs()).all(), (p, f, got)


def test_turned_back(H):
    """Negated positions undo a turn, up to what two roundings leave."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(50, 4, 128, generator=gen).to(F).cuda()
    freqs, p = H.rotary_frequencies(128), torch.arange(0, 50 * 999, 999, dtype=torch.int32, device="cuda")
    there = H.rotary(freqs, p, x, interleaved=True)
    back = H.rotary(freqs, -p, there, interleaved=True)
    size = x.double().abs().view(50, 4, 64, 2).sum(-1).repeat_interleave(2, -1)
    # a rounding of each of the two numbers on the way there, one on the way back, and 2^-20 for the rest
    assert ((back.double() - x.double()).abs() <= (3 * 2.0 ** -11 + 2.0 ** -20) * size + 2.0 ** -23).all()


def test_infinities_and_nan_stay_in_their_pair(H):
    x = torch.ones(2, 2, 64, dtype=F, device="cuda")
    x[0, 0, 3], x[1, 1, 40] = math.inf, math.nan
    freqs = H.rotary_frequencies(64)
    got = H.rotary(freqs, i32([5, 6]), x)
    ref = H.rotary(freqs, i32([5, 6]), torch.ones_like(x))
    touched = torch.zeros(2, 2, 64, dtype=torch.bool)
    touched[0, 0, 3] = touched[0, 0, 35] = touched[1, 1, 40] = touched[1, 1, 8] = True
    assert torch.equal(got.cpu()[~touched], ref.cpu()[~touched]) and not torch.isfinite(got.cpu()[touched]).any()


def test_nothing_to_turn(H):
    freqs = H.rotary_frequencies(64)
    q = torch.empty(0, 4, 64, dtype=F, device="cuda")
    assert H.rotary(freqs, i32([]), q).shape == q.shape
    q = torch.empty(3, 0, 64, dtype=F, device="cuda")
    assert H.rotary(freqs, i32([1, 2, 3]), q).shape == q.shape


def test_the_binding_refuses(H):
    freqs, p = H.rotary_frequencies(64), i32([1, 2])
    q = torch.zeros(2, 4, 64, dtype=F, device="cuda")
    for args, kw in (((freqs.cpu(), p, q), {}), ((freqs.float(), p, q), {}), ((freqs[::2], p, q), {}), ((freqs, p[:1], q), {}),
                     ((freqs, p.long(), q), {}), ((freqs, p, q.float()), {}), ((freqs, p, q[0]), {}), ((freqs, p, q.transpose(1, 2)), {}),
                     ((freqs, p, q, q.bfloat16()), {}), ((freqs, p, q, q[:1]), {}), ((freqs, p, q, q[..., :32]), {}),
                     ((freqs, p, q), dict(q_out=q[:, :2])), ((freqs, p, q), dict(k_out=q)), ((freqs, p, q[..., :62]), {}),
                     ((freqs, p, q), dict(scale=math.inf)), ((freqs, p, q), dict(q_out=q.cpu()))):
        with pytest.raises(H.HQQError):
            H.hqq_rotary(*args, **kw)
