"""Scores hundreds apart, which grow, fall and jump along the sequence: the moving maximum and what
follows it (sums, outputs, pieces that are joined). Keys are whole numbers on their grids and queries
whole numbers, so that sums over groups are exact and the bound is a small part of the outputs."""
import pytest
import torch

import cache_bound as CB
import cache_ref as R
from test_gpu_cache_ranges import held_cache, i32

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


# dtype, nbits, dim, group, heads, query heads to each, tokens, new ones, width of the table: tiles of
# 16 rows, whole and in pieces; of 32; of 128, or of 32 and 64 for heads of 256
FORMS = [
    (F, 4, 128, 64, 2, 1, 400, 7, 400), (B, 8, 64, 32, 2, 2, 400, 8, 400), (B, 4, 256, 32, 1, 1, 400, 9, 400),
    (B, 8, 128, 128, 1, 8, 2500, 1, 2512), (F, 4, 128, 32, 1, 4, 2500, 3, 2512), (F, 8, 256, 64, 2, 2, 1500, 3, 1504),
    (B, 4, 128, 32, 256, 1, 400, 100, 1024), (F, 8, 64, 64, 256, 1, 400, 100, 1024),
    (B, 4, 128, 64, 256, 1, 400, 128, 2048), (F, 8, 64, 32, 256, 1, 400, 128, 2048), (F, 4, 128, 128, 256, 1, 400, 128, 2048),
    (B, 8, 256, 128, 256, 1, 200, 30, 1024), (F, 4, 256, 64, 256, 1, 200, 60, 2048),
]


@pytest.mark.parametrize("scene", ["growing", "falling", "jumping", "one at the end", "up and down"])
@pytest.mark.parametrize("dtype,nbits,dim,group,heads,per,n,new,width", FORMS)
def test_scores_far_apart(H, scene, dtype, nbits, dim, group, heads, per, n, new, width):
    gen = torch.Generator().manual_seed(dim + nbits + len(scene))
    top, t = 2 ** nbits - 1, torch.arange(n) / n
    part = {"growing": t, "falling": 1 - t, "jumping": torch.rand(n, generator=gen), "up and down": (1 - (8 * t % 2 - 1).abs()),
            "one at the end": (torch.arange(n) == n - 1).float()}[scene]
    # codes: 8 dimensions follow the scene, the others are random; 0 and the last in every group
    codes = torch.randint(0, top + 1, (n, heads, dim), generator=gen).double()
    codes[:, :, 2:10] = (part * top).round()[:, None, None].double()
    codes = codes.reshape(n, heads, -1, group)
    codes[..., 0], codes[..., 1] = 0, top
    base = -(top + 1) // 2 * torch.randint(0, 2, (n, heads, dim // group, 1), generator=gen).double()
    k = (codes + base).reshape(n, heads, dim)
    v = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64) + torch.randn(heads, dim, generator=gen)
    q = torch.randint(-1, 2, (new, heads * per, dim), generator=gen).float()
    q[..., 2:10] = torch.randint(1, 4, (new, heads * per, 1), generator=gen).float()
    scale = 1.0 if nbits == 4 else 2.0 ** -4        # the scene's dimensions: 120 to 382 from end to end
    cache, table = held_cache(H, dtype, nbits, group, 16, width, k, v, gen)
    held = R.Held(cache)
    q = q.to(dtype).cuda()
    for s in (scale, -scale):
        lse = torch.empty(new, heads * per, dtype=torch.float32, device="cuda")
        out = H.cache_attention(cache, i32(table), i32([n]), q, lse=lse, scale=s)
        ref = CB.attention(held, table, [n], None, q, s, whole=True)
        assert ref[2].max() < 0.1 * ref[0].square().mean().sqrt(), float(ref[2].max())
        CB.check(out, lse, ref, torch.ones(new, dtype=torch.bool))
