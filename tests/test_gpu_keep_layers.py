"""Accepted tokens kept in caches that lie one behind another in one allocation."""
import pytest
import torch

from test_gpu_cache import i32, layout
from test_gpu_tree import check_kept, some

pytestmark = pytest.mark.gpu

PARTS = ("k_codes", "v_codes", "k_meta", "v_meta")


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq


def test_layers_of_one_allocation(H):
    gen = torch.Generator().manual_seed(1)
    table, n_pages, _ = layout([50, 33], 16, gen)
    caches = some(H, 5, torch.float16, 4, 128, 64, 16, 2, n_pages, gen)
    whole = {x: torch.stack([c[x] for c in caches]) for x in PARTS}
    stacked = [dict(caches[0], **{x: whole[x][i] for x in PARTS}) for i in range(5)]
    check_kept(H, stacked[::-1], table, [50, 33], [0, 20, 30], 30, [[1, 4, 9], [0, 7, -1]])


@pytest.mark.parametrize("part", PARTS)
def test_shared_buffers_are_refused(H, part):
    gen = torch.Generator().manual_seed(2)
    a, b = some(H, 2, torch.float16, 4, 128, 64, 16, 2, 4, gen)
    before = [{x: c[x].clone() for x in PARTS} for c in (a, b)]
    with pytest.raises(H.HQQError, match="overlap"):
        H.hqq_cache_keep([a, dict(b, **{part: a[part]})], i32([[0, 1]]), i32([30]), i32([[2, 5]]), 9)
    assert all(torch.equal(c[x].view(torch.uint8), y[x].view(torch.uint8)) for c, y in zip((a, b), before) for x in PARTS)
