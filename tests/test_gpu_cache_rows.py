"""Calls of many rows write and read back several heads of a token at a time: every code, grid and row
against the definition, with numbers of heads and tokens that leave the last ones short."""
import pytest
import torch

import cache_ref as R
from test_gpu_cache import cumulated, expect_written, i32, layout, poison, same_bits

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16
# dtype, nbits, dim, group, page, heads, lens, new (None: as long as the sequence); 2^22 numbers and
# more are read so, 2^23 and more written too
ROWS = [
    (F, 4, 128, 64, 64, 7, [6000, 3501, 1], None),
    (B, 8, 128, 128, 16, 5, [9000, 4121], [9000, 4119]),
    (B, 4, 64, 32, 32, 5, [20000, 7003], None),
    (F, 8, 64, 64, 128, 9, [15001], [14999]),
    (B, 4, 256, 128, 64, 6, [5001, 500], None),
    (F, 8, 256, 32, 16, 7, [4700, 11], None),
    (F, 4, 128, 32, 256, 34, [1000] * 2 + [30], None),
    (B, 8, 64, 64, 64, 3, [40000, 3911], [39999, 3911]),
    # read so and not written so
    (F, 4, 128, 128, 64, 7, [4000, 1003], None),
    (B, 8, 256, 64, 32, 5, [3333], None),
]


@pytest.mark.parametrize("dtype,nbits,dim,group,page,heads,lens,new", ROWS)
def test_many_rows(H, dtype, nbits, dim, group, page, heads, lens, new):
    gen = torch.Generator().manual_seed(dim + nbits + heads)
    new = lens if new is None else new
    table, n_pages, _ = layout(lens, page, gen)
    cu = cumulated(new)
    n = cu[-1]
    assert n * heads * dim >= 1 << 22
    cache = poison(H.alloc_cache(n_pages, page, heads, dim, nbits, group, dtype))
    # parts of a wider tensor, and three rows of no sequence
    wide = (torch.randn(n + 3, 2 * heads + 2, dim, generator=gen) * (1 + torch.rand(2 * heads + 2, 1, generator=gen))).to(dtype).cuda()
    k, v = wide[:, :heads], wide[:, heads + 1:2 * heads + 1]
    want = expect_written(cache, k, v, R.where(table, lens, cu, n, page, n_pages) + [None] * 3)
    H.hqq_cache_write(cache, i32(table), i32(lens), k, v, cu_tokens=i32(cu))
    for name, x in want.items():
        assert same_bits(cache[name], x), name
    back = torch.full((n + 3, 2, heads + 1, dim), 9.0, dtype=dtype, device="cuda")
    H.hqq_cache_read(cache, i32(table), i32(lens), back[:, 0, :heads], back[:, 1, :heads], cu_tokens=i32(cu))
    for j, x in enumerate((k, v)):
        assert same_bits(back[:n, j, :heads], R.value(*R.grid(x[:n].cpu(), nbits, group)).to(dtype))
    assert (back[n:] == 9).all() and (back[:, :, heads] == 9).all()


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    return hqq
