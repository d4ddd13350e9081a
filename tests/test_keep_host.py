"""Caches that share memory, as hqq_cache_keep refuses them (no GPU needed)."""
import pytest

from test_cache_host import cache, seqs
from test_serving_host import H, keep       # noqa: F401 (H is a fixture)

CODES, GRIDS = 10 * 2 * 16 * 128 // 2, 10 * 2 * 16 * 2 * 4      # bytes of the buffers of cache()


def apart(base):
    """A cache's buffers from here, one behind another."""
    return dict(k_codes=base, v_codes=base + CODES, k_meta=base + 2 * CODES, v_meta=base + 2 * CODES + GRIDS)


ONE, TWO = apart(1 << 20), apart((1 << 20) + 2 * (CODES + GRIDS))


@pytest.mark.parametrize("part", ["k_codes", "v_codes", "k_meta", "v_meta"])
def test_caches_that_share_a_buffer_are_refused(H, part):       # noqa: F811
    def refused(second, first=ONE):
        for a, b in ((first, second), (second, first)):
            assert keep(H, [cache(H, **a), cache(H, **b)], seqs(H)) == H.HQQ_ERR_ARG and "overlap" in H.hqq_last_error()
    size = CODES if part.endswith("codes") else GRIDS
    refused(dict(TWO, **{part: ONE[part]}))
    refused(dict(TWO, **{part: ONE[part] + size - 16}))
    refused(dict(TWO, **{part: ONE["k_codes"] + 16}))           # of another kind
    refused(dict(TWO, **{part: ONE["v_meta"] + GRIDS - 16}))
    refused(ONE)
    # a cache in itself, and the last of many
    other = "v_codes" if part == "k_codes" else "k_codes"
    assert keep(H, [cache(H, **dict(ONE, **{part: ONE[other]}))], seqs(H)) == H.HQQ_ERR_ARG and "overlap" in H.hqq_last_error()
    many = [cache(H, **apart((i + 1) << 20)) for i in range(900)]
    bad = dict(apart(1000 << 20), **{part: (500 << 20) + 32})
    assert keep(H, many + [cache(H, **bad)], seqs(H)) == H.HQQ_ERR_ARG and "overlap" in H.hqq_last_error()
