"""Caches that share memory, as hqq_cache_keep refuses them (no GPU needed)."""
import os
import re
import subprocess

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


def test_moved_codes_stay_in_registers(tmp_path):
    """No instance of the kernel takes LDS or scratch memory."""
    from calibration_free_weight_amd import build as hb
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    out = tmp_path / "keep.s"
    subprocess.check_call([hipcc, *hb.HIPCC_FLAGS, "-w", "--offload-device-only", "-S", "-I", os.path.join(hb.ROOT, "include"),
                           "-I", os.path.join(hb.PKG, "csrc"), "-o", str(out), os.path.join(hb.PKG, "csrc", "hqq_keep.hip")])
    sizes = re.findall(r"\.(?:group|private)_segment_fixed_size:\s+(\d+)", out.read_text())
    assert len(sizes) == 8 and set(sizes) == {"0"}
