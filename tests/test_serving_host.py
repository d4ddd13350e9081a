"""Rotary positions, prompt attention, tree attention and keeping accepted tokens on the host: what
their entry points refuse (no GPU needed), and the frequencies."""
import ctypes as C
import math
import os

import pytest
import torch

from test_cache_host import BAD_CACHE, BAD_SEQS, cache, seqs

P = 0x10000


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    if not os.path.exists(hqq.LIB_PATH):
        from calibration_free_weight_amd import build
        build.build()
    return hqq


# ---- rotary ----------------------------------------------------------------------------------
def rotary(H, rows=None, **kw):
    a = dict(freqs=P, rotary_dim=64, interleaved=0, scale=1.0, positions=P, n_tokens=5, head_dim=128, dtype=0, n_rows=None)
    a.update(kw)
    rows = [{}] if rows is None else rows
    arr = (H.hqq_rotary_rows * max(len(rows), 1))()
    for i, r in enumerate(rows):
        x = dict(in_=P, in_token_stride=512, in_head_stride=128, out=2 * P, out_token_stride=512, out_head_stride=128, n_heads=4)
        x.update(r)
        arr[i] = H.hqq_rotary_rows(**x)
    return H.lib().hqq_rotary(a["freqs"], a["rotary_dim"], a["interleaved"], a["scale"], a["positions"], a["n_tokens"],
                              a["head_dim"], a["dtype"], arr, len(rows) if a["n_rows"] is None else a["n_rows"], None)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=130), dict(rotary_dim=-2), dict(head_dim=1026, rotary_dim=64),
    dict(head_dim=62), dict(dtype=2), dict(dtype=-1), dict(interleaved=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(n_tokens=-1), dict(n_tokens=(1 << 24) + 1), dict(n_rows=-1), dict(n_rows=3),
    dict(freqs=None), dict(freqs=P + 4), dict(positions=None), dict(positions=P + 2),
    dict(rows=[dict(in_=None)]), dict(rows=[dict(out=None)]), dict(rows=[dict(in_=P + 1)]), dict(rows=[dict(out=P + 1)]),
    dict(rows=[dict(n_heads=-1)]), dict(rows=[dict(n_heads=4097)]), dict(rows=[dict(in_token_stride=-8)]),
    dict(rows=[dict(out_head_stride=(1 << 36) + 8)]), dict(rows=[dict(out=P, out_token_stride=520)]),
    dict(rows=[{}, dict(out=P, out_head_stride=136)])], ids=str)
def test_rotary_refuses(H, kw):
    assert rotary(H, **kw) == H.HQQ_ERR_ARG and H.hqq_last_error()


def test_rotary_with_nothing_to_do(H):
    null = dict(in_=None, out=None)
    assert rotary(H, rows=[]) == 0 and rotary(H, rows=[], freqs=None, positions=None) == 0
    assert rotary(H, rows=[null], n_tokens=0, freqs=None, positions=None) == 0
    assert rotary(H, rows=[dict(null, n_heads=0)] * 2) == 0 and H.hqq_last_error() == ""


def freqs(H, *a):
    out = (C.c_uint64 * 600)()
    return H.lib().hqq_rotary_frequencies(*a, out), list(out)


@pytest.mark.parametrize("bad", [(0, 1e4, 1.0, 0, 1.0, 4.0), (63, 1e4, 1.0, 0, 1.0, 4.0), (1026, 1e4, 1.0, 0, 1.0, 4.0),
                                 (64, 0.5, 1.0, 0, 1.0, 4.0), (64, math.nan, 1.0, 0, 1.0, 4.0),
                                 (64, math.inf, 1.0, 0, 1.0, 4.0), (64, 1e4, 0.5, 0, 1.0, 4.0), (64, 1e4, math.nan, 0, 1.0, 4.0),
                                 (64, 1e4, 2.0, -1, 1.0, 4.0), (64, 1e4, 2.0, 100, 4.0, 4.0), (64, 1e4, 2.0, 100, -1.0, 4.0),
                                 (64, 1e4, 2.0, 100, 1.0, math.inf), (64, 1e4, 2.0, 100, math.nan, 4.0)])
def test_frequencies_refused(H, bad):
    assert freqs(H, *bad)[0] == H.HQQ_ERR_ARG and H.hqq_last_error()


def test_frequencies_without_an_array(H):
    assert H.lib().hqq_rotary_frequencies(64, 1e4, 1.0, 0, 1.0, 4.0, None) == H.HQQ_ERR_ARG


@pytest.mark.parametrize("dim,theta,factor,length,low,high", [
    (128, 1e4, 1.0, 0, 1.0, 4.0), (2, 1.0, 1.0, 0, 1.0, 4.0), (64, 5e5, 8.0, 8192, 1.0, 4.0),
    (96, 1e6, 3.5, 0, 7.0, 3.0), (1024, 1e4, 40.0, 4096, 1.0, 32.0), (128, 1e4, 4.0, 10 ** 12, 1.0, 4.0)])
def test_frequencies(H, dim, theta, factor, length, low, high):
    st, got = freqs(H, dim, theta, factor, length, low, high)
    assert st == 0 and got[dim // 2:] == [0] * (600 - dim // 2)
    for i in range(dim // 2):
        f = theta ** (-2 * i / dim)
        s = min(1.0, max(0.0, (length * f / (2 * math.pi) - low) / (high - low))) if length else 0.0
        want = f * ((1 - s) / factor + s) / (2 * math.pi) * 2.0 ** 64
        # double's 53 bits in theta's power, whose exponent is up to 21, and in what follows
        assert abs(got[i] - want) <= 2.0 ** -46 * want * factor + 1, i


def test_frequencies_of_the_binding(H):
    t = H.rotary_frequencies(64, theta=1e4, device="cpu")
    assert t.dtype == torch.int64 and t.tolist() == [x - (1 << 64) if x >> 63 else x for x in freqs(H, 64, 1e4, 1.0, 0, 1.0, 4.0)[1][:32]]
    for bad in (0, 7, -2):
        with pytest.raises(H.HQQError):
            H.rotary_frequencies(bad, device="cpu")


# ---- prompts ---------------------------------------------------------------------------------
def prompt(H, **kw):
    a = dict(q=(P, 512, 128), k=(P, 256, 128), v=(P, 256, 128), n=6, hq=4, hk=2, dim=128, dtype=0, cu=None, seqs=2,
             scale=1.0, out=(2 * P, 512, 128), lse=None)
    a.update(kw)
    return H.lib().hqq_prompt_attention(*a["q"], *a["k"], *a["v"], a["n"], a["hq"], a["hk"], a["dim"], a["dtype"], a["cu"],
                                        a["seqs"], a["scale"], *a["out"], a["lse"], None)


@pytest.mark.parametrize("kw", [
    dict(hq=3), dict(hq=0), dict(hq=-2), dict(hk=0), dict(hk=1025, hq=1025), dict(hq=(1 << 20) + 2), dict(dim=96), dict(dim=0), dict(dim=512),
    dict(dtype=2), dict(dtype=-1), dict(seqs=-1), dict(seqs=4097), dict(n=-1), dict(n=(1 << 24) + 2), dict(n=7),
    dict(cu=P + 2), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(lse=P + 2),
    dict(n=1 << 24, hq=128, hk=2), dict(k=(P, (1 << 22) + 8, 128)), dict(v=(P, (1 << 22) + 8, 128)),
    *[{x: y} for x in ("q", "k", "v", "out") for y in ((None, 512, 128), (P + 8, 512, 128), (P, 511, 128), (P, 512, 4), (P, -512, 128),
                                                       (P, 512, 1 << 37))]], ids=str)
def test_prompt_refuses(H, kw):
    assert prompt(H, **kw) == H.HQQ_ERR_ARG and H.hqq_last_error()


def test_prompt_with_nothing_to_do(H):
    null = dict(q=(None, 0, 0), k=(None, 0, 0), v=(None, 0, 0), out=(None, 0, 0))
    assert prompt(H, n=0, **null) == 0 and prompt(H, seqs=0, **null) == 0 and H.hqq_last_error() == ""


# ---- trees -----------------------------------------------------------------------------------
def tree(H, c, s, t=P, words=1, heads=4, scale=1.0, ws=P, wb=1 << 40, q=(P, 512, 128), out=(2 * P, 512, 128), lse=None):
    cr, sr = (None if c is None else C.byref(c)), (None if s is None else C.byref(s))
    return H.lib().hqq_cache_attention_tree(cr, sr, t, words, *q, heads, scale, *out, lse, ws, wb, None)


@pytest.mark.parametrize("kw", [dict(t=None), dict(t=P + 4), dict(words=0), dict(words=-1), dict(words=257), dict(heads=3),
                                dict(heads=0), dict(scale=float("nan")), dict(q=(None, 512, 128)), dict(q=(P + 8, 512, 128)),
                                dict(out=(P, 511, 128)), dict(lse=P + 2), dict(ws=P + 16)], ids=str)
def test_tree_refuses(H, kw):
    assert tree(H, cache(H), seqs(H, max_pages=64), **kw) == H.HQQ_ERR_ARG and H.hqq_last_error()


def test_tree_workspace_and_nothing_to_do(H):
    s = seqs(H, max_pages=64)
    need = H.lib().hqq_cache_attention_workspace(C.byref(cache(H)), C.byref(s), 4, 0)
    assert need > 0
    assert tree(H, cache(H), s, ws=None) == H.HQQ_ERR_WORKSPACE and tree(H, cache(H), s, wb=need - 1) == H.HQQ_ERR_WORKSPACE
    assert tree(H, cache(H), seqs(H, n_tokens=0), t=None) == 0


@pytest.mark.parametrize("bad", BAD_CACHE + [None])
def test_bad_caches_are_refused(H, bad):
    c = None if bad is None else cache(H, **bad)
    assert tree(H, c, seqs(H)) == H.HQQ_ERR_ARG and "cache" in H.hqq_last_error()
    assert keep(H, [c], seqs(H)) == H.HQQ_ERR_ARG and "cache" in H.hqq_last_error()
    if c is not None:
        assert keep(H, [cache(H), c], seqs(H)) == H.HQQ_ERR_ARG and "cache" in H.hqq_last_error()


@pytest.mark.parametrize("bad", BAD_SEQS + [None])
def test_bad_sequences_are_refused(H, bad):
    s = None if bad is None else seqs(H, **bad)
    assert tree(H, cache(H), s) == H.HQQ_ERR_ARG and "seqs" in H.hqq_last_error()
    assert keep(H, [cache(H)], s) == H.HQQ_ERR_ARG and "seqs" in H.hqq_last_error()


# ---- accepted tokens -------------------------------------------------------------------------
def keep(H, caches, s, kept=P, most=3, out=2 * P, n=None):
    arr = None
    if caches and caches[0] is not None:
        arr = (H.hqq_cache * len(caches))(*caches)
    return H.lib().hqq_cache_keep(arr, len(caches) if n is None else n, None if s is None else C.byref(s), kept, most, out, None)


def test_keep_refuses(H):
    one = [cache(H)]
    for kw in (dict(kept=None), dict(kept=P + 2), dict(most=-1), dict(most=(1 << 24) + 1), dict(out=P + 2), dict(out=0x6000), dict(out=0x6004), dict(out=0x5ffc),
               dict(n=0), dict(n=-1), dict(n=1025)):
        assert keep(H, one, seqs(H), **kw) == H.HQQ_ERR_ARG and H.hqq_last_error(), kw
    other = dict(k_codes=0x8000)
    for differs in (dict(n_pages=11), dict(page_size=32), dict(n_heads=3), dict(head_dim=64), dict(nbits=8), dict(group_size=32), dict(dtype=1)):
        assert keep(H, [cache(H), cache(H, **other, **differs)], seqs(H)) == H.HQQ_ERR_ARG and "same" in H.hqq_last_error()
    assert keep(H, [cache(H, **other), cache(H), cache(H, **other)], seqs(H)) == H.HQQ_ERR_ARG and "differ" in H.hqq_last_error()
    assert keep(H, one, seqs(H, n_tokens=0, lens=None)) == H.HQQ_ERR_ARG       # lens_out comes of them
    assert keep(H, one, seqs(H, n_seqs=0, table=None, lens=None), kept=None) == 0


def test_packed_rows_are_the_struct(H):
    a = (1, 2, 3, 4, 5, 6, 7)
    assert H._pack_rotary(*a) == bytes(H.hqq_rotary_rows(*a))
