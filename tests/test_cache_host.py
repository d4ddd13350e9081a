"""The quantized key/value cache on the host: refusals of its entry points (no GPU needed), and
the index arithmetic of its kernels on tables, lengths and row offsets of any contents."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import cache_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def H():
    from calibration_free_weight_amd import hqq
    if not os.path.exists(hqq.LIB_PATH):
        from calibration_free_weight_amd import build
        build.build()
    return hqq


def cache(H, **kw):
    base = dict(k_codes=0x1000, v_codes=0x2000, k_meta=0x3000, v_meta=0x4000, n_pages=10, page_size=16,
                n_heads=2, head_dim=128, nbits=4, group_size=64, dtype=0)
    base.update(kw)
    return H.hqq_cache(**base)


def seqs(H, **kw):
    base = dict(table=0x5000, lens=0x6000, cu_tokens=None, n_seqs=2, max_pages=4, n_tokens=2)
    base.update(kw)
    return H.hqq_seqs(**base)


BAD_CACHE = [dict(head_dim=96), dict(head_dim=0), dict(nbits=3), dict(nbits=2), dict(group_size=16),
             dict(head_dim=64, group_size=128), dict(group_size=0), dict(dtype=2), dict(dtype=-1),
             dict(page_size=8), dict(page_size=48), dict(page_size=8192), dict(n_heads=0), dict(n_heads=1025),
             dict(n_pages=0), dict(n_pages=1 << 31), dict(k_codes=None), dict(v_codes=None), dict(k_meta=None),
             dict(v_meta=None), dict(k_codes=0x1008), dict(v_meta=0x4004)]
BAD_SEQS = [dict(n_seqs=-1), dict(n_seqs=4097), dict(n_tokens=-1), dict(n_tokens=(1 << 24) + 2),
            dict(max_pages=-1), dict(max_pages=1 << 27), dict(table=None), dict(lens=None), dict(lens=0x6002),
            dict(table=0x5001), dict(cu_tokens=0x7002), dict(n_tokens=3)]


def calls(H, c, s):
    """Every entry point on this cache and these sequences: (name, status)."""
    L, p = H.lib(), 0x10000
    cr, sr = (None if c is None else C.byref(c)), (None if s is None else C.byref(s))
    rows = (p, 256, 128)
    return [("write", L.hqq_cache_write(cr, sr, *rows, *rows, None)),
            ("read", L.hqq_cache_read(cr, sr, *rows, *rows, None)),
            ("attention", L.hqq_cache_attention(cr, sr, *rows, 4, 1.0, *rows, None, p, 1 << 40, None)),
            ("prefix", L.hqq_cache_attention_prefix(cr, sr, p, 4, 10, *rows, 4, 1.0, *rows, None, p, 1 << 40, None))]


@pytest.mark.parametrize("bad", BAD_CACHE + [None])
def test_bad_caches_are_refused(H, bad):
    c = None if bad is None else cache(H, **bad)
    for name, st in calls(H, c, seqs(H)):
        assert st == H.HQQ_ERR_ARG and "cache" in H.hqq_last_error(), name
    assert H.lib().hqq_cache_attention_workspace(None if c is None else C.byref(c), C.byref(seqs(H)), 4, 0) == 0


@pytest.mark.parametrize("bad", BAD_SEQS + [None])
def test_bad_sequences_are_refused(H, bad):
    s = None if bad is None else seqs(H, **bad)
    for name, st in calls(H, cache(H), s):
        assert st == H.HQQ_ERR_ARG and "seqs" in H.hqq_last_error(), name


def test_nothing_to_do_is_ok_without_buffers(H):
    for s in (seqs(H, n_seqs=0, table=None, lens=None), seqs(H, n_tokens=0, table=None, lens=None)):
        for name, st in calls(H, cache(H), s):
            assert st == H.HQQ_OK and H.hqq_last_error() == "", name


def test_bad_rows_and_plans_are_refused(H):
    L, p, big = H.lib(), 0x10000, 1 << 40
    c, s = C.byref(cache(H)), C.byref(seqs(H))
    good = (p, 256, 128)
    for bad in ((None, 256, 128), (p + 8, 256, 128), (p, 255, 128), (p, 256, 4), (p, -256, 128), (p, 256, -8)):
        assert L.hqq_cache_write(c, s, *bad, *good, None) == 1
        assert L.hqq_cache_read(c, s, *good, *bad, None) == 1
        assert L.hqq_cache_attention(c, s, *bad, 4, 1.0, *good, None, p, big, None) == 1
        assert L.hqq_cache_attention(c, s, *good, 4, 1.0, *bad, None, p, big, None) == 1

    def att(heads=4, scale=1.0, lse=None, ws=p, wb=big, pages=p, n=4, plen=10):
        return L.hqq_cache_attention_prefix(c, s, pages, n, plen, *good, heads, scale, *good, lse, ws, wb, None)
    for kw in (dict(heads=3), dict(heads=0), dict(heads=-2), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=3e38), dict(heads=(1 << 20) + 2),
               dict(lse=p + 2), dict(ws=p + 16), dict(pages=None), dict(pages=p + 1), dict(plen=-1), dict(plen=65),
               dict(n=-1), dict(n=1 << 28)):
        assert att(**kw) == H.HQQ_ERR_ARG, kw
    need = L.hqq_cache_attention_workspace(c, s, 4, 10)
    assert need > 0
    assert att(ws=None) == H.HQQ_ERR_WORKSPACE and att(wb=need - 1) == H.HQQ_ERR_WORKSPACE
    # more than a launch takes
    wide, many = C.byref(cache(H, n_heads=64, head_dim=256)), C.byref(seqs(H, n_tokens=1 << 24))
    for f in (L.hqq_cache_write, L.hqq_cache_read):
        assert f(wide, many, p, 0, 0, p, 0, 0, None) == H.HQQ_ERR_UNSUPPORTED
    assert L.hqq_cache_attention(c, many, p, 0, 0, 66, 1.0, *good, None, p, big, None) == H.HQQ_ERR_ARG
    # work counted beyond 32 bits
    s = C.byref(seqs(H, n_seqs=1, n_tokens=1 << 24, max_pages=1 << 26))
    assert L.hqq_cache_attention(c, s, *good, 64, 1.0, *good, None, p, big, None) == H.HQQ_ERR_UNSUPPORTED


DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include <random>
#include "hqq_cache.h"
using namespace hqq;
static void need(bool ok, const char *what) { if (!ok) { std::printf("FAILED: %s\n", what); std::exit(1); } }
int main()
{
    std::mt19937 r(1);
    const int edge[] = {0, 1, -1, 5, 16, 17, INT32_MAX, INT32_MIN, INT32_MAX - 1, 100, 4096, -4096};
    auto any = [&] { return r() % 2 ? edge[r() % 12] : (int)(r() % 60); };
    for (int round = 0; round < 20000; ++round) {
        const int n = 1 + r() % 9, mp = r() % 5, shift = 4 + r() % 9, pages = 1 + r() % 6;
        // exact-sized: the sanitizer sees any index outside
        std::vector<int32_t> table(n * mp), lens(n), cu(n + 1);
        for (auto &x : table) x = any();
        for (auto &x : lens) x = any();
        for (auto &x : cu) x = any();
        const bool sorted = r() % 2, uniform = r() % 4 == 0;
        if (sorted) { int at = 0; for (auto &x : cu) { x = at; at += r() % 6; } }
        const int n_tokens = uniform ? n * (int)(r() % 5) : (int)(r() % 50);
        SeqView s{table.data(), lens.data(), uniform ? nullptr : cu.data(), n, mp, n_tokens, -1, shift, pages};
        for (int b = 0; b < n; ++b) {
            const Rows x = rows_of(s, b);
            need(0 <= x.begin && x.begin <= x.end && x.end <= n_tokens, "rows in the tensors");
            const int len = len_of(s, b);
            need(0 <= len && len <= mp << shift, "length in the table");
            const int pos[] = {any(), len - 1, len, mp << shift, (mp << shift) - 1, -1, INT32_MIN, INT32_MAX};
            for (int p : pos) { const int g = page_of(s, b, p); need(g >= -1 && g < pages, "page in the cache"); }
            const int far = len - (x.end - x.begin);    // the smallest position a row can have
            need(far >= -n_tokens, "positions in 32 bits");
        }
        // offsets that do not fall leave no more rows than there are; those that do are found
        int64_t all = 0;
        bool falls = false;
        for (int b = 0; b < n; ++b) { all += rows_of(s, b).end - rows_of(s, b).begin; falls = falls || falls_at(s, b); }
        need(falls || all <= n_tokens, "rows counted once");
        need(!falls || !(sorted || uniform), "offsets that rise");
        for (int i = 0; i < n_tokens + 2; ++i) {
            const int b = seq_at(s, i);
            need(b >= 0 && b < n, "sequence of a row");
            if ((sorted || uniform) && i < n_tokens) {
                int want = -1;
                for (int k = 0; k < n; ++k) if (rows_of(s, k).begin <= i && i < rows_of(s, k).end) want = k;
                if (want >= 0) need(b == want, "the row's sequence");
            }
        }
    }
    for (int round = 0; round < 200000; ++round) {
        // runs: every unit is in one, and none is empty
        const int U = 1 + r() % (round % 3 ? 300 : 2000000000), W = runs_of(1 + r() % 2000, U);
        const int u = r() % U, w = run_of(u, W, U), any_run = r() % W;
        need(w >= 0 && w < W && first_unit(w, W, U) <= u && u < first_unit(w + 1, W, U), "a unit's run");
        need(first_unit(0, W, U) == 0 && first_unit(W, W, U) == U, "all units");
        need(first_unit(any_run, W, U) < first_unit(any_run + 1, W, U), "no empty run");
        const int len = r() % 2 ? (int)(r() % 1000) : INT32_MAX - (int)(r() % 1000), unit = 128 << r() % 4;
        const int n = units_along(len, unit);
        need(n >= 1 && (int64_t)n * unit >= len && (n == 1 || (int64_t)(n - 1) * unit < len), "units of a length");
    }
    for (int dim : {64, 128, 256}) for (int nbits : {4, 8}) {
        const int page = 64, bytes = page * dim * nbits / 8;
        std::vector<char> k(bytes), v(bytes);
        for (int t = 0; t < page; ++t) {
            for (int a = 0; a < 4; ++a) for (int m = 0; m < dim / 32; ++m)
                for (int x = 0; x < nbits; ++x) { char &c = k[k_unit_at(t, a, m, dim, nbits) + x]; need(!c, "key bytes apart"); c = 1; }
            for (int q = 0; q < 16; ++q)
                for (int x = 0; x < dim * nbits / 128; ++x) { char &c = v[v_row_at(t, q, dim, nbits) + x]; need(!c, "value bytes apart"); c = 1; }
        }
        for (char c : k) need(c, "all key bytes");
        for (char c : v) need(c, "all value bytes");
    }
    std::puts("ok");
}
"""


def test_indexes_stay_in_their_buffers(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    inc = os.path.join(ROOT, "calibration_free_weight_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-g", "-D_GLIBCXX_ASSERTIONS", "-fsanitize=address,undefined",
                           "-fno-sanitize-recover=all", "-I", inc, "-o", str(exe), str(src)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr[-2000:]


@pytest.mark.parametrize("nbits,dim,g", [(4, 128, 64), (8, 64, 32), (4, 256, 128), (4, 64, 32)])
def test_reference_layout_is_a_bijection(nbits, dim, g):
    q = torch.randint(0, 2 ** nbits, (2, 3, 16, dim))
    for w in "kv":
        buf = R.codes_to_pages(q, nbits, g, w)
        assert torch.equal(R.pages_to_codes(buf, 16, dim, nbits, g, w), q)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nbits", [4, 8])
def test_reference_grid_bound(dtype, nbits):
    """Half a step, whatever the values; the step is the smallest that reaches the maximum."""
    gen = torch.Generator().manual_seed(nbits)
    x = torch.cat([torch.randn(50, 128, generator=gen) * 10.0 ** e for e in (-6, -3, 0, 3)]).to(dtype)
    q, step, base = R.grid(x, nbits, 64)
    assert q.min() == 0 and q.max() <= 2 ** nbits - 1
    err = (R.value(q, step, base) - x.double()).abs().reshape(-1, 2, 64)
    assert (err <= step[..., None] / 2).all()
    smaller = (step.to(dtype).view(torch.int16) - 1).view(dtype).double()
    span = x.double().reshape(-1, 2, 64).amax(-1) - base
    assert (smaller * (2 ** nbits - 1) < span).all()


def test_packed_structs_are_the_structs(H):
    """The binding's packed bytes are what the C structures hold."""
    a = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11)
    assert H._pack_cache(*a) == bytes(H.hqq_cache(*a))
    b = (1, 2, 3, 4, 5, 6)
    assert H._pack_seqs(*b) == bytes(H.hqq_seqs(*b))
