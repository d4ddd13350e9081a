"""Which numbers a rotary call turns and copies, counted on the host."""
import os
import subprocess

import pytest

from test_serving_host import H, P, rotary      # noqa: F401 (H is a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "hqq_rotary.h"
using namespace hqq;
static void need(bool ok, const char *what) { if (!ok) { std::printf("FAILED: %s\n", what); std::exit(1); } }

template <bool NEIGHBOURS>
static void count(int dim, int rotary, const int (&heads)[2], const bool (&in_place)[2])
{
    const int pairs = rotary / 2;
    RotaryHeads x[2];
    std::vector<char> turned[2], copied[2];
    for (int i = 0; i < 2; ++i) {
        x[i] = rotary_heads(heads[i], pairs, in_place[i] ? 0 : dim - rotary);
        turned[i].resize(heads[i] * dim);
        copied[i].resize(heads[i] * dim);
    }
    const int before = heads[0] * x[0].per_head, units = before + heads[1] * x[1].per_head;
    for (int j = 0; j < units; ++j) {
        const RotaryUnit u = rotary_unit<NEIGHBOURS>(x, pairs, before, j);
        need(u.tensor == 0 || u.tensor == 1, "a tensor of the call");
        need(u.head >= 0 && u.head < heads[u.tensor], "a head of the tensor");
        const int n = u.wide ? 8 : 1;
        auto mark = [&](std::vector<char> &v, int d) {
            need(d >= 0 && d < dim, "a dimension of the head");
            char &c = v[u.head * dim + d];
            need(!c, "no dimension twice");
            c = 1;
        };
        if (u.pair < 0) {
            need(u.d0 == u.d1, "one place");
            for (int e = 0; e < n; ++e) mark(copied[u.tensor], u.d0 + e);
            continue;
        }
        need(u.pair + n <= pairs, "pairs that there are");
        for (int e = 0; e < n; ++e) { mark(turned[u.tensor], u.d0 + e); mark(turned[u.tensor], u.d1 + e); }
        if (NEIGHBOURS) need(u.d0 == 2 * u.pair && u.d1 == u.d0 + n, "neighbours");
        else need(u.d0 == u.pair && u.d1 == u.pair + pairs, "halves");
    }
    for (int i = 0; i < 2; ++i)
        for (int h = 0; h < heads[i]; ++h)
            for (int d = 0; d < dim; ++d) {
                need(turned[i][h * dim + d] == (d < rotary), "the first dimensions are turned");
                need(copied[i][h * dim + d] == (d >= rotary && !in_place[i]), "the others are copied, in place left alone");
            }
}

int main()
{
    const int sizes[][2] = {{128, 128}, {128, 64}, {64, 32}, {128, 2}, {64, 62}, {96, 48}, {80, 26}, {65, 64}, {31, 30}, {256, 254}, {1024, 512}, {2, 2}, {17, 16}};
    const int heads[][2] = {{1, 0}, {4, 1}, {3, 3}, {1, 7}};
    const bool places[][2] = {{false, false}, {true, false}, {false, true}, {true, true}};
    for (auto &s : sizes) for (auto &h : heads) for (auto &p : places) {
        count<false>(s[0], s[1], h, p);
        count<true>(s[0], s[1], h, p);
    }
    // rows that share a number, against all pairs of them
    for (int n = 1; n <= 7; ++n) for (int h = 1; h <= 6; ++h) for (int w : {1, 2, 3, 5})
        for (int ts = 0; ts < 24; ++ts) for (int hs = 0; hs < 24; ++hs) {
            bool meet = false;
            for (int i = 0; i < n * h; ++i) for (int j = 0; j < i; ++j)
                meet = meet || std::abs((i / h - j / h) * ts + (i % h - j % h) * hs) < w;
            need(rows_meet(n, h, ts, hs, w) == meet, "rows that meet");
        }
    const int64_t far = int64_t(1) << 36;
    need(!rows_meet(1 << 24, 4096, far, 1024, 1024) && !rows_meet(1 << 24, 4096, 1024, far, 1024), "long strides");
    need(rows_meet(1 << 24, 4096, far, far, 1024) && rows_meet(1 << 24, 4096, 1024, 1024 << 10, 1024), "long strides that meet");
    std::puts("ok");
}
"""


def test_what_a_call_turns_and_copies(tmp_path):
    """Each pair once, and the dimensions behind them once, or in place not at all: of each tensor for
    itself, whatever the call does with the other one."""
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    inc = os.path.join(ROOT, "calibration_free_weight_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-g", "-D_GLIBCXX_ASSERTIONS", "-fsanitize=address,undefined",
                           "-fno-sanitize-recover=all", "-I", inc, "-o", str(exe), str(src)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr[-2000:]


OVER = dict(out=P)          # in place, of 5 tokens and 4 heads of 128, 64 of them turned


@pytest.mark.parametrize("rows", [
    [dict(OVER, in_token_stride=0, out_token_stride=0)], [dict(OVER, in_head_stride=0, out_head_stride=0)],
    [dict(OVER, in_head_stride=63, out_head_stride=63)], [dict(OVER, in_token_stride=63, out_token_stride=63)],
    [dict(OVER, in_token_stride=192, out_token_stride=192)],                # a token's second head and the next one's first
    [dict(out_token_stride=0)], [dict(out_head_stride=0)], [dict(out_head_stride=127)], [dict(out_token_stride=511)],
    [{}, dict(in_=5 * P, out=4 * P, out_head_stride=0)], [dict(OVER), dict(OVER)], [{}, {}]], ids=str)
def test_outputs_that_overlap_are_refused(H, rows):     # noqa: F811
    assert rotary(H, rows=rows) == H.HQQ_ERR_ARG and "overlap" in H.hqq_last_error()


def test_more_rows_than_a_launch_takes(H):      # noqa: F811
    """Heads of 64 that are turned in place have four units: 64 of them 256, 33 of them 132."""
    rows = lambda heads: [dict(out=P, in_token_stride=1 << 20, out_token_stride=1 << 20, n_heads=heads)]
    for heads, n in ((64, 1 << 24), (33, 1 << 24), (65, 1 << 23), (128, 1 << 23), (4096, 1 << 18)):
        assert rotary(H, rows=rows(heads), n_tokens=n) == H.HQQ_ERR_UNSUPPORTED, heads
