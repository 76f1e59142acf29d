"""What the operators around attention work out on the host (csrc/token_rules.h),
compiled by itself and asked for its answers."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include "token_rules.h"
using namespace rz::rules;
extern "C" {

void runs(int heads, int lanes, long long tokens, int warps, int *out)
{
    const Runs r = head_runs(heads, lanes, tokens, warps);
    out[0] = r.chunks;
    out[1] = r.chunk;
}
// token counts below `most` whose runs of heads do not all have some, or do not add up
int bad_runs(int heads, int lanes, int most, int warps)
{
    int bad = 0;
    for (int t = 1; t < most; t++) {
        const Runs r = head_runs(heads, lanes, t, warps);
        bad += r.chunk < 1 || r.chunks < 1 || (r.chunks - 1) * r.chunk >= heads || r.chunks * r.chunk < heads;
    }
    return bad;
}
// looks of a wait that began at times[0] until it gives up, at most n - 1; 0: it does not
int looks(const unsigned long long *times, int n, unsigned long long limit)
{
    WaitClock clock(times[0]);
    for (int i = 1; i < n; i++)
        if (clock.over(times[i], limit)) return i;
    return 0;
}

}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("rules")
    (at / "rules.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "bilinear_image_resize_gb300", "csrc")
    subprocess.run([cc, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", csrc, str(at / "rules.cpp"), "-o",
                    str(at / "rules.so")], check=True)
    return ctypes.CDLL(str(at / "rules.so"))


@pytest.mark.parametrize("lanes", [1, 2, 4, 8, 16, 32])
def test_every_run_of_heads_has_some(rules, lanes):
    """Whatever the heads and the tokens: two walks of the gradient rely on it."""
    for heads in (*range(1, 130), 255, 256, 1000, 4095, 65536):
        assert rules.bad_runs(heads, lanes, 2500, 8) == 0, heads


# (heads of queries, of keys, lanes of a head, tokens): runs that once left the last one empty
ONCE_EMPTY = [(12, 12, 32, 256), (2, 2, 32, 900), (32, 8, 16, 289), (16, 16, 32, 196), (16, 16, 16, 256), (20, 20, 16, 288)]


@pytest.mark.parametrize("q, k, lanes, tokens", ONCE_EMPTY)
def test_runs_are_copied_as_they_are_used(rules, q, k, lanes, tokens):
    """The gradient's two walks, step by step: what is copied into a place is what is read from it."""
    out = (ctypes.c_int * 2)()
    rules.runs(q + k, lanes, ctypes.c_longlong(tokens), 8, out)
    chunks, chunk = out
    heads, at_once, items = q + k, 32 // lanes, tokens * chunks
    step = min(-(-items // 8), 304) * 8
    assert chunks > 1 and items > 0
    for warp in range(step):
        copied, used = [], []
        for item in range(warp, items, step):
            h0 = item % chunks * chunk
            h1 = min(heads, h0 + chunk)
            at = h0
            while True:
                to = min(h1, q) if at < q else h1
                copied.append((item, at))
                at = min(at + at_once, to)
                if at >= h1:
                    break
            for p0, p1 in ((h0, min(h1, q)), (max(h0, q), h1)):
                used += [(item, f) for f in range(p0, p1, at_once)]
        assert copied == used


def looks(rules, times, limit=10 ** 9):
    return rules.looks((ctypes.c_ulonglong * len(times))(*times), len(times), ctypes.c_ulonglong(limit))


def test_a_wait_gives_up_after_a_second_of_its_own(rules):
    ms = 10 ** 6
    times = [5 + i * ms // 2 for i in range(2100)]
    assert looks(rules, times) == 2001                        # looks every half millisecond
    # another program's slice of 1.5 s, and one of an hour, between two looks: neither uses the second up
    away = [5, 5 + ms, 5 + ms + 1500 * ms, 5 + 3_600_000 * ms]
    away += [away[-1] + i * ms // 2 for i in range(1, 500)]
    assert looks(rules, away) == 0
    # but a wait whose looks are always late ends too, after a hundred of them
    assert looks(rules, [i * 3000 * ms for i in range(200)]) == 101
    # a clock that passes 2^64: look i is at 5 ns + (i - 1) ms, which passes 50 ms with the 51st
    assert looks(rules, [(1 << 64) - 5] + [i * ms for i in range(100)], 50 * ms) == 51
