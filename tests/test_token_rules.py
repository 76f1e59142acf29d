"""What the map operators work out in plain C++ (csrc/token_rules.h),
compiled by itself and asked for its answers."""
import ctypes
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

import token_reference as tok
from conftest import ROOT

SOURCE = r"""
#include <cstddef>
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
unsigned long long turn(double base, double scale, int j, int pairs)
{
    unsigned long long all[128];
    turns_of(base, scale, pairs, all);
    return all[j];
}
// asks for (device, function, bytes) three ints at a time; the device `failing` refuses. asked[i]: bytes that call i asked for, 0 none,
// -1 refused
void grants(const int *calls, int n, int failing, int *asked)
{
    Granted g;
    for (int i = 0; i < n; i++) {
        const int *c = calls + 3 * i;
        asked[i] = 0;
        if (g.have(c[0], reinterpret_cast<const void *>(static_cast<size_t>(c[1])), c[2], [&](int bytes) {
                asked[i] = bytes;
                return c[0] == failing ? 7 : 0;
            }) == 7)
            asked[i] = -1;
    }
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
    subprocess.run([cc, "-std=c++17", "-O3", "-Wall", "-Werror", "-shared", "-fPIC", "-I", csrc, str(at / "rules.cpp"), "-o",
                    str(at / "rules.so")], check=True)
    lib = ctypes.CDLL(str(at / "rules.so"))
    lib.turn.restype = ctypes.c_ulonglong
    lib.turn.argtypes = [ctypes.c_double, ctypes.c_double, ctypes.c_int, ctypes.c_int]
    return lib


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


def test_steps_of_positions_are_exact_turns(rules):
    """In 2^-64 of a turn, against sixty digits: within two of them and 2^-92 of the step, so that 2^31 positions stay within 2^-31."""
    rng = random.Random(4)
    cases = [(base, scale, j, pairs) for base in (10000.0, 500000.0, 100.0, 1.0, 2.0, 0.5) for scale in (1.0, -1.0, 9.0, 1000.0, 0.125)
             for pairs in (1, 2, 16, 37, 64, 128) for j in sorted({0, 1, pairs // 2, pairs - 1}) if j < pairs]
    cases += [(10.0 ** rng.uniform(-300, 300), rng.choice([-1, 1]) * 10.0 ** rng.uniform(-20, 20), rng.randrange(128), 128) for _ in range(200)]
    cases += [(rng.uniform(1, 1e6), rng.uniform(-1e6, 1e6), rng.randrange(p), p) for p in (3, 5, 24, 100, 127) for _ in range(40)]
    for base, scale, j, pairs in cases:
        step = tok.step_in_turns(base, scale, j, pairs)
        if abs(step) > 1 << 28:
            continue                                          # less than 2^-63 is left of a turn
        off = (Fraction(rules.turn(base, scale, j, pairs), 1 << 64) - step) % 1
        off = min(off, 1 - off)
        assert off <= Fraction(2, 1 << 64) + abs(step) / (1 << 92), (base, scale, j, pairs, float(off * 2 ** 64))


def test_steps_past_the_range(rules):
    assert rules.turn(1e-300, 1e300, 127, 128) == 0 and rules.turn(5e-324, 1.0, 1, 2) >= 0
    assert rules.turn(1e-300, -1e300, 0, 1) >= 0 and rules.turn(1e308, 1e-300, 127, 128) == 0
    assert rules.turn(1.0, 0.0, 3, 7) == 0


def test_shared_memory_is_asked_for_once_and_again_for_more(rules):
    calls = [(0, 1, 100), (0, 1, 100), (0, 1, 90), (0, 1, 120), (0, 1, 100), (0, 1, 120), (0, 2, 100), (1, 1, 100), (1, 1, 121), (2, 1, 50), (2, 1, 50)]
    flat = (ctypes.c_int * (3 * len(calls)))(*(v for c in calls for v in c))
    asked = (ctypes.c_int * len(calls))()
    rules.grants(flat, len(calls), 2, asked)
    assert list(asked) == [100, 0, 0, 120, 0, 0, 100, 100, 121, -1, -1]
