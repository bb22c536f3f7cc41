"""The whole-number rules of the attention kernels and the pool's, run on the host with every overflow and division by zero trapped."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_routing_moe_gb300", "csrc")
PRELUDE = """
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "ranges.h"
using namespace moe;
#define CHECK(x) do { if (!(x)) { std::printf("%s fails\\n", #x); std::exit(1); } } while (0)
"""


def _run(tmp_path, body):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PRELUDE + "int main() {" + body + "return 0; }\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout or "trapped (%d)" % r.returncode


def test_the_traps_work(tmp_path):
    with pytest.raises(AssertionError, match="trapped"):
        _run(tmp_path, "volatile int x = INT_MIN; x = x - 5;")


def test_pages_of_any_length(tmp_path):
    _run(tmp_path, """
    for (int len : {0, 1, 63, 64, 65, 1 << 20, INT_MAX - 64, INT_MAX - 63, INT_MAX - 62, INT_MAX}) CHECK(pages_of(len) == (len + 63ll) / 64);
    """)


def test_rows_of_any_starts(tmp_path):
    """Starts, lengths and tables of any numbers, the ends of their type among them."""
    _run(tmp_path, """
    const int v[] = {INT_MIN, INT_MIN + 1, -100, -1, 0, 1, 5, 63, 64, 100, 101, INT_MAX - 64, INT_MAX - 1, INT_MAX};
    for (int q0 : v) for (int q1 : v) for (int len : v) for (int T : {0, 1, 100, INT_MAX}) for (int mp : {0, 1, 2, INT_MAX}) {
        const bool want = q0 >= 0 && q1 >= q0 && q1 <= T && len >= 0 && (long long)len <= 64ll * mp;
        CHECK(rows_fit(q0, q1, len, T, mp) == want);
    }
    """)


def test_windows_of_any_size(tmp_path):
    """Rows before their sequence and windows near the largest number among them: what the kernels compute, place - window + 1,
    neither overflows nor hides what the caller's window shows."""
    _run(tmp_path, """
    for (int mp : {0, 1, 2, 40, (1 << 25) - 1, 1 << 25, INT_MAX}) for (int T : {1, 6, 1000, 1 << 20})
    for (int w : {0, 1, 2, 63, 64, 65, 127, 128, 129, 2560, INT_MAX - 250, INT_MAX - 63, INT_MAX - 1, INT_MAX}) {
        const int k = kernel_window(w, T, mp);
        const long long tokens = 64ll * mp;
        if (k < 0) { CHECK(tokens > w && w + (long long)T > INT_MAX); continue; }
        for (long long p : {-(long long)T, -1ll, 0ll, 1ll, 62ll, 63ll, 64ll, 200ll, tokens - 1}) {
            if (p >= tokens || p > INT_MAX) continue;
            const long long first = w > 0 && p - w + 1 > 0 ? p - w + 1 : 0;
            const int got = k > 0 && (int)p - k + 1 > 0 ? (int)p - k + 1 : 0;
            CHECK(got == first);
        }
    }
    """)


def test_ctas_of_a_tile(tmp_path):
    """Every CTA that holds a piece of a tile finds the same ones, with more tiles than CTAs (no CTA for each) among the cases."""
    _run(tmp_path, """
    unsigned x = 1;
    for (int round = 0; round < 3000; ++round) {
        const int grid = 152, tiles = 1 + (x = x * 1664525u + 1013904223u) / 65536 % 400, most = 1 + (x = x * 1664525u + 1013904223u) / 65536 % 300;
        long long total = 0, begin[400], units[400];
        for (int i = 0; i < tiles; ++i) { begin[i] = total; total += units[i] = 1 + (x = x * 1664525u + 1013904223u) / 65536 % most; }
        long long share = (total + grid - 1) / grid;
        if (share < 8) share = 8;
        for (int i = 0; i < tiles; ++i) {
            const int b0 = begin[i] / share, b1 = (begin[i] + units[i] - 1) / share;
            for (int b = b0; b <= b1; ++b) {
                const CtaRange r = tile_ctas(false, b, grid / tiles, share, share * b, begin[i], units[i]);
                CHECK(r.first == b0 && r.last == b1);
            }
        }
        const int per_item = grid / tiles;
        if (per_item < 16) continue;
        share = (most + per_item - 1) / per_item;
        if (share < 8) share = 8;
        for (int i = 0; i < tiles; ++i)
            for (int j = 0; j * share < most; ++j) {
                const CtaRange r = tile_ctas(true, i * per_item + j, per_item, share, (long long)i * most + j * share, (long long)i * most, most);
                CHECK(r.first == i * per_item && r.last == i * per_item + (most - 1) / share && r.last < (i + 1) * per_item);
            }
    }
    // far into a long sequence of units
    const CtaRange r = tile_ctas(false, 100, 0, 3000000000ll / 152, 3000000000ll / 152 * 100, 3000000000ll / 152 * 99 + 5, 40000000);
    CHECK(r.first == 99 && r.last == 101);
    """)
