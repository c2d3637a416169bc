"""The page-table entries that attention within a window with first tokens looks up: those of pages with a token that a new
token of the sequence sees, and no others.  The rules are the kernel's (csrc/serve/kv_walk.cuh), compiled for the host and
gone through as its copies do, step by step and half by half, with the entry after a page's loaded ahead."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include "kv_walk.cuh"
#include <cstdio>
#include <set>
using namespace arcs;
int main() {
    long calls = 0;
    for (int shift = 4; shift <= 5; ++shift)
    for (int ps = 16; ps <= 64; ps *= 2)
    for (int pos = 0; pos < 260; pos += pos < 70 ? 1 : 7)
    for (int n = 1; n <= 40; n += n < 3 ? 1 : 12)
    for (int window = 1; window < 120; window += window < 35 ? 3 : 17)
    for (int front = 1; front < 150; front += front < 50 ? 3 : 29) {
        // as load_seq has it
        const int step0 = pos + 1 > window ? (pos + 1 - window) >> shift : 0;
        const int steps = ((front - 1) >> shift) + 1, sinks = steps < step0 ? steps : step0;
        const int all = ((pos + n + (1 << shift) - 1) >> shift) - step0 + sinks;
        std::set<int> seen;  // pages that a row sees
        for (int p = pos; p < pos + n; ++p)
            for (int j = 0; j <= p; ++j)
                if (j > p - window || j < front) seen.insert(j / ps);
        for (int tile = 0; tile < n; tile += 3) {  // tiles of three tokens' rows
            const int last = pos + (tile + 3 < n ? tile + 3 : n) - 1, first = pos + tile - window + 1;
            for (int s = 0; s < all; ++s)
                for (int half = 0; half < 1 << (shift - 4); ++half) {
                    const int tok = sinks_token(s, sinks, step0, shift) + 16 * half;
                    if (shift > 4 && sinks_unseen(tok, first, last, front)) continue;
                    const int next = (tok / ps + 1) * ps;
                    ++calls;
                    if (!seen.count(tok / ps) || (sinks_ahead(tok, next, last, front) && !seen.count(next / ps))) {
                        std::printf("shift %d page %d pos %d n %d window %d front %d tile %d: token %d\n", shift, ps, pos, n, window, front, tile, tok);
                        return 1;
                    }
                }
        }
    }
    std::printf("%ld\n", calls);
    return 0;
}
"""


def test_no_entry_between_first_tokens_and_window_is_looked_up(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "walk.cpp").write_text(PROGRAM)
    inc = os.path.join(ROOT, "device_logits_sampling_gb300", "csrc", "serve")
    exe = str(tmp_path / "walk")
    subprocess.run([gxx, "-std=c++17", "-O2", "-x", "c++", "-I", inc, "-o", exe, str(tmp_path / "walk.cpp")], check=True)
    got = subprocess.run([exe], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout
    assert int(got.stdout) > 1_000_000
