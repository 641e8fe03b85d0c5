"""The counting of tiles sent for and still on their way (csrc/tile_ring.h), run on the host: whichever fetch a producer
gives up at, what it waits for before it ends is exactly what was sent and may not have arrived."""
import os
import shutil
import subprocess

import pytest

import paged_kv_cache_121_gb300 as pa

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include "tile_ring.h"

// A producer of three rings: units of one or two held tiles and some streamed ones, given up at fetch `stop`.
static bool run(unsigned seed, int held_buffers, int str_slots, int stop) {
    srand(seed);
    pa::TileRing rings[3] = {pa::TileRing(held_buffers), pa::TileRing(held_buffers), pa::TileRing(str_slots)};
    std::set<int> sent[3];
    int fetches = 0;
    bool ok = true;
    auto fetch = [&](int r) {   // as the kernel does: the slot, the phase to wait for, then the copies or none
        const int n = rings[r].sent, slots = rings[r].slots;
        if (rings[r].slot() != n % slots) return false;
        if (rings[r].empty_parity() != (n < slots ? -1 : (n / slots - 1) & 1)) return false;
        ok = fetches++ != stop;
        if (ok) sent[r].insert(n);
        rings[r].count(ok);
        return true;
    };
    for (int unit = 0; ok && unit < 12; ++unit) {
        const int held = 1 + rand() % 2, streamed = rand() % 7;
        for (int i = 0; i < held && ok; ++i)
            if (!fetch(i)) return false;
        for (int i = 0; i < streamed && ok; ++i)
            if (!fetch(2)) return false;
    }
    for (int r = 0; r < 3; ++r) {
        const int slots = rings[r].slots;
        if (rings[r].sent != static_cast<int>(sent[r].size())) return false;
        // a tile that was sent and is not among those waited for has had its slot taken again, by a tile sent later
        for (int n : sent[r])
            if (n < rings[r].first_left() && !sent[r].count(n + slots)) return false;
        for (int n = rings[r].first_left(); n < rings[r].sent; ++n)
            if (!sent[r].count(n) || rings[r].full_parity(n) != ((n / slots) & 1)) return false;
    }
    return true;
}

int main() {
    for (unsigned seed = 0; seed < 200; ++seed)
        for (int held = 1; held <= 2; ++held)
            for (int slots = 2; slots <= 11; slots += 3)
                for (int stop = -1; stop < 60; ++stop)
                    if (!run(seed, held, slots, stop)) {
                        std::printf("seed %u, held %d, slots %d, given up at %d\n", seed, held, slots, stop);
                        return 1;
                    }
    return 0;
}
"""


def test_what_is_waited_for_is_what_was_sent(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    include = os.path.join(os.path.dirname(pa.__file__), "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", include, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
