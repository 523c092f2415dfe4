"""The schedule of the fp8 products on the host: its units are cut without a gap or an overlap, the parts of a
tile are counted as the joining worker counts them, and an item is the same whether a warp steps to it or
looks it up after it gave up a wait (all warps of a CTA have to go through the same barriers)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <vector>
#include "fp8_tiles.cuh"
using namespace coli::fp8;

static void fail(const char* what, int tiles, int kb, int G, int slices)
{
    printf("%s: tiles %d, K steps %d, workers %d, slices %d\n", what, tiles, kb, G, slices);
    exit(1);
}

static void check(int tiles, int kb, int G, int least, int join, int slices)
{
    std::vector<int> seen((size_t)tiles * kb, 0);
    std::map<int, int> parts, first;                   // of a split tile: parts, its first part's worker
    for (int c = 0; c < G; c++) {
        Schedule s, fixed;
        s.init(tiles, kb, G, c, least, join, slices);
        fixed = s;
        Item it, same;
        int i = 0;
        for (; s.next(it); i++) {
            if (!fixed.at(i, same) || same.tile != it.tile || same.kb0 != it.kb0 || same.kb1 != it.kb1 || same.slice != it.slice)
                fail("an item looked up is another", tiles, kb, G, slices);
            if (it.tile < 0 || it.tile >= tiles || it.kb0 < 0 || it.kb1 > kb || it.kb0 >= it.kb1)
                fail("an item lies outside", tiles, kb, G, slices);
            for (int k = it.kb0; k < it.kb1; k++) seen[(size_t)it.tile * kb + k]++;
            if (it.kb1 - it.kb0 == kb || slices > 1) continue;
            const int o0 = s.owner(it.tile * kb), o1 = s.owner(it.tile * kb + kb - 1);
            if (c < o0 || c > o1 || (it.kb0 == 0) != (c == o0)) fail("a part's worker", tiles, kb, G, slices);
            if (parts.count(it.tile) && first[it.tile] != o0) fail("a tile's first worker", tiles, kb, G, slices);
            first[it.tile] = o0;
            parts[it.tile]++;
            if (it.kb1 == kb && o1 != c) fail("a tile's last worker", tiles, kb, G, slices);
        }
        if (fixed.at(i, same)) fail("an item too many", tiles, kb, G, slices);
    }
    for (int n : seen)
        if (n != 1) fail("a unit missed or done twice", tiles, kb, G, slices);
    std::map<int, int> tickets;
    for (auto& t : parts) {
        Schedule s;
        s.init(tiles, kb, G, 0, least, join, slices);
        if (t.second != s.owner(t.first * kb + kb - 1) - s.owner(t.first * kb) + 1) fail("parts", tiles, kb, G, slices);
        if (tickets[first[t.first]]++) fail("two split tiles count on one ticket", tiles, kb, G, slices);
    }
}

int main()
{
    int n = 0;
    for (int G : {1, 2, 74, 147, 148})
        for (int tiles : {0, 1, 2, 3, 7, 47, 48, 73, 74, 75, 96, 147, 148, 149, 190, 256, 333, 1025})
            for (int kb : {1, 2, 3, 4, 5, 8, 13, 14, 16, 48, 129})
                for (int l : {2, 4, 6})
                    for (int join : {3, 12, 14}) {
                        check(tiles, kb, G, l, join, 1);
                        n++;
                    }
    for (int G : {74, 148})
        for (int tiles : {1, 3, 18, 36, 37, 74})
            for (int kb : {8, 16, 48, 131})
                for (int slices = 2; slices <= kb / 4 && tiles * slices <= G; slices++) {
                    check(tiles, kb, G, 4, 14, slices);
                    n++;
                }
    printf("ok %d\n", n);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from int4_routed_expert_gemv_b200 import build
    d = tmp_path_factory.mktemp("schedule")
    src, exe = str(d / "schedule.cu"), str(d / "schedule")
    with open(src, "w") as f:
        f.write(PROGRAM)
    r = subprocess.run([build.nvcc(), *build.NVCC_FLAGS, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_schedule(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout
