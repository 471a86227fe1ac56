"""The order of the products of the shared attention's prefix kernel (csrc/fa_shared_order.h), compiled
for the host and walked through: no product waits for a tile whose slot a later product gives back,
for every ring length that the kernel has; and what its warps keep about tiles in use holds."""
import subprocess

import pytest

from online_softmax_tiled_attn_gb300 import binding

CSRC = binding.build_lib.CSRC

PROGRAM = """
#define __device__
#define __forceinline__ inline
#include "fa_shared_order.h"
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#define CHECK(x) if (!(x)) { std::printf("slots %d, %s\\n", slots, #x); return false; }
struct Item { int n; bool halves; };

// Walks through the items as the kernel does.  false: a product asks for a tile for which the ring has
// no slot before a later product, or something kept is wrong.
bool walk(int slots, const std::vector<Item>& items) {
    std::vector<char> given_back;  // of each tile of the ring, in the order of first uses
    for (const Item& it : items) {
        std::vector<int> tile_of[2];  // K and V tiles: their number in the ring
        for (auto& t : tile_of) t.assign(it.n, -1);
        int done[2][2] = {};  // S and P V products of a group
        int at[2][2] = {};    // K and V of the tile that a group works on, as the issuing warp keeps them
        int base = 0;         // the loading warp's first of three tiles whose pages it holds
        const bool ok = osm::for_steps(it.n, it.halves, [&](auto x, int u, int t, bool first, bool last) {
            constexpr int w = decltype(x)::w;
            constexpr bool pv = decltype(x)::pv;
            // P(u) lies over S(u): P V(u) follows S(u), and S(u + 1) follows P V(u)
            CHECK(u == done[w][pv] && (pv ? done[w][0] == u + 1 : done[w][1] == u));
            ++done[w][pv];
            CHECK(t >= 0 && t < it.n && (it.halves ? t == u : t == 2 * u + w));
            if (first) {
                const int e = static_cast<int>(given_back.size());
                CHECK(e < slots || given_back[e - slots]);
                CHECK(tile_of[pv][t] == -1);
                tile_of[pv][t] = e;
                given_back.push_back(0);
                at[w][pv] = e;
                if (it.halves) at[1][pv] = e;
                if (t > base + 1) ++base;
                CHECK(t == base || t == base + 1);
            }
            CHECK(tile_of[pv][t] >= 0 && at[w][pv] == tile_of[pv][t]);
            CHECK(!given_back[at[w][pv]]);
            if (last) given_back[at[w][pv]] = 1;
            return true;
        });
        if (!ok) return false;
        for (auto& tiles : tile_of)
            for (int e : tiles) CHECK(e >= 0 && given_back[e]);
        for (int w = 0; w < 2; ++w)
            for (int n : done[w]) CHECK(n == osm::steps_of(it.n, it.halves, w));
    }
    return true;
}

bool all(int slots) {
    for (int n = 1; n <= 300; ++n)
        for (bool halves : {false, true})
            if (!walk(slots, {{n, halves}})) return false;
    for (int a = 1; a <= 12; ++a)
        for (int b = 1; b <= 12; ++b)
            for (int h = 0; h < 4; ++h)
                if (!walk(slots, {{a, (h & 1) != 0}, {b, (h & 2) != 0}, {a, (h & 1) == 0}})) return false;
    std::mt19937 r(1);
    for (int i = 0; i < 3000; ++i) {
        std::vector<Item> items(2 + r() % 6);
        for (Item& it : items) it = {static_cast<int>(1 + r() % 9), r() % 2 != 0};
        if (!walk(slots, items)) return false;
    }
    return true;
}

int main(int argc, char** argv) {
    if (argc == 2) return all(std::atoi(argv[1])) ? 0 : 1;
    for (int d : {64, 128})
        for (bool int4 : {false, true})
            if (!all(osm::sh_slots(d, int4))) return 1;
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    folder = tmp_path_factory.mktemp("order")
    (folder / "main.cpp").write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}",
                        str(folder / "main.cpp"), "-o", str(folder / "main")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(folder / "main")


def run(*args):
    return subprocess.run(args, capture_output=True, text=True, timeout=60)


def test_the_kernels_rings(program):
    r = run(program)
    assert r.returncode == 0, r.stdout


def test_the_walk_finds_a_ring_that_is_too_short(program):
    """One slot cannot hold the tiles of two products that wait for one another; two can."""
    r = run(program, "1")
    assert r.returncode == 1 and "given_back" in r.stdout
    assert run(program, "2").returncode == 0
