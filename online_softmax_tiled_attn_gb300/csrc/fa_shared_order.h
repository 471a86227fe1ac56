// fa_shared_order.h -- the order of the products of the prefix kernel (fa_shared.cu) over an item's
// tiles, which its loading, expanding and issuing warps all follow, and the length of its ring of
// tiles.  A tile's slot is given back with its last product, and a wait for a slot that a later product
// gives back would never end: tests/test_shared_order_cpu.py compiles this header for the host and
// checks that none is asked for.
#pragma once

namespace osm {

// Tiles that the ring holds: what shared memory has room for beside the queries (two tiles) and, in 4
// bits, the tiles as they are stored.
constexpr int sh_slots(int d, bool int4) { return d == 128 ? (int4 ? 3 : 5) : (int4 ? 8 : 10); }

// Steps of group w in an item of n tiles: all tiles or every other one.
__device__ __forceinline__ int steps_of(int n, bool halves, int w) {
    return halves ? n : (n + 1 - w) / 2;
}

// The products of an item in their order: use(product, u, tile, first use of the tile's K or V, last
// use of it).
template <int W, bool PV>
struct Product {
    static constexpr int w = W;     // group
    static constexpr bool pv = PV;  // P V, or S
};
template <typename Use>
__device__ __forceinline__ bool for_steps(int n, bool halves, const Use& use) {
    const int na = steps_of(n, halves, 0), nb = steps_of(n, halves, 1);
    auto call = [&](auto x, int u) {
        constexpr int w = decltype(x)::w;
        return use(x, u, halves ? u : 2 * u + w, w == 0 || !halves, w == 1 || !halves);
    };
    for (int u = -1; u < na; ++u) {
        if (u >= 0 && !call(Product<0, true>(), u)) return false;
        if (u + 1 < na && !call(Product<0, false>(), u + 1)) return false;
        if (u >= 0 && u < nb && !call(Product<1, true>(), u)) return false;
        if (u + 1 < nb && !call(Product<1, false>(), u + 1)) return false;
    }
    return true;
}

}  // namespace osm
