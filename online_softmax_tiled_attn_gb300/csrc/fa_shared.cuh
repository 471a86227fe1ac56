// fa_shared.cuh -- what the kernels of fa_fwd_paged_shared hand to one another.
//
// Plan (fa_shared.cu): which sequences share how many tokens.  A shared group is a run of sequences
// with `tiles` common tiles of 128 tokens; its rows over all its sequences, (sequence, query, query
// head of the key/value head), are taken 256 at a time, and an item is (group, key/value head, block
// of rows).  All tiles of all items, in order, are cut into equal shares, one a CTA of the prefix
// kernel (fa_shared.cu), which leaves the rows' states (m, l, O unnormalised, m in log2 units); the
// kernel over the sequences' own tokens (fa_paged.cu) joins them.
//
// States.  An item within one share: at the row's own place (two of them, see below).  One that spans
// shares: for each of its shares at the CTA's edge places, [0] of an item that began earlier, [1] of
// one that begins there and goes on.  A block of more than 128 rows gives its halves to the CTA's two
// softmax groups, which see every tile; a smaller one gives its rows to both groups, which take the
// tiles in turn, so it has two states.
#pragma once

#include <cstdint>

namespace osm {

constexpr int kShTile = 128;   // tokens a tile
constexpr int kShRows = 256;   // rows of a block
constexpr int kShHalf = 128;

// One shared group, made by the plan on the device.
struct ShGroup {
    long long unit0;  // tiles of the items of the groups before
    int first, count; // its sequences
    int tiles;
    int pad;
};

// The workspace's parts as kernel parameters.
struct ShView {
    const int32_t* skip;    // [B] common tokens of each sequence (0: none; a multiple of kShTile)
    const int32_t* group;   // [B] its group (where skip is not 0)
    const ShGroup* groups;  // [n + 1]; the last one's unit0 is the number of units
    const int32_t* n;       // groups
    float* edge_o;          // [ctas][2][2][kShHalf][d]
    float2* edge_ml;        // [ctas][2][2][kShHalf]
    float* row_o;           // [B * H * Nq][2][d]
    float2* row_ml;         // [B * H * Nq][2]
    int ctas;               // of the prefix kernel
    int rows_per_seq;       // Nq * H / H_kv
    int H_kv;
};

__device__ __forceinline__ int sh_blocks(const ShView& s, const ShGroup& g) {
    return (g.count * s.rows_per_seq + kShRows - 1) / kShRows;
}

// Tiles a CTA takes: at least kShLeast, so that a short prefix does not leave more states to join
// than it saves time.
constexpr int kShLeast = 2;
__device__ __forceinline__ long long sh_share(long long units, int ctas) {
    const long long s = (units + ctas - 1) / ctas;
    return s > kShLeast ? s : kShLeast;
}

// The same for the kernel over the sequences' own tokens: at least a tile a warp.
constexpr int kOwnWarps = 4;
__device__ __forceinline__ long long own_share(long long units, int ctas) {
    const long long s = (units + ctas - 1) / ctas;
    return s > kOwnWarps ? s : kOwnWarps;
}

}  // namespace osm
