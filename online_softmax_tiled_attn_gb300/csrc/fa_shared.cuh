// fa_shared.cuh -- what the kernels of fa_fwd_paged_shared hand to one another.
//
// Plan (fa_shared.cu): which sequences share how many tokens.  A shared group is a run of sequences
// with `tiles` common tiles of 128 tokens; its rows over all its sequences, (sequence, query, query
// head of the key/value head), are taken 256 at a time, and an item is (group, key/value head, block
// of rows).  The items are cut into units of a few tiles each, and each CTA of the prefix kernel
// (fa_shared.cu) takes as many units in a row, `share` of them.  It leaves the rows' states (m, l, O
// unnormalised, m in log2 units); the kernel over the sequences' own tokens (fa_paged.cu) leaves
// theirs, and a last one joins them.
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
// The kernel over the own tokens: its CTAs' shares are equal numbers of units, a unit a tile of an item
// and this many in front of each item's tiles, for what an item costs a CTA whatever it holds (some 4.5
// us, 30 tiles).  With tiles alone, a CTA whose share is many short items was the last by far: 64
// sequences behind 16384 common bf16 tokens, half of them with 1000 tokens of their own and half with
// 10, 288 us (fa_fwd_paged 259), now 68; 4 bits and three queries 561 (328), now 108.  30 units leave
// the CTAs within a long item, which pay for their start as well, with too many tiles: 4 bits, 8 with
// 4000 and 56 with 10 behind 32768 112 us, with 16 units 91, with 8 77; but bf16, three queries, half
// with 1000 131, 131 and 183, and 8 x 8192 in 4 bits without common tokens 37, 36 and 37.
constexpr int kOwnItemUnits = 16;

// Made by the plan on the device.
struct alignas(16) ShHead {
    long long units;  // of all groups
    int groups;
    int share;            // units that a CTA of the prefix kernel takes
    long long own_share;  // of which a CTA of the kernel over the sequences' own tokens takes
    int piece;            // tiles of a unit of a block of more than 128 rows
    int small_piece;      // and of one of fewer
    long long own_units;  // of the own tokens of all sequences (see kOwnItemUnits)
};
struct alignas(16) ShGroup {
    long long unit0;   // units of the items of the groups before
    int first, count;  // its sequences
    int tiles;
};
struct alignas(16) ShSeq {  // of a sequence
    long long own0;         // units of the own tokens of the sequences before (see kOwnItemUnits)
    long long unit0;        // of its group
    int skip;               // common tokens (0: none, and no group; a multiple of kShTile)
    int first, count;       // its group's sequences
    int pad;
};

// The workspace's parts as kernel parameters.
struct ShView {
    const ShHead* head;
    const ShGroup* groups;
    const ShSeq* seqs;
    float* edge_o;          // [ctas][2][2][kShHalf][d]
    float2* edge_ml;        // [ctas][2][2][kShHalf]
    float* row_o;           // [B * H * Nq][2][d]
    float2* row_ml;         // [B * H * Nq][2]
    int ctas;               // of the prefix kernel
    int B;
    int rows_per_seq;       // Nq * H / H_kv
    int H_kv;
};

// a / b for a quotient far below 2^31, without the call that a 64-bit division is.
__device__ __forceinline__ int divide(long long a, long long b) {
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

// Units of an item.
__device__ __forceinline__ int sh_units(int tiles, int piece) {
    return piece == 1 ? tiles : (tiles + piece - 1) / piece;
}

// A group's units on one key/value head: those of its blocks of more than 128 rows, then those of the
// last block if it has fewer.
struct ShCut {
    int big, units, small_units, per;
};
__device__ __forceinline__ ShCut sh_cut(int group_rows, int tiles, int piece, int small_piece) {
    const int rest = group_rows % kShRows;
    ShCut c;
    c.big = group_rows / kShRows + (rest > kShHalf);
    c.units = sh_units(tiles, piece);
    c.small_units = rest > 0 && rest <= kShHalf ? sh_units(tiles, small_piece) : 0;
    c.per = c.big * c.units + c.small_units;
    return c;
}

}  // namespace osm
