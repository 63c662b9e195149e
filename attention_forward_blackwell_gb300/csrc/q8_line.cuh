// The line of key blocks that the CTAs of decode_q8.cu share, and a CTA's way along it:
// whole-number arithmetic alone, for the kernels and, as plain C++, for checks on the host.
//
// A unit (batch entry, key/value head, tile of query rows) has one block of keys at least.
// The units, one after the other, form a line that is cut into pieces, one per CTA.
#pragma once

#ifdef __CUDACC__
#define FA_LINE_FN __host__ __device__ __forceinline__
#else
#include <algorithm>
#define FA_LINE_FN inline
#endif

namespace fa {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kQ8Lead = 2;        // blocks that a unit's set-up and merge are worth
constexpr int kLeastKeys = 256;   // of a piece
constexpr int kManyBlocks = 48;   // a CTA's share from which part of it goes in small pieces

// Keys of a block, four slices.
constexpr int q8_block(int head_dim) { return head_dim == 256 ? 64 : 128; }

// CTAs of an SM: what the registers of a warp leave.  16 rows with two parts in
// hand and two CTAs at head_dim 128 took 66 us where one part and three took 76
// (16 x 1K to 16K keys x 8 heads; at 64, three for four, 43 for 65).
constexpr int q8_ctas(int head_dim, int tile) {
    return head_dim == 256 ? 2 : (head_dim == 64 ? 5 : 4) - (tile == 32 ? 3 : tile / 8);
}

// Most keys of a table: positions go up to the end of the block behind the last one, and a
// block's, a window's or the queries' length away from a key; all of them stay in 32 bits.
constexpr int kQ8MostKeys = 0x7fffffff - 4095;   // 2^31 - 4096

// Levels of small pieces, for the SMs that are done with their own first, where there may be
// much and bytes bound it: with more rows, or fewer and larger CTAs, SMs end together and
// pieces only cost.  us without / with them, 8 heads: 64 x 1K to 16K keys at head_dim 128
// 183 / 178, 300 x 1 to 12K 568 / 537, at 64 303 / 289; 16 rows, 64 x 1K to 16K at 128 191 / 200,
// at 64 124 / 139; 8 rows at 256 338 / 344, 16 x 1K to 16K 96 / 113
inline int q8_levels(int head_dim, int tile, double blocks, int slots) {
    return tile == 8 && head_dim < 256 && blocks >= (double)kManyBlocks * slots ? 2 : 0;
}

FA_LINE_FN int q8_unit_blocks(int span, int block) { return max(1, (span + block - 1) / block); }

// How the line, `all` long, is cut: a unit takes a lead of kQ8Lead, what its set-up and
// merge are worth, and its blocks; the line is cut into `slots` pieces of `big`, then
// `small` ones up to its end.  Or, with `aligned` blocks to a piece, unit by unit (the
// line then counts pieces).
struct Line {
    int all, slots, big, small, aligned;
    FA_LINE_FN int lead() const { return aligned > 0 ? 0 : kQ8Lead; }
    FA_LINE_FN int of_unit(int nb) const {   // what a unit of nb blocks takes of the line
        return aligned > 0 ? (nb + aligned - 1) / aligned : nb + kQ8Lead;
    }
    FA_LINE_FN int from(int x) const {   // where piece x starts
        if (aligned > 0) return min(x, all);
        const long long at = x < slots ? (long long)x * big
                                       : (long long)slots * big + (long long)(x - slots) * small;
        return (int)(at < all ? at : (long long)all);
    }
    FA_LINE_FN int piece_of(int pos) const {
        if (aligned > 0) return pos;
        // (slots * big < all + slots + big: within 32 bits as unsigned)
        const unsigned bigs = (unsigned)slots * (unsigned)big;
        return (unsigned)pos < bigs ? pos / big : slots + (int)(((unsigned)pos - bigs) / (unsigned)small);
    }
};

// The cut of `total` blocks of `units` units, key blocks of `block` keys.  count(s): the
// pieces that units cut every s blocks make.
//
// Pieces that end with their units save the set-up and merge of a second segment, worth
// about two blocks: taken where such pieces, one for every CTA at most, are no more
// than that much longer.  A long line may leave a quarter of itself to small pieces, for
// the SMs that are done with their own first.
template <class Count>
FA_LINE_FN Line q8_cut(int total, int units, int slots, int levels, int block, Count&& count) {
    Line line;
    line.all = total + kQ8Lead * units;
    line.slots = slots;
    line.aligned = 0;
    const int share = (int)(((unsigned)line.all + (unsigned)slots - 1) / (unsigned)slots);
    const int least = max(1, kLeastKeys / block);
    line.small = levels > 0 && share >= kManyBlocks ? share / (4 * levels) : 0;
    line.big = max(share - levels * line.small, least);
    if (line.small == 0 && units <= slots) {
        const int cut = max((total + slots - 1) / slots, least);
        for (int s = cut; s <= cut + kQ8Lead && line.aligned == 0; ++s) {
            const int all = count(s);
            if (all <= slots) {
                line.aligned = s;
                line.all = all;
            }
        }
    }
    line.small = max(line.small, 1);
    return line;
}

// Blocks before a place on an uneven line: `at` from the start of a unit, which starts at
// `start` behind `units` others.
FA_LINE_FN int q8_blocks_before(int start, int units, int at) {
    return start - kQ8Lead * units + max(0, at - kQ8Lead);
}

// Blocks of a joined split, `chunk` of each unit from block `at` on, where the unit has nb.
FA_LINE_FN int q8_joined_blocks(int nb, int at, int chunk) { return max(0, min(chunk, nb - at)); }

// A CTA's part of a unit of nb blocks, from block kb on, when `left` of the CTA's are to
// come: how many, and whether some of the next unit follow.  (A joined split past the end of
// a short sequence has kb > nb and none left.)
struct Segment {
    int n;
    bool more;
};
FA_LINE_FN Segment q8_segment(int nb, int kb, int left) {
    Segment s;
    s.n = max(0, min(nb - kb, left));
    s.more = left > s.n;
    return s;
}

// The pieces that hold blocks of a unit of nb blocks that starts at `from` on the line:
// the first one, their number, and whether the first is its CTA's second slot (it holds
// what comes before the unit, which ends with a block).
struct Pieces {
    int first, count, second;
    FA_LINE_FN int slot(int k) const { return k == 0 ? 2 * first + second : 2 * (first + k); }
};
FA_LINE_FN Pieces q8_pieces(const Line& line, int from, int nb) {
    Pieces p;
    p.first = line.piece_of(from + line.lead());
    p.count = line.piece_of(from + line.of_unit(nb) - 1) - p.first + 1;
    p.second = from > line.from(p.first) ? 1 : 0;
    return p;
}

}  // namespace fa
