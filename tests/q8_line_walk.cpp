// The 8-bit decode's CTAs walked on the host, by the arithmetic that its kernels run
// (csrc/q8_line.cuh): built and called by test_q8_line.py.
#include <vector>

#include "q8_line.cuh"

using namespace fa;

namespace {

// Units of all sequences, in their order: blocks and places on the line.
struct Units {
    std::vector<int> nb;
    int per;   // of a sequence
    Units(const int* spans, int B, int units, int block) : per(units) {
        for (int b = 0; b < B; ++b)
            for (int u = 0; u < units; ++u) nb.push_back(q8_unit_blocks(spans[b], block));
    }
    int count() const { return (int)nb.size(); }
};

// A CTA's segments from block kb of unit u on.  taken[unit][block] counts who works on it;
// slot(unit, second segment or later) is called for the units that do not end here or
// did not start here.  False where queries of a unit past the last are asked for.
template <class Part>
bool walk(const Units& all, int u, int kb, int blocks, std::vector<std::vector<int>>& taken, Part&& part) {
    int left = blocks, index = 0;
    do {
        if (u >= all.count()) return false;
        const Segment s = q8_segment(all.nb[u], kb, left);
        if (s.n < 0 || (s.n > 0 && kb + s.n > all.nb[u])) return false;
        for (int i = 0; i < s.n; ++i) ++taken[u][kb + i];
        if (s.n != all.nb[u]) part(u, kb, s.n, index);
        if (s.more && u + 1 >= all.count()) return false;
        left -= s.n;
        kb = 0;
        ++index;
        ++u;
    } while (left > 0);
    return true;
}
std::vector<std::vector<int>> counts(const Units& all) {
    std::vector<std::vector<int>> t;
    for (int n : all.nb) t.emplace_back(n, 0);
    return t;
}
int once(const std::vector<std::vector<int>>& taken) {
    for (auto& u : taken)
        for (int c : u)
            if (c != 1) return 2;
    return 0;
}

}  // namespace

extern "C" {

// Joined splits, `chunk` blocks each, `splits` to a unit.  0: every block has one split and
// no CTA asks for queries that are not there.
int walk_joined(const int* spans, int B, int units, int block, int chunk, int splits) {
    const Units all(spans, B, units, block);
    auto taken = counts(all);
    for (int b = 0; b < B; ++b)
        for (int u = 0; u < units; ++u)
            for (int x = 0; x < splits; ++x) {
                const int unit = b * units + u, at = x * chunk;
                if (!walk(all, unit, at, q8_joined_blocks(all.nb[unit], at, chunk), taken,
                          [](int, int, int, int) {}))
                    return 1;
                // (a split has its own unit alone)
                if (q8_segment(all.nb[unit], at, q8_joined_blocks(all.nb[unit], at, chunk)).more) return 3;
            }
    return once(taken);
}

// The line: cut[0..4] all, big, small, aligned, share of a CTA.  0: every block has one piece,
// and the merge reads each unit's pieces where they were left.
int walk_line(const int* spans, int B, int units, int block, int slots, int levels, int* cut) {
    const Units all(spans, B, units, block);
    long long total = 0;
    for (int n : all.nb) total += n;
    const Line line = q8_cut((int)total, all.count(), slots, levels, block, [&](int s) {
        int n = 0;
        for (int nb : all.nb) n += (nb + s - 1) / s;
        return n;
    });
    cut[0] = line.all, cut[1] = line.big, cut[2] = line.small, cut[3] = line.aligned;
    cut[4] = (int)((total + (long long)kQ8Lead * all.count() + slots - 1) / slots);
    std::vector<int> start;
    int end = 0;
    for (int n : all.nb) {
        start.push_back(end);
        end += line.of_unit(n);
    }
    if (end != line.all) return 4;
    const int ctas = slots * (1 + levels);
    if (line.from(ctas) != line.all) return 5;   // some of it has no piece
    auto taken = counts(all);
    std::vector<std::vector<std::vector<int>>> slot_of(all.count());   // of a unit: {kb, n, slot}, in order
    auto unit_at = [&](int pos) {
        int u = 0;
        while (u + 1 < all.count() && start[u + 1] <= pos) ++u;
        return u;
    };
    for (int x = 0; x < ctas; ++x) {
        const int begin = line.from(x), stop = line.from(x + 1);
        if (begin >= line.all) continue;
        if (line.piece_of(begin) != x || line.piece_of(stop - 1) != x) return 6;
        const int u = unit_at(begin);
        int kb, blocks;
        if (line.aligned > 0) {
            kb = (begin - start[u]) * line.aligned;
            blocks = std::min(line.aligned, all.nb[u] - kb);
        } else {
            const int to = stop < line.all ? unit_at(stop) : 0;
            const int before = q8_blocks_before(start[u], u, begin - start[u]);
            const int after = stop < line.all ? q8_blocks_before(start[to], to, stop - start[to])
                                              : line.all - kQ8Lead * all.count();
            kb = std::max(0, begin - start[u] - kQ8Lead);
            blocks = after - before;
        }
        if (blocks < 0) return 7;
        if (blocks == 0) continue;
        if (!walk(all, u, kb, blocks, taken, [&](int unit, int at, int n, int index) {
                slot_of[unit].push_back({at, n, 2 * x + (index > 0)});
            }))
            return 1;
    }
    if (const int bad = once(taken)) return bad;
    for (int u = 0; u < all.count(); ++u) {
        const Pieces pc = q8_pieces(line, start[u], all.nb[u]);
        if (slot_of[u].empty()) {
            if (pc.count != 1) return 8;
            continue;
        }
        if (pc.count != (int)slot_of[u].size()) return 9;
        for (int k = 0; k < pc.count; ++k)
            if (pc.slot(k) != slot_of[u][k][2]) return 10;
    }
    return 0;
}

int line_ctas(int head_dim, int tile) { return q8_ctas(head_dim, tile); }
int line_block(int head_dim) { return q8_block(head_dim); }
int line_levels(int head_dim, int tile, double blocks, int slots) { return q8_levels(head_dim, tile, blocks, slots); }
int line_unit_blocks(int span, int block) { return q8_unit_blocks(span, block); }
int line_many() { return kManyBlocks; }

}  // extern "C"
