// Attention of rows that share spans of keys, on the tensor cores (head_dim
// 64, 128 and 256): a tree of drafted tokens over a cache (MODE kSpanTree), and
// a sliding window whose first keys stay visible (kSpanWindow; prompts, chunks
// of prompts and single tokens).
//
// Rows.  All query heads of a key/value head read the same keys, so a tile of
// 128 rows holds several of them.  For a tree the rows [b, hk * group ..
// + group, 0 .. T) of Q and O lie side by side in memory, one matrix of group *
// T rows; a tile is 128 of them whatever T is, and row r of the matrix is node
// r % T.  For a window a tile is `group` heads x P = 128 / group positions
// (row r: head r / P, position r % P of the tile), so that the keys it visits,
// window + P, grow least.
//
// Keys.  A tile visits positions [0, span) of an axis of its own: for a window
// the first keys rounded up to a box of rows, then, skipping what no row sees,
// the keys from its first row's window on, rounded down to one (span_geometry);
// a tree visits every key.  So no block is spent on the few first keys alone,
// and blocks of 256 keys waste less of a window than their size suggests.
// Only the blocks at the borders are masked.
//
// What bounds it: per key of a key/value head 4 d bytes of K and V are read
// and 4 d operations per row done, so up to about 270 rows that share it
// memory is the bound and past it the tensor cores (1865 TFLOP/s over 6793
// GB/s, both measured).  The blocks are therefore spread evenly over the SMs:
// the units' (batch entry, key/value head, tile) blocks, one after the other,
// form one line of N blocks, and CTA x takes the blocks [x quota, (x + 1)
// quota), quota = ceil(N / CTAs), whatever the sequences' lengths (which only
// the device knows).  A unit that lies in one CTA is finished there; of the
// others each CTA writes its piece's unnormalised O, row max and row sum, and
// span_combine_kernel merges the pieces, in their order (the result does not
// depend on timing).  A tree of several tiles gives each to a CTA of a group
// that walks the same keys at the same time, so that K and V come from HBM
// once and from L2 after that (64 nodes x 8 heads over 8 x 4K to 8K keys at
// head_dim 128: 95 us; one tile after the other read them three times and took
// 20 more).
//
// Inside a CTA: the roles and barriers of the 256-key prefill kernel (see
// prefill_wide.cuh), which this one follows: S = Q K^T of the next block is
// issued once the softmax has read this block's scores into registers; two
// warpgroups share each row's softmax; P has tensor memory of its own.  Key
// blocks are 256 keys (one N = 256 score instruction per 16 head dims), 128 at
// head_dim 256, whose 256 O columns leave no room for more.
//
#include "prefill.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

template <int D>
struct SpanTraits {
    static constexpr int BM = 128;                  // rows of a tile = TMEM lanes
    static constexpr int BN = D == 256 ? 128 : 256; // keys of a block
    static constexpr int HK = BN / 2;               // keys of a softmax half
    static constexpr int NCH = D / 64;              // 64-column chunks of a row
    static constexpr int CHUNK = 128 * 128;         // one chunk of the Q tile, bytes
    static constexpr int QTILE = NCH * CHUNK;
    static constexpr int SLOT = 32768;              // ring slot, bytes
    static constexpr int KCHUNK = BN * 128;         // one chunk of a K block, bytes
    static constexpr int KCH = SLOT / KCHUNK;       // chunks of a K slot
    static constexpr int KP = NCH / KCH;            // slots of a K block
    static constexpr int VKEYS = SLOT / (NCH * 128);// keys of a V slot
    static constexpr int VCHUNK = VKEYS * 128;
    static constexpr int VP = BN / VKEYS;           // slots of a V block
    static constexpr int NSLOT = D == 64 ? 6 : (D == 128 ? 5 : 4);
    static constexpr int THREADS = 512;
    static constexpr int CORR_WG = 2;
    static constexpr int MMA_WARP = 12;
    static constexpr int LOAD_WARP = 13;
    static constexpr int ITEM_WARP = 14;
    static constexpr int LOAD2_WARP = 15;
    static constexpr int D_COLS = D;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t S_COL = 0;
    static constexpr uint32_t P_COL = BN;           // BN / 2 columns of bf16 pairs
    static constexpr uint32_t O_COL = D == 256 ? 256 : 384;
    static constexpr int SMEM_Q = QTILE;
    static constexpr int SMEM_RING = NSLOT * SLOT;
    static constexpr int SMEM_AUX = 8192;
    static constexpr int STAGE = 2048;              // O staging per correction warp
    static constexpr int SMEM_TOTAL = 1024 + SMEM_Q + SMEM_RING + SMEM_AUX + 4 * STAGE;
    static constexpr uint32_t SOFTMAX_REGS = 168, CORR_REGS = 96, OTHER_REGS = 80;
    static_assert(8 * 32 * SOFTMAX_REGS + 4 * 32 * CORR_REGS + 4 * 32 * OTHER_REGS <= THREADS * 128,
                  "register split exceeds the launch allocation");
    static_assert(KP * KCH == NCH && VP * VKEYS == BN, "slots must cover a block");
    static_assert(P_COL + BN / 2 <= O_COL && O_COL + D <= TMEM_COLS, "S, P and O must fit");
    static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA exceeds the sm_103 limit");
};

constexpr int kSpanSlots = 6;

// Wait sites of the segment queue (after those of the other kernels).
constexpr unsigned kSiteItem = 64, kSiteItemRead = 65;

// A segment of a CTA: consecutive key blocks of a unit, one tile's share of a
// (batch entry, key/value head).
struct SpanItem {
    int b, u;        // batch entry, unit of it
    int kb, n, nb;   // first block, blocks on the line (0: the CTA has no more), the unit's
    int m;           // blocks that hold keys of the tile
    int index;       // segments before it
    int hk, tile;
    int head, skip;  // position x of its axis: key x below head, key x + skip from there on
    int span;        // positions that a row may see
    int end;         // position of the sequence's end
    int gap;         // decode: no row sees a position from `first` up to here
    int rows, keys;  // the sequence's (see SpanSeq)
    int q0, k0, cap;
};
constexpr int kItems = 4;    // segments known ahead

struct SpanAux {
    SpanItem items[kItems];
    uint64_t bar_item[kItems];        // segment written (scheduler)
    uint64_t bar_item_read[kItems];   // and read by every warp that works on it
    uint64_t bar_q;
    uint64_t bar_full[kSpanSlots];
    uint64_t bar_empty[kSpanSlots];
    uint64_t bar_s_full;
    uint64_t bar_xm[2];
    uint64_t bar_p_ready[2];
    uint64_t bar_corrected[2];
    uint64_t bar_pv_done[2];
    uint64_t bar_fin;
    uint64_t bar_qfree;
    uint64_t bar_odrained;
    uint64_t bar_drain;
    uint32_t tmem_base;
    int abort_flag;
    int start_b;              // the CTA's first block: its batch entry,
    int start_off;            // and blocks of that entry's units before it
    float xm[2][2][128];      // [J & 1][half][row] block maxima
    float mb_l[2][128];       // [half][row] row sums of a segment
};

// A sequence: query rows (nodes) and keys, in packed tensors its first query
// and key token, and the rows that are computed (packed: at most the launch's).
struct SpanSeq {
    int rows, keys, q0, k0, cap;
};
template <int MODE>
__device__ __forceinline__ SpanSeq span_seq(const SpanArgs& a, int b) {
    SpanSeq q{a.Sq, a.Sk, 0, 0, 0};
    if (MODE == kSpanTree) {
        if (a.tree_lens != nullptr) q.rows = max(0, min(a.tree_lens[b], a.Sq));
    } else if (a.cu_seqlens_q != nullptr) {   // (clamped: bad offsets stay inside the tensors)
        q.q0 = min(max(a.cu_seqlens_q[b], 0), a.total_q);
        q.rows = min(max(a.cu_seqlens_q[b + 1], q.q0), a.total_q) - q.q0;
    }
    if (a.seqlens_k != nullptr) {
        q.keys = max(0, min(a.seqlens_k[b], a.Sk));
    } else if (MODE == kSpanWindow && a.cu_seqlens_k != nullptr) {
        q.k0 = min(max(a.cu_seqlens_k[b], 0), a.total_k);
        q.keys = min(max(a.cu_seqlens_k[b + 1], q.k0), a.total_k) - q.k0;
    }
    q.cap = min(q.rows, a.Sq);
    return q;
}
// Units of a batch entry -- a window's tiles, a tree's groups of group_ctas tiles,
// of each key/value head -- and the key blocks each counts for on the line: a
// bound for a window (its tiles near the start have fewer), one at least, so
// that rows without keys are written too.
template <int MODE>
__device__ __forceinline__ int span_groups(const SpanArgs& a, const SpanSeq& q) {
    if (q.cap == 0) return 0;
    if (MODE == kSpanTree) return a.tile_groups;
    return (int)((unsigned)(q.cap + a.P - 1) / (unsigned)a.P);
}
template <int MODE>
__device__ __forceinline__ int span_units(const SpanArgs& a, const SpanSeq& q) {
    return a.Hkv * span_groups<MODE>(a, q);
}
template <class T, int MODE>
__device__ __forceinline__ int span_blocks(const SpanArgs& a, const SpanSeq& q) {
    int keys = q.keys;
    if (MODE == kSpanWindow && a.causal) keys = min(keys, a.window_keys);
    return max(1, (keys + T::BN - 1) / T::BN);
}

__device__ __forceinline__ int span_key(const SpanItem& s, int x) {
    return x < s.head ? x : x + s.skip;
}

// The axis of the keys of the unit whose first tile is t0.
template <class T, int MODE>
__device__ __forceinline__ void span_geometry(const SpanArgs& a, int t0, SpanItem& s) {
    s.head = s.skip = s.gap = 0;
    if constexpr (MODE == kSpanTree) {
        s.span = s.end = s.keys;
    } else {
        const int off = s.keys - s.rows;   // bottom-right alignment
        const int p0 = t0 * a.P + off;     // keys of the unit's first and last row
        const int p1 = min((t0 + 1) * a.P, s.cap) - 1 + off;
        const int last = a.causal ? min(s.keys - 1, p1) : s.keys - 1;
        const int lo = max(0, p0 - a.window + 1), base = lo & -a.box;
        if (a.head_keys < base) {
            s.head = a.head_keys;
            s.skip = base - s.head;
        }
        if (a.decode) s.gap = lo - s.skip;
        s.span = max(0, last + 1 - s.skip);
        s.end = s.keys - s.skip;
    }
    const int real = (s.span + T::BN - 1) / T::BN;
    s.m = max(0, min(s.kb + s.n, real) - s.kb);
}

// Where a segment's Q tile lies in its tensor map.
template <class T, int MODE>
__device__ __forceinline__ void span_q_at(const SpanArgs& a, const SpanItem& s, int& row,
                                          int& plane) {
    row = s.tile * T::BM;   // tree: rows of the matrix; window: positions x heads
    plane = s.b * a.Hkv + s.hk;
    if (MODE == kSpanWindow) {
        row = s.q0 + s.tile * a.P;
        plane = (a.cu_seqlens_q != nullptr ? 0 : s.b * a.Hq) + s.hk * a.group;
    }
}

// Scheduler's warp: places the CTA on the line of blocks -- each lane sums the
// blocks of its share of the batch, and the lane whose share holds the CTA's
// first block finds it there -- then (one lane) walks the CTA's blocks, writes
// its segments ahead of the roles and loads each one's Q as soon as the segment
// before has issued its last score MMA (the producers, busy with slots, would
// come to it later).  Numbers of blocks are below 2^31 (span_ok sees to it).
template <class T, int MODE>
__device__ void span_item_role(const SpanMaps& tm, const SpanArgs& a, SpanAux* aux, uint32_t sQ,
                               const WaitCtx& wc) {
    const int lane = threadIdx.x & 31;
    const int per = (a.B + 31) >> 5, b0 = lane * per, b1 = min(b0 + per, a.B);
    int mine = 0, at = 0, beg = 0, left = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        // pass 0: the lane's blocks; pass 1: the batch entry that holds block beg
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const SpanSeq q = span_seq<MODE>(a, b);
            const int v = span_units<MODE>(a, q) * span_blocks<T, MODE>(a, q);
            if (pass == 0) {
                mine += v;
            } else {
                if (at <= beg && beg < at + v) {
                    aux->start_b = b;
                    aux->start_off = beg - at;
                }
                at += v;
            }
        }
        if (pass == 0) {
            at = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            const int all = __shfl_sync(0xffffffffu, at, 31);
            at -= mine;
            const unsigned groups = (unsigned)gridDim.x / (unsigned)a.group_ctas;
            const int quota = (int)(((unsigned)all + groups - 1) / groups);
            // (below all where the CTA has blocks; large products stay in range)
            const long long from = (long long)quota * (int)(blockIdx.x / (unsigned)a.group_ctas);
            beg = (int)min(from, (long long)all);
            left = min(quota, all - beg);
            if (blockIdx.x == 0 && lane == 0)   // (for the combine kernel)
                a.head[2 * gridDim.x] = make_int4(quota, 0, 0, 0);
            if (per == 1) {   // (no second pass)
                if (at <= beg && beg < at + mine) {
                    aux->start_b = b0;
                    aux->start_off = beg - at;
                }
                break;
            }
        }
    }
    __syncwarp();
    if (lane == 0) {
        int tiles = 0, kq = 0;   // tile numbers of a key/value head's units
        const int first = (int)(blockIdx.x % (unsigned)a.group_ctas);
        const uint32_t bar_q = smem_u32(&aux->bar_q);
        SpanItem s{};
        s.b = aux->start_b - 1;
        s.hk = a.Hkv;      // (the line starts with a batch entry)
        s.n = 1;
#pragma unroll 1
        for (int i = 0;; ++i) {
            if (s.n > 0) {   // segment i
                s.kb = 0;
                if (left > 0) {
                    s.tile += a.group_ctas;
                    ++s.u;
                    if (s.tile >= tiles) {
                        s.tile = first;
                        ++s.hk;
                    }
                    if (s.hk >= a.Hkv) {   // the next batch entry that has units
                        int groups;
#pragma unroll 1
                        do {
                            const SpanSeq q = span_seq<MODE>(a, ++s.b);
                            groups = span_groups<MODE>(a, q);
                            s.nb = span_blocks<T, MODE>(a, q);
                            s.rows = q.rows;
                            s.keys = q.keys;
                            s.q0 = q.q0;
                            s.k0 = q.k0;
                            s.cap = q.cap;
                        } while (groups == 0 && s.b + 1 < a.B);
                        s.u = s.hk = 0;
                        tiles = groups * a.group_ctas;
                        s.tile = first;
                        if (i == 0) {   // where on the line the CTA starts
                            s.u = (int)((unsigned)aux->start_off / (unsigned)s.nb);
                            s.kb = aux->start_off - s.u * s.nb;
                            s.hk = (int)((unsigned)s.u / (unsigned)groups);
                            s.tile += (s.u - s.hk * groups) * a.group_ctas;
                        }
                    }
                }
                s.n = max(0, min(s.nb - s.kb, left));
                left -= s.n;
                s.index = i;
                span_geometry<T, MODE>(a, s.tile - first, s);
                const int slot = i % kItems;
                if (i >= kItems && !mbar_wait_lane(smem_u32(&aux->bar_item_read[slot]),
                                                   (uint32_t)((i / kItems - 1) & 1), wc,
                                                   kErrWaitTimeout | kSiteItemRead))
                    break;
                aux->items[slot] = s;
                mbar_arrive(smem_u32(&aux->bar_item[slot]));
            }
            // Q of segment i into L2, and of segment i - 1 into shared memory (the
            // first at once)
#pragma unroll 1
            for (int behind = 0; behind < 2; ++behind) {
                const SpanItem& g = aux->items[(i + kItems - behind) % kItems];
                const bool load = behind > 0 || i == 0;
                if ((behind > 0 && i < 2) || g.n == 0 || g.m == 0 || (behind == 0 && s.n == 0))
                    continue;
                int row, q_plane;
                span_q_at<T, MODE>(a, g, row, q_plane);
                if (load) {
                    if (kq > 0 && !mbar_wait_lane(smem_u32(&aux->bar_qfree), (uint32_t)((kq - 1) & 1),
                                                  wc, kErrWaitTimeout | kSiteLoadQfree)) {
                        s.n = 0;   // given up
                        left = -1;
                        break;
                    }
                    mbar_arrive_expect_tx(bar_q, (uint32_t)a.q_bytes);
                    ++kq;
                }
#pragma unroll 1
                for (int q = 0; q < T::NCH; ++q) {
                    if (load)
                        tma_load_3d(sQ + q * T::CHUNK, &tm.q, q * 64, row, q_plane, bar_q);
                    else
                        tma_prefetch_l2_3d(&tm.q, q * 64, row, q_plane);
                }
            }
            if (left < 0 || (i >= 1 && aux->items[(i + kItems - 1) % kItems].n == 0)) break;
        }
        if (kq > 0) mbar_wait_drain(bar_q, (uint32_t)((kq - 1) & 1), a.wait_limit_ns);
    }
    __syncwarp();
}

// Segment i, for one lane (the caller then counts it as read) or a warp.
// False at the end, or if the wait gave up.
__device__ __forceinline__ bool span_item_lane(SpanAux* aux, int i, const WaitCtx& wc, SpanItem& s) {
    if (!mbar_wait_lane(smem_u32(&aux->bar_item[i % kItems]), (uint32_t)((i / kItems) & 1), wc,
                        kErrWaitTimeout | kSiteItem))
        return false;
    s = aux->items[i % kItems];
    return s.n > 0;
}
__device__ __forceinline__ bool span_item(SpanAux* aux, int i, const WaitCtx& wc, SpanItem& s) {
    if (!mbar_wait(smem_u32(&aux->bar_item[i % kItems]), (uint32_t)((i / kItems) & 1), wc,
                   kErrWaitTimeout | kSiteItem))
        return false;
    s = aux->items[i % kItems];
    mbar_arrive_warp(smem_u32(&aux->bar_item_read[i % kItems]));
    return s.n > 0;
}

// Tile row r (window: head g = r / P of the group, position gp = r % P of the
// tile): its query head, and its index among the rows of O and in the LSE;
// whether it is a row of the sequence.
template <class T, int MODE>
__device__ __forceinline__ bool span_row(const SpanArgs& a, int cap, int q0, int b, int hk, int tile,
                                         int r, int g, int gp, int& h, size_t& o_row,
                                         size_t& lse_at) {
    bool real;
    int pos;
    if constexpr (MODE == kSpanTree) {
        const int row = tile * T::BM + r;
        h = row / a.Sq;
        pos = row - h * a.Sq;
        h += hk * a.group;
        real = row < a.group * a.Sq && pos < cap;
    } else {
        h = hk * a.group + g;
        pos = tile * a.P + gp;
        real = g < a.group && pos < cap;
        if (a.cu_seqlens_q != nullptr) {
            o_row = (size_t)(q0 + pos) * a.Hq + h;
            lse_at = (size_t)h * a.total_q + q0 + pos;
            return real;
        }
    }
    o_row = lse_at = ((size_t)b * a.Hq + h) * a.Sq + pos;
    return real;
}

// Producers: per segment K_0, then K_{j+1} and V_j for every block j, slot
// after slot of one ring, two warps in turn (each waits a slot free, counts its
// bytes and copies).  Keys that lie together come as one copy per chunk of a
// slot; those of pages, and of a block on both sides of a window's gap, as boxes
// of a.box rows, one or two per lane.  A slot takes its warp 500 to 700 cycles of waits and issue one
// after the other: one warp for the four slots of a block took as long as the
// block's softmax.  The code is kept to a few hundred bytes, with what does not
// change from slot to slot in registers: the softmax's straight code keeps
// evicting it (about 0.3 cycles a byte).
template <class T, int MODE, bool PAGED>
__device__ void span_load_role(int part, const SpanMaps& tm, const SpanArgs& a, SpanAux* aux,
                               uint32_t sRing, const WaitCtx& wc, unsigned long long* tr) {
    const int lane = threadIdx.x & 31;
    const int box_shift = __ffs(a.box) - 1;   // (a power of two)
    const bool one = elect_one();
    // the boxes of a block, lane l's the l-th and the (l + 32)-th: K slots hold
    // all of them, one chunk or more each; V slot h the boxes [h vboxes, (h + 1)
    // vboxes)
    const int boxes = T::BN >> box_shift, vboxes_shift = __ffs(T::VKEYS >> box_shift) - 1;
    const uint32_t bars = smem_u32(&aux->bar_full[0]);
    const uint32_t empty_off = smem_u32(&aux->bar_empty[0]) - bars;
    int slot = 0, used = 0;   // the next slot, slots before it
    uint32_t phase = 1;   // parity of the phase in which the slot's last contents are released
    uint32_t dst, bar;
    // the next slot: false where it is the other warp's, else it is free and its
    // bytes are counted
    bool ok = true;
    auto acquire = [&]() -> bool {
        const bool its = (used & 1) == part;
        bar = bars + slot * 8;
        dst = sRing + slot * T::SLOT;
        if (its) {
            ok = ok && mbar_wait(bar + empty_off, phase, wc, kErrWaitTimeout | kSiteLoadEmpty);
            if (!ok) return false;
            if (one) {
                trace_mark(tr, kTrLoad, slot, 0);
                mbar_arrive_expect_tx(bar, (uint32_t)T::SLOT);
            }
        }
        ++used;
        if (++slot == T::NSLOT) {
            slot = 0;
            phase ^= 1u;
        }
        __syncwarp();
        return its;
    };
    SpanItem s;
    for (int i = 0; ok && span_item(aux, i, wc, s); ++i) {
        if (s.m == 0) continue;
        const int plane = (a.cu_seqlens_k != nullptr ? 0 : s.b * a.Hkv) + s.hk;
        // where the lane's boxes of a block lie in the tensor map (past the span,
        // or no page: a plane that does not exist, which reads as zeros); v: of
        // block j, k: of j + 1
        int k_row[2] = {0, 0}, k_plane[2] = {0, 0}, v_row[2], v_plane[2];
#pragma unroll 1
        for (int j = -2; j < s.m && ok; ++j) {
            // page numbers are fetched a block ahead
            int n_row[2] = {0, 0}, n_plane[2] = {a.planes, a.planes};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int box = lane + 32 * e;
                const int xb = (s.kb + j + 2) * T::BN + (box << box_shift);
                if (box < boxes && xb < s.span) {
                    const int key = span_key(s, xb);
                    n_row[e] = s.k0 + key;
                    n_plane[e] = plane;
                    if (PAGED) {
                        const unsigned at = (unsigned)key / (unsigned)a.page_size;
                        const int page = a.block_table[(size_t)s.b * a.max_pages + at];
                        n_row[e] = key - (int)at * a.page_size;
                        n_plane[e] =
                            (unsigned)page < (unsigned)a.num_pages ? page * a.Hkv + s.hk : a.planes;
                    }
                }
            }
            if (j >= -1) {
                const int x0 = (s.kb + j) * T::BN;   // block j
                if (j + 1 < s.m) {
                    const int x1 = x0 + T::BN;
                    const bool in_boxes = PAGED || (MODE == kSpanWindow && x1 < s.head && x1 + T::BN > s.head);
#pragma unroll 1
                    for (int c = 0; c < T::KP && ok; ++c) {
                        if (!acquire()) continue;
                        if (in_boxes) {
#pragma unroll 1
                            for (int box = lane; box < boxes; box += 32) {
                                const uint32_t to = dst + ((uint32_t)(box << box_shift) << 7);
                                const int y = box < 32 ? k_row[0] : k_row[1];
                                const int z = box < 32 ? k_plane[0] : k_plane[1];
#pragma unroll
                                for (int q = 0; q < T::KCH; ++q) {
                                    const int col = (c * T::KCH + q) * 64;
                                    tma_load_3d(to + q * T::KCHUNK, &tm.k_box, col, y, z, bar);
                                }
                            }
                        } else if (one) {
                            const int row = s.k0 + span_key(s, x1);
#pragma unroll
                            for (int q = 0; q < T::KCH; ++q)
                                tma_load_3d(dst + q * T::KCHUNK, &tm.k, (c * T::KCH + q) * 64, row,
                                            plane, bar);
                        }
                    }
                }
                if (j >= 0) {
#pragma unroll 1
                    for (int h = 0; h < T::VP && ok; ++h) {
                        const int xv = x0 + h * T::VKEYS;
                        if (!acquire()) continue;
                        if (PAGED || (MODE == kSpanWindow && xv < s.head && xv + T::VKEYS > s.head)) {
#pragma unroll 1
                            for (int box = lane; box < boxes; box += 32) {
                                if (box >> vboxes_shift != h) continue;
                                const uint32_t to =
                                    dst + ((uint32_t)((box - (h << vboxes_shift)) << box_shift) << 7);
                                const int y = box < 32 ? v_row[0] : v_row[1];
                                const int z = box < 32 ? v_plane[0] : v_plane[1];
#pragma unroll
                                for (int q = 0; q < T::NCH; ++q)
                                    tma_load_3d(to + q * T::VCHUNK, &tm.v_box, q * 64, y, z, bar);
                            }
                        } else if (one) {
                            const int row = s.k0 + span_key(s, xv);
#pragma unroll
                            for (int q = 0; q < T::NCH; ++q)
                                tma_load_3d(dst + q * T::VCHUNK, &tm.v, q * 64, row, plane, bar);
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v_row[e] = k_row[e];
                v_plane[e] = k_plane[e];
                k_row[e] = n_row[e];
                k_plane[e] = n_plane[e];
            }
        }
    }
    // every copy issued must have landed before the CTA exits
    if (one) {
#pragma unroll 1
        for (int q = used > T::NSLOT ? used - T::NSLOT : 0; q < used; ++q) {
            if ((q & 1) != part) continue;
            mbar_wait_drain(bars + ring_slot<T>(q) * 8, ring_phase<T>(q), a.wait_limit_ns);
        }
    }
    __syncwarp();
}

// Whether the block of positions x0 on holds values that must be zeroed.
template <class T>
__device__ __forceinline__ bool span_zeroes(const SpanArgs& a, const SpanItem& s, int x0) {
    return s.end < x0 + T::BN || (x0 < s.gap && x0 + T::BN > a.first);
}

// MMA issue (one lane): S(J+1), then PV(J), as in the 256-key prefill kernel.
template <class T, int MODE>
__device__ void span_mma_role(const SpanArgs& a, SpanAux* aux, uint32_t tmem, uint32_t sQ,
                              uint32_t sRing, const WaitCtx& wc, unsigned long long* tr) {
    if (!elect_one()) {
        __syncwarp();
        return;
    }
    const uint32_t qd0 = sdesc_lo_sw128(sQ, 16);
    const uint32_t kd0 = sdesc_lo_sw128(sRing, 16);
    const uint32_t vd0 = sdesc_lo_sw128(sRing, T::VCHUNK);
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, T::BN, false, false);
    constexpr uint32_t idesc_v = idesc_bf16_f32(128, T::D_COLS, false, true);
    int p = 0;
    auto next_slot = [&](unsigned site) -> bool {
        if (!mbar_wait_lane(smem_u32(&aux->bar_full[ring_slot<T>(p)]), ring_phase<T>(p), wc,
                            kErrWaitTimeout | site))
            return false;
        tc_fence_after();
        return true;
    };
    auto slot_desc = [&](uint32_t d0) { return d0 + (uint32_t)((ring_slot<T>(p) * T::SLOT) >> 4); };
    auto release_slot = [&] {
        tc_commit(smem_u32(&aux->bar_empty[ring_slot<T>(p)]));
        ++p;
    };
    int J0 = 0, kq = 0;
    bool ok = true;
    SpanItem s;
    for (int i = 0; ok && span_item_lane(aux, i, wc, s); ++i) {
        const int n = s.m;
        mbar_arrive(smem_u32(&aux->bar_item_read[i % kItems]));
        if (n == 0) continue;
        if (!mbar_wait_lane(smem_u32(&aux->bar_q), (uint32_t)(kq & 1), wc,
                            kErrWaitTimeout | kSiteMmaQ))
            break;
        tc_fence_after();
#pragma unroll 1
        for (int j = -1; j < n && ok; ++j) {
            if (j + 1 < n) {   // S(J + 1)
                const int J = J0 + j + 1;
                trace_mark(tr, kTrMma, J, 0);
                // the softmax has read S(J) out of the buffer
                if (J > 0 &&
                    !mbar_wait_lane(smem_u32(&aux->bar_xm[(J - 1) & 1]),
                                    (uint32_t)(((J - 1) >> 1) & 1), wc,
                                    kErrWaitTimeout | kSiteMmaSfree)) {
                    ok = false;
                    break;
                }
                // the correction warps have the row maxima of S(J - 2), in whose
                // place those of S(J) will be written
                if (J > 1 &&
                    !mbar_wait_lane(smem_u32(&aux->bar_corrected[J & 1]),
                                    (uint32_t)(((J - 2) >> 1) & 1), wc,
                                    kErrWaitTimeout | kSiteMmaSfree)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                trace_mark(tr, kTrMma, J, 1);
#pragma unroll
                for (int c = 0; c < T::KP && ok; ++c) {
                    if (!next_slot(kSiteMmaK)) {
                        ok = false;
                        break;
                    }
                    trace_mark(tr, kTrMma, J, 2 + c);
                    const uint32_t kd = slot_desc(kd0), qd = qd0 + c * kstep_off(4 * T::KCH);
#pragma unroll
                    for (int kin = 0; kin < 4 * T::KCH; ++kin)
                        umma_ss_lo(tmem + T::S_COL, qd + kstep_off(kin),
                                   kd + (uint32_t)(((kin >> 2) * T::KCHUNK + (kin & 3) * 32) >> 4),
                                   idesc_s, (c | kin) > 0 ? 1u : 0u);
                    release_slot();
                }
                if (!ok) break;
                tc_commit(smem_u32(&aux->bar_s_full));
                if (j + 2 == n) tc_commit(smem_u32(&aux->bar_qfree));   // Q no longer read
            }
            if (j < 0) continue;
            const int J = J0 + j;   // PV(J)
            if (!mbar_wait_lane(smem_u32(&aux->bar_p_ready[J & 1]), (uint32_t)((J >> 1) & 1), wc,
                                kErrWaitTimeout | kSiteMmaP)) {
                ok = false;
                break;
            }
            trace_mark(tr, kTrMma, J, 4);
            // O rebased, values zeroed (the first block of a segment needs
            // neither as a rule, and the correction warps may still be busy with
            // the last segment's end)
            if ((j > 0 || span_zeroes<T>(a, s, s.kb * T::BN)) &&
                !mbar_wait_lane(smem_u32(&aux->bar_corrected[J & 1]), (uint32_t)((J >> 1) & 1), wc,
                                kErrWaitTimeout | kSiteMmaP)) {
                ok = false;
                break;
            }
            if (j == 0 && kq > 0 &&   // the previous segment's O has been read out
                !mbar_wait_lane(smem_u32(&aux->bar_odrained), (uint32_t)((kq - 1) & 1), wc,
                                kErrWaitTimeout | kSiteMmaOdrained)) {
                ok = false;
                break;
            }
            tc_fence_after();
            trace_mark(tr, kTrMma, J, 5);
#pragma unroll
            for (int hh = 0; hh < T::VP; ++hh) {
                if (!next_slot(kSiteMmaV)) {
                    ok = false;
                    break;
                }
                trace_mark(tr, kTrMma, J, 6 + hh);
                const uint32_t vd = slot_desc(vd0);
                const uint32_t pcol = tmem + T::P_COL + (uint32_t)(hh * (T::VKEYS / 2));
#pragma unroll
                for (int kk = 0; kk < T::VKEYS / 16; ++kk)
                    umma_ts_lo(tmem + T::O_COL, pcol + kk * 8, vd + (uint32_t)((kk * 2048) >> 4),
                               idesc_v, (j | hh | kk) > 0 ? 1u : 0u);
                release_slot();
            }
            if (ok) tc_commit(smem_u32(&aux->bar_pv_done[J & 1]));
        }
        J0 += n;
        ++kq;
    }
    const uint32_t drain = smem_u32(&aux->bar_drain);
    tc_commit(drain);
    mbar_wait_drain(drain, 0, a.wait_limit_ns);
    __syncwarp();
}

// Visibility of the 32 keys from offset o after node 0 on (o < 0: keys before
// the tree, all seen): bits of the row's mask words; keys past the last node
// are not there.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* words, int nodes, int o) {
    auto word = [&](int w) -> uint32_t {
        if (w < 0) return 0xffffffffu;
        const int rest = nodes - w * 32;
        if (rest <= 0) return 0u;
        const uint32_t x = words[w];
        return rest < 32 ? x & ((1u << rest) - 1u) : x;
    };
    const int w = o >> 5;   // (rounds down)
    return __funnelshift_r(word(w), word(w + 1), (uint32_t)o & 31u);
}

// Softmax of one segment by warpgroup h (keys [HK h, HK h + HK) of every
// block; thread = row); see wide_softmax_unit.
template <class T, int MODE>
__device__ bool span_softmax_segment(int h, const SpanArgs& a, const SpanItem& s, int gp, SpanAux* aux,
                                     uint32_t tmem, const WaitCtx& wc, int J0, int kq,
                                     unsigned long long* tr) {
    constexpr int HK = T::HK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((warp & 3) != 0 || lane != 0) tr = nullptr;
    const int trole = h == 0 ? kTrSoftmax0 : kTrSoftmax1;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // what the row sees: a tree's node its mask words from position node0 on,
    // before it everything; a window's row the positions below fa and [lo, lim]
    // (rows that do not exist: as some row)
    const uint32_t* words = nullptr;
    int node0 = 0, fa = 0, lo = 0, lim = 0;
    if constexpr (MODE == kSpanTree) {
        words = a.tree_mask + s.b * a.tree_stride +
                (long long)((s.tile * T::BM + r) % a.Sq) * a.tree_words;
        node0 = s.keys - s.rows;
    } else {
        const int p = s.tile * a.P + gp + s.keys - s.rows;   // the row's key
        const int last = a.causal ? min(s.keys - 1, p) : s.keys - 1;
        fa = min(a.first, last + 1);
        lim = last - s.skip;
        lo = max(p - a.window + 1 - s.skip, s.head);
    }
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    for (int j = 0; j < s.m; ++j) {
        const int J = J0 + j;
        const int sb = J & 1;
        const uint32_t par = (uint32_t)((J >> 1) & 1);
        uint32_t u[HK / 32][32];
        if (!mbar_wait(smem_u32(&aux->bar_s_full), (uint32_t)(J & 1), wc,
                       kErrWaitTimeout | kSiteSmS))
            return false;
        trace_mark(tr, trole, J, 0);
        tc_fence_after();
        const int x0 = (s.kb + j) * T::BN + h * HK;   // first position of the half
        const bool masked = MODE == kSpanTree ? x0 + HK > node0   // the nodes' own keys, or past
                                              : (x0 < lo || x0 + HK - 1 > lim) && x0 + HK > fa;
        if (__any_sync(0xffffffffu, masked)) {
            // a block at the border: scores that the row does not see become
            // -inf in tensor memory, 32 at a time (a loop of a kilobyte of
            // instructions; selects on the 128 registers below take five, which
            // the instruction cache has no room for; with the scheduler warp this
            // took a window's prompts from 123 to 99 us)
#pragma unroll 1
            for (int q = 0; q < HK / 32; ++q) {
                const int xq = x0 + 32 * q;
                uint32_t vis, w[32];
                if constexpr (MODE == kSpanTree)
                    vis = tree_bits(words, s.rows, xq - node0);
                else
                    vis = low_bits(fa - xq) | (low_bits(lim + 1 - xq) & ~low_bits(lo - xq));
                if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
                const uint32_t col = lane_base + T::S_COL + h * HK + q * 32;
                tmem_ld32(col, w);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) w[c] = ((vis >> c) & 1u) ? w[c] : 0xff800000u;
                tmem_st32(col, w);
            }
            tmem_wait_st();
        }
        float mq[HK / 64];
#pragma unroll
        for (int q = 0; q < HK / 64; ++q)
            mq[q] = tmem_ld64_max(lane_base + T::S_COL + h * HK + q * 64,
                                  *reinterpret_cast<uint32_t(*)[2][32]>(&u[2 * q][0]));
        tmem_wait_ld();
        trace_mark(tr, trole, J, 1);
        float x[HK];
#pragma unroll
        for (int c = 0; c < HK; ++c) x[c] = __uint_as_float(u[c >> 5][c & 31]);
        const float mx_h = fmaxf(mq[0], mq[HK / 64 - 1]);
        trace_mark(tr, trole, J, 2);
        aux->xm[sb][h][r] = mx_h;
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_xm[sb]));
        if (!mbar_wait(smem_u32(&aux->bar_xm[sb]), par, wc, kErrWaitTimeout | kSiteSmXm))
            return false;
        trace_mark(tr, trole, J, 3);
        const float m_new = fmaxf(m_run, fmaxf(mx_h, aux->xm[sb][h ^ 1][r]) * sl2);
        float alpha = 1.f;
        if (m_new > m_run + kRescaleThreshold) {
            alpha = ex2_approx(m_run - m_new);   // 0 when m_run = -inf
            m_run = m_new;
        }
        const float base = (m_run == -INFINITY) ? 0.f : m_run;
        const float2 sl2x2 = make_float2(sl2, sl2);
        const float2 nbase = make_float2(-base, -base);
        float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        uint32_t pk[HK / 64][32];
        const uint32_t pcol = lane_base + T::P_COL + h * (HK / 2);
#pragma unroll
        for (int c = 0; c < HK / 2; ++c) {
            const float2 xv = ffma2(make_float2(x[2 * c], x[2 * c + 1]), sl2x2, nbase);
            const float2 pv = make_float2(ex2_approx(xv.x), ex2_approx(xv.y));
            rs[c & 3] = fadd2(rs[c & 3], pv);
            pk[c >> 5][c & 31] = pack_bf16x2(pv.x, pv.y);
            if (c == 31) trace_mark(tr, trole, J, 4);
            if (c == 31) {   // P(J) overwrites P(J-1) once PV(J-1) has read it
                if (J > 0) {
                    if (!mbar_wait(smem_u32(&aux->bar_pv_done[(J - 1) & 1]),
                                   (uint32_t)(((J - 1) >> 1) & 1), wc,
                                   kErrWaitTimeout | kSiteSmPv))
                        return false;
                    tc_fence_after();
                }
                trace_mark(tr, trole, J, 5);
                tmem_st32(pcol, pk[0]);
            }
        }
        const float2 rs01 = fadd2(rs[0], rs[1]), rs23 = fadd2(rs[2], rs[3]);
        const float2 rsum = fadd2(rs01, rs23);
        l_run = fmaf(l_run, alpha, rsum.x + rsum.y);
        if constexpr (HK == 128) tmem_st32(pcol + 32, pk[1]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_p_ready[sb]));
        trace_mark(tr, trole, J, 6);
    }
    // the previous segment's statistics must have been read
    if (kq > 0 && !mbar_wait(smem_u32(&aux->bar_odrained), (uint32_t)((kq - 1) & 1), wc,
                             kErrWaitTimeout | kSiteSmOdrained))
        return false;
    aux->mb_l[h][r] = l_run;
    mbar_arrive_warp(smem_u32(&aux->bar_fin));
    return true;
}

// Sum and max (log2 units) of a row with its head's sink logit, one more term
// without a value.  Returns what O (in basis m) is multiplied by.
// (sink: the logit of the row's head, -inf without sinks).
__device__ __forceinline__ float span_normaliser(float sink, float& l, float& m) {
    float scale = 1.f;
    if (sink != -INFINITY) {
        const float sg = sink * kLog2e;
        const float m2 = fmaxf(m, sg);
        if (m2 == -INFINITY) return 0.f;
        scale = (m == -INFINITY) ? 0.f : ex2_approx(m - m2);
        l = l * scale + ex2_approx(sg - m2);
        m = m2;
    }
    return l > 0.f ? scale / l : 0.f;
}

// Writes the calling warp's 32 rows of O (times inv_l, bf16; have false:
// zeros) to the rows o_row of each lane's own row, 32 columns at a time through
// the warp's 2 KB staging area: a lane writes its row's 64 bytes in 16-byte
// granules, XOR-ed with the row against bank conflicts, and each store
// instruction writes 64 bytes of 8 rows.
template <class T>
__device__ __forceinline__ void span_store_o(uint32_t lane_base, const SpanArgs& a, bool have,
                                             bool real, size_t o_row, float inv_l,
                                             uint32_t stage, uint32_t drained) {
    const int lane = threadIdx.x & 31;
    if (!have) {   // a unit without keys
        if (real)
#pragma unroll 1
            for (int c = 0; c < T::D_COLS; c += 8)
                *reinterpret_cast<uint4*>(a.o + o_row * T::D_COLS + c) = make_uint4(0, 0, 0, 0);
        return;
    }
    const unsigned rows = __ballot_sync(0xffffffffu, real);
    uint16_t* to[4];   // the rows (and columns) that this lane stores
#pragma unroll
    for (int k = 0; k < 4; ++k)
        to[k] = a.o +
                (size_t)__shfl_sync(0xffffffffu, (unsigned long long)o_row, k * 8 + (lane >> 2)) *
                    T::D_COLS +
                (lane & 3) * 8;
    uint32_t v[32];
    tmem_ld32(lane_base + T::O_COL, v);
#pragma unroll 1
    for (int c0 = 0; c0 < T::D_COLS; c0 += 32) {
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                                   make_float2(inv_l, inv_l), make_float2(0.f, 0.f));
            pk[e] = pack_bf16x2(y.x, y.y);
        }
        if (c0 + 32 < T::D_COLS) {
            tmem_ld32(lane_base + T::O_COL + c0 + 32, v);   // lands meanwhile
        } else {   // O is free for the next segment
            tc_fence_before();
            mbar_arrive_warp(drained);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stage + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)),
                         "r"(pk[4 * g]), "r"(pk[4 * g + 1]), "r"(pk[4 * g + 2]), "r"(pk[4 * g + 3])
                         : "memory");
        __syncwarp();
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int rr = k * 8 + (lane >> 2), g = lane & 3;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[k].x), "=r"(x[k].y), "=r"(x[k].z), "=r"(x[k].w)
                         : "r"(stage + rr * 64 + ((g ^ ((rr >> 1) & 3)) << 4))
                         : "memory");
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((rows >> (k * 8 + (lane >> 2))) & 1u)
                *reinterpret_cast<uint4*>(to[k] + c0) = x[k];
        __syncwarp();
    }
}

// Correction of one segment (thread = row): rebases O when the running max
// moved; at its end writes O and LSE of a whole unit, or the piece's
// unnormalised O, max and sum.
template <class T, int MODE>
__device__ bool span_correction_segment(const SpanArgs& a, const SpanItem& s, int g, int gp, SpanAux* aux,
                                        uint32_t tmem, uint32_t sRing, const WaitCtx& wc, int J0,
                                        int kq, int p0, unsigned long long* tr) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((warp & 3) != 0 || lane != 0) tr = nullptr;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY;
    for (int j = 0; j < s.m; ++j) {
        const int J = J0 + j;
        const int sb = J & 1;
        if (!mbar_wait(smem_u32(&aux->bar_xm[sb]), (uint32_t)((J >> 1) & 1), wc,
                       kErrWaitTimeout | kSiteCorrMbox))
            return false;
        const float m_new = fmaxf(m_run, fmaxf(aux->xm[sb][0][r], aux->xm[sb][1][r]) * sl2);
        float alpha = 1.f;
        if (m_new > m_run + kRescaleThreshold) {
            alpha = ex2_approx(m_run - m_new);
            m_run = m_new;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha < 1.f)) {
            if (!mbar_wait(smem_u32(&aux->bar_pv_done[(J - 1) & 1]),
                           (uint32_t)(((J - 1) >> 1) & 1), wc, kErrWaitTimeout | kSiteCorrPv))
                return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < T::D_COLS / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(lane_base + T::O_COL + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                tmem_st32(lane_base + T::O_COL + c * 32, v);
            }
            tmem_wait_st();
        }
        // value rows past the sequence's end, and (decode) those between the
        // first keys and the window, may hold anything, and zero times a
        // non-finite value would poison O: zeroed here, before PV(J) is let go
        const int x0 = (s.kb + j) * T::BN;
        if (span_zeroes<T>(a, s, x0)) {
            // (V_j's slots come after K_{j+1}'s)
            int pv = p0 + j * (T::KP + T::VP) + (j + 1 < s.m ? 2 : 1) * T::KP;
            // (the slots' contents before V_j are at most V_{j-1}: past that, full
            // means V_j)
            bool landed = j == 0 || mbar_wait(smem_u32(&aux->bar_pv_done[(J - 1) & 1]),
                                              (uint32_t)(((J - 1) >> 1) & 1), wc,
                                              kErrWaitTimeout | kSiteCorrPv);
#pragma unroll 1
            for (int hh = 0; hh < T::VP && landed; ++hh, ++pv) {
                const int xv = x0 + hh * T::VKEYS;   // first position of the slot
                landed = mbar_wait(smem_u32(&aux->bar_full[ring_slot<T>(pv)]), ring_phase<T>(pv), wc,
                                   kErrWaitTimeout | kSiteLoadTail);
                const uint32_t slot = sRing + ring_slot<T>(pv) * T::SLOT;
#pragma unroll 1
                for (int g = r; g < T::VKEYS * 8; g += T::BM) {
                    const int x = xv + (g >> 3);
                    if (x < s.end && (x < a.first || x >= s.gap)) continue;
#pragma unroll 1
                    for (int q = 0; q < T::NCH; ++q)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         slot + q * T::VCHUNK + g * 16),
                                     "r"(0)
                                     : "memory");
                }
            }
            if (!landed) return false;
            fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_corrected[sb]));
    }
    // (what the end needs from memory, while the last PV runs)
    int head;
    size_t o_row, lse_at;
    const bool real =
        span_row<T, MODE>(a, s.cap, s.q0, s.b, s.hk, s.tile, r, g, gp, head, o_row, lse_at);
    const float sink = a.sinks != nullptr && real ? a.sinks[head] : -INFINITY;
    float l = 0.f, m = m_run;
    const int Jl = J0 + s.m - 1;
    if (s.m > 0) {   // (else a unit, or a piece of one, without keys)
        if (!mbar_wait(smem_u32(&aux->bar_fin), (uint32_t)(kq & 1), wc,
                       kErrWaitTimeout | kSiteEpiMbox))
            return false;
        l = aux->mb_l[0][r] + aux->mb_l[1][r];
        if (!mbar_wait(smem_u32(&aux->bar_pv_done[Jl & 1]), (uint32_t)((Jl >> 1) & 1), wc,
                       kErrWaitTimeout | kSiteEpiPv))
            return false;
        tc_fence_after();
        trace_mark(tr, kTrCorr, Jl, 0);
    }
    const uint32_t drained = smem_u32(&aux->bar_odrained);
    if (s.n < s.nb) {   // a piece
        const int slot = 2 * (int)blockIdx.x + (s.index > 0);
        float4* po = reinterpret_cast<float4*>(a.part_o + (size_t)slot * (T::D_COLS * T::BM));
#pragma unroll 1
        for (int c64 = 0; c64 < (s.m > 0 ? T::D_COLS / 64 : 0); ++c64) {
            uint32_t v[2][32];
            tmem_ld64(lane_base + T::O_COL + c64 * 64, v);
            tmem_wait_ld();
            if (c64 == T::D_COLS / 64 - 1) {
                tc_fence_before();
                mbar_arrive_warp(drained);
            }
            if (!real) continue;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const uint32_t* x = &v[q >> 3][4 * (q & 7)];
                po[(size_t)(c64 * 16 + q) * T::BM + r] =
                    make_float4(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]),
                                __uint_as_float(x[3]));
            }
        }
        float* ml = a.part_ml + (size_t)slot * 2 * T::BM;
        ml[r] = m;
        ml[T::BM + r] = l;
        if (r == 0) a.head[slot] = make_int4(s.b, s.u, s.n, s.kb == 0 ? s.nb : 0);
    } else {
        const float inv_l = span_normaliser(sink, l, m);
        span_store_o<T>(lane_base, a, s.m > 0, real, o_row, inv_l,
                        sRing + T::SMEM_RING + T::SMEM_AUX + (warp & 3) * T::STAGE, drained);
        if (real) a.lse[lse_at] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
    }
    if (s.m > 0) trace_mark(tr, kTrCorr, Jl, 1);
    return true;
}

template <int D, int MODE, bool PAGED>
__global__ void __launch_bounds__(SpanTraits<D>::THREADS, 1)
    span_kernel(const __grid_constant__ SpanMaps tm, const SpanArgs a) {
    using T = SpanTraits<D>;
    static_assert(sizeof(SpanAux) <= T::SMEM_AUX && T::NSLOT <= kSpanSlots, "auxiliary block");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sRing = sQ + T::SMEM_Q;
    auto* aux = reinterpret_cast<SpanAux*>(smem_raw + (sQ - raw) + T::SMEM_Q + T::SMEM_RING);
    const int warp = threadIdx.x >> 5;
    const int wg = warp >> 2;
    dependents_may_start();
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&aux->bar_q), 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(smem_u32(&aux->bar_item[i]), 1);
            mbar_init(smem_u32(&aux->bar_item_read[i]), 15);   // warps that read it
        }
        for (int i = 0; i < T::NSLOT; ++i) {
            mbar_init(smem_u32(&aux->bar_full[i]), 1);
            mbar_init(smem_u32(&aux->bar_empty[i]), 1);
        }
        mbar_init(smem_u32(&aux->bar_s_full), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&aux->bar_xm[i]), 8);
            mbar_init(smem_u32(&aux->bar_p_ready[i]), 8);
            mbar_init(smem_u32(&aux->bar_corrected[i]), 4);
            mbar_init(smem_u32(&aux->bar_pv_done[i]), 1);
        }
        mbar_init(smem_u32(&aux->bar_fin), 8);
        mbar_init(smem_u32(&aux->bar_qfree), 1);
        mbar_init(smem_u32(&aux->bar_odrained), 4);
        mbar_init(smem_u32(&aux->bar_drain), 1);
        aux->abort_flag = 0;
        aux->start_b = 0;
        aux->start_off = 0;
        mbar_fence_init();
    }
    if (warp == T::MMA_WARP) {
        tmem_alloc(smem_u32(&aux->tmem_base), T::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == T::LOAD_WARP && (threadIdx.x & 31) == 0) {
        tma_prefetch_desc(&tm.q);
        tma_prefetch_desc(PAGED ? &tm.k_box : &tm.k);
        tma_prefetch_desc(PAGED ? &tm.v_box : &tm.v);
    }
    wait_for_previous();   // (what is above overlaps the kernel before)
    if (threadIdx.x == 0)
        a.head[2 * blockIdx.x] = a.head[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = aux->tmem_base;
    const WaitCtx wc{smem_u32(&aux->abort_flag), (uint32_t)a.wait_limit_ns, a.err_word};
    if (FA_PREFILL_TRACE && a.trace != nullptr && (int)blockIdx.x == a.trace_block && threadIdx.x == 0)
        trace_mark(a.trace, kTrCorr, 250, 0);
    unsigned long long* tr =
        FA_PREFILL_TRACE && a.trace != nullptr && (int)blockIdx.x == a.trace_block ? a.trace : nullptr;
    if (wg < 2) {
        setmaxnreg_inc<T::SOFTMAX_REGS>();
        int J0 = 0, kq = 0;
        const int gp = MODE == kSpanWindow ? (int)(threadIdx.x & 127) % a.P : 0;
        SpanItem s;
        for (int i = 0; span_item(aux, i, wc, s); ++i) {
            if (s.m == 0) continue;
            if (!span_softmax_segment<T, MODE>(wg, a, s, gp, aux, tmem, wc, J0, kq, tr)) break;
            J0 += s.m;
            ++kq;
        }
    } else if (wg == T::CORR_WG) {
        setmaxnreg_dec<T::CORR_REGS>();
        int J0 = 0, kq = 0;
        const int g = MODE == kSpanWindow ? (int)(threadIdx.x & 127) / a.P : 0;
        const int gp = MODE == kSpanWindow ? (int)(threadIdx.x & 127) % a.P : 0;
        SpanItem s;
        for (int i = 0; span_item(aux, i, wc, s); ++i) {
            if (!span_correction_segment<T, MODE>(a, s, g, gp, aux, tmem,
                                                  sRing, wc, J0, kq, J0 * (T::KP + T::VP), tr))
                break;
            J0 += s.m;
            kq += s.m > 0;
        }
    } else {
        setmaxnreg_dec<T::OTHER_REGS>();
        if (warp == T::MMA_WARP)
            span_mma_role<T, MODE>(a, aux, tmem, sQ, sRing, wc, tr);
        else if (warp == T::ITEM_WARP)
            span_item_role<T, MODE>(tm, a, aux, sQ, wc);
        else if (warp == T::LOAD_WARP || warp == T::LOAD2_WARP)
            span_load_role<T, MODE, PAGED>(warp == T::LOAD_WARP ? 0 : 1, tm, a, aux, sRing, wc, tr);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == T::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, T::TMEM_COLS);
    }
}

// Merges the pieces of the unit that starts in CTA blockIdx.x of the split
// kernel and goes on in the next ones of its place in the groups (16 columns
// per CTA here, thread = row).
template <int D, int MODE>
__global__ void __launch_bounds__(128) span_combine_kernel(const SpanArgs a) {
    using T = SpanTraits<D>;
    dependents_may_start();
    wait_for_previous();
    const int r = threadIdx.x, c16 = blockIdx.y, G = gridDim.x;
    const int step = a.group_ctas;
    // (what the pieces' addresses need, in one latency)
    int slot = 2 * blockIdx.x;
    const int4 h0 = a.head[slot], h1 = a.head[slot + 1];
    const int quota = a.head[2 * G].x;
    const bool second = !(h0.z > 0 && h0.w > h0.z);
    const int4 hd = second ? h1 : h0;
    slot += second;
    if (!(hd.z > 0 && hd.w > hd.z)) return;
    const int b = hd.x, u = hd.y, nb = hd.w;
    if ((unsigned)b >= (unsigned)a.B) return;
    const SpanSeq seq = span_seq<MODE>(a, b);   // (its loads run with the pieces')
    float M = -INFINITY, L = 0.f;
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    // the pieces: hd.z blocks here, then a full CTA's share each, as the first
    // segments of the next CTAs (their number is known without reading them,
    // so that four at a time are in flight)
    const int pieces = min(1 + (nb - hd.z + quota - 1) / max(quota, 1), (G - (int)blockIdx.x + step - 1) / step);
    for (int k0 = 0; k0 < pieces; k0 += 4) {
        float mk[4], lk[4];
        float4 v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = min(k0 + e, pieces - 1);
            const int at = k == 0 ? slot : 2 * ((int)blockIdx.x + k * step);
            const float* ml = a.part_ml + (size_t)at * 2 * T::BM;
            const float4* po = reinterpret_cast<const float4*>(a.part_o + (size_t)at * (D * T::BM));
            mk[e] = k0 + e < pieces ? ml[r] : -INFINITY;
            lk[e] = ml[T::BM + r];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[e][q] = po[(size_t)(c16 * 4 + q) * T::BM + r];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (mk[e] == -INFINITY) continue;   // no keys, or no piece
            const float m2 = fmaxf(M, mk[e]);
            const float sc = (M == -INFINITY) ? 0.f : ex2_approx(M - m2);
            const float wk = ex2_approx(mk[e] - m2);
            M = m2;
            L = fmaf(L, sc, wk * lk[e]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[4 * q + 0] = fmaf(acc[4 * q + 0], sc, wk * v[e][q].x);
                acc[4 * q + 1] = fmaf(acc[4 * q + 1], sc, wk * v[e][q].y);
                acc[4 * q + 2] = fmaf(acc[4 * q + 2], sc, wk * v[e][q].z);
                acc[4 * q + 3] = fmaf(acc[4 * q + 3], sc, wk * v[e][q].w);
            }
        }
    }
    if ((unsigned)u >= (unsigned)span_units<MODE>(a, seq)) return;
    const int groups = span_groups<MODE>(a, seq);
    const int tile = u % groups * step + (int)blockIdx.x % step;
    int h;
    size_t o_row, lse_at;
    const int g = MODE == kSpanWindow ? r / a.P : 0, gp = MODE == kSpanWindow ? r % a.P : 0;
    if (!span_row<T, MODE>(a, seq.cap, seq.q0, b, u / groups, tile, r, g, gp, h, o_row, lse_at))
        return;
    const float inv_l = span_normaliser(a.sinks != nullptr ? a.sinks[h] : -INFINITY, L, M);
    uint4* dst = reinterpret_cast<uint4*>(a.o + o_row * D + c16 * 16);
#pragma unroll
    for (int g = 0; g < 2; ++g)
        dst[g] = make_uint4(pack_bf16x2(acc[8 * g + 0] * inv_l, acc[8 * g + 1] * inv_l),
                            pack_bf16x2(acc[8 * g + 2] * inv_l, acc[8 * g + 3] * inv_l),
                            pack_bf16x2(acc[8 * g + 4] * inv_l, acc[8 * g + 5] * inv_l),
                            pack_bf16x2(acc[8 * g + 6] * inv_l, acc[8 * g + 7] * inv_l));
    if (c16 == 0) a.lse[lse_at] = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
}

template <int D, int MODE, bool PAGED>
cudaError_t launch_span_mode(const SpanLaunch& p, cudaStream_t s) {
    using T = SpanTraits<D>;
    cudaError_t e = cudaFuncSetAttribute(span_kernel<D, MODE, PAGED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         T::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    e = launch_dependent(span_kernel<D, MODE, PAGED>, dim3(p.ctas), dim3(T::THREADS), T::SMEM_TOTAL,
                         s, p.maps, p.args);
    if (e != cudaSuccess) return e;
    return launch_dependent(span_combine_kernel<D, MODE>, dim3(p.ctas, D / 16), dim3(T::BM), 0, s,
                            p.args);
}

template <int D>
cudaError_t launch_span_impl(const SpanLaunch& p, cudaStream_t s) {
    const bool paged = p.args.block_table != nullptr;
    if (p.args.tree_mask == nullptr)
        return paged ? launch_span_mode<D, kSpanWindow, true>(p, s)
                     : launch_span_mode<D, kSpanWindow, false>(p, s);
    return paged ? launch_span_mode<D, kSpanTree, true>(p, s)
                 : launch_span_mode<D, kSpanTree, false>(p, s);
}

}  // namespace

cudaError_t launch_span(const SpanLaunch& p, int head_dim, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_span_impl<64>(p, s);
        case 128: return launch_span_impl<128>(p, s);
        case 256: return launch_span_impl<256>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
