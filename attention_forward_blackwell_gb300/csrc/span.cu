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
// once (one tile after the other, a 64-node tree of 8 heads read them three
// times and took 117 us instead of %GROUPED%).
//
// Inside a CTA: the roles and barriers of the 256-key prefill kernel (see
// prefill_wide.cuh), which this one follows: S = Q K^T of the next block is
// issued once the softmax has read this block's scores into registers; two
// warpgroups share each row's softmax; P has tensor memory of its own.  Key
// blocks are 256 keys (one N = 256 score instruction per 16 head dims), 128 at
// head_dim 256, whose 256 O columns leave no room for more.
//
// Boxes (BOXED): a box of the tensor maps is as many rows as always lie
// together -- of one page, of one side of the window's gap -- one lane of the
// producer per box, page numbers fetched a block ahead.
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
    static constexpr int D_COLS = D;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t S_COL = 0;
    static constexpr uint32_t P_COL = BN;           // BN / 2 columns of bf16 pairs
    static constexpr uint32_t O_COL = D == 256 ? 256 : 384;
    static constexpr int SMEM_Q = QTILE;
    static constexpr int SMEM_RING = NSLOT * SLOT;
    static constexpr int SMEM_AUX = 8192;
    static constexpr int SMEM_TOTAL = 1024 + SMEM_Q + SMEM_RING + SMEM_AUX;
    static constexpr uint32_t SOFTMAX_REGS = 168, CORR_REGS = 96, OTHER_REGS = 80;
    static_assert(8 * 32 * SOFTMAX_REGS + 4 * 32 * CORR_REGS + 4 * 32 * OTHER_REGS <= THREADS * 128,
                  "register split exceeds the launch allocation");
    static_assert(KP * KCH == NCH && VP * VKEYS == BN, "slots must cover a block");
    static_assert(P_COL + BN / 2 <= O_COL && O_COL + D <= TMEM_COLS, "S, P and O must fit");
    static_assert(SMEM_TOTAL <= 232448, "shared memory per CTA exceeds the sm_103 limit");
};

constexpr int kSpanSlots = 6;

struct SpanAux {
    uint64_t bar_q;
    uint64_t bar_full[kSpanSlots];
    uint64_t bar_empty[kSpanSlots];
    uint64_t bar_s_full;
    uint64_t bar_xm[2];
    uint64_t bar_p_ready[2];
    uint64_t bar_pv_done[2];
    uint64_t bar_fin;
    uint64_t bar_qfree;
    uint64_t bar_odrained;
    uint64_t bar_tail;
    uint64_t bar_drain;
    uint32_t tmem_base;
    int abort_flag;
    int start_b;              // the CTA's first unit: batch entry,
    int start_n;              // (the CTA's blocks in all)
    long long start_off;      // and blocks of that entry's units before its own
    long long scan[16];
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
// Units of a batch entry, and the key blocks each counts for on the line: a
// bound for a window (its tiles near the start have fewer), one at least, so
// that rows without keys are written too.
template <int MODE>
__device__ __forceinline__ int span_units(const SpanArgs& a, const SpanSeq& q) {
    if (q.cap == 0) return 0;
    return a.Hkv * (MODE == kSpanTree ? a.tile_groups : (q.cap + a.P - 1) / a.P);
}
template <class T, int MODE>
__device__ __forceinline__ int span_blocks(const SpanArgs& a, const SpanSeq& q) {
    int keys = q.keys;
    if (MODE == kSpanWindow && a.causal) keys = min(keys, a.window_keys);
    return max(1, (keys + T::BN - 1) / T::BN);
}

// The CTA's segments in turn: `n` consecutive key blocks from kb on of a
// unit with nb blocks, m of them real.
struct SpanSeg {
    int b, u;        // batch entry, unit of it
    int kb, n, nb;
    int left;        // blocks of the CTA after this segment
    int index;       // segments before it
    SpanSeq q;
    int units;       // of the batch entry
    // the unit's tile (see span_geometry)
    int hk, tile, m;
    int head, skip;  // position x of its axis: key x below head, key x + skip from there on
    int span;        // positions that a row may see
    int end;         // position of the sequence's end
};

__device__ __forceinline__ int span_key(const SpanSeg& s, int x) {
    return x < s.head ? x : x + s.skip;
}

// The tile of unit s.u and the axis of its keys.
template <class T, int MODE>
__device__ __forceinline__ void span_geometry(const SpanArgs& a, SpanSeg& s) {
    s.head = s.skip = 0;
    if constexpr (MODE == kSpanTree) {
        s.hk = s.u / a.tile_groups;
        s.tile = (s.u % a.tile_groups) * a.group_ctas + (int)blockIdx.x % a.group_ctas;
        s.span = s.end = s.tile < a.tiles ? s.q.keys : 0;
    } else {
        const int tiles = (s.q.cap + a.P - 1) / a.P;
        s.hk = s.u / tiles;
        s.tile = s.u % tiles;
        const int off = s.q.keys - s.q.rows;   // bottom-right alignment
        const int p0 = s.tile * a.P + off;     // keys of the tile's first and last row
        const int p1 = min(s.tile * a.P + a.P, s.q.cap) - 1 + off;
        const int last = a.causal ? min(s.q.keys - 1, p1) : s.q.keys - 1;
        const int base = max(0, p0 - a.window + 1) / a.box * a.box;
        if (a.head_keys < base) {
            s.head = a.head_keys;
            s.skip = base - s.head;
        }
        s.span = max(0, last + 1 - s.skip);
        s.end = s.q.keys - s.skip;
    }
    const int real = (s.span + T::BN - 1) / T::BN;
    s.m = max(0, min(s.kb + s.n, real) - s.kb);
}

template <class T, int MODE>
__device__ __forceinline__ bool span_first(const SpanArgs& a, const SpanAux* aux, SpanSeg& s) {
    s.left = aux->start_n;
    if (s.left <= 0) return false;
    s.b = aux->start_b;
    s.q = span_seq<MODE>(a, s.b);
    s.units = span_units<MODE>(a, s.q);
    s.nb = span_blocks<T, MODE>(a, s.q);
    s.u = (int)(aux->start_off / s.nb);
    s.kb = (int)(aux->start_off % s.nb);
    s.n = min(s.nb - s.kb, s.left);
    s.left -= s.n;
    s.index = 0;
    span_geometry<T, MODE>(a, s);
    return true;
}
template <class T, int MODE>
__device__ __forceinline__ bool span_next(const SpanArgs& a, SpanSeg& s) {
    if (s.left <= 0) return false;
    s.kb = 0;
    if (++s.u == s.units) {
        s.u = 0;
        do {
            if (++s.b >= a.B) return false;   // (never: `left` counts blocks that are there)
            s.q = span_seq<MODE>(a, s.b);
            s.units = span_units<MODE>(a, s.q);
        } while (s.units == 0);
        s.nb = span_blocks<T, MODE>(a, s.q);
    }
    s.n = min(s.nb, s.left);
    s.left -= s.n;
    ++s.index;
    span_geometry<T, MODE>(a, s);
    return true;
}

// Tile row r: its query head, position (node), and index among the rows of O
// (the LSE's too, but of packed tensors); whether it is a row of the sequence.
template <class T, int MODE>
__device__ __forceinline__ bool span_row(const SpanArgs& a, const SpanSeq& q, int b, int hk,
                                         int tile, int r, int& h, int& pos, size_t& o_row,
                                         size_t& lse_at) {
    bool real;
    if constexpr (MODE == kSpanTree) {
        const int row = tile * T::BM + r;
        h = hk * a.group + row / a.Sq;
        pos = row % a.Sq;
        real = row < a.group * a.Sq && pos < q.cap;
    } else {
        const int g = r / a.P;
        h = hk * a.group + g;
        pos = tile * a.P + r % a.P;
        real = g < a.group && pos < q.cap;
        if (a.cu_seqlens_q != nullptr) {
            o_row = (size_t)(q.q0 + pos) * a.Hq + h;
            lse_at = (size_t)h * a.total_q + q.q0 + pos;
            return real;
        }
    }
    o_row = lse_at = ((size_t)b * a.Hq + h) * a.Sq + pos;
    return real;
}

// Places the CTA on the line of blocks (all threads): the sequences' blocks
// are summed, then the one that holds the CTA's first block is found.
template <class T, int MODE>
__device__ void span_place(const SpanArgs& a, SpanAux* aux) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto scan = [&](long long v, long long& total) -> long long {   // exclusive, over the block
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) aux->scan[warp] = x;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < T::THREADS / 32; ++w) {
            const long long y = aux->scan[w];
            if (w < warp) before += y;
            total += y;
        }
        return before + x - v;
    };
    auto blocks_of = [&](int b) -> long long {   // of all of a batch entry's units
        if (b >= a.B) return 0;
        const SpanSeq q = span_seq<MODE>(a, b);
        return (long long)span_units<MODE>(a, q) * span_blocks<T, MODE>(a, q);
    };
    long long all = 0, mine = 0, total;
    for (int b = threadIdx.x; b < a.B; b += T::THREADS) mine += blocks_of(b);
    scan(mine, all);
    const int group_ctas = MODE == kSpanTree ? a.group_ctas : 1;
    const int groups = (int)gridDim.x / group_ctas;
    const long long quota = (all + groups - 1) / groups;
    const long long beg = quota * ((int)blockIdx.x / group_ctas);
    if (threadIdx.x == 0) aux->start_n = (int)max(0ll, min(quota, all - beg));
    long long base = 0;
    for (int b0 = 0; b0 < a.B && base <= beg; b0 += T::THREADS) {
        const int b = b0 + threadIdx.x;
        const long long v = blocks_of(b);
        const long long at = base + scan(v, total);
        if (at <= beg && beg < at + v) {
            aux->start_b = b;
            aux->start_off = beg - at;
        }
        base += total;
    }
    __syncthreads();
}

// Producer: per segment K_0, Q, then K_{j+1} and V_j for every block j.
template <class T, int MODE, bool BOXED>
__device__ void span_load_role(const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                               const CUtensorMap* tm_v, const SpanArgs& a, SpanAux* aux,
                               uint32_t sQ, uint32_t sRing, const WaitCtx& wc) {
    const int lane = threadIdx.x & 31;
    const uint32_t bar_q = smem_u32(&aux->bar_q);
    if (lane == 0) {
        tma_prefetch_desc(tm_q);
        tma_prefetch_desc(tm_k);
        tma_prefetch_desc(tm_v);
    }
    int p = 0, ntail = 0, kq = 0;
    bool ok = true;
    SpanSeg s;
    for (bool more = span_first<T, MODE>(a, aux, s); more && ok; more = span_next<T, MODE>(a, s)) {
        if (s.m == 0) continue;
        const int plane = (a.cu_seqlens_k != nullptr ? 0 : s.b * a.Hkv) + s.hk;
        // BOXED: lane i's box of block j, positions [i box, (i + 1) box) of it:
        // where it lies in the tensor map (past the span, or no page: a plane
        // that does not exist, which reads as zeros)
        const int boxes = BOXED ? T::BN / a.box : 0;
        struct Box {
            int row, plane;
        };
        auto box_of = [&](int j) -> Box {
            const int x = (s.kb + j) * T::BN + lane * a.box;
            Box at{0, a.planes};
            if (lane < boxes && x < s.span) {
                const int key = span_key(s, x);
                if (a.block_table == nullptr) {
                    at = Box{s.q.k0 + key, plane};
                } else {
                    const int page = a.block_table[(size_t)s.b * a.max_pages + key / a.page_size];
                    if ((unsigned)page < (unsigned)a.num_pages)
                        at = Box{key % a.page_size, page * a.Hkv + s.hk};
                }
            }
            return at;
        };
        auto acquire = [&](uint32_t& dst, uint32_t& full) -> bool {
            const uint32_t slot = ring_slot<T>(p);
            if (!mbar_wait(smem_u32(&aux->bar_empty[slot]), ring_phase<T>(p) ^ 1u, wc,
                           kErrWaitTimeout | kSiteLoadEmpty))
                return false;
            dst = sRing + slot * T::SLOT;
            full = smem_u32(&aux->bar_full[slot]);
            return true;
        };
        auto load_k = [&](int j, int c, const Box& at) -> bool {
            uint32_t dst, full;
            if (!acquire(dst, full)) return false;
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)T::SLOT);
            if constexpr (BOXED) {
                __syncwarp();
                if (lane < boxes) {
#pragma unroll
                    for (int q = 0; q < T::KCH; ++q)
                        tma_load_3d(dst + q * T::KCHUNK + lane * a.box * 128, tm_k,
                                    (c * T::KCH + q) * 64, at.row, at.plane, full);
                }
            } else if (lane == 0) {
#pragma unroll
                for (int q = 0; q < T::KCH; ++q)
                    tma_load_3d(dst + q * T::KCHUNK, tm_k, (c * T::KCH + q) * 64,
                                (s.kb + j) * T::BN, plane, full);
            }
            __syncwarp();
            ++p;
            return true;
        };
        auto load_v = [&](int j, int hh, const Box& at) -> bool {
            uint32_t dst, full;
            if (!acquire(dst, full)) return false;
            const int r0 = (s.kb + j) * T::BN + hh * T::VKEYS;   // first position of the slot
            const int rv = s.end - r0;                           // keys of the sequence in it
            const bool tail = rv < T::VKEYS;
            const uint32_t bar = tail ? smem_u32(&aux->bar_tail) : full;
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)T::SLOT);
            if constexpr (BOXED) {
                __syncwarp();
                const int per = T::VKEYS / a.box, i = lane - hh * per;
                if (i >= 0 && i < per) {
#pragma unroll
                    for (int q = 0; q < T::NCH; ++q)
                        tma_load_3d(dst + q * T::VCHUNK + i * a.box * 128, tm_v, q * 64, at.row,
                                    at.plane, bar);
                }
            } else if (lane == 0) {
#pragma unroll
                for (int q = 0; q < T::NCH; ++q)
                    tma_load_3d(dst + q * T::VCHUNK, tm_v, q * 64, r0, plane, bar);
            }
            if (tail) {
                // rows past the sequence may hold anything, and zero times a
                // non-finite value would poison O: zeroed before publication
                if (!mbar_wait(bar, (uint32_t)(ntail & 1), wc, kErrWaitTimeout | kSiteLoadTail))
                    return false;
                ++ntail;
                const int z0 = rv > 0 ? rv : 0;
#pragma unroll
                for (int q = 0; q < T::NCH; ++q)
                    for (int g = z0 * 8 + lane; g < T::VKEYS * 8; g += 32)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         dst + q * T::VCHUNK + g * 16),
                                     "r"(0)
                                     : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            }
            __syncwarp();
            ++p;
            return true;
        };
        // boxes of the block whose V is loaded next, and of the next one
        Box at0 = box_of(0);
        Box at1 = s.m > 1 ? box_of(1) : at0;
        for (int c = 0; c < T::KP && ok; ++c) ok = load_k(0, c, at0);
        if (!ok) break;
        if (kq > 0 && !mbar_wait(smem_u32(&aux->bar_qfree), (uint32_t)((kq - 1) & 1), wc,
                                 kErrWaitTimeout | kSiteLoadQfree))
            break;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, (uint32_t)a.q_bytes);
            int row = s.tile * T::BM, q_plane = s.b * a.Hkv + s.hk;   // tree: rows of the matrix
            if (MODE == kSpanWindow) {   // positions x heads
                row = s.q.q0 + s.tile * a.P;
                q_plane = (a.cu_seqlens_q != nullptr ? 0 : s.b * a.Hq) + s.hk * a.group;
            }
#pragma unroll
            for (int q = 0; q < T::NCH; ++q)
                tma_load_3d(sQ + q * T::CHUNK, tm_q, q * 64, row, q_plane, bar_q);
        }
        __syncwarp();
        ++kq;
        for (int j = 0; j < s.m && ok; ++j) {
            const Box at2 = j + 2 < s.m ? box_of(j + 2) : at1;
            if (j + 1 < s.m)
                for (int c = 0; c < T::KP && ok; ++c) ok = load_k(j + 1, c, at1);
            for (int hh = 0; hh < T::VP && ok; ++hh) ok = load_v(j, hh, at0);
            at0 = at1;
            at1 = at2;
        }
    }
    // every copy issued must have landed before the CTA exits
    if (lane == 0) {
        if (kq > 0) mbar_wait_drain(bar_q, (uint32_t)((kq - 1) & 1), a.wait_limit_ns);
        for (int q = p > T::NSLOT ? p - T::NSLOT : 0; q < p; ++q)
            mbar_wait_drain(smem_u32(&aux->bar_full[ring_slot<T>(q)]), ring_phase<T>(q),
                            a.wait_limit_ns);
    }
    __syncwarp();
}

// MMA issue (one lane): S(J+1), then PV(J), as in the 256-key prefill kernel.
template <class T, int MODE>
__device__ void span_mma_role(const SpanArgs& a, SpanAux* aux, uint32_t tmem, uint32_t sQ,
                              uint32_t sRing, const WaitCtx& wc) {
    const int lane = threadIdx.x & 31;
    if (lane != 0) {
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
    auto score = [&](int J) -> bool {
        if (J > 0) {   // the softmax has read S(J-1) out of the buffer
            if (!mbar_wait_lane(smem_u32(&aux->bar_xm[(J - 1) & 1]), (uint32_t)(((J - 1) >> 1) & 1),
                                wc, kErrWaitTimeout | kSiteMmaSfree))
                return false;
            tc_fence_after();
        }
        for (int c = 0; c < T::KP; ++c) {
            if (!next_slot(kSiteMmaK)) return false;
            const uint32_t kd = slot_desc(kd0);
#pragma unroll
            for (int kin = 0; kin < 4 * T::KCH; ++kin) {
                const int kk = c * 4 * T::KCH + kin;
                umma_ss_lo(tmem + T::S_COL, qd0 + kstep_off(kk),
                           kd + (uint32_t)(((kin >> 2) * T::KCHUNK + (kin & 3) * 32) >> 4), idesc_s,
                           kk > 0 ? 1u : 0u);
            }
            tc_commit(smem_u32(&aux->bar_empty[ring_slot<T>(p)]));
            ++p;
        }
        tc_commit(smem_u32(&aux->bar_s_full));
        return true;
    };
    int J0 = 0, kq = 0;
    bool ok = true;
    SpanSeg s;
    for (bool more = span_first<T, MODE>(a, aux, s); more && ok; more = span_next<T, MODE>(a, s)) {
        const int n = s.m;
        if (n == 0) continue;
        if (!mbar_wait_lane(smem_u32(&aux->bar_q), (uint32_t)(kq & 1), wc,
                            kErrWaitTimeout | kSiteMmaQ))
            break;
        tc_fence_after();
        if (!score(J0)) break;
        if (n == 1) tc_commit(smem_u32(&aux->bar_qfree));   // Q no longer read
        for (int j = 0; j < n && ok; ++j) {
            const int J = J0 + j;
            if (j + 1 < n) {
                if (!score(J + 1)) {
                    ok = false;
                    break;
                }
                if (j + 2 == n) tc_commit(smem_u32(&aux->bar_qfree));
            }
            if (!mbar_wait_lane(smem_u32(&aux->bar_p_ready[J & 1]), (uint32_t)((J >> 1) & 1), wc,
                                kErrWaitTimeout | kSiteMmaP)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (j == 0 && kq > 0) {   // the previous segment's O has been read out
                if (!mbar_wait_lane(smem_u32(&aux->bar_odrained), (uint32_t)((kq - 1) & 1), wc,
                                    kErrWaitTimeout | kSiteMmaOdrained)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            for (int hh = 0; hh < T::VP; ++hh) {
                if (!next_slot(kSiteMmaV)) {
                    ok = false;
                    break;
                }
                const uint32_t vd = slot_desc(vd0);
#pragma unroll
                for (int kk = 0; kk < T::VKEYS / 16; ++kk)
                    umma_ts_lo(tmem + T::O_COL,
                               tmem + T::P_COL + (uint32_t)((hh * (T::VKEYS / 16) + kk) * 8),
                               vd + (uint32_t)((kk * 2048) >> 4), idesc_v,
                               (j > 0 || hh > 0 || kk > 0) ? 1u : 0u);
                tc_commit(smem_u32(&aux->bar_empty[ring_slot<T>(p)]));
                ++p;
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

// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// Softmax of one segment by warpgroup h (keys [HK h, HK h + HK) of every
// block; thread = row); see wide_softmax_unit.
template <class T, int MODE>
__device__ bool span_softmax_segment(int h, const SpanArgs& a, const SpanSeg& s, SpanAux* aux,
                                     uint32_t tmem, const WaitCtx& wc, int J0, int kq) {
    constexpr int HK = T::HK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
        node0 = s.q.keys - s.q.rows;
    } else {
        const int p = s.tile * a.P + r % a.P + s.q.keys - s.q.rows;   // the row's key
        const int last = a.causal ? min(s.q.keys - 1, p) : s.q.keys - 1;
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
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < HK / 64; ++q)
            tmem_ld64(lane_base + T::S_COL + h * HK + q * 64,
                      *reinterpret_cast<uint32_t(*)[2][32]>(&u[2 * q][0]));
        tmem_wait_ld();
        float x[HK];
#pragma unroll
        for (int c = 0; c < HK; ++c) x[c] = __uint_as_float(u[c >> 5][c & 31]);
        const int x0 = (s.kb + j) * T::BN + h * HK;   // first position of the half
        const bool masked = MODE == kSpanTree ? x0 + HK > node0   // the nodes' own keys, or past
                                              : (x0 < lo || x0 + HK - 1 > lim) && x0 + HK > fa;
        if (masked) {
#pragma unroll
            for (int q = 0; q < HK / 32; ++q) {
                const int xq = x0 + 32 * q;
                uint32_t vis;
                if constexpr (MODE == kSpanTree)
                    vis = tree_bits(words, s.q.rows, xq - node0);
                else
                    vis = low_bits(fa - xq) | (low_bits(lim + 1 - xq) & ~low_bits(lo - xq));
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    x[32 * q + c] = ((vis >> c) & 1u) ? x[32 * q + c] : -INFINITY;
            }
        }
        float mq[HK / 32];
#pragma unroll
        for (int q = 0; q < HK / 32; ++q) {
            float m = fmax3(x[32 * q], x[32 * q + 1], x[32 * q + 2]);
#pragma unroll
            for (int c = 3; c < 31; c += 2) m = fmax3(m, x[32 * q + c], x[32 * q + c + 1]);
            mq[q] = fmaxf(m, x[32 * q + 31]);
        }
        float mx_h = fmaxf(mq[0], mq[1]);
        if constexpr (HK == 128) mx_h = fmaxf(fmax3(mx_h, mq[2], mq[3]), mx_h);
        aux->xm[sb][h][r] = mx_h;
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_xm[sb]));
        if (!mbar_wait(smem_u32(&aux->bar_xm[sb]), par, wc, kErrWaitTimeout | kSiteSmXm))
            return false;
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
            if (c == 31) {   // P(J) overwrites P(J-1) once PV(J-1) has read it
                if (J > 0) {
                    if (!mbar_wait(smem_u32(&aux->bar_pv_done[(J - 1) & 1]),
                                   (uint32_t)(((J - 1) >> 1) & 1), wc,
                                   kErrWaitTimeout | kSiteSmPv))
                        return false;
                    tc_fence_after();
                }
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
__device__ __forceinline__ float span_normaliser(const float* sinks, int h, float& l, float& m) {
    float scale = 1.f;
    if (sinks != nullptr) {
        const float sg = sinks[h] * kLog2e;
        const float m2 = fmaxf(m, sg);
        if (m2 == -INFINITY) return 0.f;
        scale = (m == -INFINITY) ? 0.f : ex2_approx(m - m2);
        l = l * scale + ex2_approx(sg - m2);
        m = m2;
    }
    return l > 0.f ? scale / l : 0.f;
}

// Correction of one segment (thread = row): rebases O when the running max
// moved; at its end writes O and LSE of a whole unit, or the piece's
// unnormalised O, max and sum.
template <class T, int MODE>
__device__ bool span_correction_segment(const SpanArgs& a, const SpanSeg& s, SpanAux* aux,
                                        uint32_t tmem, const WaitCtx& wc, int J0, int kq) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_p_ready[sb]));
    }
    float l = 0.f, m = m_run;
    if (s.m > 0) {   // (else a unit, or a piece of one, without keys)
        if (!mbar_wait(smem_u32(&aux->bar_fin), (uint32_t)(kq & 1), wc,
                       kErrWaitTimeout | kSiteEpiMbox))
            return false;
        l = aux->mb_l[0][r] + aux->mb_l[1][r];
        const int Jl = J0 + s.m - 1;
        if (!mbar_wait(smem_u32(&aux->bar_pv_done[Jl & 1]), (uint32_t)((Jl >> 1) & 1), wc,
                       kErrWaitTimeout | kSiteEpiPv))
            return false;
        tc_fence_after();
    }
    int head, pos;
    size_t o_row, lse_at;
    const bool real = span_row<T, MODE>(a, s.q, s.b, s.hk, s.tile, r, head, pos, o_row, lse_at);
    if (s.n < s.nb) {   // a piece
        const int slot = 2 * (int)blockIdx.x + (s.index > 0);
        float4* po = reinterpret_cast<float4*>(a.part_o + (size_t)slot * (T::D_COLS * T::BM));
#pragma unroll 1
        for (int c32 = 0; c32 < (s.m > 0 ? T::D_COLS / 32 : 0); ++c32) {
            uint32_t v[32];
            tmem_ld32(lane_base + T::O_COL + c32 * 32, v);
            tmem_wait_ld();
            if (!real) continue;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                po[(size_t)(c32 * 8 + q) * T::BM + r] =
                    make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
        }
        float* ml = a.part_ml + (size_t)slot * 2 * T::BM;
        ml[r] = m;
        ml[T::BM + r] = l;
        if (r == 0) a.head[slot] = make_int4(s.b, s.u, s.n, s.kb == 0 ? s.nb : 0);
    } else {
        const float inv_l = span_normaliser(real ? a.sinks : nullptr, head, l, m);
        store_o_rows_direct<T>(lane_base, T::O_COL, a.o + o_row * T::D_COLS, real, s.m, inv_l, 0,
                               T::D_COLS / 32);
        if (real) a.lse[lse_at] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
    }
    if (s.m > 0) {
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&aux->bar_odrained));
    }
    return true;
}

template <int D, int MODE, bool BOXED>
__global__ void __launch_bounds__(SpanTraits<D>::THREADS, 1)
    span_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const SpanArgs a) {
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
        for (int i = 0; i < T::NSLOT; ++i) {
            mbar_init(smem_u32(&aux->bar_full[i]), 1);
            mbar_init(smem_u32(&aux->bar_empty[i]), 1);
        }
        mbar_init(smem_u32(&aux->bar_s_full), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&aux->bar_xm[i]), 8);
            mbar_init(smem_u32(&aux->bar_p_ready[i]), 12);
            mbar_init(smem_u32(&aux->bar_pv_done[i]), 1);
        }
        mbar_init(smem_u32(&aux->bar_fin), 8);
        mbar_init(smem_u32(&aux->bar_qfree), 1);
        mbar_init(smem_u32(&aux->bar_odrained), 4);
        mbar_init(smem_u32(&aux->bar_tail), 1);
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
    wait_for_previous();   // (what is above overlaps the kernel before)
    if (threadIdx.x == 0)
        a.head[2 * blockIdx.x] = a.head[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    span_place<T, MODE>(a, aux);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = aux->tmem_base;
    const WaitCtx wc{smem_u32(&aux->abort_flag), (uint32_t)a.wait_limit_ns, a.err_word};
    if (wg < 2) {
        setmaxnreg_inc<T::SOFTMAX_REGS>();
        int J0 = 0, kq = 0;
        SpanSeg s;
        for (bool more = span_first<T, MODE>(a, aux, s); more; more = span_next<T, MODE>(a, s)) {
            if (s.m == 0) continue;
            if (!span_softmax_segment<T, MODE>(wg, a, s, aux, tmem, wc, J0, kq)) break;
            J0 += s.m;
            ++kq;
        }
    } else if (wg == T::CORR_WG) {
        setmaxnreg_dec<T::CORR_REGS>();
        int J0 = 0, kq = 0;
        SpanSeg s;
        for (bool more = span_first<T, MODE>(a, aux, s); more; more = span_next<T, MODE>(a, s)) {
            if (MODE == kSpanTree && s.tile >= a.tiles) continue;   // a group's spare CTA
            if (!span_correction_segment<T, MODE>(a, s, aux, tmem, wc, J0, kq)) break;
            J0 += s.m;
            kq += s.m > 0;
        }
    } else {
        setmaxnreg_dec<T::OTHER_REGS>();
        if (warp == T::MMA_WARP)
            span_mma_role<T, MODE>(a, aux, tmem, sQ, sRing, wc);
        else if (warp == T::LOAD_WARP)
            span_load_role<T, MODE, BOXED>(&tm_q, &tm_k, &tm_v, a, aux, sQ, sRing, wc);
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
    const int step = MODE == kSpanTree ? a.group_ctas : 1;
    int slot = 2 * blockIdx.x;
    int4 hd = a.head[slot];
    if (!(hd.z > 0 && hd.w > hd.z)) hd = a.head[++slot];
    if (!(hd.z > 0 && hd.w > hd.z)) return;
    const int b = hd.x, u = hd.y, nb = hd.w;
    if ((unsigned)b >= (unsigned)a.B) return;
    const SpanSeq seq = span_seq<MODE>(a, b);
    if ((unsigned)u >= (unsigned)span_units<MODE>(a, seq)) return;
    const int tiles = MODE == kSpanTree ? a.tile_groups : (seq.cap + a.P - 1) / a.P;
    const int tile = MODE == kSpanTree
                         ? u % tiles * a.group_ctas + (int)blockIdx.x % a.group_ctas
                         : u % tiles;
    int h, pos;
    size_t o_row, lse_at;
    if (!span_row<T, MODE>(a, seq, b, u / tiles, tile, r, h, pos, o_row, lse_at)) return;
    float M = -INFINITY, L = 0.f;
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    int x = blockIdx.x;
    for (int done = 0; done < nb && x < G; x += step) {
        if (x > (int)blockIdx.x) slot = 2 * x;   // it goes on as the next CTA's first segment
        const int n = a.head[slot].z;
        if (n <= 0) break;
        done += n;
        const float* ml = a.part_ml + (size_t)slot * 2 * T::BM;
        const float4* po = reinterpret_cast<const float4*>(a.part_o + (size_t)slot * (D * T::BM));
        const float mk = ml[r], lk = ml[T::BM + r];
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = po[(size_t)(c16 * 4 + q) * T::BM + r];
        if (mk == -INFINITY) continue;
        const float m2 = fmaxf(M, mk);
        const float sc = (M == -INFINITY) ? 0.f : ex2_approx(M - m2);
        const float wk = ex2_approx(mk - m2);
        M = m2;
        L = fmaf(L, sc, wk * lk);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            acc[4 * q + 0] = fmaf(acc[4 * q + 0], sc, wk * v[q].x);
            acc[4 * q + 1] = fmaf(acc[4 * q + 1], sc, wk * v[q].y);
            acc[4 * q + 2] = fmaf(acc[4 * q + 2], sc, wk * v[q].z);
            acc[4 * q + 3] = fmaf(acc[4 * q + 3], sc, wk * v[q].w);
        }
    }
    const float inv_l = span_normaliser(a.sinks, h, L, M);
    uint4* dst = reinterpret_cast<uint4*>(a.o + o_row * D + c16 * 16);
#pragma unroll
    for (int g = 0; g < 2; ++g)
        dst[g] = make_uint4(pack_bf16x2(acc[8 * g + 0] * inv_l, acc[8 * g + 1] * inv_l),
                            pack_bf16x2(acc[8 * g + 2] * inv_l, acc[8 * g + 3] * inv_l),
                            pack_bf16x2(acc[8 * g + 4] * inv_l, acc[8 * g + 5] * inv_l),
                            pack_bf16x2(acc[8 * g + 6] * inv_l, acc[8 * g + 7] * inv_l));
    if (c16 == 0) a.lse[lse_at] = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
}

template <int D, int MODE, bool BOXED>
cudaError_t launch_span_mode(const SpanLaunch& p, cudaStream_t s) {
    using T = SpanTraits<D>;
    cudaError_t e = cudaFuncSetAttribute(span_kernel<D, MODE, BOXED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         T::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    e = launch_dependent(span_kernel<D, MODE, BOXED>, dim3(p.ctas), dim3(T::THREADS), T::SMEM_TOTAL,
                         s, p.tm_q, p.tm_k, p.tm_v, p.args);
    if (e != cudaSuccess) return e;
    return launch_dependent(span_combine_kernel<D, MODE>, dim3(p.ctas, D / 16), dim3(T::BM), 0, s,
                            p.args);
}

template <int D>
cudaError_t launch_span_impl(const SpanLaunch& p, cudaStream_t s) {
    if (p.args.tree_mask == nullptr) return launch_span_mode<D, kSpanWindow, true>(p, s);
    return p.args.box > 0 ? launch_span_mode<D, kSpanTree, true>(p, s)
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
