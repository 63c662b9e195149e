// Attention of a tree of drafted tokens over a cache, on the tensor cores
// (head_dim 64, 128 and 256).
//
// All query rows of a key/value head (group heads x T nodes) see the same
// keys up to the tree, and lie side by side in memory: the rows
// [b, hk * group .. + group, 0 .. T) of Q and O are one matrix of
// R = group * T rows.  A tile is 128 of them, whatever T is; row r of the
// matrix is node r % T.  Only the last keys, the nodes' own, are masked, by
// the bits of the row's node.
//
// What bounds it: per key of a key/value head 4 d bytes of K and V are read
// and 4 d R operations done, so up to about 270 rows memory is the bound and
// past it the tensor cores (1865 TFLOP/s over 6793 GB/s, both measured).  The
// keys are therefore spread evenly over the SMs: with nb_b key blocks per
// unit (batch entry, key/value head, row tile), the units' blocks, one after
// the other, form one line of N blocks, and CTA x takes the blocks
// [x quota, (x + 1) quota), quota = ceil(N / CTAs), whatever the sequences'
// lengths (which only the device knows).  A unit that lies in one CTA is
// finished there; of the others each CTA writes its piece's unnormalised O,
// row max and row sum, and tree_combine_kernel merges the pieces, in their
// order (the result does not depend on timing).
//
// Inside a CTA: the roles and barriers of the 256-key prefill kernel (see
// prefill_wide.cuh), which this one follows: S = Q K^T of the next block is
// issued once the softmax has read this block's scores into registers; two
// warpgroups share each row's softmax; P has tensor memory of its own.  Key
// blocks are 256 keys (one N = 256 score instruction per 16 head dims), 128 at
// head_dim 256, whose 256 O columns leave no room for more.
//
// Paged caches: a box of the tensor maps is as many rows of one page as the
// page's size allows (the largest power of two that divides it, 8 at least),
// one lane of the producer per box, the page numbers fetched a block ahead.
#include "prefill.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

template <int D>
struct TreeTraits {
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

constexpr int kTreeSlots = 6;

struct TreeAux {
    uint64_t bar_q;
    uint64_t bar_full[kTreeSlots];
    uint64_t bar_empty[kTreeSlots];
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

// Keys and nodes of sequence b.
__device__ __forceinline__ int tree_keys(const TreeArgs& a, int b) {
    return a.seqlens_k != nullptr ? max(0, min(a.seqlens_k[b], a.Sk)) : a.Sk;
}
__device__ __forceinline__ int tree_count(const TreeArgs& a, int b) {
    return a.tree_lens != nullptr ? max(0, min(a.tree_lens[b], a.T)) : a.T;
}
// Key blocks of each of sequence b's units.
template <class T>
__device__ __forceinline__ int tree_blocks(const TreeArgs& a, int b) {
    return tree_count(a, b) > 0 ? (tree_keys(a, b) + T::BN - 1) / T::BN : 0;
}

// The CTA's segments in turn: `n` consecutive key blocks from kb on of a
// unit with nb blocks.
struct TreeSeg {
    int b, u;        // batch entry, unit of it: hk * tiles + tile
    int kb, n, nb;
    int L, nodes;
    int left;        // blocks of the CTA after this segment
    int index;       // segments before it
};
template <class T>
__device__ __forceinline__ bool tree_first(const TreeArgs& a, const TreeAux* aux, TreeSeg& s) {
    s.left = aux->start_n;
    if (s.left <= 0) return false;
    s.b = aux->start_b;
    s.nb = tree_blocks<T>(a, s.b);
    s.u = (int)(aux->start_off / s.nb);
    s.kb = (int)(aux->start_off % s.nb);
    s.L = tree_keys(a, s.b);
    s.nodes = tree_count(a, s.b);
    s.n = min(s.nb - s.kb, s.left);
    s.left -= s.n;
    s.index = 0;
    return true;
}
template <class T>
__device__ __forceinline__ bool tree_next(const TreeArgs& a, TreeSeg& s) {
    if (s.left <= 0) return false;
    s.kb = 0;
    if (++s.u == a.units) {
        s.u = 0;
        do {
            if (++s.b >= a.B) return false;   // (never: `left` counts real blocks)
            s.nb = tree_blocks<T>(a, s.b);
        } while (s.nb == 0);
        s.L = tree_keys(a, s.b);
        s.nodes = tree_count(a, s.b);
    }
    s.n = min(s.nb, s.left);
    s.left -= s.n;
    ++s.index;
    return true;
}

// Places the CTA on the line of blocks (all threads): the sequences' blocks
// are summed, then the one that holds the CTA's first block is found.
template <class T>
__device__ void tree_place(const TreeArgs& a, TreeAux* aux) {
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
    long long all = 0, mine = 0, total;
    for (int b = threadIdx.x; b < a.B; b += T::THREADS)
        mine += (long long)tree_blocks<T>(a, b) * a.units;
    scan(mine, all);
    long long quota = (all + gridDim.x - 1) / gridDim.x;
    if (quota < a.min_quota) quota = a.min_quota;
    const long long beg = quota * blockIdx.x;
    if (threadIdx.x == 0) aux->start_n = (int)max(0ll, min(quota, all - beg));
    long long base = 0;
    for (int b0 = 0; b0 < a.B && base <= beg; b0 += T::THREADS) {
        const int b = b0 + threadIdx.x;
        const long long v = b < a.B ? (long long)tree_blocks<T>(a, b) * a.units : 0;
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
template <class T, bool PAGED>
__device__ void tree_load_role(const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                               const CUtensorMap* tm_v, const TreeArgs& a, TreeAux* aux,
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
    TreeSeg s;
    for (bool more = tree_first<T>(a, aux, s); more && ok; more = tree_next<T>(a, s)) {
        const int hk = s.u / a.tiles, tile = s.u % a.tiles;
        const int plane = s.b * a.Hkv + hk;
        // PAGED: lane i's box of block j, rows [i box, (i + 1) box) of it: the
        // plane of its page (past the sequence, or no page: a plane that does
        // not exist, which reads as zeros)
        const int boxes = PAGED ? T::BN / a.box : 0;
        auto box_plane = [&](int j) -> int {
            const int key = (s.kb + j) * T::BN + lane * a.box;
            int pl = a.num_pages * a.Hkv;
            if (lane < boxes && key < s.L) {
                const int page = a.block_table[(size_t)s.b * a.max_pages + key / a.page_size];
                if ((unsigned)page < (unsigned)a.num_pages) pl = page * a.Hkv + hk;
            }
            return pl;
        };
        auto box_row = [&](int j) { return ((s.kb + j) * T::BN + lane * a.box) % a.page_size; };
        auto acquire = [&](uint32_t& dst, uint32_t& full) -> bool {
            const uint32_t slot = ring_slot<T>(p);
            if (!mbar_wait(smem_u32(&aux->bar_empty[slot]), ring_phase<T>(p) ^ 1u, wc,
                           kErrWaitTimeout | kSiteLoadEmpty))
                return false;
            dst = sRing + slot * T::SLOT;
            full = smem_u32(&aux->bar_full[slot]);
            return true;
        };
        auto load_k = [&](int j, int c, int pl) -> bool {
            uint32_t dst, full;
            if (!acquire(dst, full)) return false;
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)T::SLOT);
            if constexpr (PAGED) {
                __syncwarp();
                if (lane < boxes) {
#pragma unroll
                    for (int q = 0; q < T::KCH; ++q)
                        tma_load_3d(dst + q * T::KCHUNK + lane * a.box * 128, tm_k,
                                    (c * T::KCH + q) * 64, box_row(j), pl, full);
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
        auto load_v = [&](int j, int hh, int pl) -> bool {
            uint32_t dst, full;
            if (!acquire(dst, full)) return false;
            const int r0 = (s.kb + j) * T::BN + hh * T::VKEYS;   // first key of the slot
            const int rv = s.L - r0;                             // its valid keys
            const bool tail = rv < T::VKEYS;
            const uint32_t bar = tail ? smem_u32(&aux->bar_tail) : full;
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)T::SLOT);
            if constexpr (PAGED) {
                __syncwarp();
                const int per = T::VKEYS / a.box, i = lane - hh * per;
                if (i >= 0 && i < per) {
#pragma unroll
                    for (int q = 0; q < T::NCH; ++q)
                        tma_load_3d(dst + q * T::VCHUNK + i * a.box * 128, tm_v, q * 64,
                                    box_row(j), pl, bar);
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
        // page planes of the block whose V is loaded next, and of the next one
        int pl0 = PAGED ? box_plane(0) : 0;
        int pl1 = PAGED && s.n > 1 ? box_plane(1) : 0;
        for (int c = 0; c < T::KP && ok; ++c) ok = load_k(0, c, pl0);
        if (!ok) break;
        if (kq > 0 && !mbar_wait(smem_u32(&aux->bar_qfree), (uint32_t)((kq - 1) & 1), wc,
                                 kErrWaitTimeout | kSiteLoadQfree))
            break;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, (uint32_t)T::QTILE);
#pragma unroll
            for (int q = 0; q < T::NCH; ++q)
                tma_load_3d(sQ + q * T::CHUNK, tm_q, q * 64, tile * T::BM, plane, bar_q);
        }
        __syncwarp();
        ++kq;
        for (int j = 0; j < s.n && ok; ++j) {
            const int pl2 = PAGED && j + 2 < s.n ? box_plane(j + 2) : 0;
            if (j + 1 < s.n)
                for (int c = 0; c < T::KP && ok; ++c) ok = load_k(j + 1, c, pl1);
            for (int hh = 0; hh < T::VP && ok; ++hh) ok = load_v(j, hh, pl0);
            pl0 = pl1;
            pl1 = pl2;
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
template <class T>
__device__ void tree_mma_role(const TreeArgs& a, TreeAux* aux, uint32_t tmem, uint32_t sQ,
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
    TreeSeg s;
    for (bool more = tree_first<T>(a, aux, s); more && ok; more = tree_next<T>(a, s)) {
        const int n = s.n;
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

// Softmax of one segment by warpgroup h (keys [HK h, HK h + HK) of every
// block; thread = row); see wide_softmax_unit.
template <class T>
__device__ bool tree_softmax_segment(int h, const TreeArgs& a, const TreeSeg& s, TreeAux* aux,
                                     uint32_t tmem, const WaitCtx& wc, int J0, int kq) {
    constexpr int HK = T::HK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int node = ((s.u % a.tiles) * T::BM + r) % a.T;   // (rows past the last: any row's words)
    const uint32_t* words = a.tree_mask + s.b * a.tree_stride + (long long)node * a.tree_words;
    const int node0 = s.L - s.nodes;
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY, l_run = 0.f;
    for (int j = 0; j < s.n; ++j) {
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
        const int kv0 = (s.kb + j) * T::BN + h * HK;   // first key of the half
        if (kv0 + HK > node0) {                        // the nodes' own keys, or past them
#pragma unroll
            for (int q = 0; q < HK / 32; ++q) {
                const uint32_t vis = tree_bits(words, s.nodes, kv0 + 32 * q - node0);
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
__device__ __forceinline__ float tree_normaliser(const float* sinks, int h, float& l, float& m) {
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
template <class T>
__device__ bool tree_correction_segment(const TreeArgs& a, const TreeSeg& s, TreeAux* aux,
                                        uint32_t tmem, const WaitCtx& wc, int J0, int kq) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY;
    for (int j = 0; j < s.n; ++j) {
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
    if (!mbar_wait(smem_u32(&aux->bar_fin), (uint32_t)(kq & 1), wc, kErrWaitTimeout | kSiteEpiMbox))
        return false;
    float l = aux->mb_l[0][r] + aux->mb_l[1][r];
    float m = m_run;
    const int Jl = J0 + s.n - 1;
    if (!mbar_wait(smem_u32(&aux->bar_pv_done[Jl & 1]), (uint32_t)((Jl >> 1) & 1), wc,
                   kErrWaitTimeout | kSiteEpiPv))
        return false;
    tc_fence_after();
    const int row = (s.u % a.tiles) * T::BM + r;   // of the key/value head's rows
    const int hk = s.u / a.tiles;
    const bool real = row < a.rows && row % a.T < s.nodes;
    if (s.n < s.nb) {   // a piece
        const int slot = 2 * (int)blockIdx.x + (s.index > 0);
        float4* po = reinterpret_cast<float4*>(a.part_o + (size_t)slot * (T::D_COLS * T::BM));
#pragma unroll 1
        for (int c32 = 0; c32 < T::D_COLS / 32; ++c32) {
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
        const float inv_l = tree_normaliser(a.sinks, hk * a.group + row / a.T, l, m);
        const size_t at = ((size_t)s.b * a.Hkv + hk) * a.rows + row;
        store_o_rows_direct<T>(lane_base, T::O_COL, a.o + at * T::D_COLS, real, s.n, inv_l, 0,
                               T::D_COLS / 32);
        if (real) a.lse[at] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
    }
    tc_fence_before();
    mbar_arrive_warp(smem_u32(&aux->bar_odrained));
    return true;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(TreeTraits<D>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
    using T = TreeTraits<D>;
    static_assert(sizeof(TreeAux) <= T::SMEM_AUX && T::NSLOT <= kTreeSlots, "auxiliary block");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sRing = sQ + T::SMEM_Q;
    auto* aux = reinterpret_cast<TreeAux*>(smem_raw + (sQ - raw) + T::SMEM_Q + T::SMEM_RING);
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
    tree_place<T>(a, aux);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = aux->tmem_base;
    const WaitCtx wc{smem_u32(&aux->abort_flag), (uint32_t)a.wait_limit_ns, a.err_word};
    if (wg < 2) {
        setmaxnreg_inc<T::SOFTMAX_REGS>();
        int J0 = 0, kq = 0;
        TreeSeg s;
        for (bool more = tree_first<T>(a, aux, s); more; more = tree_next<T>(a, s)) {
            if (!tree_softmax_segment<T>(wg, a, s, aux, tmem, wc, J0, kq)) break;
            J0 += s.n;
            ++kq;
        }
    } else if (wg == T::CORR_WG) {
        setmaxnreg_dec<T::CORR_REGS>();
        int J0 = 0, kq = 0;
        TreeSeg s;
        for (bool more = tree_first<T>(a, aux, s); more; more = tree_next<T>(a, s)) {
            if (!tree_correction_segment<T>(a, s, aux, tmem, wc, J0, kq)) break;
            J0 += s.n;
            ++kq;
        }
    } else {
        setmaxnreg_dec<T::OTHER_REGS>();
        if (warp == T::MMA_WARP)
            tree_mma_role<T>(a, aux, tmem, sQ, sRing, wc);
        else if (warp == T::LOAD_WARP)
            tree_load_role<T, PAGED>(&tm_q, &tm_k, &tm_v, a, aux, sQ, sRing, wc);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == T::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, T::TMEM_COLS);
    }
}

// Merges the pieces of the unit that starts in CTA blockIdx.x of the split
// kernel and goes on in the next ones (16 columns per CTA here, thread = row),
// and writes the rows of sequences without keys.
template <int D>
__global__ void __launch_bounds__(128) tree_combine_kernel(const TreeArgs a) {
    using T = TreeTraits<D>;
    dependents_may_start();
    wait_for_previous();
    const int r = threadIdx.x, c16 = blockIdx.y, G = gridDim.x;
    for (int b = blockIdx.x; b < a.B; b += G) {
        const int nodes = tree_count(a, b);
        if (nodes == 0 || tree_keys(a, b) > 0) continue;
        for (long long i = r; i < (long long)a.Hkv * a.rows; i += T::BM) {
            if (i % a.T >= nodes) continue;
            const size_t at = (size_t)b * a.Hkv * a.rows + i;
            uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + c16 * 16);
            dst[0] = dst[1] = make_uint4(0, 0, 0, 0);
            float l = 0.f, m = -INFINITY;
            tree_normaliser(a.sinks, (int)(i / a.T), l, m);
            if (c16 == 0) a.lse[at] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
        }
    }
    int slot = 2 * blockIdx.x;
    int4 hd = a.head[slot];
    if (!(hd.z > 0 && hd.w > hd.z)) hd = a.head[++slot];
    if (!(hd.z > 0 && hd.w > hd.z)) return;
    const int b = hd.x, u = hd.y, nb = hd.w;
    if ((unsigned)b >= (unsigned)a.B || (unsigned)u >= (unsigned)a.units) return;
    const int row = (u % a.tiles) * T::BM + r;
    if (row >= a.rows || row % a.T >= tree_count(a, b)) return;
    float M = -INFINITY, L = 0.f;
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    int x = blockIdx.x;
    for (int done = 0; done < nb && x < G; ++x) {
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
    const int hk = u / a.tiles;
    const float inv_l = tree_normaliser(a.sinks, hk * a.group + row / a.T, L, M);
    const size_t at = ((size_t)b * a.Hkv + hk) * a.rows + row;
    uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + c16 * 16);
#pragma unroll
    for (int g = 0; g < 2; ++g)
        dst[g] = make_uint4(pack_bf16x2(acc[8 * g + 0] * inv_l, acc[8 * g + 1] * inv_l),
                            pack_bf16x2(acc[8 * g + 2] * inv_l, acc[8 * g + 3] * inv_l),
                            pack_bf16x2(acc[8 * g + 4] * inv_l, acc[8 * g + 5] * inv_l),
                            pack_bf16x2(acc[8 * g + 6] * inv_l, acc[8 * g + 7] * inv_l));
    if (c16 == 0) a.lse[at] = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_tree_impl(const TreeLaunch& p, cudaStream_t s) {
    using T = TreeTraits<D>;
    const auto kern = p.args.block_table != nullptr ? tree_kernel<D, true> : tree_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         T::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(p.ctas), dim3(T::THREADS), T::SMEM_TOTAL, s, p.tm_q, p.tm_k,
                         p.tm_v, p.args);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_combine_kernel<D>, dim3(p.ctas, D / 16), dim3(T::BM), 0, s, p.args);
}

}  // namespace

cudaError_t launch_tree(const TreeLaunch& p, int head_dim, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_tree_impl<64>(p, s);
        case 128: return launch_tree_impl<128>(p, s);
        case 256: return launch_tree_impl<256>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
