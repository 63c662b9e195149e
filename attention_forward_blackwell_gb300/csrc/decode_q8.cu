// Decode attention over a paged cache held in 8 bits, for sm_103a.
//
// Half the bytes of decode.cu's caches for a key, so that twice as many keys a
// second have to be turned into operands: what decides is how few instructions
// that takes.  The split over the keys, the merge by LSE and the joined splits
// are decode.cu's; what differs:
//
//   - The keys are the M side of the products: S^T [16 keys x 8 rows] = K Q^T and
//     O^T [16 dims x 8 rows] += V^T P^T, so that 8 query rows (a group of 8 heads)
//     fill the instruction, where rows on M would leave half of it empty.
//   - A sum may be taken in any order, so the operands are laid out for the loads:
//     a lane's 16 codes of a key (16 bytes) are its share of four steps of the score
//     product, the rows of Q permuted alike; a lane's 16 dims of four keys are its
//     share of 8 tiles of O^T, two byte permutes for two pairs of keys.
//     A conversion (two codes to fp16, exact) per register of an operand is all the
//     rest; products of e4m3 values with fp16 P and Q are exact, their sums fp32.
//     (Scores by e4m3 products, each query as two codes, need no conversion of keys,
//     but products of both kinds in one loop cost more than that: 202 us where fp16
//     alone took 194.)
//   - Q in fp16: each row times a power of two that brings its largest element
//     into [1, 2), so 8 bits of fraction stay of every element down to 2^-14 of
//     it; below, the error is 2^-25 of the largest, that of an fp32 sum.
//   - Scales.  A key's score is multiplied by its scale.  A value's scale goes into
//     its probability, p_j v_j = (p_j s_j) code_j, and fp16 has to hold that
//     product whatever the scales are: it is exp2(score_j + log2 s_j - m'), with a
//     running maximum m' of its own beside that of the softmax's sum, so that
//     the largest terms of O always lie in the upper binades; 2^6 of headroom is
//     used (kLift), 2^8 of growth allowed before both are moved on (kGrow).
//   - The row maxima of a slice are never taken: lanes check their own exponents
//     against the bounds and vote; a shuffle tree follows only where one is over.
//     Scores and exponents are computed two rows an instruction.
//
// Work.  The sequences' lengths are known to the device only, and differ.  A unit
// (batch entry, key/value head, tile of query rows) counts its blocks of keys; the
// units' blocks, one after the other, form a line that is cut into equal pieces, one
// per CTA, as many CTAs as fit the SMs at once (as in span.cu; q8_line.cuh has the
// arithmetic and its choices).  A unit that lies in one piece is finished there; of the others each CTA
// writes what it has, normalised, with its LSE, and a second kernel merges them in
// their order.  (The split kernel's grid, one CTA of 256 keys and more for every
// piece of the longest possible sequence, took 195 us for 64 x 1K to 16K keys x 8
// heads at head_dim 128, now 178, 6.4 TB/s, and 213 for one of 130,000 keys x 2 heads
// at 256, now 35.  Merged by the CTA that writes a unit's last piece, without a second
// kernel: 189, for the fences and counts stop its ring.)  Neither kernel lets the
// next start early: its CTAs would take the places of this one's later pieces (195).
// Short caches are split over the CTAs of a cluster instead, which merge without a
// second kernel, as decode.cu's joined splits (2,000 keys x 8 heads 6.7 us).
//
// A warp takes a slice of every block through a ring of its own.  Tensor copies
// fill it, one lane for every box of rows that lie together (a page's, up to 32),
// so that a slice costs the warp a few instructions where 16-byte copies by all
// lanes took a third of all it issues; copies run ahead over the ends of units,
// and the page numbers of a slice are fetched while the one before is issued.
// What a box brings beside keys that some row sees may be anything: scores are
// replaced, values zeroed, at the borders alone.
#include <atomic>

#include "common.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "q8_line.cuh"

namespace fa {
namespace {

constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kLog2ef = 1.44269504088896340736f;
constexpr float kGrow = 8.0f;   // log2
constexpr float kLift = 6.0f;
constexpr float kFar = 3.0e38f;  // minus a base of a row that has seen nothing

constexpr unsigned kSiteQ8 = 72; // wait site of the ring

// Rows that a CTA of n joined splits holds for its part of a tile's R, n pieces of each.
// (Not a row more than the most of any n: at head_dim 64 and 128 the CTAs of an SM fill its
// shared memory to the last kilobyte.)
constexpr int join_rows(int R) {
    int most = 0;
    for (int n = 1; n <= kJoinSplits; ++n) most = (R + n - 1) / n * n > most ? (R + n - 1) / n * n : most;
    return most;
}

template <int D, int NR>
struct Q8Traits {
    static constexpr int WARPS = 4;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int R = 8 * NR;                    // rows of a tile
    static constexpr int SUB = D == 256 ? 1 : 2;        // 16-key parts of a slice
    static constexpr int KB = 16 * SUB;                 // keys of a slice
    static constexpr int BLOCK = WARPS * KB;            // keys of a block
    static constexpr int SUMS = NR == 1 ? 2 : 1;         // of a score, side by side
    static constexpr int SW = SUB;                       // parts worked on together
    static constexpr bool KEEP = NR == 1 || (D != 256 && NR == 2);   // exponents kept over the vote
    static constexpr int PITCH = D == 64 ? 64 : 128;    // bytes of a box's row
    static constexpr int CHUNK = KB * PITCH;            // a box of a slice's rows
    static constexpr int SLICE = KB * D;                // bytes of a slice of keys, or of values
    static constexpr int STAGE = 2 * SLICE;
    static constexpr int STAGES = D == 64 ? 3 : 2;
    static constexpr int WARP_RING = STAGES * STAGE;
    static constexpr int SCALE_BYTES = 2 * KB * 4;      // of a slot's keys and values
    static constexpr int SCALES = WARPS * WARP_RING;    // behind the ring
    static constexpr int WARP_SCALES = STAGES * SCALE_BYTES;
    static constexpr int BARS = SCALES + WARPS * WARP_SCALES;   // a barrier a slot, the abort flag
    static constexpr int LINE = BARS + (WARPS * STAGES + 1) * 8;
    static constexpr int RING = (LINE + 32 + 15) / 16 * 16;
    static constexpr int JOIN_ROWS = join_rows(R);
    static constexpr int JOIN_LSE = (JOIN_ROWS * 4 + 15) / 16 * 16;
    static constexpr int JOIN = JOIN_LSE + JOIN_ROWS * D * 4;
    static constexpr int MT = D / 16;                   // tiles of O^T
    static constexpr int MIN_CTAS = q8_ctas(D, R);      // of an SM
    static_assert(BLOCK == q8_block(D), "keys of a block");
    // the merge of 8 rows goes through the slot that was read last
    static_assert(8 * D * 4 <= STAGE && 16 * 4 <= SCALE_BYTES, "merge buffer");
};

// Place of granule g (16 bytes) of key row `key` in a slice: the copies' swizzle.
// S^T row g holds key slice_key(g), whose order lets the lanes of a quarter warp that
// read together hit all banks, in keys (rows of two lanes' groups) and in values
// (rows of four lanes).
template <int D>
__device__ __forceinline__ uint32_t place_of(int key, int g) {
    if (D == 64) return (uint32_t)(key * 64 + ((g ^ ((key >> 1) & 3)) << 4));
    return (uint32_t)((g >> 3) * Q8Traits<D, 1>::CHUNK + key * 128 + (((g & 7) ^ (key & 7)) << 4));
}
template <int D>
__device__ __forceinline__ int slice_key(int g) {
    return D == 64 ? g : g ^ ((g & 1) << 2);
}

// Keys that a sequence's splits walk, as in decode.cu: positions [0, span) stand
// for the keys [0, head) and [base, L); lo: the first key of some row's window.
struct Axis {
    int head, base, span, lo;
    __device__ __forceinline__ int key(int x) const { return x < head ? x : x - head + base; }
};
__device__ __forceinline__ Axis key_axis(const DecodeQ8Args& a, int L) {
    Axis s{0, 0, L, 0};
    if (a.window <= 0) return s;
    s.lo = max(0, L - a.Sq - a.window + 1);
    s.base = s.lo & ~63;
    if (a.first > 0) s.head = ((a.first - 1) | 63) + 1;
    if (a.first > L || s.head >= s.base) {
        if (a.first > 0) s.base = 0;
        s.head = 0;
    }
    s.span = s.head + (L - s.base);
    return s;
}

__device__ __forceinline__ uint32_t pack_halves(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ int keys_of(const DecodeQ8Args& a, int b) {
    return max(0, min(a.seqlens_k[b], a.Sk));
}

// Blocks of a unit of batch entry b.
template <int BLOCK>
__device__ __forceinline__ int blocks_of(const DecodeQ8Args& a, int b) {
    return q8_unit_blocks(key_axis(a, keys_of(a, b)).span, BLOCK);
}

// Sum of f(blocks of a unit of entry b) over the entries [b0, b1).
template <int BLOCK, class F>
__device__ __forceinline__ int sum_blocks(const DecodeQ8Args& a, int b0, int b1, F&& f) {
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += f(blocks_of<BLOCK>(a, b));
    return sum;
}

// (Leads, us without / with: 300 x 10 to 4,000 keys x 2 heads at head_dim 128 86.5 / 57.9;
// 128 x 100 to 800 x 8 42.4 / 36.4, at 256 78.3 / 58.9; a lead of one block 35.4 and 62.9
// there, of three 35.7 and 58.3; 16 x 1K to 16K x 8 at 128 53.9 / 54.2.)
//
// The line's cut, by a warp together, each lane with its share of the batch.  mine: what
// this lane's entries take of the line.
template <int BLOCK>
__device__ __forceinline__ Line cut_line(const DecodeQ8Args& a, int& mine) {
    const int lane = threadIdx.x & 31, units = a.Hkv * a.tiles;
    const int per = (a.B + 31) >> 5, b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
    const int blocks = units * sum_blocks<BLOCK>(a, b0, b1, [](int nb) { return nb; });
    int pieces = 0;   // of this lane's entries, of the cut tried last
    const Line line = q8_cut(__reduce_add_sync(0xffffffffu, blocks), a.B * units, a.slots, a.levels, BLOCK,
                             [&](int s) {
                                 pieces = units * sum_blocks<BLOCK>(a, b0, b1, [&](int nb) { return (nb + s - 1) / s; });
                                 return __reduce_add_sync(0xffffffffu, pieces);
                             });
    mine = line.aligned > 0 ? pieces : blocks + kQ8Lead * units * max(0, b1 - b0);
    return line;
}

// Where position pos < line.all lies: batch entry, unit, the unit's start on the line,
// place in it, and its blocks.  (A warp together; mine: of cut_line.)
struct Spot {
    int b, u, start, at, nb;
};
template <int BLOCK>
__device__ __forceinline__ Spot find_on_line(const DecodeQ8Args& a, const Line& line, int mine, int pos) {
    const int lane = threadIdx.x & 31, units = a.Hkv * a.tiles;
    int end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
    }
    const bool here = end - mine <= pos && pos < end;
    const int from_lane = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    int at = end - mine, b = lane * ((a.B + 31) >> 5), nb = 1;
    if (here) {
        for (;; ++b) {
            nb = blocks_of<BLOCK>(a, b);
            if (pos < at + units * line.of_unit(nb)) break;
            at += units * line.of_unit(nb);
        }
    }
    Spot p;
    p.b = __shfl_sync(0xffffffffu, b, from_lane);
    p.nb = __shfl_sync(0xffffffffu, nb, from_lane);
    p.start = __shfl_sync(0xffffffffu, at, from_lane);
    const int len = line.of_unit(p.nb);
    p.u = (pos - p.start) / len;
    p.start += p.u * len;
    p.at = pos - p.start;
    return p;
}

template <int D, int NR>
__global__ void __launch_bounds__(Q8Traits<D, NR>::THREADS, Q8Traits<D, NR>::MIN_CTAS)
    decode_q8_kernel(const __grid_constant__ DecodeQ8Maps tm, const DecodeQ8Args a) {
    using T = Q8Traits<D, NR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(smem), bars = base + T::BARS + warp * T::STAGES * 8;
    const WaitCtx wc{base + T::BARS + T::WARPS * T::STAGES * 8, (uint32_t)a.wait_limit_ns, a.err_word};
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::WARPS * T::STAGES; ++i) mbar_init(base + T::BARS + i * 8, 1);
        st_volatile_shared(wc.abort_flag, 0);
        mbar_fence_init();
        tma_prefetch_desc(&tm.k);
        tma_prefetch_desc(&tm.v);
    }
    __syncthreads();
    wait_for_previous();   // (what is above overlaps the kernel before)
    const bool joined = a.joined != 0;
    const int units = a.Hkv * a.tiles;
    Spot spot;
    int blocks;   // of this CTA
    auto* const kept = reinterpret_cast<Line*>(smem + T::LINE);   // (for the end of segments)
    if (joined) {   // grid (splits of a unit, units, batch entries), the splits a cluster
        cluster_arrive();   // (waited for before the first write to another)
        const int nb = blocks_of<T::BLOCK>(a, blockIdx.z), n = a.chunk / T::BLOCK;
        spot.b = blockIdx.z;
        spot.u = blockIdx.y;
        spot.at = (int)blockIdx.x * n;
        blocks = q8_joined_blocks(nb, spot.at, n);
    } else {
        int mine;
        if (a.head != nullptr && threadIdx.x == 0) a.head[blockIdx.x] = make_int4(0, 0, 0, 0);
        const Line line = cut_line<T::BLOCK>(a, mine);
        const int begin = line.from(blockIdx.x);
        if (begin >= line.all) return;
        const int end = line.from(blockIdx.x + 1);
        blocks = line.all - kQ8Lead * a.B * units;   // before the end, where the line ends there
#pragma unroll 1
        for (int side = end < line.all && line.aligned == 0 ? 1 : 0; side >= 0; --side) {
            spot = find_on_line<T::BLOCK>(a, line, mine, side ? end : begin);
            // blocks before the position: those of the units before, and of its own
            const int before = q8_blocks_before(spot.start, spot.b * units + spot.u, spot.at);
            blocks = side ? before : blocks - before;
        }
        if (line.aligned > 0) {
            spot.at *= line.aligned;
            blocks = min(line.aligned, spot.nb - spot.at);
        } else {
            spot.at = max(0, spot.at - kQ8Lead);
        }
        if (blocks == 0) return;   // (a piece within a lead)
        if (threadIdx.x == 0) *kept = line;
    }

    // ------------------------------------------------ ring
    const uint32_t ring = base + warp * T::WARP_RING, scales = base + T::SCALES + warp * T::WARP_SCALES;
    // The producer's place on the line: unit lu of batch entry lb, block lk; and
    // this lane's key (lane, of 16: lane & 15) of the slice looked up last: its page,
    // -1 where no row sees it, and its row there.  Nothing waits for the page before
    // the slice is issued.
    int lb = spot.b, lu = spot.u, lk = spot.at, l_head = lu / a.tiles;
    Axis la = key_axis(a, keys_of(a, lb));
    const int lane_key = lane & (T::KB - 1);
    int page = -1, page_head = 0;
    unsigned page_row = 0;
    auto look_up = [&]() {
        if (lk * T::BLOCK >= la.span && lk > 0) {   // the next unit
            lk = 0;
            if (++lu == units) {
                lu = 0;
                la = key_axis(a, keys_of(a, ++lb));
            }
            l_head = lu / a.tiles;
        }
        const int x = lk * T::BLOCK + T::KB * warp + lane_key;
        const int key = la.key(x);
        page = -1;
        page_head = l_head;
        ++lk;
        // (a box whose first key no row sees may hold some that a row does)
        const int last = key | (a.box - 1);
        if (x >= la.span || (last < la.lo && key >= a.first)) return;
        const unsigned p = a.by_page((unsigned)key);
        page_row = (unsigned)key - p * (unsigned)a.page_size;
        page = a.block_table[(size_t)lb * a.max_pages + p];
    };
    const int box = min(a.box, T::KB);
    const bool copies = lane < T::KB && (lane & (box - 1)) == 0 && (D != 64 || box > 1);
    int issued = 0, in_slot = 0, out_slot = 0;
    uint32_t out_phase = 0;
    bool ok = true;
    auto issue = [&]() {   // the slice looked up, and the look-up of the next
        if (ok && issued < blocks) {
            const bool there = (unsigned)page < (unsigned)a.num_pages;   // (no page: reads as zeros)
            const int plane = page * a.Hkv + page_head;
            const uint32_t bar = bars + in_slot * 8, to = ring + in_slot * T::STAGE;
            if (D == 64 && box == 1) {
                // single rows of 64 bytes: shorter than a tensor copy's alignment
                if (lane == 0) mbar_arrive(bar);
#pragma unroll
                for (int u = 0; u < T::KB / 8; ++u) {
                    const int key = (lane >> 2) + 8 * u, gr = lane & 3;
                    const int z = __shfl_sync(0xffffffffu, there ? plane : -1, key);
                    const unsigned y = __shfl_sync(0xffffffffu, page_row, key);
                    const size_t src = z < 0 ? 0 : ((size_t)z * a.page_size + y) * 64 + gr * 16;
                    cp_async_16(to + place_of<64>(key, gr), a.k + src, z < 0 ? 0u : 16u);
                    cp_async_16(to + T::SLICE + place_of<64>(key, gr), a.v + src, z < 0 ? 0u : 16u);
                }
            } else if (lane == 0) {
                mbar_arrive_expect_tx(bar, T::STAGE);
            }
            __syncwarp();
            if (copies) {
                const int z = there ? plane : a.planes, y = there ? (int)page_row : 0;
                const uint32_t row = to + lane * T::PITCH;
#pragma unroll
                for (int c = 0; c < (D + 127) / 128; ++c) {
                    tma_load_3d(row + c * T::CHUNK, &tm.k, c * 128, y, z, bar);
                    tma_load_3d(row + T::SLICE + c * T::CHUNK, &tm.v, c * 128, y, z, bar);
                }
            }
            // scales: one of the slice's keys and one of its values where they have no
            // more (every key's to the same place would be one after the other)
            if (!a.flat || lane_key == 0) {
                const size_t at = there ? (size_t)plane * a.blocks + a.by_block(page_row) : 0;
                const uint32_t slot = scales + in_slot * T::SCALE_BYTES + lane_key * 4, size = there ? 4u : 0u;
                if (T::KB == 32 || lane < 16) cp_async_4(slot, a.k_scale + at, size);
                if (T::KB == 32 || lane >= 16) cp_async_4(slot + T::KB * 4, a.v_scale + at, size);
            }
            if (++issued < blocks) look_up();
        }
        cp_async_commit();
        if (++in_slot == T::STAGES) in_slot = 0;
    };
    if (blocks > 0) look_up();
#pragma unroll 1
    for (int s = 0; s < T::STAGES - 1; ++s) issue();
    // places in a slot that this lane reads: keys kg, kg + 8 (16-byte granules, 64 dims
    // on: ^ 64), values of S^T rows 2 t, 2 t + 1 (and + 8)
    const int kg = slice_key<D>(g), v0 = slice_key<D>(2 * t), v1 = slice_key<D>(2 * t + 1);
    const uint32_t k_at = place_of<D>(kg, t);
    const uint32_t v0_at = D == 64 ? place_of<64>(v0, g >> 1) + (g & 1) * 8 : place_of<D>(v0, g);
    const uint32_t v1_at = D == 64 ? place_of<64>(v1, g >> 1) + (g & 1) * 8 : place_of<D>(v1, g);
    const uint32_t scale_at = a.flat ? 0 : kg * 4;
    const uint32_t scale_step = a.flat ? 0 : 32;   // eight keys on

    // This lane's words of query row nr 8 + g of a tile: of each 64 dims the 16 from
    // 16 t on (zeros where there is no such row).
    auto load_query = [&](int b, int hkv, int rbase, int nr, uint32_t (&w)[D / 64][8]) {
        const int pr = rbase + nr * 8 + g;
        const bool real = pr < a.rows;
        const int h = hkv * a.group + pr / a.Sq;
        const uint4* q = reinterpret_cast<const uint4*>(
            a.q + (real ? (((size_t)b * a.Hq + h) * a.Sq + pr % a.Sq) * D : 0) + t * 16);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (real) {
                x = q[c * 8];
                y = q[c * 8 + 1];
            }
            w[c][0] = x.x, w[c][1] = x.y, w[c][2] = x.z, w[c][3] = x.w;
            w[c][4] = y.x, w[c][5] = y.y, w[c][6] = y.z, w[c][7] = y.w;
        }
    };
    // (of a tile of eight rows, the next segment's come while this one is merged)
    uint32_t qw[D / 64][8];
    if (NR == 1) load_query(spot.b, spot.u / a.tiles, spot.u % a.tiles * T::R, 0, qw);

    // ------------------------------------------------ segments: a unit's blocks here
    int left = blocks, b = spot.b, at_unit = spot.u, kb = spot.at, index = 0;
#pragma unroll 1
    do {
        const int L = keys_of(a, b);
        const Axis axis = key_axis(a, L);
        const int nb = q8_unit_blocks(axis.span, T::BLOCK);
        const Segment here = q8_segment(nb, kb, left);
        const int n = here.n;
        const int hkv = at_unit / a.tiles, rbase = (at_unit - hkv * a.tiles) * T::R;
        // ------------------------------------------------ queries
        // B fragments: lane (g, t) has row nr 8 + g, of each 64 dims the 16 from 16 t on
        uint32_t qb[NR][D / 64][8];
        float2 unit[NR];     // scores of rows 2 t, 2 t + 1 are sums times this (log2 units)
        int place[NR][2];    // the rows' keys
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (NR > 1) load_query(b, hkv, rbase, nr, qw);
            const uint32_t(&w)[D / 64][8] = qw;
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    most = fmax3(most, fabsf(__uint_as_float(w[c][e] << 16)),
                                 fabsf(__uint_as_float(w[c][e] & 0xffff0000u)));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // the largest element into [1, 2) (a row of zeros: as it is; exponents whose
            // power would not be a normal number stay short of that)
            int ex = (int)(__float_as_uint(most) >> 23) - 127;
            ex = most == 0.f ? 0 : max(-125, min(ex, 125));
            const float by = __uint_as_float((uint32_t)(127 - ex) << 23);
            const float back = __uint_as_float((uint32_t)(127 + ex) << 23) * a.scale_log2;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    qb[nr][c][e] = pack_halves(__uint_as_float(w[c][e] << 16) * by,
                                               __uint_as_float(w[c][e] & 0xffff0000u) * by);
            unit[nr].x = __shfl_sync(0xffffffffu, back, 8 * t);
            unit[nr].y = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) place[nr][e] = (rbase + nr * 8 + 2 * t + e) % a.Sq + L - a.Sq;
        }
        // keys [all_lo, all_hi) are seen by every row of the sequence, as those below
        // all_first are
        const int all_hi = a.causal ? L - a.Sq + 1 : L;
        const int all_lo = a.window > 0 ? L - a.window : 0;
        const int all_first = min(a.first, all_hi);

        float oacc[NR][T::MT][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int j = 0; j < T::MT; ++j)
                oacc[nr][j][0] = oacc[nr][j][1] = oacc[nr][j][2] = oacc[nr][j][3] = 0.f;
        // of rows 2 t, 2 t + 1: minus the base of the sum, kLift minus that of O (both the
        // same in all lanes of a row), and this lane's part of the sum
        float2 nm[NR], qv[NR], l[NR];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            nm[nr] = qv[nr] = make_float2(kFar, kFar);
            l[nr] = make_float2(0.f, 0.f);
        }

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            issue();   // (into the slot of the block before this one, which every lane has read)
            cp_async_wait<T::STAGES - 1>();
            ok = ok && mbar_wait(bars + out_slot * 8, out_phase, wc, kErrWaitTimeout | kSiteQ8);
            __syncwarp();
            const uint32_t sk0 = ring + out_slot * T::STAGE + k_at, sv0 = ring + out_slot * T::STAGE + T::SLICE;
            const uint32_t sc0 = scales + out_slot * T::SCALE_BYTES + scale_at;
            const int x0 = (kb + i) * T::BLOCK + T::KB * warp;   // the slice's first position, and key
            const int key0 = axis.key(x0);
            const bool whole = x0 + T::KB <= axis.span && key0 + T::KB <= all_hi &&
                               (key0 >= all_lo || key0 + T::KB <= all_first);
            if (!whole) {
                // values that no row sees may be anything, and zero times that would
                // poison O: zeros in their place (a lane per key, a row's granules)
                if (lane < T::KB) {
                    const int key = key0 + lane;
                    if (x0 + lane >= axis.span || (key < axis.lo && key >= a.first)) {
                        const uint32_t at = ring + out_slot * T::STAGE + T::SLICE + lane * T::PITCH;
#pragma unroll 1
                        for (int e = 0; e < D / 16; ++e)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             at + e / (T::PITCH / 16) * T::CHUNK + e % (T::PITCH / 16) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();   // (copies will write here)
                __syncwarp();
            }
#pragma unroll 1
            for (int part = 0; part < T::SUB; part += T::SW) {
                float2 s[T::SW][NR][2];   // scores: of key kg + 8 f in rows 2 t, 2 t + 1
                float lv[T::SW][2];       // log2 of the values' scales
#pragma unroll
                for (int w = 0; w < T::SW; ++w) {
                    const int u16 = 16 * (part + w);
                    float sums[T::SUMS][NR][4];
#pragma unroll
                    for (int i = 0; i < T::SUMS; ++i)
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr)
                            sums[i][nr][0] = sums[i][nr][1] = sums[i][nr][2] = sums[i][nr][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint32_t at = (sk0 ^ ((c & 1) * 64)) + (c >> 1) * T::CHUNK + u16 * T::PITCH;
                        const uint4 x = lds128(at), y = lds128(at + 8 * T::PITCH);
                        const uint32_t xx[4] = {x.x, x.y, x.z, x.w}, yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t a0 = q8_halves(xx[e]), a1 = q8_halves(yy[e]);
                            const uint32_t a2 = q8_halves_up(xx[e]), a3 = q8_halves_up(yy[e]);
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
                                mma_f16_16816(sums[(4 * c + e) % T::SUMS][nr], a0, a1, a2, a3, qb[nr][c][2 * e],
                                              qb[nr][c][2 * e + 1]);
                        }
                    }
                    auto sum_of = [&](int nr, int f) {
                        float2 x = make_float2(sums[0][nr][2 * f], sums[0][nr][2 * f + 1]);
#pragma unroll
                        for (int i = 1; i < T::SUMS; ++i)
                            x = fadd2(x, make_float2(sums[i][nr][2 * f], sums[i][nr][2 * f + 1]));
                        return x;
                    };
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const uint32_t at = sc0 + (2 * (part + w) + f) * scale_step;
                        const float ks = lds32(at);
                        lv[w][f] = lg2_approx(lds32(at + T::KB * 4));
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr)
                            s[w][nr][f] = fmul2(sum_of(nr, f), fmul2(unit[nr], make_float2(ks, ks)));
                    }
                    if (!whole) {
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int at = u16 + kg + 8 * f, key = key0 + at;
                            const bool real = x0 + at < axis.span;
                            // (a scale that belongs to no key of some row may be anything)
                            if (!real || (key < axis.lo && key >= a.first)) lv[w][f] = 0.f;
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int p = place[nr][e];
                                    const bool seen = real && (!a.causal || key <= p) &&
                                                      (a.window <= 0 || key > p - a.window || key < a.first);
                                    float& x = e == 0 ? s[w][nr][f].x : s[w][nr][f].y;
                                    x = seen ? x : -INFINITY;
                                }
                        }
                    }
                }
                // exponents of the probabilities, and of those times the values' scales
                // (kept over the vote where registers allow, else computed again)
                float2 px[T::SW][NR][2], py[T::SW][NR][2];
                auto exponents = [&](int w, int nr, int f) {
                    px[w][nr][f] = fadd2(s[w][nr][f], nm[nr]);
                    py[w][nr][f] = fadd2(s[w][nr][f], fadd2(qv[nr], make_float2(lv[w][f], lv[w][f])));
                };
                float most = -INFINITY, most_v = -INFINITY;
#pragma unroll
                for (int w = 0; w < T::SW; ++w)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            exponents(w, nr, f);
                            most = fmax3(most, px[w][nr][f].x, px[w][nr][f].y);
                            most_v = fmax3(most_v, py[w][nr][f].x, py[w][nr][f].y);
                        }
                if (__any_sync(0xffffffffu, most > kGrow || most_v > kGrow + kLift)) {
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = -INFINITY, y = -INFINITY;
#pragma unroll
                            for (int w = 0; w < T::SW; ++w)
#pragma unroll
                                for (int f = 0; f < 2; ++f) {
                                    const float z = e == 0 ? s[w][nr][f].x : s[w][nr][f].y;
                                    x = fmaxf(x, z);
                                    y = fmaxf(y, z + lv[w][f]);
                                }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) {
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
                            }
                            float& old = e == 0 ? nm[nr].x : nm[nr].y;
                            float& old_v = e == 0 ? qv[nr].x : qv[nr].y;
                            const float now = fminf(old, -x), now_v = fminf(old_v, kLift - y);
                            float& sum = e == 0 ? l[nr].x : l[nr].y;
                            sum *= ex2_approx(now - old);
                            const float by = ex2_approx(now_v - old_v);
                            old = now;
                            old_v = now_v;
#pragma unroll
                            for (int j = 0; j < T::MT; ++j) {
                                oacc[nr][j][e] *= by;
                                oacc[nr][j][2 + e] *= by;
                            }
                        }
                    if (T::KEEP) {
#pragma unroll
                        for (int w = 0; w < T::SW; ++w)
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                exponents(w, nr, 0);
                                exponents(w, nr, 1);
                            }
                    }
                }
#pragma unroll
                for (int w = 0; w < T::SW; ++w) {
                    const int u16 = 16 * (part + w);
                    uint32_t pb[NR][2];
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            if (!T::KEEP) exponents(w, nr, f);
                            const float2 x = px[w][nr][f], y = py[w][nr][f];
                            l[nr] = fadd2(l[nr], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                            pb[nr][f] = movmatrix_trans(pack_halves(ex2_approx(y.x), ex2_approx(y.y)));
                        }
                    // O^T += V^T P^T: lane (g, t) has 16 dims (64: 8) of four keys
                    auto add = [&](int j, uint32_t x0_, uint32_t x1_, uint32_t y0_, uint32_t y1_) {
                        // words of four dims of the keys: tiles j (dims 0, 1) and j + 1 (dims 2, 3)
                        const uint32_t xl = __byte_perm(x0_, x1_, 0x5140), xh = __byte_perm(x0_, x1_, 0x7362);
                        const uint32_t yl = __byte_perm(y0_, y1_, 0x5140), yh = __byte_perm(y0_, y1_, 0x7362);
                        const uint32_t a0 = q8_halves(xl), a1 = q8_halves_up(xl);
                        const uint32_t a2 = q8_halves(yl), a3 = q8_halves_up(yl);
                        const uint32_t b0 = q8_halves(xh), b1 = q8_halves_up(xh);
                        const uint32_t b2 = q8_halves(yh), b3 = q8_halves_up(yh);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            mma_f16_16816(oacc[nr][j], a0, a1, a2, a3, pb[nr][0], pb[nr][1]);
                            mma_f16_16816(oacc[nr][j + 1], b0, b1, b2, b3, pb[nr][0], pb[nr][1]);
                        }
                    };
                    const uint32_t sv = sv0 + u16 * T::PITCH;
                    if constexpr (D == 64) {
                        const uint2 x0_ = lds64(sv + v0_at), x1_ = lds64(sv + v1_at);
                        const uint2 y0_ = lds64(sv + v0_at + 8 * T::PITCH), y1_ = lds64(sv + v1_at + 8 * T::PITCH);
                        add(0, x0_.x, x1_.x, y0_.x, y1_.x);
                        add(2, x0_.y, x1_.y, y0_.y, y1_.y);
                    } else {
#pragma unroll
                        for (int c = 0; c < D / 128; ++c) {
                            const uint32_t at = sv + c * T::CHUNK;
                            const uint4 x0_ = lds128(at + v0_at), x1_ = lds128(at + v1_at);
                            const uint4 y0_ = lds128(at + v0_at + 8 * T::PITCH);
                            const uint4 y1_ = lds128(at + v1_at + 8 * T::PITCH);
                            add(c * 8, x0_.x, x1_.x, y0_.x, y1_.x);
                            add(c * 8 + 2, x0_.y, x1_.y, y0_.y, y1_.y);
                            add(c * 8 + 4, x0_.z, x1_.z, y0_.z, y1_.z);
                            add(c * 8 + 6, x0_.w, x1_.w, y0_.w, y1_.w);
                        }
                    }
                }
            }
            __syncwarp();
            if (++out_slot == T::STAGES) {
                out_slot = 0;
                out_phase ^= 1u;
            }
        }

        // the next segment
        const bool last_unit = at_unit + 1 == units;
        const int next_b = last_unit ? b + 1 : b, next_unit = last_unit ? 0 : at_unit + 1;
        if (NR == 1 && here.more)
            load_query(next_b, next_unit / a.tiles, next_unit % a.tiles * T::R, 0, qw);

        // ------------------------------------------------ merge of the warps
        // eight rows at a time through the slot that was read last, which is free until
        // the next block is begun: [8][D] O (columns turned by the row
        // against bank conflicts), and row maxima and sums through its scales
        const int last_slot = (out_slot == 0 ? T::STAGES : out_slot) - 1;
        const float* merge0 = reinterpret_cast<const float*>(smem + last_slot * T::STAGE);
        float* mine = reinterpret_cast<float*>(smem + warp * T::WARP_RING + last_slot * T::STAGE);
        constexpr int WF = T::WARP_RING / 4, WS = T::WARP_SCALES / 4;   // floats from warp to warp
        const float* ml0 = reinterpret_cast<const float*>(smem + T::SCALES + last_slot * T::SCALE_BYTES);
        float* ml = reinterpret_cast<float*>(smem + T::SCALES + warp * T::WARP_SCALES +
                                             last_slot * T::SCALE_BYTES);
        const int valid_rows = min(T::R, a.rows - rbase);
        const bool whole_unit = n == nb;
        // joined: split s finishes the rows [s own, (s + 1) own) (see decode.cu)
        const int split = blockIdx.x;
        const int own = joined ? (T::R + a.n_splits - 1) / a.n_splits : 1;
        const uint32_t jl = smem_u32(smem) + T::RING, jo = jl + T::JOIN_LSE;
        auto row_id = [&](int r) {
            const int pr = rbase + r;
            return ((size_t)b * a.Hq + hkv * a.group + pr / a.Sq) * a.Sq + pr % a.Sq;
        };
        const int part = 2 * (int)blockIdx.x + (index > 0);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (nr * 8 >= valid_rows) break;
            if (joined && nr == 0) cluster_wait();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = e == 0 ? l[nr].x : l[nr].y;
                const float to_m = e == 0 ? nm[nr].x : nm[nr].y, to_v = e == 0 ? qv[nr].x : qv[nr].y;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const int r = 2 * t + e;
                if (g == 0) {
                    ml[r] = -to_m;
                    ml[8 + r] = sum;
                }
                // O in the base of the sum (a row without keys: 0 times 1 or 0)
                const float by = ex2_approx(to_m - to_v);
#pragma unroll
                for (int j = 0; j < T::MT; ++j) {
                    const int dim = D == 64 ? g * 8 + 2 * j : (j >> 3) * 128 + g * 16 + 2 * (j & 7);
                    *reinterpret_cast<float2*>(mine + r * D + ((dim + 4 * r) & (D - 1))) =
                        make_float2(oacc[nr][j][e] * by, oacc[nr][j][2 + e] * by);
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int e = threadIdx.x * 4; e < 8 * D; e += T::THREADS * 4) {
                const int r8 = e / D, c = e % D, r = nr * 8 + r8;
                if (r >= valid_rows) break;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < T::WARPS; ++w) M = fmaxf(M, ml0[w * WS + r8]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                const size_t row = row_id(r);
                const bool sink = whole_unit && !joined && a.sinks != nullptr;
                const float sg = sink ? a.sinks[hkv * a.group + (rbase + r) / a.Sq] * kLog2ef : -INFINITY;
                M = fmaxf(M, sg);   // (finite: at least -kFar)
                float sum = ex2_approx(sg - M);
#pragma unroll
                for (int w = 0; w < T::WARPS; ++w) {
                    const float f = ex2_approx(ml0[w * WS + r8] - M);
                    const float4 x = *reinterpret_cast<const float4*>(merge0 + w * WF + r8 * D +
                                                                      ((c + 4 * r8) & (D - 1)));
                    sum = fmaf(f, ml0[w * WS + 8 + r8], sum);
                    o.x = fmaf(f, x.x, o.x);
                    o.y = fmaf(f, x.y, o.y);
                    o.z = fmaf(f, x.z, o.z);
                    o.w = fmaf(f, x.w, o.w);
                }
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                const float lse2 = sum > 0.f ? M + lg2_approx(sum) : -INFINITY;
                if (joined) {
                    const int to = r / own, at = split * own + r - to * own;
                    cluster_write4(jo + (at * D + c) * 4, to, o);
                    if (c == 0) cluster_write(jl + at * 4, to, lse2);
                } else if (whole_unit) {
                    *reinterpret_cast<uint2*>(a.o + row * D + c) =
                        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                    if (c == 0) a.lse[row] = lse2 * kLn2f;
                } else {
                    *reinterpret_cast<float4*>(a.part_o + ((size_t)part * T::R + r) * D + c) = o;
                    if (c == 0) a.part_lse[(size_t)part * T::R + r] = lse2;
                }
            }
            fence_proxy_async_smem();   // (copies will write here)
            __syncthreads();
        }
        if (joined) {
            cluster_sync_all();
#pragma unroll 1
            for (int e = threadIdx.x * 4; e < own * D; e += T::THREADS * 4) {
                const int k = e / D, c = e % D, r = split * own + k;
                if (r >= valid_rows) break;
                const uint8_t* from = smem + T::RING;
                const float sg = a.sinks != nullptr ? a.sinks[hkv * a.group + (rbase + r) / a.Sq] * kLog2ef : -INFINITY;
                float x[kJoinSplits], M = sg, sum = 0.f;
                float4 y[kJoinSplits], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < kJoinSplits; ++s) {
                    x[s] = -INFINITY;
                    y[s] = o;
                    if (s < a.n_splits) {
                        x[s] = *reinterpret_cast<const float*>(from + (s * own + k) * 4);
                        y[s] = *reinterpret_cast<const float4*>(from + T::JOIN_LSE + ((s * own + k) * D + c) * 4);
                    }
                    M = fmaxf(M, x[s]);
                }
                if (M != -INFINITY) {
                    sum = ex2_approx(sg - M);
#pragma unroll
                    for (int s = 0; s < kJoinSplits; ++s) {
                        const float f = ex2_approx(x[s] - M);
                        sum += f;
                        o.x = fmaf(f, y[s].x, o.x);
                        o.y = fmaf(f, y[s].y, o.y);
                        o.z = fmaf(f, y[s].z, o.z);
                        o.w = fmaf(f, y[s].w, o.w);
                    }
                }
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                const size_t row = row_id(r);
                *reinterpret_cast<uint2*>(a.o + row * D + c) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (c == 0) a.lse[row] = sum > 0.f ? (M + lg2_approx(sum)) * kLn2f : -INFINITY;
            }
            break;
        }
        // (the unit starts here and goes on: what the merge by pieces has to know)
        if (kb == 0 && !whole_unit && a.head != nullptr && threadIdx.x == 0) {
            const Line cut = *kept;
            const int from = cut.aligned > 0 ? (int)blockIdx.x : cut.from(blockIdx.x + 1) - n - kQ8Lead;
            const Pieces pc = q8_pieces(cut, from, nb);
            a.head[blockIdx.x] = make_int4(b, at_unit, pc.count, pc.second);
        }
        left -= n;
        kb = 0;
        ++index;
        at_unit = next_unit;
        b = next_b;
    } while (left > 0);
    cp_async_wait<0>();
    if (!ok) {   // given up: what was asked for must have landed before the CTA exits
#pragma unroll 1
        for (int q = max(0, issued - T::STAGES); q < issued; ++q)
            mbar_wait_drain(bars + q % T::STAGES * 8, (uint32_t)(q / T::STAGES) & 1u, a.wait_limit_ns);
    }
}

// Merge of units in a few pieces: CTA (piece that such a unit starts in, eight rows
// of its tile), a warp per row.
template <int D>
__global__ void __launch_bounds__(256) combine_few_kernel(const DecodeQ8Args a, int tile) {
    constexpr int PER = D / 32;   // columns of a lane, two side by side
    wait_for_previous();
    const int4 hd = a.head[blockIdx.x];   // batch entry, unit, pieces, the first's slot
    if (hd.z < 2) return;
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int hkv = hd.y / a.tiles, pr = (hd.y - hkv * a.tiles) * tile + r;
    if (pr >= a.rows) return;
    const Pieces pc{(int)blockIdx.x, hd.z, hd.w};
    const int h = hkv * a.group + pr / a.Sq;
    const float sg = a.sinks != nullptr ? a.sinks[h] * kLog2ef : -INFINITY;
    float M = sg, sum = sg == -INFINITY ? 0.f : 1.f, acc[PER];   // (the sink's own term)
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < pc.count; k0 += 4) {   // (four in flight)
        float x[4];
        float2 y[4][PER / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const size_t at = (size_t)pc.slot(min(k0 + k, pc.count - 1)) * tile + r;
            x[k] = k0 + k < pc.count ? a.part_lse[at] : -INFINITY;
#pragma unroll
            for (int e = 0; e < PER / 2; ++e)
                y[k][e] = *reinterpret_cast<const float2*>(a.part_o + at * D + e * 64 + 2 * lane);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (x[k] == -INFINITY) continue;
            const float top = fmaxf(M, x[k]), old = ex2_approx(M - top), f = ex2_approx(x[k] - top);
            M = top;
            sum = fmaf(sum, old, f);
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) {
                acc[2 * e] = fmaf(acc[2 * e], old, f * y[k][e].x);
                acc[2 * e + 1] = fmaf(acc[2 * e + 1], old, f * y[k][e].y);
            }
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const size_t row = ((size_t)hd.x * a.Hq + h) * a.Sq + pr % a.Sq;
#pragma unroll
    for (int e = 0; e < PER / 2; ++e)
        *reinterpret_cast<uint32_t*>(a.o + row * D + e * 64 + 2 * lane) =
            pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0) a.lse[row] = sum > 0.f ? (M + lg2_approx(sum)) * kLn2f : -INFINITY;
}

// Merge of few units in many pieces: CTA (unit, row), sixteen warps over the pieces, each
// with a base of its own, merged at the end.
constexpr int kCombineWarps = 16;
template <int D, int BLOCK>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_q8_kernel(const DecodeQ8Args a, int tile) {
    constexpr int PER = D / 32;   // columns of a lane, two side by side
    __shared__ float other[kCombineWarps][D], base[kCombineWarps], weight[kCombineWarps];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
    const int units = a.Hkv * a.tiles, b = (int)blockIdx.x / units, u = (int)blockIdx.x - b * units;
    const int hkv = u / a.tiles, pr = (u - hkv * a.tiles) * tile + r;
    if (pr >= a.rows) return;
    int mine;
    const Line line = cut_line<BLOCK>(a, mine);
    const int nb = blocks_of<BLOCK>(a, b), len = line.of_unit(nb);
    int before = 0;   // its batch entry's place on the line
    for (int i = lane; i < b; i += 32)
        before += units * line.of_unit(blocks_of<BLOCK>(a, i));
    before = __reduce_add_sync(0xffffffffu, before);
    const Pieces pc = q8_pieces(line, before + u * len, nb);
    if (pc.count < 2) return;
    const int h = hkv * a.group + pr / a.Sq;
    auto at = [&](int k) { return (size_t)pc.slot(k) * tile + r; };
    // the warp's pieces: warp, warp + 16, ...; lane l has the weight of the l-th
    float M = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int k0 = warp; k0 < pc.count; k0 += 32 * kCombineWarps) {
        const int its = k0 + lane * kCombineWarps;
        const float x = its < pc.count ? a.part_lse[at(its)] : -INFINITY;
        float top = fmaxf(x, M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top == -INFINITY) continue;
        const float old = ex2_approx(M - top), w = ex2_approx(x - top);
        M = top;
        sum *= old;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= old;
        const int n = min(32, (pc.count - k0 + kCombineWarps - 1) / kCombineWarps);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float f = __shfl_sync(0xffffffffu, w, k);
            const float* po = a.part_o + at(k0 + k * kCombineWarps) * D + 2 * lane;
            sum += f;
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const float2 y = *reinterpret_cast<const float2*>(po + e * 32);
                acc[e] = fmaf(f, y.x, acc[e]);
                acc[e + 1] = fmaf(f, y.y, acc[e + 1]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        *reinterpret_cast<float2*>(&other[warp][e * 32 + 2 * lane]) = make_float2(acc[e], acc[e + 1]);
    if (lane == 0) {
        base[warp] = M;
        weight[warp] = sum;
    }
    __syncthreads();
    const int c = threadIdx.x * 2;
    if (c >= D) return;
    const float sg = a.sinks != nullptr ? a.sinks[h] * kLog2ef : -INFINITY;
    M = sg;
    for (int w = 0; w < kCombineWarps; ++w) M = fmaxf(M, base[w]);
    float2 o = make_float2(0.f, 0.f);
    sum = 0.f;
    if (M != -INFINITY) {
        sum = ex2_approx(sg - M);
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) {
            const float f = ex2_approx(base[w] - M);
            sum = fmaf(f, weight[w], sum);
            o.x = fmaf(f, other[w][c], o.x);
            o.y = fmaf(f, other[w][c + 1], o.y);
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const size_t row = ((size_t)b * a.Hq + h) * a.Sq + pr % a.Sq;
    *reinterpret_cast<uint32_t*>(a.o + row * D + c) = pack_bf16x2(o.x * inv, o.y * inv);
    if (c == 0) a.lse[row] = sum > 0.f ? (M + lg2_approx(sum)) * kLn2f : -INFINITY;
}

// (What is asked of the runtime once per device: a small call takes seven microseconds.)
constexpr int kAlign = 1024, kDevices = 64;

// Lets the kernel have the shared memory that it takes on the current device.
template <int D, int NR>
cudaError_t allow_shared(int& dev) {
    using T = Q8Traits<D, NR>;
    static std::atomic<bool> allowed[kDevices];
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < kDevices;
    if (!keep || !allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(decode_q8_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kAlign + T::RING + T::JOIN);
        if (e != cudaSuccess) return e;
        if (keep) allowed[dev].store(true, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

// Clusters of n CTAs that the current device holds at once (0: not known).
template <int D, int NR>
int clusters_at_once(int n) {
    using T = Q8Traits<D, NR>;
    static std::atomic<int> known[kDevices][kJoinSplits + 1];
    int dev = 0, count = 0;
    if (n < 1 || n > kJoinSplits || allow_shared<D, NR>(dev) != cudaSuccess) return 0;
    const bool keep = dev >= 0 && dev < kDevices;
    if (keep) count = known[dev][n].load(std::memory_order_relaxed);
    if (count > 0) return count;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)n;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((unsigned)n);
    config.blockDim = dim3(T::THREADS);
    config.dynamicSmemBytes = kAlign + T::RING + T::JOIN;
    config.attrs = &attr;
    config.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&count, decode_q8_kernel<D, NR>, &config) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (keep) known[dev][n].store(count, std::memory_order_relaxed);
    return count;
}

template <int D, int NR>
cudaError_t launch_tile(const DecodeQ8Launch& p, cudaStream_t s) {
    using T = Q8Traits<D, NR>;
    const DecodeQ8Args& a = p.args;
    int dev = 0;
    cudaError_t e = allow_shared<D, NR>(dev);
    if (e != cudaSuccess) return e;
    if (a.joined)
        return launch_dependent_clusters(
            decode_q8_kernel<D, NR>, (unsigned)a.n_splits,
            dim3((unsigned)a.n_splits, (unsigned)(a.Hkv * a.tiles), (unsigned)a.B), dim3(T::THREADS),
            kAlign + T::RING + T::JOIN, s, p.maps, a);
    e = launch_dependent(decode_q8_kernel<D, NR>, dim3((unsigned)a.n_splits), dim3(T::THREADS),
                         kAlign + T::RING, s, p.maps, a);
    if (e != cudaSuccess) return e;
    if (a.head != nullptr)
        return launch_dependent(combine_few_kernel<D>, dim3((unsigned)a.n_splits, (unsigned)(T::R / 8)), dim3(256),
                                0, s, a, (int)T::R);
    return launch_dependent(combine_q8_kernel<D, T::BLOCK>,
                            dim3((unsigned)(a.B * a.Hkv * a.tiles), (unsigned)T::R), dim3(kCombineWarps * 32), 0,
                            s, a, (int)T::R);
}

template <int D>
cudaError_t launch_dim(const DecodeQ8Launch& p, cudaStream_t s) {
    switch (p.tile) {
        case 8: return launch_tile<D, 1>(p, s);
        case 16: return launch_tile<D, 2>(p, s);
        default:
            if constexpr (D == 64) return launch_tile<D, 4>(p, s);
            else return cudaErrorInvalidValue;
    }
}

}  // namespace

int decode_q8_clusters(int head_dim, int tile, int n) {
    switch (head_dim) {
        case 64:
            return tile == 8    ? clusters_at_once<64, 1>(n)
                   : tile == 16 ? clusters_at_once<64, 2>(n)
                                : clusters_at_once<64, 4>(n);
        case 128: return tile == 8 ? clusters_at_once<128, 1>(n) : clusters_at_once<128, 2>(n);
        default: return tile == 8 ? clusters_at_once<256, 1>(n) : clusters_at_once<256, 2>(n);
    }
}

cudaError_t launch_decode_q8(const DecodeQ8Launch& p, int head_dim, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_dim<64>(p, s);
        case 128: return launch_dim<128>(p, s);
        case 256: return launch_dim<256>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
