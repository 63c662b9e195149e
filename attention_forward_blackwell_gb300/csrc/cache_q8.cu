// Appending to and reading from a paged cache held in 8 bits (fa_cache_append_q8,
// fa_cache_read_q8).
//
// The cache: codes [num_pages, hkv, page_size, d] in e4m3 and scales [num_pages,
// hkv, page_size / block] in fp32, one for `block` keys of a head.  A scale that
// the append chooses is a power of two (q8_scale): a code then carries the same
// three bits of fraction whatever the scale, and rows that lay in a block before
// are taken to a larger one exactly (but for what falls below the smallest normal
// code), so that nothing is lost by appending row by row.  It goes by the lengths
// of the pairs, which a rotation does not change: the scale of a block does not
// depend on its rows' positions, nor on the last bits of a sine.
#include "../../include/fa.h"
#include "q8.cuh"
#include "rope.cuh"

namespace fa {
namespace {

struct Q8Cache {
    uint8_t* codes[2];         // of keys and values
    float* scales[2];
    PageTable pages;
    int hkv, block;
    int blocks;                // of a page
    FastDiv by_block;          // by block
};

// ------------------------------------------------------------ append ----

struct AppendArgs {
    Q8Cache c;
    Turn turn;
    int tasks;                 // of a row: d / 16
    const int* lens;
    int n;
    const int* n_new;          // [batch] or nullptr (n)
    const int* copies;         // [batch, 3] or nullptr
    const int* positions;      // nullptr: lens[b] + i
    long long position_stride;
    const uint4* src[3];       // new keys, new values, queries; strides in granules of 8
    long long ss[3][3];
    int hq;
    uint4* q_out;              // [batch, hq, n, d]
    FastDiv by_tasks, by_hq;
    int units;                 // blocks that an entry's new rows may lie in
    int kv_ctas;               // CTAs along y that append; the rest turn queries
};

// Tasks that a thread keeps between the two passes over a block (a unit's in a warp, in
// a CTA).  More cost a CTA's registers more than they spare (head_dim 128, 64 keys to a
// block, 8 heads: 64 entries x 64 tokens 12.0 us with four, 10.6 with two, 10.9 with one;
// 16 x 2,048 51.8, 50.6, 53.1).
constexpr int kKeptWarp = 4, kKeptCta = 2;
// A unit has 128 threads where it keeps them busy with at most kPasses tasks each and
// there are more than kFewUnits units of keys an SM, else 256: 8 x 600 tokens x 8
// heads 11.8 us with 128, 12.4 with 256; 1 x 2,048 7.3 and 6.6; at head_dim 256, 8 x 600 x 4
// heads 13.7 and 12.0.
constexpr int kPasses = 4, kFewUnits = 4;

// Codes of a granule, its elements times inv.
__device__ __forceinline__ uint2 codes_of(const Granule& x, float inv) {
    const float2 i2 = both(inv);
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fmul2(make_float2(x.even[i], x.odd[i]), i2);
    return make_uint2(q8_codes(y[0].x, y[0].y, y[1].x, y[1].y), q8_codes(y[2].x, y[2].y, y[3].x, y[3].y));
}
// Largest square of a granule's elements, and of its interleaved pairs' lengths.
// (Products of bf16 values are exact in fp32, a sum of two rounds once.)
__device__ __forceinline__ float square_of(const Granule& x) {
    float m = fmax3(fabsf(x.even[0]), fabsf(x.odd[0]), fabsf(x.even[1]));
    m = fmax3(m, fabsf(x.odd[1]), fabsf(x.even[2]));
    m = fmax3(m, fabsf(x.odd[2]), fabsf(x.even[3]));
    m = fmaxf(m, fabsf(x.odd[3]));
    return m * m;
}
__device__ __forceinline__ float square_of_pairs(const float (&x)[4], const float (&y)[4]) {
    const float2 a0 = make_float2(x[0], x[1]), a1 = make_float2(x[2], x[3]);
    const float2 b0 = make_float2(y[0], y[1]), b1 = make_float2(y[2], y[3]);
    const float2 p = ffma2(a0, a0, fmul2(b0, b0)), q = ffma2(a1, a1, fmul2(b1, b1));
    return fmax3(fmaxf(p.x, p.y), q.x, q.y);
}

// Queries of batch entry b: as in rope.cu, a task a thread.
template <bool INTERLEAVED>
__device__ void append_queries(const AppendArgs& a, int b, int len, int n) {
    const unsigned all = (unsigned)n * (unsigned)(a.hq * a.tasks);   // (below 2^31: the host sees to it)
    const long long cta = (long long)(blockIdx.y - a.kv_ctas) * gridDim.x + blockIdx.x;
    const long long step = (long long)(gridDim.y - a.kv_ctas) * gridDim.x * blockDim.x;
    for (long long e_ = cta * blockDim.x + threadIdx.x; e_ < (long long)all; e_ += step) {
        const unsigned e = (unsigned)e_;
        const unsigned r = a.by_tasks(e), i = a.by_hq(r);
        const int j = (int)(e - r * (unsigned)a.tasks), h = (int)(r - i * (unsigned)a.hq);
        const TaskAt at = task_at<INTERLEAVED>(a.turn.rot, a.tasks, j);
        const uint4* from = a.src[2] + b * a.ss[2][0] + h * a.ss[2][1] + (long long)i * a.ss[2][2];
        uint4* to = a.q_out + (((long long)b * a.hq + h) * a.n + (int)i) * (2 * a.tasks);
        uint4 u = from[at.a >> 3], w = from[at.b >> 3];
        if (at.turned_a || at.turned_b) {
            Angles g;
            angles_of<INTERLEAVED>(a.turn, at,
                                   a.positions != nullptr ? a.positions[b * a.position_stride + i]
                                                          : (int)((unsigned)len + i),
                                   g);
            Granule x = unpack8(u), y = unpack8(w);
            turn_task<INTERLEAVED>(at, g, x, y);
            u = pack8(x);
            w = pack8(y);
        }
        to[at.a >> 3] = u;
        to[at.b >> 3] = w;
    }
}

// A unit is a block of an entry's keys or of its values, of a head; WARP: a warp has
// one, four a CTA (few rows), else a CTA.  CTA (block, heads and keys or values -- past
// kv_ctas: queries --, batch entry).  Two passes over the new rows of a block: their
// reach, then their codes; the first tasks that a thread has of them stay in registers in
// between, the others are read again (from L1 or L2).  A block has one writer, so nothing
// is atomic.  Single tokens are bound by a chain of loads (length, page, scale; the rows,
// and the angles that need only the length, come beside it): 128 tokens x 8 heads, with
// 32 heads of queries, 4.4 us.  Chunks move 3 bytes an element and are bound
// by the instructions, half of them for the angles: 16 x 2,048 tokens x 8 heads of 128
// 50.6 us, 4.0 TB/s.  (Four heads of keys to a CTA by the same angles, read again for
// the codes, took 52.3 there and 14.8 for 11.7 at 8 x 600: fewer CTAs, more registers.)
template <bool INTERLEAVED, bool WARP>
__global__ void append_q8_kernel(const AppendArgs a) {
    constexpr int kKept = WARP ? kKeptWarp : kKeptCta;
    __shared__ float most[8];
    dependents_may_start();
    wait_for_previous();
    const Q8Cache& c = a.c;
    const int b = blockIdx.z;
    const int start = max(a.lens[b], 0);
    int n = max(0, min(a.n_new != nullptr ? a.n_new[b] : a.n, a.n));
    if ((int)blockIdx.y >= a.kv_ctas) {
        if (n > 0) append_queries<INTERLEAVED>(a, b, start, n);
        return;
    }
    const int T = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int which = WARP ? blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.y;
    if (WARP && which >= 2 * c.hkv) return;
    const int h = which >> 1, kind = which & 1;
    // (what lies behind the table has no page; len + n stays in 32 bits)
    const int room = c.pages.max_pages * c.pages.page_size, len = min(start, room);
    n = min(n, room - len);
    uint8_t* const codes = kind == 0 ? c.codes[0] : c.codes[1];
    float* const scales = kind == 0 ? c.scales[0] : c.scales[1];
    const int d = a.tasks * 16, num_pages = c.pages.num_pages;
    auto row_of = [&](int page, int row) {
        return codes + (((size_t)page * c.hkv + h) * c.pages.page_size + row) * d;
    };
    auto scale_of = [&](int page, int block) {
        return scales + ((size_t)page * c.hkv + h) * c.blocks + block;
    };
    const int first0 = (int)c.by_block((unsigned)len) * c.block;   // the open block: where the next key goes
    // the page that reserve replaced: its rows below `copied` come along
    int from = -1, copied = 0;
    bool moved = false;   // the open block's earlier rows are taken by the unit that fills it
    if (a.copies != nullptr) {
        from = a.copies[3 * b];
        const int to = a.copies[3 * b + 1];
        copied = min(a.copies[3 * b + 2], c.pages.page_size);
        if ((unsigned)from >= (unsigned)num_pages || (unsigned)to >= (unsigned)num_pages || from == to)
            copied = 0;
        int page0 = -1, row0 = 0;
        key_page(c.pages, b, first0, page0, row0);
        moved = copied > 0 && page0 == to && len > first0 && row0 + (len - first0) == copied;
        if ((int)blockIdx.x >= a.units) {   // a whole block of a replaced page
            const int block = blockIdx.x - a.units, at = block * c.block;
            const int rows = min(c.block, copied - at);
            if (rows <= 0 || (moved && at == row0)) return;
            const uint4* s = reinterpret_cast<const uint4*>(row_of(from, at));
            uint4* t = reinterpret_cast<uint4*>(row_of(to, at));
            for (int e = tid; e < rows * a.tasks; e += T) t[e] = s[e];
            if (tid == 0) *scale_of(to, block) = *scale_of(from, block);
            return;
        }
    }
    const long long first_ = first0 + (long long)blockIdx.x * c.block;
    const int first = (int)min(first_, (long long)room);
    const int lo = max(first, len), hi = (int)min(first_ + c.block, (long long)len + n);
    const bool takes_over = moved && blockIdx.x == 0;
    if (lo >= hi && !takes_over) return;
    const uint4* src = (kind == 0 ? a.src[0] : a.src[1]) + b * a.ss[kind][0] + h * a.ss[kind][1];
    const long long step = a.ss[kind][2];
    const int rot = kind == 0 ? a.turn.rot : 0;
    // a thread has one task of the rows i0, i0 + slots, ...: what goes by the task alone
    // is worked out once
    const int slots = (int)a.by_tasks((unsigned)T), slot = (int)a.by_tasks((unsigned)tid), rows = max(0, hi - lo);
    const int i0 = slot < slots ? slot : rows;
    const TaskAt at = task_at<INTERLEAVED>(rot, a.tasks, tid - slot * a.tasks);
    const bool turned = at.turned_a || at.turned_b;
    const uint4* const mine = src + (lo - len + i0) * step + (at.a >> 3);
    const int apart = (at.b - at.a) >> 3;
    const long long stride = slots * step;
    uint4 ka[kKept], kb[kKept];
    auto load = [&](int k, uint4& u, uint4& w) {   // of row i0 + k slots
        const uint4* r = mine + k * stride;
        u = r[0];
        w = r[apart];
    };
    auto angles = [&](int k, Angles& g) {
        const int new_row = lo - len + i0 + k * slots;
        angles_of<INTERLEAVED>(a.turn, at,
                               a.positions != nullptr ? a.positions[b * a.position_stride + new_row]
                                                      : (int)((unsigned)start + new_row),
                               g);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (i0 + k * slots < rows) load(k, ka[k], kb[k]);
    int page, row;   // (a block lies in one page)
    const bool there = key_page(c.pages, b, first, page, row);
    Angles g;
    if (turned && i0 < rows) angles(0, g);
    if (!there) return;
    const int block = (int)c.by_block((unsigned)row);
    const int old_page = takes_over ? from : page;
    const float before = lo > first ? *scale_of(old_page, block) : 0.f;
    float square = 0.f;
    const float f2 = a.turn.factor * a.turn.factor;
    auto reach = [&](const uint4& u, const uint4& w) {
        const Granule x = unpack8(u), y = unpack8(w);
        float turned_most = 0.f, rest = 0.f;
        if (INTERLEAVED) {
            if (at.turned_a) turned_most = square_of_pairs(x.even, x.odd);
            else rest = square_of(x);
            if (at.turned_b) turned_most = fmaxf(turned_most, square_of_pairs(y.even, y.odd));
            else rest = fmaxf(rest, square_of(y));
        } else if (at.turned_a) {
            turned_most = fmaxf(square_of_pairs(x.even, y.even), square_of_pairs(x.odd, y.odd));
        } else {
            rest = fmaxf(square_of(x), square_of(y));
        }
        square = fmaxf(square, fmaxf(turned_most * f2, rest));
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (i0 + k * slots < rows) reach(ka[k], kb[k]);
    for (int k = kKept; i0 + k * slots < rows; ++k) {
        uint4 u, w;
        load(k, u, w);
        reach(u, w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square = fmaxf(square, __shfl_xor_sync(0xffffffffu, square, o));
    if (!WARP) {
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = square;
        __syncthreads();   // (every thread has read `before` too)
        for (int w = 0; w < T / 32; ++w) square = fmaxf(square, most[w]);
    }
    const float now = hi > lo ? fmaxf(before, q8_scale(square)) : before;
    const float inv = 1.f / now;
    uint8_t* const to = row_of(page, row + (lo - first) + i0);
    auto store = [&](int k, const uint4& u, const uint4& w) {
        Granule x = unpack8(u), y = unpack8(w);
        if (turned) turn_task<INTERLEAVED>(at, g, x, y);
        uint8_t* const r = to + (size_t)(k * slots) * d;
        *reinterpret_cast<uint2*>(r + at.a) = codes_of(x, inv);
        *reinterpret_cast<uint2*>(r + at.b) = codes_of(y, inv);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        if (i0 + k * slots >= rows) break;
        if (k > 0 && turned) angles(k, g);
        store(k, ka[k], kb[k]);
    }
    for (int k = kKept; i0 + k * slots < rows; ++k) {
        uint4 u, w;
        load(k, u, w);
        if (turned) angles(k, g);
        store(k, u, w);
    }
    // rows that lay in the block before
    if (lo > first && (now != before || takes_over)) {
        const uint4* s = reinterpret_cast<const uint4*>(row_of(old_page, row));
        uint4* t = reinterpret_cast<uint4*>(row_of(page, row));
        const float ratio = before * inv;
        for (int e = tid; e < (lo - first) * a.tasks; e += T) {
            const uint4 u = s[e];
            uint32_t r[4] = {u.x, u.y, u.z, u.w};
            if (now != before) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[4];
                    q8_floats(r[k], x);
                    r[k] = q8_codes(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
                }
            }
            t[e] = make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
    if (tid == 0 && (now != before || takes_over)) *scale_of(page, block) = now;
}

// -------------------------------------------------------------- read ----

struct ReadArgs {
    Q8Cache c;
    int tasks;
    int tokens;                // of a CTA
    FastDiv by_hkv;
    const int* cu;             // [batch + 1]
    int total;
    uint4* out[2];             // [total, hkv, d] bf16
};

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 64;   // of a CTA, all heads, at most
// Tasks (16 codes) a thread has in flight, for long reads.  us with one, two, three and four:
// 16 x 5,000 tokens x 8 heads of 128 86.2, 74.3, 74.5, 74.4; 8 x 2,500 x 8 23.4, 19.3, 19.4, 18.9;
// x 4 heads of 256 23.1, 19.0, 19.0, 18.4.  Short ones lose what long ones gain, in CTAs:
// 8 x 2,500 x 2 heads of 128 6.4, 5.6, 5.5, 6.5; 1 x 4,000 x 8 5.3, 5.0, 5.3, 6.1.
constexpr int kReadFlight = 4;
// Below as many CTAs an SM they take fewer tokens: 1,000 tokens x 8 heads 3.4 us so,
// 3.9 with half as many, 4.5 with four times; 8 x 2,500 tokens x 2 heads 6.5, 6.5, 6.0.
constexpr int kReadCtas = 2;

// CTA (tokens of a sequence, keys or values, batch entry).  Where the tokens lie is
// looked up once, by a thread each; then tasks of two granules of 8 codes, half a row
// apart as in rope.cuh: 8 bytes in and 16 out each.  3 bytes move for an element, and
// what can hold them up is the instructions: 16 x 5,000 tokens x 8 heads of 128 take
// 74.3 us, 6.6 TB/s, 99% of a copy's rate (one granule a thread with its page and
// address worked out for each: 82.2).
__global__ void __launch_bounds__(kReadThreads) read_q8_kernel(const ReadArgs a) {
    __shared__ long long code_at[kReadTokens], scale_at[kReadTokens];   // of head 0; -1: no page
    dependents_may_start();
    wait_for_previous();
    const Q8Cache& c = a.c;
    const int b = blockIdx.z, kind = blockIdx.y, t0 = blockIdx.x * a.tokens;
    const int q0 = min(max(a.cu[b], 0), a.total);
    const int len = min(max(a.cu[b + 1], q0), a.total) - q0;
    const int count = min(a.tokens, len - t0);
    if (count <= 0) return;
    const int G = 2 * a.tasks;   // granules of a row
    const size_t head_step = (size_t)c.pages.page_size * G;
    if ((int)threadIdx.x < count) {
        int page, row;
        const bool there = key_page(c.pages, b, (long long)t0 + threadIdx.x, page, row);
        code_at[threadIdx.x] = there ? (long long)(page * (size_t)c.hkv * head_step + (size_t)row * G) : -1;
        if (there) scale_at[threadIdx.x] = (long long)page * c.hkv * c.blocks + c.by_block((unsigned)row);
    }
    __syncthreads();
    const int slots = kReadThreads / a.tasks, slot = threadIdx.x / a.tasks, j = threadIdx.x - slot * a.tasks;
    if (slot >= slots) return;
    const uint2* const codes = reinterpret_cast<const uint2*>(kind == 0 ? c.codes[0] : c.codes[1]) + j;
    const float* const scales = kind == 0 ? c.scales[0] : c.scales[1];
    uint4* const out = (kind == 0 ? a.out[0] : a.out[1]) + (size_t)(q0 + t0) * c.hkv * G + j;
    const int rows = count * c.hkv;   // (token, head), the head fastest
    for (int r0 = slot; r0 < rows; r0 += kReadFlight * slots) {
        uint2 u[kReadFlight], w[kReadFlight];
        float s[kReadFlight];
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const int r = r0 + k * slots;
            u[k] = w[k] = make_uint2(0, 0);
            s[k] = 0.f;
            if (r >= rows) continue;
            const int t = (int)a.by_hkv((unsigned)r), h = r - t * c.hkv;
            const long long at = code_at[t];
            if (at < 0) continue;
            const uint2* const p = codes + (at + h * head_step);
            u[k] = p[0];
            w[k] = p[a.tasks];
            s[k] = scales[scale_at[t] + h * c.blocks];
        }
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const int r = r0 + k * slots;
            if (r >= rows) continue;
            uint4* const to = out + (size_t)r * G;
            const float2 by = both(s[k]);
            auto four = [&](uint32_t four_codes) {
                const float2 x = fmul2(halves_to_floats(q8_halves(four_codes)), by);
                const float2 y = fmul2(halves_to_floats(q8_halves_up(four_codes)), by);
                return make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
            };
            const uint2 u0 = four(u[k].x), u1 = four(u[k].y), w0 = four(w[k].x), w1 = four(w[k].y);
            __stcs(to, make_uint4(u0.x, u0.y, u1.x, u1.y));
            __stcs(to + a.tasks, make_uint4(w0.x, w0.y, w1.x, w1.y));
        }
    }
}

// -------------------------------------------------------------- host ----

// Checks of an 8-bit cache and its table.
fa_status check_cache(const Q8Cache& c, int head_dim) {
    const PageTable& t = c.pages;
    if (t.num_pages < 0 || c.hkv < 0 || t.page_size < 0 || t.max_pages < 0 || c.hkv > 16000)
        return FA_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim % 16 != 0 || head_dim > 2048) return FA_ERR_UNSUPPORTED;
    if (t.num_pages == 0 || c.hkv == 0 || t.page_size == 0) return FA_OK;
    if (c.block <= 0 || t.page_size % c.block != 0) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (!c.codes[i] || !c.scales[i]) return FA_ERR_INVALID_ARG;
        if (!is_aligned(c.codes[i], 16) || !is_aligned(c.scales[i], 4)) return FA_ERR_MISALIGNED;
    }
    if (t.max_pages > 0 && !t.table) return FA_ERR_INVALID_ARG;
    if (!is_aligned(t.table, 4)) return FA_ERR_MISALIGNED;
    if ((long long)t.max_pages * t.page_size >= (1ll << 31) ||
        (long long)c.block * (head_dim / 16) >= (1ll << 30))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

Q8Cache cache_of(void* k, void* v, float* ks, float* vs, int num_pages, int hkv, int page_size,
                 int block, const int* table, int max_pages) {
    Q8Cache c{};
    c.codes[0] = static_cast<uint8_t*>(k);
    c.codes[1] = static_cast<uint8_t*>(v);
    c.scales[0] = ks;
    c.scales[1] = vs;
    c.pages = PageTable{table, max_pages, page_size, num_pages, fast_div(page_size > 0 ? page_size : 1)};
    c.hkv = hkv;
    c.block = block;
    c.blocks = block > 0 ? page_size / block : 0;
    c.by_block = fast_div(block > 0 ? block : 1);
    return c;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_cache_append_q8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                             int num_pages, int hkv, int page_size, int block, int head_dim,
                             const int* block_table, int max_pages, const int* seqlens, int batch,
                             const void* k_new, const long long* k_strides, const void* v_new,
                             const long long* v_strides, int n, const int* n_new,
                             const int* copies, const fa_turn* turn, fa_stream_t stream) {
    AppendArgs a{};
    a.c = cache_of(k_cache, v_cache, k_scale, v_scale, num_pages, hkv, page_size, block, block_table,
                   max_pages);
    if (batch < 0 || batch > 65535 || n < 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(a.c, head_dim);
    if (st != FA_OK) return st;
    a.turn.factor = 1.f;
    if (turn) {
        if (turn->hq < 0 || turn->position_stride < 0) return FA_ERR_INVALID_ARG;
        if ((st = check_turn(turn->freqs, turn->rot, head_dim, turn->factor)) != FA_OK) return st;
        a.turn = Turn{turn->freqs, turn->rot, turn->interleaved ? 1 : 0, turn->factor, 1.f};
        a.positions = turn->positions;
        a.position_stride = turn->position_stride;
        a.hq = turn->hq;
    }
    if (batch == 0) return FA_OK;
    const bool pages = num_pages > 0 && hkv > 0 && page_size > 0;
    if (!pages && a.hq > 0) return FA_ERR_INVALID_ARG;   // queries come beside keys
    if (!pages || (n == 0 && !copies)) return FA_OK;
    if (!seqlens || (max_pages > 0 && !block_table)) return FA_ERR_INVALID_ARG;
    if (!is_aligned(seqlens, 4) || !is_aligned(n_new, 4) || !is_aligned(copies, 4) ||
        !is_aligned(a.positions, 4))
        return FA_ERR_MISALIGNED;
    // (keys of a sequence, new ones among them, are counted in 32 bits)
    if (n >= (1 << 30)) return FA_ERR_INVALID_ARG;
    a.tasks = head_dim / 16;
    a.by_tasks = fast_div(a.tasks);
    a.by_hq = fast_div(a.hq > 0 ? a.hq : 1);
    if ((double)n * a.hq * a.tasks >= 2147483648.0) return FA_ERR_INVALID_ARG;
    if (n > 0) {
        const void* src[3] = {k_new, v_new, a.hq > 0 ? turn->q : nullptr};
        const long long* ss[3] = {k_strides, v_strides, a.hq > 0 ? turn->q_strides : nullptr};
        for (int i = 0; i < (a.hq > 0 ? 3 : 2); ++i) {
            if (!src[i] || !ss[i]) return FA_ERR_INVALID_ARG;
            if (!is_aligned(src[i], 16)) return FA_ERR_MISALIGNED;
            a.src[i] = static_cast<const uint4*>(src[i]);
            for (int k = 0; k < 3; ++k) {
                if (ss[i][k] % 8 != 0) return FA_ERR_MISALIGNED;
                a.ss[i][k] = ss[i][k] / 8;
            }
        }
        if (a.hq > 0) {
            if (!turn->q_out) return FA_ERR_INVALID_ARG;
            if (!is_aligned(turn->q_out, 16)) return FA_ERR_MISALIGNED;
            a.q_out = static_cast<uint4*>(turn->q_out);
        }
    }
    a.lens = seqlens;
    a.n = n;
    a.n_new = n_new;
    a.copies = copies;
    a.units = n > 0 ? (n + block - 2) / block + 1 : 1;
    const long long x = (long long)a.units + (copies ? a.c.blocks : 0);
    if (x >= (1ll << 31)) return FA_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = sm103_or_status(sms)) != FA_OK) return st;
    // a warp for a unit where it keeps all of its rows
    const int unit_rows = n < block ? n : block;
    const bool warp = unit_rows <= 32 / a.tasks * kKeptWarp;
    const bool many = (long long)batch * a.units * hkv > (long long)kFewUnits * sms;
    const int threads = warp || (many && unit_rows <= 128 / a.tasks * kPasses) ? 128 : 256;
    a.kv_ctas = warp ? (2 * hkv + 3) / 4 : 2 * hkv;
    long long q_ctas = 0;
    if (a.hq > 0 && n > 0) {
        q_ctas = ((long long)n * a.hq * a.tasks + threads * x - 1) / (threads * x);
        if (q_ctas > 4096) q_ctas = 4096;
    }
    const dim3 grid((unsigned)x, (unsigned)(a.kv_ctas + q_ctas), (unsigned)batch);
    void (*kernel)(AppendArgs) =
        a.turn.interleaved ? (warp ? append_q8_kernel<true, true> : append_q8_kernel<true, false>)
                           : (warp ? append_q8_kernel<false, true> : append_q8_kernel<false, false>);
    const cudaError_t e = launch_dependent(kernel, grid, dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_read_q8(const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, int num_pages, int hkv, int page_size, int block,
                           int head_dim, const int* block_table, int max_pages,
                           const int* cu_seqlens, int batch, int max_seqlen, int total, void* k_out,
                           void* v_out, fa_stream_t stream) {
    ReadArgs a{};
    a.c = cache_of(const_cast<void*>(k_cache), const_cast<void*>(v_cache), const_cast<float*>(k_scale),
                   const_cast<float*>(v_scale), num_pages, hkv, page_size, block, block_table,
                   max_pages);
    if (batch < 0 || batch > 65535 || max_seqlen < 0 || total < 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(a.c, head_dim);
    if (st != FA_OK) return st;
    if (batch == 0 || total == 0 || hkv == 0) return FA_OK;
    if (max_seqlen == 0 || !cu_seqlens || !k_out || !v_out) return FA_ERR_INVALID_ARG;
    if (!is_aligned(cu_seqlens, 4) || !is_aligned(k_out, 16) || !is_aligned(v_out, 16))
        return FA_ERR_MISALIGNED;
    if (num_pages == 0 || page_size == 0) a.c.pages.max_pages = 0;   // (no page: every key reads as zeros)
    a.tasks = head_dim / 16;
    a.by_hkv = fast_div(hkv);
    a.cu = cu_seqlens;
    a.total = total;
    a.out[0] = static_cast<uint4*>(k_out);
    a.out[1] = static_cast<uint4*>(v_out);
    int sms = 0;
    if ((st = sm103_or_status(sms)) != FA_OK) return st;
    const int longest = max_seqlen < total ? max_seqlen : total;
    // tokens that give each thread what it has in flight, fewer where the CTAs are few
    a.tokens = kReadFlight * (kReadThreads / a.tasks) / hkv;
    if (a.tokens > kReadTokens) a.tokens = kReadTokens;
    while (a.tokens > 1 && 2ll * total / a.tokens < kReadCtas * sms) a.tokens /= 2;
    if (a.tokens < 1) a.tokens = 1;
    const dim3 grid((unsigned)((longest - 1) / a.tokens + 1), 2, (unsigned)batch);
    const cudaError_t e = launch_dependent(read_q8_kernel, grid, dim3(kReadThreads), 0,
                                           reinterpret_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
