// Rotation of queries and keys by their positions (fa_rope), and the append
// that turns keys on their way into a paged cache and queries beside them
// (fa_cache_append_rope).
//
// Each element is read once and written once, 4 bytes moved for 3 operations:
// bound by the memory (8,192 tokens x 40 heads of 128: 27.0 us, 6.2 TB/s, 93% of a
// copy's).  What could hold it up is the angles, 15 instructions a pair; they are the
// same for all heads of a token, so a thread takes one task (16 elements, 8 pairs) of
// up to kHeads heads of a token, computes their angles once while the rows are on their
// way, and turns them one after the other.  Where there are few rows, threads take one
// head each: a call is then bound by the chain of its loads, and every row is in flight
// at once (one token x 40 heads: 2.1 us on the device).  Rows that pass through once are
// loaded and stored as such: 28.5 us there without.  (64 threads a CTA: 28.1 where 256
// took 29.5.)
#include "../../include/fa.h"
#include "rope.cuh"

namespace fa {
namespace {

constexpr int kThreads = 64;
constexpr int kStreams = 3;

// Rows of one kind: [batch, heads, n, d] with strides in granules; dst null: to
// the paged cache `pages`.
struct Rows {
    const uint4* src;
    uint4* dst;
    uint4* pages;
    long long ss[3], ds[3];    // batch, head, token
    int heads;
    int turned;
};
struct RopeArgs {
    Rows rows[kStreams];       // heads 0: none
    Turn turn;
    int tasks;                 // of a row: d / 16
    int heads;                 // of all streams
    int n;                     // rows of a batch entry, at most
    const int* n_new;          // [batch] or nullptr (n)
    const int* positions;      // row i of entry b at positions[b * position_stride + i], or
    long long position_stride;
    const int* lens;           // (positions null) at lens[b] + i
    // cache
    PageTable pages;
    int hkv;
    const int* copies;         // [batch, 3] or nullptr
    int row_ctas;              // CTAs along x that turn rows; the rest copy
    int by_token;              // neighbouring threads take neighbouring tokens, not heads
    FastDiv by_tasks, by_inner;   // by tasks, and by what goes round next: groups or tokens
};

// CTA (rows of an entry, batch entry), threads over (token, group of heads, task), the
// task fastest -- 8 threads read the halves of a row of 128 elements -- then what
// lies next in memory, the heads of a token or the tokens of a head.
template <int HEADS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, HEADS > 1 ? 13 : 20) rope_kernel(const RopeArgs a) {
    dependents_may_start();
    wait_for_previous();
    const int b = blockIdx.y, page_size = a.pages.page_size;
    if ((int)blockIdx.x >= a.row_ctas) {   // rows [0, c) of a page that reserve replaced
        const int src = a.copies[3 * b], dst = a.copies[3 * b + 1];
        const int c = min(a.copies[3 * b + 2], page_size);
        if ((unsigned)src >= (unsigned)a.pages.num_pages || (unsigned)dst >= (unsigned)a.pages.num_pages ||
            src == dst)
            return;
        const int per = a.tasks * 2, part = c * per;      // granules of a row, of a head
        const size_t page = (size_t)a.hkv * page_size * per;
        const long long step = (long long)(gridDim.x - a.row_ctas) * kThreads;
        for (long long e = (long long)(blockIdx.x - a.row_ctas) * kThreads + threadIdx.x;
             e < (long long)part * a.hkv; e += step) {
            const int h = (int)(e / part);
            const size_t at = (size_t)h * page_size * per + (size_t)(e - (long long)h * part);
            const uint4 k = a.rows[0].pages[src * page + at], v = a.rows[1].pages[src * page + at];
            a.rows[0].pages[dst * page + at] = k;
            a.rows[1].pages[dst * page + at] = v;
        }
        return;
    }
    const int n = min(a.n_new != nullptr ? a.n_new[b] : a.n, a.n);
    const int groups = (a.heads + HEADS - 1) / HEADS;
    const unsigned x = blockIdx.x * kThreads + threadIdx.x;   // (below 2^31: the host sees to it)
    const unsigned row = a.by_tasks(x), outer = a.by_inner(row);
    const int j = (int)(x - row * (unsigned)a.tasks);
    const int inner = (int)(row - outer * (unsigned)(a.by_token ? a.n : groups));
    const int i = a.by_token ? inner : (int)outer, g = a.by_token ? (int)outer : inner;
    if (i >= n || g >= groups) return;
    const TaskAt at = task_at<INTERLEAVED>(a.turn.rot, a.tasks, j);
    const int ga = at.a >> 3, gb = at.b >> 3;   // granules of a row
    uint4 xa[HEADS], xb[HEADS];
    uint4* to[HEADS];
    bool turned[HEADS];
    const int len = a.lens != nullptr ? max(a.lens[b], 0) : 0;
    // the rows of heads g, g + groups, ...
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        int h = g + u * groups;
        to[u] = nullptr;
        turned[u] = false;
        if (h >= a.heads) continue;
        int s = 0;
        while (s < kStreams - 1 && h >= a.rows[s].heads) h -= a.rows[s++].heads;
        const Rows& r = a.rows[s];
        const uint4* from = r.src + b * r.ss[0] + h * r.ss[1] + i * r.ss[2];
        xa[u] = HEADS > 1 ? __ldcs(from + ga) : from[ga];
        xb[u] = HEADS > 1 ? __ldcs(from + gb) : from[gb];
        turned[u] = (at.turned_a || at.turned_b) && r.turned;
        if (r.dst != nullptr) {
            to[u] = r.dst + b * r.ds[0] + h * r.ds[1] + i * r.ds[2];
        } else {
            int page, row;
            if (key_page(a.pages, b, (long long)len + i, page, row))
                to[u] = r.pages + (((size_t)page * a.hkv + h) * page_size + row) * (2 * a.tasks);
        }
    }
    Angles angles;
    if (at.turned_a || at.turned_b)
        angles_of<INTERLEAVED>(a.turn, at, a.positions != nullptr ? a.positions[b * a.position_stride + i]
                                                               : (int)((unsigned)len + i),
                               angles);
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        if (to[u] == nullptr) continue;
        if (turned[u]) {
            Granule p = unpack8(xa[u]), q = unpack8(xb[u]);
            turn_task<INTERLEAVED>(at, angles, p, q);
            xa[u] = pack8(p);
            xb[u] = pack8(q);
        }
        if (HEADS > 1) {
            __stcs(to[u] + ga, xa[u]);
            __stcs(to[u] + gb, xb[u]);
        } else {
            to[u][ga] = xa[u];
            to[u][gb] = xb[u];
        }
    }
}

fa_status strides_of(const long long* strides, long long (&to)[3]) {
    for (int i = 0; i < 3; ++i) {
        if (strides[i] % 8 != 0) return FA_ERR_MISALIGNED;
        to[i] = strides[i] / 8;
    }
    return FA_OK;
}

// Heads of a thread: four past 1,280 tasks (of 16 elements) an SM, else one.  us for
// 1, 2, 4, 5 and 8 heads: 8,192 tokens x 40 heads of 128 40.7, 30.9, 28.5, 29.3, 31.7;
// 4 x 2,047 x 32 heads of 96, interleaved, 20.5, 17.9, 17.6, 18.4, 20.5.  One head
// / four, by tokens x 40 heads of 128: 256 4.6 / 5.1, 512 5.3 / 5.9, 600 6.0 / 6.0,
// 700 6.8 / 6.2, 1,000 8.0 / 6.5, 4,000 22.9 / 15.4.
constexpr int kHeads = 4;
constexpr long long kManyTasks = 1280;

fa_status launch_rope(RopeArgs& a, int batch, cudaStream_t s) {
    int sms = 0;
    const fa_status st = sm103_or_status(sms);
    if (st != FA_OK) return st;
    const long long rows = (long long)a.n * a.tasks;
    const bool many = rows * a.heads * batch >= kManyTasks * sms;
    const int per = many ? kHeads : 1;
    const long long ctas = (rows * ((a.heads + per - 1) / per) + kThreads - 1) / kThreads;
    long long copy_ctas = 0;
    if (a.copies != nullptr) {
        copy_ctas = ((long long)a.pages.page_size * a.tasks * 2 * a.hkv + 4 * kThreads - 1) / (4 * kThreads);
        if (copy_ctas > 64) copy_ctas = 64;
    }
    if (ctas * kThreads >= (1ll << 31)) return FA_ERR_INVALID_ARG;   // (rows of one entry, 16 elements each)
    if (ctas + copy_ctas == 0) return FA_OK;
    a.row_ctas = (int)ctas;
    a.by_token = a.n > 0 && a.rows[0].ss[2] < a.rows[0].ss[1] ? 1 : 0;
    a.by_tasks = fast_div(a.tasks);
    a.by_inner = fast_div(a.by_token ? a.n : (a.heads + per - 1) / per);
    void (*kernel)(RopeArgs) =
        a.turn.interleaved ? (many ? rope_kernel<kHeads, true> : rope_kernel<1, true>)
                           : (many ? rope_kernel<kHeads, false> : rope_kernel<1, false>);
    const cudaError_t e = launch_dependent(kernel, dim3((unsigned)(ctas + copy_ctas), (unsigned)batch),
                                           dim3(kThreads), 0, s, a);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rope(const void* q, const long long* q_strides, void* q_out,
                  const long long* q_out_strides, int hq, const void* k, const long long* k_strides,
                  void* k_out, const long long* k_out_strides, int hk, int batch, int n, int head_dim,
                  const int* positions, long long position_stride, const long long* freqs, int rot,
                  int interleaved, int inverse, float factor, fa_stream_t stream) {
    if (batch < 0 || n < 0 || hq < 0 || hk < 0 || position_stride < 0) return FA_ERR_INVALID_ARG;
    if (batch > 65535) return FA_ERR_INVALID_ARG;
    fa_status st = check_turn(freqs, rot, head_dim, factor);
    if (st != FA_OK) return st;
    if (batch == 0 || n == 0 || hq + (long long)hk == 0) return FA_OK;
    if (hq + (long long)hk > 65535) return FA_ERR_INVALID_ARG;
    if (!positions) return FA_ERR_INVALID_ARG;
    if (!is_aligned(positions, 4)) return FA_ERR_MISALIGNED;
    RopeArgs a{};
    const void* src[2] = {q, k};
    void* dst[2] = {q_out, k_out};
    const long long* ss[2] = {q_strides, k_strides};
    const long long* ds[2] = {q_out_strides, k_out_strides};
    const int heads[2] = {hq, hk};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        if (!src[i] || !dst[i] || !ss[i] || !ds[i]) return FA_ERR_INVALID_ARG;
        if (!is_aligned(src[i], 16) || !is_aligned(dst[i], 16)) return FA_ERR_MISALIGNED;
        Rows& r = a.rows[i];
        r.src = static_cast<const uint4*>(src[i]);
        r.dst = static_cast<uint4*>(dst[i]);
        if ((st = strides_of(ss[i], r.ss)) != FA_OK || (st = strides_of(ds[i], r.ds)) != FA_OK) return st;
        r.heads = heads[i];
        r.turned = 1;
    }
    a.turn = Turn{freqs, rot, interleaved ? 1 : 0, factor, inverse ? -1.f : 1.f};
    a.tasks = head_dim / 16;
    a.heads = hq + hk;
    a.n = n;
    a.positions = positions;
    a.position_stride = position_stride;
    return launch_rope(a, batch, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_cache_append_rope(void* k_cache, void* v_cache, int num_pages, int hkv, int page_size,
                               int head_dim, const int* block_table, int max_pages,
                               const int* seqlens, int batch, const void* k_new,
                               const long long* k_strides, const void* v_new,
                               const long long* v_strides, int n, const int* n_new,
                               const int* copies, const fa_turn* turn, fa_stream_t stream) {
    if (batch < 0 || num_pages < 0 || hkv < 0 || page_size < 0 || max_pages < 0 || n < 0 || !turn)
        return FA_ERR_INVALID_ARG;
    if (batch > 65535 || hkv > 20000 || turn->hq < 0 || turn->hq > 20000 || turn->position_stride < 0)
        return FA_ERR_INVALID_ARG;
    fa_status st = check_turn(turn->freqs, turn->rot, head_dim, turn->factor);
    if (st != FA_OK) return st;
    if (hkv == 0 && turn->hq > 0) return FA_ERR_INVALID_ARG;
    if (batch == 0 || hkv == 0) return FA_OK;
    if (!seqlens || ((num_pages > 0 || copies) && (!k_cache || !v_cache || !block_table)))
        return FA_ERR_INVALID_ARG;
    if (num_pages > 0 && page_size == 0) return FA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size >= (1ll << 31) ||
        (long long)page_size * (head_dim / 8) >= (1ll << 31) - (1 << 16))
        return FA_ERR_INVALID_ARG;
    if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(block_table, 4) ||
        !is_aligned(seqlens, 4) || !is_aligned(n_new, 4) || !is_aligned(copies, 4) ||
        !is_aligned(turn->positions, 4))
        return FA_ERR_MISALIGNED;
    RopeArgs a{};
    a.rows[0].pages = static_cast<uint4*>(k_cache);
    a.rows[1].pages = static_cast<uint4*>(v_cache);
    if (n > 0) {
        const void* src[3] = {k_new, v_new, turn->q};
        const long long* ss[3] = {k_strides, v_strides, turn->q_strides};
        const int heads[3] = {hkv, hkv, turn->hq};
        for (int i = 0; i < 3; ++i) {
            if (heads[i] == 0) continue;
            if (!src[i] || !ss[i]) return FA_ERR_INVALID_ARG;
            if (!is_aligned(src[i], 16)) return FA_ERR_MISALIGNED;
            a.rows[i].src = static_cast<const uint4*>(src[i]);
            if ((st = strides_of(ss[i], a.rows[i].ss)) != FA_OK) return st;
            a.rows[i].heads = heads[i];
            a.rows[i].turned = i != 1;
        }
        if (turn->hq > 0) {
            if (!turn->q_out) return FA_ERR_INVALID_ARG;
            if (!is_aligned(turn->q_out, 16)) return FA_ERR_MISALIGNED;
            a.rows[2].dst = static_cast<uint4*>(turn->q_out);
            a.rows[2].ds[2] = head_dim / 8;
            a.rows[2].ds[1] = (long long)n * (head_dim / 8);
            a.rows[2].ds[0] = a.rows[2].ds[1] * turn->hq;
        }
    } else if (!copies) {
        return FA_OK;
    }
    a.turn = Turn{turn->freqs, turn->rot, turn->interleaved ? 1 : 0, turn->factor, 1.f};
    a.tasks = head_dim / 16;
    a.heads = 2 * hkv + turn->hq;
    a.n = n;
    a.n_new = n_new;
    a.positions = turn->positions;
    a.position_stride = turn->position_stride;
    a.lens = seqlens;
    a.hkv = hkv;
    // (without pages the table may be absent)
    a.pages = PageTable{block_table, num_pages > 0 ? max_pages : 0, page_size, num_pages,
                        fast_div(page_size > 0 ? page_size : 1)};
    a.copies = num_pages > 0 ? copies : nullptr;
    return launch_rope(a, batch, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
