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
    int num_pages, hkv, page_size, block;
    int blocks;                // of a page
    const int* table;
    int max_pages;
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
    int units;                 // blocks that an entry's new rows may lie in
};

// Granules of a row that a thread keeps between the two passes over a block.
constexpr int kKept = 4;

// Codes of 16 elements in two granules' places (8 bytes each).
__device__ __forceinline__ void store_codes(uint8_t* row, const TaskAt& at, const float (&x)[8],
                                            const float (&y)[8], float inv) {
    const uint2 u = make_uint2(q8_codes(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                               q8_codes(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
    const uint2 w = make_uint2(q8_codes(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                               q8_codes(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    if (at.b == at.a + 8) {
        *reinterpret_cast<uint4*>(row + at.a) = make_uint4(u.x, u.y, w.x, w.y);
    } else {
        *reinterpret_cast<uint2*>(row + at.a) = u;
        *reinterpret_cast<uint2*>(row + at.b) = w;
    }
}

// Queries of batch entry b: as in rope.cu, a task a thread.
template <bool INTERLEAVED>
__device__ void append_queries(const AppendArgs& a, int b, int len, int n) {
    const long long all = (long long)n * a.hq * a.tasks;
    for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < all;
         e += (long long)gridDim.x * blockDim.x) {
        const int j = (int)(e % a.tasks);
        const long long r = e / a.tasks;
        const int i = (int)(r % n), h = (int)(r / n);
        const TaskAt at = task_at(a.turn, j);
        const uint4* from = a.src[2] + b * a.ss[2][0] + h * a.ss[2][1] + i * a.ss[2][2];
        uint4* to = a.q_out + (((long long)b * a.hq + h) * a.n + i) * (2 * a.tasks);
        uint4 u = from[at.a >> 3], w = from[at.b >> 3];
        if (at.turned) {
            Angles g;
            angles_of(a.turn, j,
                      a.positions != nullptr ? a.positions[b * a.position_stride + i] : (int)((unsigned)len + i), g);
            float x[8], y[8];
            unpack8(u, x);
            unpack8(w, y);
            turn_task(INTERLEAVED, g, x, y);
            u = pack8(x);
            w = pack8(y);
        }
        to[at.a >> 3] = u;
        to[at.b >> 3] = w;
    }
}

// CTA (block of an entry, head and keys or values -- the last y: queries --,
// batch entry).  Two passes over the new rows of a block: their reach, then their
// codes; what a thread has of them stays in registers in between, kKept tasks,
// which covers blocks of 64 keys of 128 elements, and is read again past that
// (from L1 or L2).  A block has one writer, so nothing is atomic.  Bound by the
// bytes, 3 for an element, and for single tokens by a chain of loads: length,
// page, scale and row.
template <bool INTERLEAVED>
__global__ void append_q8_kernel(const AppendArgs a) {
    __shared__ float most[8];
    dependents_may_start();
    wait_for_previous();
    const int b = blockIdx.z;
    const Q8Cache& c = a.c;
    const int start = max(a.lens[b], 0);
    int n = max(0, min(a.n_new != nullptr ? a.n_new[b] : a.n, a.n));
    if ((int)blockIdx.y == 2 * c.hkv) {
        if (n > 0) append_queries<INTERLEAVED>(a, b, start, n);
        return;
    }
    // (what lies behind the table has no page; len + n stays in 32 bits)
    const int room = c.max_pages * c.page_size, len = min(start, room);
    n = min(n, room - len);
    const int h = blockIdx.y >> 1, kind = blockIdx.y & 1;
    uint8_t* const codes = c.codes[kind];
    float* const scales = c.scales[kind];
    const int d = a.tasks * 16;
    auto row_of = [&](int page, int row) {
        return codes + (((size_t)page * c.hkv + h) * c.page_size + row) * d;
    };
    auto scale_of = [&](int page, int block) {
        return scales + ((size_t)page * c.hkv + h) * c.blocks + block;
    };
    // the page that reserve replaced: its rows below `copied` come along
    int from = -1, to = -1, copied = 0;
    if (a.copies != nullptr) {
        from = a.copies[3 * b];
        to = a.copies[3 * b + 1];
        copied = min(a.copies[3 * b + 2], c.page_size);
        if ((unsigned)from >= (unsigned)c.num_pages || (unsigned)to >= (unsigned)c.num_pages || from == to)
            copied = 0;
    }
    // the open block: page and first row where the next key goes
    const int first0 = len / c.block * c.block;
    int page0 = -1, row0 = 0;
    key_page(c.table + (size_t)b * c.max_pages, c.max_pages, c.page_size, c.num_pages, first0, page0, row0);
    // its earlier rows are taken from the replaced page by the unit that fills it
    const bool moved = copied > 0 && page0 == to && len > first0 && row0 + (len - first0) == copied;
    if ((int)blockIdx.x >= a.units) {   // a whole block of a replaced page
        const int block = blockIdx.x - a.units, at = block * c.block;
        const int rows = min(c.block, copied - at);
        if (rows <= 0 || (moved && at == row0)) return;
        const uint4* s = reinterpret_cast<const uint4*>(row_of(from, at));
        uint4* t = reinterpret_cast<uint4*>(row_of(to, at));
        for (int e = threadIdx.x; e < rows * a.tasks; e += blockDim.x) t[e] = s[e];
        if (threadIdx.x == 0) *scale_of(to, block) = *scale_of(from, block);
        return;
    }
    const long long first_ = first0 + (long long)blockIdx.x * c.block;
    const int first = (int)min(first_, (long long)room);
    const int lo = max(first, len), hi = (int)min(first_ + c.block, (long long)len + n);
    const bool takes_over = moved && blockIdx.x == 0;
    if (lo >= hi && !takes_over) return;
    int page, row;   // (a block lies in one page)
    if (!key_page(c.table + (size_t)b * c.max_pages, c.max_pages, c.page_size, c.num_pages, first, page, row))
        return;
    const int block = row / c.block;
    const int old_page = takes_over ? from : page;
    const float before = lo > first ? *scale_of(old_page, block) : 0.f;
    const uint4* src = a.src[kind] + b * a.ss[kind][0] + h * a.ss[kind][1];
    const long long step = a.ss[kind][2];
    const bool turns = kind == 0 && a.turn.rot > 0;
    const int all = max(0, hi - lo) * a.tasks;
    uint4 ka[kKept], kb[kKept];
    float square = 0.f;
    const float f2 = a.turn.factor * a.turn.factor;
    auto load = [&](int e, uint4& u, uint4& w) {
        const int i = e / a.tasks, j = e - i * a.tasks;
        const TaskAt at = task_at(a.turn, j);
        const int ga = turns ? at.a >> 3 : 2 * j, gb = turns ? at.b >> 3 : 2 * j + 1;
        const uint4* r = src + (lo - len + i) * step;
        u = r[ga];
        w = r[gb];
    };
    auto reach = [&](int e, const uint4& u, const uint4& w) {
        const int j = e % a.tasks;
        float x[8], y[8], m = 0.f;
        unpack8(u, x);
        unpack8(w, y);
        // (products of bf16 values are exact in fp32, a sum of two rounds once)
        if (turns && 16 * j < a.turn.rot) {
            if (INTERLEAVED) {
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    m = fmaxf(m, fmaf(x[k], x[k], x[k + 1] * x[k + 1]));
                    m = fmaxf(m, fmaf(y[k], y[k], y[k + 1] * y[k + 1]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaf(x[k], x[k], y[k] * y[k]));
            }
            m *= f2;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(x[k] * x[k], y[k] * y[k]));
        }
        square = fmaxf(square, m);
    };
    const int T = blockDim.x;
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int e = threadIdx.x + k * T;
        if (e < all) load(e, ka[k], kb[k]);
    }
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int e = threadIdx.x + k * T;
        if (e < all) reach(e, ka[k], kb[k]);
    }
    for (int e = threadIdx.x + kKept * T; e < all; e += T) {
        uint4 u, w;
        load(e, u, w);
        reach(e, u, w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square = fmaxf(square, __shfl_xor_sync(0xffffffffu, square, o));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = square;
    __syncthreads();   // (every thread has read `before` too)
    square = most[0];
    for (int w = 1; w < T / 32; ++w) square = fmaxf(square, most[w]);
    const float now = hi > lo ? fmaxf(before, q8_scale(square)) : before;
    const float inv = 1.f / now;
    auto store = [&](int e, const uint4& u, const uint4& w) {
        const int i = e / a.tasks, j = e - i * a.tasks;
        float x[8], y[8];
        unpack8(u, x);
        unpack8(w, y);
        TaskAt at{16 * j, 16 * j + 8, false};
        if (turns) {
            at = task_at(a.turn, j);
            if (at.turned) {
                Angles g;
                const int new_row = lo - len + i;
                angles_of(a.turn, j,
                          a.positions != nullptr ? a.positions[b * a.position_stride + new_row]
                                                 : len + new_row,
                          g);
                turn_task(INTERLEAVED, g, x, y);
            }
        }
        store_codes(row_of(page, row + (lo - first) + i), at, x, y, inv);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int e = threadIdx.x + k * T;
        if (e < all) store(e, ka[k], kb[k]);
    }
    for (int e = threadIdx.x + kKept * T; e < all; e += T) {
        uint4 u, w;
        load(e, u, w);
        store(e, u, w);
    }
    // rows that lay in the block before
    if (lo > first && (now != before || takes_over)) {
        const uint4* s = reinterpret_cast<const uint4*>(row_of(old_page, row));
        uint4* t = reinterpret_cast<uint4*>(row_of(page, row));
        const float ratio = before * inv;
        for (int e = threadIdx.x; e < (lo - first) * a.tasks; e += T) {
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
    if (threadIdx.x == 0 && (now != before || takes_over)) *scale_of(page, block) = now;
}

// -------------------------------------------------------------- read ----

struct ReadArgs {
    Q8Cache c;
    int tasks;
    const int* cu;             // [batch + 1]
    int total;
    uint4* out[2];             // [total, hkv, d] bf16
};

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 16;   // of a CTA, all heads
constexpr int kReadFlight = 4;    // granules a thread has in flight

// CTA (tokens of a sequence, keys or values, batch entry): 16 codes in, 32 bytes
// out, a granule a thread, four in flight.
__global__ void __launch_bounds__(kReadThreads) read_q8_kernel(const ReadArgs a) {
    dependents_may_start();
    wait_for_previous();
    const Q8Cache& c = a.c;
    const int b = blockIdx.z, kind = blockIdx.y;
    const int q0 = min(max(a.cu[b], 0), a.total);
    const int len = min(max(a.cu[b + 1], q0), a.total) - q0;
    const int t0 = blockIdx.x * kReadTokens, count = min(kReadTokens, len - t0);
    if (count <= 0) return;
    const int per = c.hkv * a.tasks;   // granules of a token
    const int* table = c.table + (size_t)b * c.max_pages;
    for (int e0 = threadIdx.x; e0 < count * per; e0 += kReadFlight * kReadThreads) {
        uint4 u[kReadFlight];
        float s[kReadFlight];
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const int e = e0 + k * kReadThreads;
            u[k] = make_uint4(0, 0, 0, 0);
            s[k] = 0.f;
            if (e >= count * per) continue;
            const int t = e / per, r = e - t * per, h = r / a.tasks, j = r - h * a.tasks;
            int page, row;
            if (!key_page(table, c.max_pages, c.page_size, c.num_pages, (long long)t0 + t, page, row))
                continue;
            const size_t head = (size_t)page * c.hkv + h;
            u[k] = reinterpret_cast<const uint4*>(c.codes[kind])[(head * c.page_size + row) * a.tasks + j];
            s[k] = c.scales[kind][head * c.blocks + row / c.block];
        }
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const int e = e0 + k * kReadThreads;
            if (e >= count * per) continue;
            const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
            uint32_t o[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float x[4];
                q8_floats(w[m], x);
                o[2 * m] = pack_bf16x2(x[0] * s[k], x[1] * s[k]);
                o[2 * m + 1] = pack_bf16x2(x[2] * s[k], x[3] * s[k]);
            }
            uint4* to = a.out[kind] + ((size_t)(q0 + t0) * per + e) * 2;
            to[0] = make_uint4(o[0], o[1], o[2], o[3]);
            to[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// -------------------------------------------------------------- host ----

// Checks of an 8-bit cache and its table.
fa_status check_cache(const Q8Cache& c, int head_dim) {
    if (c.num_pages < 0 || c.hkv < 0 || c.page_size < 0 || c.max_pages < 0 || c.hkv > 16000)
        return FA_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (c.num_pages == 0 || c.hkv == 0 || c.page_size == 0) return FA_OK;
    if (c.block <= 0 || c.page_size % c.block != 0) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (!c.codes[i] || !c.scales[i]) return FA_ERR_INVALID_ARG;
        if (!is_aligned(c.codes[i], 16) || !is_aligned(c.scales[i], 4)) return FA_ERR_MISALIGNED;
    }
    if (c.max_pages > 0 && !c.table) return FA_ERR_INVALID_ARG;
    if (!is_aligned(c.table, 4)) return FA_ERR_MISALIGNED;
    if ((long long)c.max_pages * c.page_size >= (1ll << 31) ||
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
    c.num_pages = num_pages;
    c.hkv = hkv;
    c.page_size = page_size;
    c.block = block;
    c.blocks = block > 0 ? page_size / block : 0;
    c.table = table;
    c.max_pages = max_pages;
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
    if ((st = sm103_or_status()) != FA_OK) return st;
    const int rows = n < block ? n : block;
    const int threads = (long long)rows * a.tasks > 128 * kKept ? 256 : 128;
    const dim3 grid((unsigned)x, (unsigned)(2 * hkv + (a.hq > 0 && n > 0 ? 1 : 0)), (unsigned)batch);
    const cudaError_t e =
        launch_dependent(a.turn.interleaved ? append_q8_kernel<true> : append_q8_kernel<false>, grid,
                         dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream), a);
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
    if (num_pages == 0 || page_size == 0) {   // (no page: every key reads as zeros)
        a.c.max_pages = 0;
        a.c.page_size = a.c.block = 1;
    }
    a.tasks = head_dim / 16;
    a.cu = cu_seqlens;
    a.total = total;
    a.out[0] = static_cast<uint4*>(k_out);
    a.out[1] = static_cast<uint4*>(v_out);
    if ((st = sm103_or_status()) != FA_OK) return st;
    const int longest = max_seqlen < total ? max_seqlen : total;
    const dim3 grid((unsigned)((longest + kReadTokens - 1) / kReadTokens), 2, (unsigned)batch);
    const cudaError_t e = launch_dependent(read_q8_kernel, grid, dim3(kReadThreads), 0,
                                           reinterpret_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
