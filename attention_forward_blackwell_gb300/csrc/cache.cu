// Operators on the pages of a key/value cache.
//
// A cache is what the paged attention reads: k_cache, v_cache
// [num_pages, hkv, page_size, d] bf16 and a block table int32[batch,
// max_pages] whose entry j is the page of keys [j page_size, (j + 1)
// page_size) of its sequence, or -1.  refs int32[num_pages] counts the table
// entries that hold a page (0: the page is free).  Everything lives on the
// device, so that a serving step that forks, grows and frees sequences needs
// no synchronisation and can be captured.
//
// Two kinds of kernels.  Table kernels (fork, reserve, free) read and write
// only the integers; fork and reserve check everything first and change all
// or nothing, free takes each entry by an atomic exchange so that a row
// listed twice is freed once.  Row kernels (append, copy, compact) move
// 16-byte granules of key and value rows; they are bound by the bytes moved,
// each read once and written once.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "common.cuh"

namespace fa {
namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;

__device__ __forceinline__ bool is_page(int e, int num_pages) {
    return (unsigned)e < (unsigned)num_pages;
}

// Exclusive prefix sum over the block's kTableThreads threads, and the
// total.  scratch: 33 ints of shared memory; two barriers inside.
__device__ __forceinline__ int block_scan(int v, int* scratch, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // the last call's readers are done
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    total = scratch[31];
    return x - v + (warp > 0 ? scratch[warp - 1] : 0);
}

struct TableArgs {
    int* refs;
    int num_pages;
    int* table;        // [batch, max_pages]
    int max_pages;
    int* lens;         // [batch]
    int batch;
    int* status;
};

// --------------------------------------------------------------- fork ----

constexpr int kForkHeld = 4;   // table entries a lane keeps from pass 1 to pass 2

// One cluster, a warp per pair.  Pass 1 checks the pairs; pass 2, if all
// passed (the cluster's first CTA holds the verdict), copies the rows and
// counts the pages.  A single CTA took 24 us for 256 pairs of 65 entries, each
// warp walking 8 of them; with more than 32 pairs eight CTAs share them (6.7 us:
// two chains of loads -- pair, rows -- around the cluster's barriers).
template <bool CLUSTER>
__global__ void __cluster_dims__(CLUSTER ? 8 : 1, 1, 1) __launch_bounds__(kTableThreads)
    cache_fork_kernel(const TableArgs t, const int* src, const int* dst, int n) {
    __shared__ int bad;
    cg::cluster_group cluster = cg::this_cluster();
    auto sync = [&] {
        if constexpr (CLUSTER) cluster.sync();
        else __syncthreads();
    };
    dependents_may_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * (kTableThreads / 32) + (threadIdx.x >> 5);
    const int warps = gridDim.x * (kTableThreads / 32);
    if (threadIdx.x == 0) bad = n;
    sync();
    int* verdict = CLUSTER ? cluster.map_shared_rank(&bad, 0) : &bad;
    int held[kForkHeld];   // the first entries of the warp's first pair, for pass 2
    int held_len = 0;
    for (int i = warp; i < n; i += warps) {
        const int s = src[i], d = dst[i];
        bool ok = (unsigned)s < (unsigned)t.batch && (unsigned)d < (unsigned)t.batch;
        if (ok) {
            if (i == warp) {
                const int* from = t.table + (size_t)s * t.max_pages;
                held_len = t.lens[s];
#pragma unroll
                for (int k = 0; k < kForkHeld; ++k)
                    held[k] = lane + 32 * k < t.max_pages ? from[lane + 32 * k] : -1;
            }
            if (t.lens[d] > 0) ok = false;
#pragma unroll 4
            for (int j = lane; j < t.max_pages; j += 32)   // dst holds nothing
                ok &= !is_page(t.table[(size_t)d * t.max_pages + j], t.num_pages);
#pragma unroll 4
            for (int j = lane; j < n; j += 32) {   // nor is any pair's src or an earlier dst
                const int sj = src[j], dj = dst[j];
                ok &= sj != d && (j >= i || dj != d);
            }
        }
        if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicMin(verdict, i);
    }
    sync();
    const int first_bad = *verdict;
    if (blockIdx.x == 0 && threadIdx.x == 0) *t.status = first_bad < n ? first_bad + 1 : 0;
    if (first_bad == n) {
        for (int i = warp; i < n; i += warps) {
            const int* from = t.table + (size_t)src[i] * t.max_pages;
            int* to = t.table + (size_t)dst[i] * t.max_pages;
            auto share = [&](int j, int e) {
                const bool page = is_page(e, t.num_pages);
                to[j] = page ? e : -1;
                if (page) atomicAdd(t.refs + e, 1);
            };
            int j0 = lane;
            if (i == warp) {
#pragma unroll
                for (int k = 0; k < kForkHeld; ++k)
                    if (lane + 32 * k < t.max_pages) share(lane + 32 * k, held[k]);
                j0 += 32 * kForkHeld;
            }
            for (int j = j0; j < t.max_pages; j += 32) share(j, from[j]);
            if (lane == 0) t.lens[dst[i]] = i == warp ? held_len : t.lens[src[i]];
        }
    }
    sync();   // the first CTA's shared memory stays until all have read it
}

// --------------------------------------------------------------- free ----

// A CTA per row, a thread per entry: bound by its three loads and the atomics
// (256 rows of 65 entries: 2.0 us).
__global__ void __launch_bounds__(256)
    cache_free_kernel(const TableArgs t, const int* rows, int n) {
    dependents_may_start();
    wait_for_previous();
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int r = rows[i];
        if ((unsigned)r >= (unsigned)t.batch) continue;
        for (int j = threadIdx.x; j < t.max_pages; j += blockDim.x) {
            const int e = atomicExch(t.table + (size_t)r * t.max_pages + j, -1);
            if (is_page(e, t.num_pages)) atomicSub(t.refs + e, 1);
        }
        if (threadIdx.x == 0) t.lens[r] = 0;
    }
}

// ------------------------------------------------------------ reserve ----

// Entries [first, last) of a row: its open page (the one its last keys fill in
// part) and those that its next `extra` keys will be written to.
struct Span {
    int first, last;
    bool fits;
};
__device__ __forceinline__ Span reserve_span(const TableArgs& t, const int* extra, int page_size,
                                             int r) {
    Span s{0, 0, true};
    const unsigned len = (unsigned)max(t.lens[r], 0), page = (unsigned)page_size;
    const int more = extra[r];
    if (more < 0) return s;
    const unsigned end = len + (unsigned)more, last = end / page + (end % page != 0);   // (below 2^32)
    s.fits = last <= (unsigned)t.max_pages;
    s.first = (int)min(len / page, (unsigned)t.max_pages);
    s.last = s.fits ? (int)last : s.first;
    return s;
}

constexpr int kLongSpan = 8;     // entries of a span that a warp shares
constexpr int kSharedList = 8192;   // most entries of a list in shared memory
constexpr int kScanPages = 16;   // pages a thread looks at in one step of the free scan

// Whether entry j of a row is needed (see below).
__device__ __forceinline__ bool reserve_needs(const TableArgs& t, const int* row, int j) {
    const int e = row[j];
    return !is_page(e, t.num_pages) || t.refs[e] > 1;
}

// Marks entry j of a row if it is needed.
__device__ __forceinline__ bool reserve_mark(const TableArgs& t, int* row, int j) {
    if (!reserve_needs(t, row, j)) return false;
    const int e = row[j];
    row[j] = is_page(e, t.num_pages) ? -2 - e : -1;
    return true;
}

// Entry j of row r, marked as needed, takes `page`.
__device__ __forceinline__ void reserve_grant(const TableArgs& t, int* row, int r, int j, int page,
                                              int first, int used, int* copies) {
    const int e = row[j];
    row[j] = page;
    t.refs[page] = 1;
    if (e <= -2) {
        atomicSub(t.refs + (-2 - e), 1);
        if (j == first && used > 0) {
            copies[3 * r] = -2 - e;
            copies[3 * r + 1] = page;
            copies[3 * r + 2] = used;
        }
    }
}

// One CTA.  Needed entries of a row's span are those that hold no page and
// those whose page another entry shares (it would be written under the
// other's eyes); in (row, entry) order they take the free pages in ascending
// order.
//   1  count the needed entries, a thread per row (a warp for a long span)
//   2  list the free pages, as many as are needed (ascending; the scan stops
//      early); where they do not suffice that is all
//   3  mark the needed entries: shared ones as -2 - page and entries that are
//      no page as -1, so that pass 4 sees the same set whatever it does to
//      refs (what pass 1 read is still in the L1 cache)
//   4  give the pages out
// The order of the pages makes it one scan over the rows and one over the pages;
// bound by the latencies of its chain (length, entry, count; scan; entry, page):
// 5.3 us for 288 rows over 17,000 pages, 4.0 for 5 rows.
__global__ void __launch_bounds__(kTableThreads)
    cache_reserve_kernel(const TableArgs t, const int* extra, int page_size, int* copies,
                         int* free_list) {
    extern __shared__ int shared_list[];
    __shared__ int scratch[33];
    if (free_list == nullptr) free_list = shared_list;
    __shared__ int long_row;   // first row whose span does not fit the table
    dependents_may_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) long_row = t.batch;
    // which of the kScanPages pages from p on are free
    const bool wide = (reinterpret_cast<uintptr_t>(t.refs) & 15u) == 0;
    auto free_pages = [&](int p) {
        unsigned is_free = 0;
        if (wide && p + kScanPages <= t.num_pages) {
#pragma unroll
            for (int q = 0; q < kScanPages / 4; ++q) {
                const int4 x = *reinterpret_cast<const int4*>(t.refs + p + 4 * q);
                is_free |= ((x.x == 0) | (x.y == 0) << 1 | (x.z == 0) << 2 | (x.w == 0) << 3)
                           << (4 * q);
            }
        } else {
            for (int q = 0; q < kScanPages && p + q < t.num_pages; ++q)
                is_free |= (unsigned)(t.refs[p + q] == 0) << q;
        }
        return is_free;
    };
    // (the first ones with the rows' loads: nothing changes refs before pass 4)
    const unsigned first_free = free_pages((int)threadIdx.x * kScanPages);
    __syncthreads();
    // sum of f(row, entry) over the span of each lane's row r, by the lanes of the
    // warp together where a span is long
    auto over_span = [&](int r, const Span& s, auto&& f) -> int {
        int* row = t.table + (size_t)r * t.max_pages;
        const bool shared_out = s.last - s.first > kLongSpan;
        int count = 0;
        if (!shared_out)
            for (int j = s.first; j < s.last; ++j) count += f(row, j);
        for (unsigned todo = __ballot_sync(0xffffffffu, shared_out); todo != 0; todo &= todo - 1) {
            const int from = __ffs(todo) - 1;
            const int first = __shfl_sync(0xffffffffu, s.first, from);
            const int last = __shfl_sync(0xffffffffu, s.last, from);
            int* its = t.table + (size_t)(r - lane + from) * t.max_pages;
            int c = 0;
            for (int j = first + lane; j < last; j += 32) c += f(its, j);
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == from) count = c;
        }
        return count;
    };
    int needed = 0;
    for (int r0 = 0; r0 < t.batch; r0 += kTableThreads) {
        const int r = r0 + threadIdx.x;
        Span s{0, 0, true};
        if (r < t.batch) s = reserve_span(t, extra, page_size, r);
        if (!s.fits) atomicMin(&long_row, r);
        const int count = over_span(r, s, [&](int* row, int j) { return reserve_needs(t, row, j); });
        int total;
        block_scan(count, scratch, total);
        needed += total;
    }
    int found = 0;
    for (int p0 = 0; p0 < t.num_pages && found < needed; p0 += kTableThreads * kScanPages) {
        const int p = p0 + (int)threadIdx.x * kScanPages;
        unsigned is_free = p0 == 0 ? first_free : free_pages(p);
        int total;
        int k = found + block_scan(__popc(is_free), scratch, total);
        for (; is_free != 0 && k < needed; is_free &= is_free - 1)
            free_list[k++] = p + __ffs(is_free) - 1;
        found += total;
    }
    const bool fits = long_row == t.batch;   // (the scans' barriers order it)
    const bool grant = fits && found >= needed;
    if (threadIdx.x == 0) *t.status = !fits ? -1 - long_row : (grant ? 0 : needed - found);
    // (the rows of one step are marked as they are counted: the scan's barriers
    // come before refs change)
    const bool at_once = t.batch <= kTableThreads;
    auto mark = [&](int* row, int j) { return reserve_mark(t, row, j); };
    for (int r0 = 0; r0 < t.batch; r0 += kTableThreads) {
        const int r = r0 + threadIdx.x;
        Span s{0, 0, true};
        if (r < t.batch) {
            copies[3 * r] = copies[3 * r + 1] = -1;
            copies[3 * r + 2] = 0;
            if (grant && !at_once) s = reserve_span(t, extra, page_size, r);
        }
        if (!at_once) over_span(r, s, mark);
    }
    if (!grant) return;
    if (!at_once) __syncthreads();   // every mark is there before refs change
    int base = 0;
    for (int r0 = 0; r0 < t.batch; r0 += kTableThreads) {
        const int r = r0 + threadIdx.x;
        Span s{0, 0, true};
        if (r < t.batch) s = reserve_span(t, extra, page_size, r);
        int* row = t.table + (size_t)r * t.max_pages;
        const bool shared_out = s.last - s.first > kLongSpan;
        const unsigned longs = __ballot_sync(0xffffffffu, shared_out);
        const int count = at_once ? over_span(r, s, mark)
                                  : over_span(r, s, [](const int* its, int j) { return its[j] < 0; });
        int total;
        int k = base + block_scan(count, scratch, total);
        base += total;
        const int used = r < t.batch ? max(t.lens[r], 0) % page_size : 0;
        if (!shared_out)
            for (int j = s.first; j < s.last; ++j)
                if (row[j] < 0)
                    reserve_grant(t, row, r, j, free_list[k++], s.first, used, copies);
        for (unsigned todo = longs; todo != 0; todo &= todo - 1) {
            const int from = __ffs(todo) - 1;
            const int first = __shfl_sync(0xffffffffu, s.first, from);
            const int last = __shfl_sync(0xffffffffu, s.last, from);
            const int its_used = __shfl_sync(0xffffffffu, used, from);
            int at = __shfl_sync(0xffffffffu, k, from);
            int* its = t.table + (size_t)(r - lane + from) * t.max_pages;
            for (int j0 = first; j0 < last; j0 += 32) {
                const int j = j0 + lane;
                const bool take = j < last && its[j] < 0;
                const unsigned who = __ballot_sync(0xffffffffu, take);
                if (take)
                    reserve_grant(t, its, r - lane + from, j,
                                  free_list[at + __popc(who & ((1u << lane) - 1u))], first, its_used,
                                  copies);
                at += __popc(who);
            }
        }
    }
}

// ------------------------------------------------------- append, copy ----

struct RowArgs {
    uint4* k;                  // caches, in 16-byte granules
    uint4* v;
    int num_pages, hkv, page_size, granules;   // granules of a row: d / 8
    const int* table;
    int max_pages;
    const int* lens;
    // append: k_new, v_new [batch, hkv, n, d] with strides (granules)
    const uint4* k_new;
    const uint4* v_new;
    long long ks[3], vs[3];    // batch, head, token
    int n;
    const int* n_new;          // [batch] or nullptr (n)
    const int* copies;         // [*, 3] or nullptr: source page, page, rows
};

constexpr int kRowThreads = 128;
constexpr int kRowChunk = 64;   // rows of a head that one CTA moves
// 16-byte granules that a thread has in flight, of K and of V each: a granule's
// way is a table entry and then the data, two latencies of memory, so one at a
// time left the memory idle (64 rows of 128 sequences x 8 heads: 9.2 us; four:
// 6.6).
constexpr int kRowFlight = 4;

// The granule of row `pos` of batch entry b, head h; false where it has no page.
__device__ __forceinline__ bool cache_row(const RowArgs& a, const int* table, int h, long long pos,
                                          size_t& at) {
    if (pos < 0 || pos >= (long long)a.max_pages * a.page_size) return false;   // (below 2^31)
    const unsigned p = (unsigned)pos, j = p / (unsigned)a.page_size;
    const int page = table[j];
    if (!is_page(page, a.num_pages)) return false;
    at = (((size_t)page * a.hkv + h) * a.page_size + (p - j * a.page_size)) * a.granules;
    return true;
}

// CTA (chunk of rows, head, batch entry).  First the entry's copy (rows
// [0, c) of a page, c the third number of copies[b]), then its new rows;
// the two never touch the same row.
__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const RowArgs a) {
    dependents_may_start();
    wait_for_previous();
    const int b = blockIdx.z, h = blockIdx.y, r0 = blockIdx.x * kRowChunk;
    const int G = a.granules;
    if (a.copies != nullptr) {
        const int src = a.copies[3 * b], dst = a.copies[3 * b + 1];
        const int rows = min(min(a.copies[3 * b + 2], a.page_size), r0 + kRowChunk);
        if (is_page(src, a.num_pages) && is_page(dst, a.num_pages) && src != dst && r0 < rows) {
            const size_t row = (size_t)a.page_size * G;
            const size_t s0 = ((size_t)src * a.hkv + h) * row, d0 = ((size_t)dst * a.hkv + h) * row;
            for (int e0 = r0 * G + threadIdx.x; e0 < rows * G; e0 += kRowFlight * kRowThreads) {
                uint4 kx[kRowFlight], vx[kRowFlight];
#pragma unroll
                for (int u = 0; u < kRowFlight; ++u) {
                    const int e = e0 + u * kRowThreads;
                    if (e < rows * G) {
                        kx[u] = a.k[s0 + e];
                        vx[u] = a.v[s0 + e];
                    }
                }
#pragma unroll
                for (int u = 0; u < kRowFlight; ++u) {
                    const int e = e0 + u * kRowThreads;
                    if (e < rows * G) {
                        a.k[d0 + e] = kx[u];
                        a.v[d0 + e] = vx[u];
                    }
                }
            }
        }
    }
    if (a.k_new == nullptr) return;
    const int n = min(min(a.n_new != nullptr ? a.n_new[b] : a.n, a.n), r0 + kRowChunk);
    if (r0 >= n) return;
    const long long len = max(a.lens[b], 0);
    const int* table = a.table + (size_t)b * a.max_pages;
    const uint4* k_new = a.k_new + b * a.ks[0] + h * a.ks[1];
    const uint4* v_new = a.v_new + b * a.vs[0] + h * a.vs[1];
    for (int e0 = r0 * G + threadIdx.x; e0 < n * G; e0 += kRowFlight * kRowThreads) {
        uint4 kx[kRowFlight], vx[kRowFlight];
        size_t to[kRowFlight];
        bool move[kRowFlight];
#pragma unroll
        for (int u = 0; u < kRowFlight; ++u) {
            const int e = e0 + u * kRowThreads, i = e / G, g = e - i * G;
            to[u] = 0;
            move[u] = e < n * G && cache_row(a, table, h, len + i, to[u]);
            to[u] += g;
            if (e < n * G) {   // (whether it has a page comes later than this)
                kx[u] = k_new[i * a.ks[2] + g];
                vx[u] = v_new[i * a.vs[2] + g];
            }
        }
#pragma unroll
        for (int u = 0; u < kRowFlight; ++u)
            if (move[u]) {
                a.k[to[u]] = kx[u];
                a.v[to[u]] = vx[u];
            }
    }
}

// ------------------------------------------------------------ compact ----

// CTA (head, batch entry): row start + keep[a] moves to row start + a (paths of
// up to 32 rows of 128 sequences x 8 heads: 3.9 us, a chain of three loads).  keep
// ascends strictly, so keep[a] >= a: a row written is never the source of a
// later a, and rows of one round are all read before any is written.
__global__ void __launch_bounds__(kRowThreads)
    cache_compact_kernel(const RowArgs a, const int* start, const int* keep, int stride,
                         const int* n_keep) {
    dependents_may_start();
    wait_for_previous();
    const int b = blockIdx.y, h = blockIdx.x;
    const int G = a.granules;
    const int n = min(n_keep[b], stride);
    const long long s0 = max(start[b], 0);
    const int* table = a.table + (size_t)b * a.max_pages;
    const int* kp = keep + (size_t)b * stride;
    for (int e0 = threadIdx.x; e0 - (int)threadIdx.x < n * G; e0 += kRowFlight * kRowThreads) {
        uint4 kx[kRowFlight], vx[kRowFlight];
        size_t to[kRowFlight];
        bool move[kRowFlight];
#pragma unroll
        for (int u = 0; u < kRowFlight; ++u) {
            const int e = e0 + u * kRowThreads, i = e / G, g = e - i * G;
            const int x = e < n * G ? kp[i] : i;
            size_t from = 0;
            to[u] = 0;
            move[u] = x > i && cache_row(a, table, h, s0 + x, from) &&
                      cache_row(a, table, h, s0 + i, to[u]);
            to[u] += g;
            if (move[u]) {
                kx[u] = a.k[from + g];
                vx[u] = a.v[from + g];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kRowFlight; ++u)
            if (move[u]) {
                a.k[to[u]] = kx[u];
                a.v[to[u]] = vx[u];
            }
        __syncthreads();
    }
}

// ---------------------------------------------------------- tree mask ----

constexpr int kMaskThreads = 256;

// Words of a tree's ancestor mask: node i sees itself and every node on the
// way up, parent after parent (parents[i] < i; anything else ends the walk,
// so a cycle cannot be followed).  A thread per node walks once, word after word,
// over parents in shared memory; a warp's rows are then written together.  Bound
// by the walk of the deepest node: 64 trees of 1,024 nodes 9.1 us, chains 32
// (a thread per word, each with a walk of its own in global memory: 15 and 739;
// words written as the walk leaves them: 31 and 168).
__global__ void __launch_bounds__(kMaskThreads)
    tree_mask_kernel(const int* parents, unsigned int* mask, int nodes, int words) {
    __shared__ int up[FA_TREE_MAX_NODES];
    __shared__ unsigned int tile[kMaskThreads / 32][32][33];
    dependents_may_start();
    wait_for_previous();
    const int* p = parents + (size_t)blockIdx.x * nodes;
    const int i = blockIdx.y * blockDim.x + threadIdx.x;
    const int last = min(nodes, (int)((blockIdx.y + 1) * blockDim.x));
    for (int x = threadIdx.x; x < last; x += blockDim.x) {
        const int v = p[x];
        up[x] = v < x ? v : -1;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = i < nodes ? i : -1;
    for (int w = words - 1; w >= 0; --w) {
        unsigned int bits = 0;
        while (x >= w * 32) {
            bits |= 1u << (x & 31);
            x = up[x];
        }
        tile[warp][lane][w] = bits;
    }
    __syncwarp();
    const int row0 = i - lane, n = min(32, nodes - row0) * words;
    unsigned int* rows = mask + ((size_t)blockIdx.x * nodes + row0) * words;
    for (int e = lane; e < n; e += 32) rows[e] = tile[warp][e / words][e % words];
}

// -------------------------------------------------------------- host ----

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fa_status launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// The kernels of this library are compiled for sm_103 only.
fa_status device_ok() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return FA_ERR_CUDA;
    return major == 10 && minor == 3 ? FA_OK : FA_ERR_UNSUPPORTED;
}

fa_status check_table(const TableArgs& t, bool need_status) {
    if (t.num_pages < 0 || t.max_pages < 0 || t.batch < 0) return FA_ERR_INVALID_ARG;
    if (t.batch > 0 && (!t.table || !t.lens || !t.refs)) return FA_ERR_INVALID_ARG;
    if (t.num_pages > 0 && !t.refs) return FA_ERR_INVALID_ARG;   // (reserve reads them at once)
    if (need_status && !t.status) return FA_ERR_INVALID_ARG;
    if (!aligned4(t.refs) || !aligned4(t.table) || !aligned4(t.lens) || !aligned4(t.status))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

// Checks of the caches and their table; noop where there is nothing to move.
fa_status check_rows(const RowArgs& a, int batch, int head_dim, bool need_table) {
    if (batch < 0 || a.num_pages < 0 || a.hkv < 0 || a.page_size < 0 || a.max_pages < 0 ||
        a.n < 0)
        return FA_ERR_INVALID_ARG;
    if (batch > 65535 || a.hkv > 65535) return FA_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim % 8 != 0) return FA_ERR_UNSUPPORTED;
    if (batch == 0 || a.num_pages == 0 || a.hkv == 0 || a.page_size == 0) return FA_OK;
    if (!a.k || !a.v || (need_table && (!a.table || !a.lens))) return FA_ERR_INVALID_ARG;
    // positions and the indexes of a head's granules stay below 2^31
    if ((long long)a.max_pages * a.page_size >= (1ll << 31) ||
        (long long)a.page_size * (head_dim / 8) >= (1ll << 31) - (1 << 16) ||
        (long long)a.n * (head_dim / 8) >= (1ll << 31) - (1 << 16))
        return FA_ERR_INVALID_ARG;
    if (!aligned16(a.k) || !aligned16(a.v) || !aligned4(a.table) || !aligned4(a.lens))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_cache_fork(int* refs, int num_pages, int* block_table, int max_pages, int* seqlens,
                        int batch, const int* src, const int* dst, int n, int* status,
                        fa_stream_t stream) {
    const TableArgs t{refs, num_pages, block_table, max_pages, seqlens, batch, status};
    fa_status st = check_table(t, true);
    if (st != FA_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst))) return FA_ERR_INVALID_ARG;
    if (!aligned4(src) || !aligned4(dst)) return FA_ERR_MISALIGNED;
    if ((st = device_ok()) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n <= kTableThreads / 32)
        return launched(launch_dependent(cache_fork_kernel<false>, dim3(1), dim3(kTableThreads), 0, s,
                                         t, src, dst, n));
    return launched(launch_dependent(cache_fork_kernel<true>, dim3(8), dim3(kTableThreads), 0, s, t,
                                     src, dst, n));
}

fa_status fa_cache_free(int* refs, int num_pages, int* block_table, int max_pages, int* seqlens,
                        int batch, const int* rows, int n, fa_stream_t stream) {
    const TableArgs t{refs, num_pages, block_table, max_pages, seqlens, batch, nullptr};
    fa_status st = check_table(t, false);
    if (st != FA_OK) return st;
    if (n < 0 || (n > 0 && !rows)) return FA_ERR_INVALID_ARG;
    if (!aligned4(rows)) return FA_ERR_MISALIGNED;
    if (n == 0 || batch == 0) return FA_OK;
    if ((st = device_ok()) != FA_OK) return st;
    return launched(launch_dependent(cache_free_kernel, dim3(n < 4096 ? n : 4096), dim3(256), 0,
                                     reinterpret_cast<cudaStream_t>(stream), t, rows, n));
}

fa_status fa_cache_reserve(int* refs, int num_pages, int* block_table, int max_pages,
                           const int* seqlens, int batch, const int* extra, int page_size,
                           int* copies, int* status, fa_stream_t stream) {
    const TableArgs t{refs, num_pages, block_table, max_pages, const_cast<int*>(seqlens), batch,
                      status};
    fa_status st = check_table(t, true);
    if (st != FA_OK) return st;
    if (page_size <= 0 || (batch > 0 && (!extra || !copies))) return FA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size >= (1ll << 31)) return FA_ERR_INVALID_ARG;
    if (!aligned4(extra) || !aligned4(copies)) return FA_ERR_MISALIGNED;
    if ((st = device_ok()) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    long long entries = (long long)batch * max_pages;
    if (entries > num_pages) entries = num_pages;
    // the list of granted pages: in shared memory where it surely fits (an
    // allocation and its release are 2 of the call's 6 us on the host)
    void* list = nullptr;
    const bool fits = entries <= kSharedList;
    if (!fits && cudaMallocAsync(&list, entries * sizeof(int), s) != cudaSuccess) return FA_ERR_CUDA;
    st = launched(launch_dependent(cache_reserve_kernel, dim3(1), dim3(kTableThreads),
                                   fits ? entries * sizeof(int) : 0, s, t, extra, page_size, copies,
                                   static_cast<int*>(list)));
    if (list != nullptr && cudaFreeAsync(list, s) != cudaSuccess) return FA_ERR_CUDA;
    return st;
}

fa_status fa_cache_append(void* k_cache, void* v_cache, int num_pages, int hkv, int page_size,
                          int head_dim, const int* block_table, int max_pages, const int* seqlens,
                          int batch, const void* k_new, const long long* k_strides,
                          const void* v_new, const long long* v_strides, int n, const int* n_new,
                          const int* copies, fa_stream_t stream) {
    RowArgs a{};
    a.k = static_cast<uint4*>(k_cache);
    a.v = static_cast<uint4*>(v_cache);
    a.num_pages = num_pages;
    a.hkv = hkv;
    a.page_size = page_size;
    a.granules = head_dim / 8;
    a.table = block_table;
    a.max_pages = max_pages;
    a.lens = seqlens;
    a.n = n;
    a.n_new = n_new;
    a.copies = copies;
    fa_status st = check_rows(a, batch, head_dim, true);
    if (st != FA_OK) return st;
    if (!aligned4(n_new) || !aligned4(copies)) return FA_ERR_MISALIGNED;
    if (batch == 0 || num_pages == 0 || hkv == 0 || page_size == 0) return FA_OK;
    if (n > 0) {
        if (!k_new || !v_new || !k_strides || !v_strides) return FA_ERR_INVALID_ARG;
        if (!aligned16(k_new) || !aligned16(v_new)) return FA_ERR_MISALIGNED;
        for (int i = 0; i < 3; ++i) {
            if (k_strides[i] % 8 != 0 || v_strides[i] % 8 != 0) return FA_ERR_MISALIGNED;
            a.ks[i] = k_strides[i] / 8;
            a.vs[i] = v_strides[i] / 8;
        }
        a.k_new = static_cast<const uint4*>(k_new);
        a.v_new = static_cast<const uint4*>(v_new);
    } else if (!copies) {
        return FA_OK;
    }
    if ((st = device_ok()) != FA_OK) return st;
    int rows = n;
    if (copies && page_size > rows) rows = page_size;
    const dim3 grid((unsigned)((rows + kRowChunk - 1) / kRowChunk), (unsigned)hkv, (unsigned)batch);
    return launched(launch_dependent(cache_append_kernel, grid, dim3(kRowThreads), 0,
                                     reinterpret_cast<cudaStream_t>(stream), a));
}

fa_status fa_cache_copy(void* k_cache, void* v_cache, int num_pages, int hkv, int page_size,
                        int head_dim, const int* copies, int n, fa_stream_t stream) {
    RowArgs a{};
    a.k = static_cast<uint4*>(k_cache);
    a.v = static_cast<uint4*>(v_cache);
    a.num_pages = num_pages;
    a.hkv = hkv;
    a.page_size = page_size;
    a.granules = head_dim / 8;
    a.copies = copies;
    fa_status st = check_rows(a, n, head_dim, false);
    if (st != FA_OK) return st;
    if (n == 0 || num_pages == 0 || hkv == 0 || page_size == 0) return FA_OK;
    if (!copies) return FA_ERR_INVALID_ARG;
    if (!aligned4(copies)) return FA_ERR_MISALIGNED;
    if ((st = device_ok()) != FA_OK) return st;
    const dim3 grid((unsigned)((page_size + kRowChunk - 1) / kRowChunk), (unsigned)hkv,
                    (unsigned)n);
    return launched(launch_dependent(cache_append_kernel, grid, dim3(kRowThreads), 0,
                                     reinterpret_cast<cudaStream_t>(stream), a));
}

fa_status fa_cache_compact(void* k_cache, void* v_cache, int num_pages, int hkv, int page_size,
                           int head_dim, const int* block_table, int max_pages, const int* start,
                           int batch, const int* keep, int keep_stride, const int* n_keep,
                           fa_stream_t stream) {
    RowArgs a{};
    a.k = static_cast<uint4*>(k_cache);
    a.v = static_cast<uint4*>(v_cache);
    a.num_pages = num_pages;
    a.hkv = hkv;
    a.page_size = page_size;
    a.granules = head_dim / 8;
    a.table = block_table;
    a.max_pages = max_pages;
    a.lens = start;
    a.n = keep_stride;
    fa_status st = check_rows(a, batch, head_dim, true);
    if (st != FA_OK) return st;
    if (batch == 0 || num_pages == 0 || hkv == 0 || page_size == 0 || keep_stride == 0)
        return FA_OK;
    if (!keep || !n_keep) return FA_ERR_INVALID_ARG;
    if (!aligned4(keep) || !aligned4(n_keep)) return FA_ERR_MISALIGNED;
    if ((st = device_ok()) != FA_OK) return st;
    return launched(launch_dependent(cache_compact_kernel, dim3((unsigned)hkv, (unsigned)batch),
                                     dim3(kRowThreads), 0, reinterpret_cast<cudaStream_t>(stream), a,
                                     start, keep, keep_stride, n_keep));
}

fa_status fa_tree_mask(const int* parents, unsigned int* mask, int batch, int nodes,
                       fa_stream_t stream) {
    if (batch < 0 || nodes < 0 || nodes > FA_TREE_MAX_NODES) return FA_ERR_INVALID_ARG;
    if (batch == 0 || nodes == 0) return FA_OK;
    if (!parents || !mask) return FA_ERR_INVALID_ARG;
    if (!aligned4(parents) || !aligned4(mask)) return FA_ERR_MISALIGNED;
    const int words = (nodes + 31) / 32;
    fa_status st = device_ok();
    if (st != FA_OK) return st;
    const int threads = nodes < kMaskThreads ? (nodes + 31) / 32 * 32 : kMaskThreads;
    return launched(launch_dependent(tree_mask_kernel,
                                     dim3((unsigned)batch, (unsigned)((nodes + threads - 1) / threads)),
                                     dim3((unsigned)threads), 0, reinterpret_cast<cudaStream_t>(stream),
                                     parents, mask, nodes, words));
}

}  // extern "C"
