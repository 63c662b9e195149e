// Rotation of positions: what the kernels that turn rows share (rope.cu,
// cache_q8.cu).
//
// A row of head_dim elements at position p has its pairs (x, y) turned by the
// angle 2 pi p F_i / 2^64 of pair i: F_i counts 2^-64 of a turn, so the product
// modulo 2^64, whole-number arithmetic, is the exact fraction of a turn however far
// the position, where the product of two fp32 numbers is off by 0.03 radians at
// position 10^6.  Half turns change the signs; what is left, a quarter of a turn at
// most either way, goes through two polynomials of its own (sine and cosine of
// pi/2 w over the square of w, interpolated at Chebyshev points in 64 bits: off by
// 6.7e-9 and 2.3e-10, 1.6e-7 with the roundings of fp32, and w itself by 2^-24).  Two
// angles an instruction for all but the whole numbers: about 15 an angle, with no
// range reduction, no branch and no selects, which the appends have too many of
// (with quarter turns, whose sines and cosines change places, one at a time, chunks of
// 8 x 1,024 tokens appended to an 8-bit cache and read back took 37.4 us for 35.7).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

// Upper half of p F modulo 2^64.
__device__ __forceinline__ uint32_t turn_of(int p, long long F) {
    const uint32_t lo = (uint32_t)F, up = (uint32_t)((uint64_t)F >> 32);
    return __umulhi((uint32_t)p, lo) + (uint32_t)p * up - (lo & (uint32_t)(p >> 31));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float with_sign(float x, uint32_t bits) {   // (bit 31 of `bits` changes it)
    return __uint_as_float(__float_as_uint(x) ^ (bits & 0x80000000u));
}
// Sines and cosines of 2 pi p F / 2^64 for two F.
__device__ __forceinline__ void turn_sincos(int p, const longlong2& F, float2& sine, float2& cosine) {
    const uint32_t t0 = turn_of(p, F.x), t1 = turn_of(p, F.y);
    const float2 w = fmul2(make_float2((float)(int)(t0 << 1), (float)(int)(t1 << 1)), both(0x1p-31f));
    const float2 v = fmul2(w, w);
    float2 s = ffma2(v, both(0x1.3e1420p-13f), both(-0x1.32531ep-8f));
    s = ffma2(v, s, both(0x1.4668f0p-4f));
    s = ffma2(v, s, both(-0x1.4abbc4p-1f));
    s = fmul2(ffma2(v, s, both(0x1.921fb6p+0f)), w);
    float2 c = ffma2(v, both(-0x1.8fb3f4p-16f), both(0x1.e126b0p-11f));
    c = ffma2(v, c, both(-0x1.55d074p-6f));
    c = ffma2(v, c, both(0x1.03c1e4p-2f));
    c = ffma2(v, c, both(-0x1.3bd3ccp+0f));
    c = ffma2(v, c, both(1.0f));
    const uint32_t h0 = t0 + 0x40000000u, h1 = t1 + 0x40000000u;
    sine = make_float2(with_sign(s.x, h0), with_sign(s.y, h1));
    cosine = make_float2(with_sign(c.x, h0), with_sign(c.y, h1));
}

// How rows are turned: the first `rot` elements of a row (a multiple of 16; 0:
// none), pair i with freqs[i], the pairs (i, i + rot / 2) or, interleaved,
// (2 i, 2 i + 1).  Sines and cosines are multiplied by `factor`; `sign` -1 turns
// back.
struct Turn {
    const long long* freqs;
    int rot;
    int interleaved;
    float factor, sign;
};

// A row is handled 16 elements a time, by tasks j < head_dim / 16: two granules of
// 8 elements (16 bytes of bf16), of which the tasks of neighbouring lanes take
// neighbouring ones, so that every load and store of a warp covers whole sectors
// (with the granules of a task side by side, each instruction left every other 16 bytes to
// the next: prompts with interleaved pairs 20 us for 15 of their bytes).  Pairs of the
// halves lie in both granules at the same place, interleaved ones within a granule.
struct TaskAt {
    int a, b;               // first elements of the granules
    bool turned_a, turned_b;
    int pair_a, pair_b;     // first pair: of both granules (8 of them), or of each (4)
};
template <bool INTERLEAVED>
__device__ __forceinline__ TaskAt task_at(int rot, int tasks, int j) {
    TaskAt at;
    if (INTERLEAVED) {
        at.a = 8 * j;
        at.b = 8 * (j + tasks);
        at.turned_a = at.a < rot;
        at.turned_b = at.b < rot;
        at.pair_a = 4 * j;
        at.pair_b = 4 * (j + tasks);
    } else {
        const bool in = 16 * j < rot;   // (else the rest of the row, which has its own halves)
        const int first = in ? 0 : rot, len = in ? rot : 16 * tasks - rot;
        at.a = first + 8 * j - (first >> 1);
        at.b = at.a + (len >> 1);
        at.turned_a = at.turned_b = in;
        at.pair_a = at.pair_b = 8 * j;
    }
    return at;
}

// Sines and cosines of a task's 8 pairs at a position, two together.
struct Angles {
    float2 s[4], c[4];
};
template <bool INTERLEAVED>
__device__ __forceinline__ void angles_of(const Turn& t, const TaskAt& at, int position, Angles& g) {
    const float2 f = both(t.factor), fs = both(t.factor * t.sign);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool second = INTERLEAVED && e >= 2;
        if (second ? !at.turned_b : !at.turned_a) continue;
        const long long* from = t.freqs + (second ? at.pair_b + 2 * e - 4 : at.pair_a + 2 * e);
        turn_sincos(position, *reinterpret_cast<const longlong2*>(from), g.s[e], g.c[e]);
        g.s[e] = fmul2(g.s[e], fs);
        g.c[e] = fmul2(g.c[e], f);
    }
}

// A granule's eight elements, those of even and of odd place.
struct Granule {
    float even[4], odd[4];
};
__device__ __forceinline__ Granule unpack8(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Granule x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.even[i] = __uint_as_float(w[i] << 16);
        x.odd[i] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return x;
}
__device__ __forceinline__ uint4 pack8(const Granule& x) {
    return make_uint4(pack_bf16x2(x.even[0], x.odd[0]), pack_bf16x2(x.even[1], x.odd[1]),
                      pack_bf16x2(x.even[2], x.odd[2]), pack_bf16x2(x.even[3], x.odd[3]));
}

// Two pairs (x, y), turned in place.  Products and sums in fp32, rounded once by whoever
// stores them.
__device__ __forceinline__ void turn_pairs(float& x0, float& x1, float& y0, float& y1, float2 s, float2 c) {
    const float2 x = make_float2(x0, x1), y = make_float2(y0, y1);
    const float2 a = ffma2(fmul2(y, s), both(-1.f), fmul2(x, c)), b = ffma2(y, c, fmul2(x, s));
    x0 = a.x;
    x1 = a.y;
    y0 = b.x;
    y1 = b.y;
}
// The turned pairs of a task, in place: x, y its granules.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_task(const TaskAt& at, const Angles& g, Granule& x, Granule& y) {
    if (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (at.turned_a)
                turn_pairs(x.even[2 * e], x.even[2 * e + 1], x.odd[2 * e], x.odd[2 * e + 1], g.s[e], g.c[e]);
            if (at.turned_b)
                turn_pairs(y.even[2 * e], y.even[2 * e + 1], y.odd[2 * e], y.odd[2 * e + 1], g.s[2 + e],
                           g.c[2 + e]);
        }
    } else if (at.turned_a) {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn_pairs(x.even[e], x.odd[e], y.even[e], y.odd[e], g.s[e], g.c[e]);
    }
}

// Place of key `pos` in a paged cache: its page and row in it; false where it has no
// page.
struct PageTable {
    const int* table;          // [batch, max_pages]
    int max_pages, page_size, num_pages;
    FastDiv by_page;           // by page_size
};
__device__ __forceinline__ bool key_page(const PageTable& t, int b, long long pos, int& page, int& row) {
    if (pos < 0 || pos >= (long long)t.max_pages * t.page_size) return false;   // (below 2^31)
    const unsigned p = (unsigned)pos, j = t.by_page(p);
    page = t.table[(size_t)b * t.max_pages + j];
    row = (int)(p - j * (unsigned)t.page_size);
    return (unsigned)page < (unsigned)t.num_pages;
}

// ------------------------------------------------------------------ host ----

inline bool is_aligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// The kernels of this library are compiled for sm_103 only; its SMs.  (Asked of the runtime
// once per device: the calls here take two microseconds.)
inline fa_status sm103_or_status(int& sms) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];   // 0: not asked yet, -1: it is another, else its SMs
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
    const bool keep = dev >= 0 && dev < kDevices;
    sms = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return FA_ERR_CUDA;
        if (major != 10 || minor != 3 || sms <= 0) sms = -1;
        if (keep) known[dev].store(sms, std::memory_order_relaxed);
    }
    return sms > 0 ? FA_OK : FA_ERR_UNSUPPORTED;
}
// Frequencies and factor of a call that turns rows (freqs NULL: none).
inline fa_status check_turn(const long long* freqs, int rot, int head_dim, float factor) {
    if (rot < 0 || rot > head_dim || (rot > 0 && !freqs)) return FA_ERR_INVALID_ARG;
    if (!(factor > 0.f) || !(factor < 3.0e38f)) return FA_ERR_INVALID_ARG;
    if (rot % 16 != 0 || head_dim <= 0 || head_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (!is_aligned(freqs, 16)) return FA_ERR_MISALIGNED;
    return FA_OK;
}

}  // namespace fa
