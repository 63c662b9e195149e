// Rotation of positions: what the kernels that turn rows share (rope.cu,
// cache_q8.cu).
//
// A row of head_dim elements at position p has its pairs (x, y) turned by the
// angle 2 pi p F_i / 2^64 of pair i: F_i counts 2^-64 of a turn, so the product
// modulo 2^64, whole-number arithmetic, is the exact fraction of a turn however far
// the position, where the product of two fp32 numbers is off by 0.03 radians at
// position 10^6.  Its two highest bits, rounded, are the quarter; the rest, at
// most an eighth of a turn, goes through two polynomials of its own (sine and
// cosine of pi/4 w over the square of w, interpolated at Chebyshev points in 64
// bits: off by 2.4e-9 and 4.8e-11, 8.3e-8 with the roundings of fp32).  Two
// products, 9 fused multiply-adds and the choice of the quarter: about 25
// instructions an angle, with no range reduction and no branch.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

// Sine and cosine of 2 pi p F / 2^64.
__device__ __forceinline__ void turn_sincos(int p, long long F, float& sine, float& cosine) {
    const uint32_t lo = (uint32_t)F, up = (uint32_t)((uint64_t)F >> 32);
    uint32_t t = __umulhi((uint32_t)p, lo) + (uint32_t)p * up;   // the product's upper half
    if (p < 0) t -= lo;
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float w = (float)(int)(t - (quarter << 30)) * 0x1p-29f;
    const float v = w * w;
    float s = fmaf(v, -0x1.2d9b4p-15f, 0x1.465ec4p-9f);
    s = fmaf(v, s, -0x1.4abbbap-4f);
    s = fmaf(v, s, 0x1.921fb6p-1f) * w;
    float c = fmaf(v, 0x1.d9c2e8p-19f, -0x1.55c57ap-12f);
    c = fmaf(v, c, 0x1.03c1dcp-6f);
    c = fmaf(v, c, -0x1.3bd3ccp-2f);
    c = fmaf(v, c, 1.0f);
    const bool odd = (quarter & 1u) != 0;
    sine = odd ? c : s;
    cosine = odd ? s : c;
    if (quarter & 2u) sine = -sine;
    if ((quarter + 1u) & 2u) cosine = -cosine;
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

// Sines and cosines of a task's 8 pairs at a position.
struct Angles {
    float s[8], c[8];
};
template <bool INTERLEAVED>
__device__ __forceinline__ void angles_of(const Turn& t, const TaskAt& at, int position, Angles& g) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const bool second = INTERLEAVED && e >= 4;
        if (second ? !at.turned_b : !at.turned_a) continue;
        const long long* from = t.freqs + (second ? at.pair_b + e - 4 : at.pair_a + e);
        const longlong2 F = *reinterpret_cast<const longlong2*>(from);
        turn_sincos(position, F.x, g.s[e], g.c[e]);
        turn_sincos(position, F.y, g.s[e + 1], g.c[e + 1]);
    }
    const float f = t.factor, fs = t.factor * t.sign;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        g.s[e] *= fs;
        g.c[e] *= f;
    }
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// The turned pairs of a task, in place: x, y its granules' elements.  Products
// and sums in fp32, rounded once by whoever stores them.
__device__ __forceinline__ void turn_pair(float& x, float& y, float s, float c) {
    const float a = x * c - y * s;
    y = y * c + x * s;
    x = a;
}
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_task(const TaskAt& at, const Angles& g, float (&x)[8], float (&y)[8]) {
    if (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (at.turned_a) turn_pair(x[2 * e], x[2 * e + 1], g.s[e], g.c[e]);
            if (at.turned_b) turn_pair(y[2 * e], y[2 * e + 1], g.s[4 + e], g.c[4 + e]);
        }
    } else if (at.turned_a) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(x[e], y[e], g.s[e], g.c[e]);
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
// The kernels of this library are compiled for sm_103 only.  (Asked of the runtime once
// per device: the calls here take two microseconds.)
inline fa_status sm103_or_status() {
    constexpr int kDevices = 64;
    static std::atomic<signed char> known[kDevices];   // 0: not asked yet, 1: it is, -1: it is not
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
    const bool keep = dev >= 0 && dev < kDevices;
    signed char is = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (is == 0) {
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return FA_ERR_CUDA;
        is = major == 10 && minor == 3 ? 1 : -1;
        if (keep) known[dev].store(is, std::memory_order_relaxed);
    }
    return is > 0 ? FA_OK : FA_ERR_UNSUPPORTED;
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
