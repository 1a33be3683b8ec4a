// fa_kv4_kernel.cuh -- a paged key/value cache held in 4 bits: writing it, reading it
// back, and attention over it.
//
// Format.  A page holds page_size tokens of every key/value head, head-major:
//   codes  [num_pages, H_kv, page_size, D/2] bytes; byte i of a token's row holds channel
//          2i in its low half and channel 2i+1 in its high half;
//   scales [num_pages, H_kv, page_size, D/32] bf16, one per 32 channels.
// With m the group's value of largest magnitude, s = -m/8 rounded to 5 significant bits
// and code c = clamp(rint(x/s), -8, 7) + 8, a code stands for (c - 8) * s.  c - 8 has at
// most 3 significant bits besides its sign (or is -8) and s has 5, so the product fits
// the 8 bits of a bf16: the value is exact in bf16, reading back rounds nothing, and the
// tensor cores get the operand that the definition names.  The sign of s puts the group's
// extreme value on the code -8, which has no positive partner; 4 + 16/32 bits an element.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace fa {
namespace kv4 {

constexpr int kGroup = 32;                       // channels per scale
constexpr uint32_t kMagLargest = 0x7b80;         // bf16 bits of 2^120: a group above it (or not finite) reads back as NaN
constexpr uint32_t kMagSmallest = 0x0a00;        // bf16 bits of 2^-107: a group below it reads back as zeros
constexpr uint32_t kScaleNaN = 0x7fc0;

// Where a position of a sequence lives: its page and the token in it.  Tokens are counted
// in 16-token tiles, the grain at which the attention kernel loads.
struct Paging {
    const int32_t* table;     // [B, max_pages], or NULL: page p of sequence b is b * max_pages + p
    int num_pages;
    int page_size;            // a multiple of 16
    int max_pages;
    uint32_t magic, shift;    // n / page_size = umulhi(n, magic) >> shift for n < 2^31 (see divisor)
};

// Exact division by d (16 <= d <= 2^31) of n < 2^31: with k = ceil(log2 d) and
// m = ceil(2^(31+k) / d) < 2^32 + 1, n m / 2^(31+k) exceeds n / d by less than
// n / 2^(31+k) <= 1 / d, which never reaches the next whole number.
inline void divisor(uint32_t d, uint32_t& magic, uint32_t& shift) {
    uint32_t k = 0;
    while ((1ull << k) < d) ++k;
    magic = (uint32_t)(((1ull << (31 + k)) + d - 1) / d);
    shift = k - 1;
}
__device__ __forceinline__ int page_div(const Paging& pg, int n, int& rem) {
    const int q = (int)(__umulhi((uint32_t)n, pg.magic) >> pg.shift);
    rem = n - q * pg.page_size;
    return q;
}

// Page number of the p-th page of sequence b (p < max_pages); -1 if the table names none.
__device__ __forceinline__ int page_of(const Paging& pg, int b, int p) {
    const long long at = (long long)b * pg.max_pages + p;
    if (pg.table == nullptr) return at < pg.num_pages ? (int)at : -1;
    const int page = __ldg(pg.table + at);
    return page >= 0 && page < pg.num_pages ? page : -1;
}

__device__ __forceinline__ int clamped(const int32_t* p, int b, int top) {
    if (p == nullptr) return top;
    const int v = __ldg(p + b);
    return v < 0 ? 0 : (v > top ? top : v);
}

// ---------------------------------------------------------------- codes to bf16
// The code at bits 4i .. 4i+3 of each half of w, as the bf16 pair (c - 8) * s: bits 3..6 of
// a bf16 with the exponent of 16 weigh 8, 4, 2, 1, so the code placed there reads 16 + c,
// and (16 + c) * s - 24 * s is exact (5 + 5 bits, then 5 significant bits of 24 s).
// i is a constant wherever this is called.
__device__ __forceinline__ uint32_t codes_to_bf16x2(int i, uint32_t w, uint32_t s2, uint32_t m24s2) {
    uint32_t t = i == 0 ? w << 3 : w >> (4 * i - 3);
    asm("lop3.b32 %0, %0, 0x00780078, 0x41804180, 0xEA;" : "+r"(t));   // (t & mask) | 16.0
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(t), "r"(s2), "r"(m24s2));
    return r;
}
__device__ __forceinline__ uint32_t minus_24(uint32_t s2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(s2), "r"(0xC1C0C1C0u));
    return r;
}

// ---------------------------------------------------------------- writing the cache
struct AppendParams {
    const uint4* k;            // bf16 [B, H_kv, N, D], 8 channels a uint4
    const uint4* v;
    uint32_t* k_codes;
    uint16_t* k_scales;
    uint32_t* v_codes;
    uint16_t* v_scales;
    const int32_t* key_lens;   // lengths with the new tokens
    const int32_t* new_lens;   // or NULL: N
    Paging pg;
    int H_kv, N;
    long long rows;            // B * H_kv * N
};

// One thread quantises 8 channels of a token; the four threads of a group agree on the
// scale with two shuffles.  The magnitudes compare as integers, with "positive" as the
// lowest bit, so one maximum finds m and its sign, and what is not finite is largest.
__device__ __forceinline__ void quantise8(uint4 x, uint32_t& word, uint32_t& scale) {
    const uint32_t xv[4] = {x.x, x.y, x.z, x.w};
    uint32_t key = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        key = __vmaxu2(key, ((xv[e] << 1) & 0xfffefffeu) | ((~xv[e] >> 15) & 0x00010001u));
    key = __vmaxu2(key, __shfl_xor_sync(0xffffffffu, key, 1));
    key = __vmaxu2(key, __shfl_xor_sync(0xffffffffu, key, 2));
    key = max(key & 0xffffu, key >> 16);
    const uint32_t mag = key >> 1;
    // RNE of the 8-bit significand to 5 bits (a carry raises the exponent), over 8, sign turned
    const uint32_t five = (mag + 3u + ((mag >> 3) & 1u)) & ~7u;
    scale = mag > kMagLargest ? kScaleNaN : (mag < kMagSmallest ? 0u : (five - (3u << 7)) | ((key & 1u) << 15));
    if (mag > kMagLargest || mag < kMagSmallest) {
        word = 0x88888888u;
        return;
    }
    const float inv = __fdiv_rn(1.f, __uint_as_float(scale << 16));
    word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = __uint_as_float((e & 1) ? (xv[e >> 1] & 0xffff0000u) : (xv[e >> 1] << 16));
        // rint(x / s), ties to even, without a division: x/s is k + 1/2 or at least 1/510
        // away from it (8-bit x, 5-bit s), so the product rounded once to a grid of 2^-11
        // (6144 + .) lands on the tie exactly when the quotient does
        float q = __fadd_rn(__fmaf_rn(f, inv, 6144.f), -6144.f);
        q = fminf(fmaxf(q, -8.f), 7.f);
        word |= (__float_as_uint(__fadd_rn(q, 12582920.f)) & 15u) << (4 * e);   // 1.5 * 2^23 + 8
    }
}

// Bound by memory: 4 D bytes read and 9 D / 8 written a token and head.
template <int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    constexpr int kLanes = D / 8;      // threads per row
    const long long row = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const int sub = threadIdx.x % kLanes;
    const bool in = row < p.rows;
    const long long bh = in ? row / p.N : 0;
    const int n = in ? (int)(row - bh * p.N) : 0;
    const int b = (int)(bh / p.H_kv), h = (int)(bh - (long long)b * p.H_kv);
    const int nl = clamped(p.new_lens, b, p.N);
    const long long pos = (long long)__ldg(p.key_lens + b) - nl + n;
    bool there = in && n < nl && pos >= 0 && pos < (long long)p.pg.max_pages * p.pg.page_size;
    int off = 0, page = -1;
    if (there) {
        const int pi = page_div(p.pg, (int)pos, off);
        page = page_of(p.pg, b, pi);
        there = page >= 0;
    }
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (there) {
        kx = __ldg(p.k + row * kLanes + sub);
        vx = __ldg(p.v + row * kLanes + sub);
    }
    uint32_t kw, ks, vw, vs;
    quantise8(kx, kw, ks);
    quantise8(vx, vw, vs);
    if (!there) return;
    const long long tok = ((long long)page * p.H_kv + h) * p.pg.page_size + off;
    p.k_codes[tok * kLanes + sub] = kw;
    p.v_codes[tok * kLanes + sub] = vw;
    if ((sub & 3) == 0) {
        p.k_scales[tok * (D / kGroup) + (sub >> 2)] = (uint16_t)ks;
        p.v_scales[tok * (D / kGroup) + (sub >> 2)] = (uint16_t)vs;
    }
}

// ---------------------------------------------------------------- reading it back
struct ReadParams {
    const uint32_t* k_codes;
    const uint16_t* k_scales;
    const uint32_t* v_codes;
    const uint16_t* v_scales;
    const int32_t* key_lens;
    const int32_t* first;      // first position of each sequence, or NULL: 0
    uint4* k;                  // bf16 [B, H_kv, N, D]
    uint4* v;
    Paging pg;
    int H_kv, N;
    long long rows;
};

__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint32_t scale) {
    const uint32_t s2 = scale | (scale << 16), z2 = minus_24(s2);
    const uint32_t a = codes_to_bf16x2(0, w, s2, z2), b = codes_to_bf16x2(1, w, s2, z2);   // channels (0,4), (1,5)
    const uint32_t c = codes_to_bf16x2(2, w, s2, z2), d = codes_to_bf16x2(3, w, s2, z2);   // (2,6), (3,7)
    return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632),
                      __byte_perm(c, d, 0x7632));
}

// Bound by memory: 9 D / 8 bytes read and 4 D written a token and head.
template <int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams p) {
    constexpr int kLanes = D / 8;
    const long long row = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const int sub = threadIdx.x % kLanes;
    if (row >= p.rows) return;
    const long long bh = row / p.N;
    const int n = (int)(row - bh * p.N);
    const int b = (int)(bh / p.H_kv), h = (int)(bh - (long long)b * p.H_kv);
    const int top = p.pg.max_pages * p.pg.page_size;
    const int kl = clamped(p.key_lens, b, top);
    const long long pos = (p.first != nullptr ? (long long)__ldg(p.first + b) : 0) + n;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (pos >= 0 && pos < kl) {
        int off;
        const int page = page_of(p.pg, b, page_div(p.pg, (int)pos, off));
        if (page >= 0) {
            const long long tok = ((long long)page * p.H_kv + h) * p.pg.page_size + off;
            const uint32_t kw = __ldg(p.k_codes + tok * kLanes + sub), vw = __ldg(p.v_codes + tok * kLanes + sub);
            const uint32_t ks = __ldg(p.k_scales + tok * (D / kGroup) + (sub >> 2));
            const uint32_t vs = __ldg(p.v_scales + tok * (D / kGroup) + (sub >> 2));
            k = dequantise8(kw, ks);
            v = dequantise8(vw, vs);
        }
    }
    p.k[row * kLanes + sub] = k;
    p.v[row * kLanes + sub] = v;
}

}  // namespace kv4
}  // namespace fa
