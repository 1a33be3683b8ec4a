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
// s is at most 2^117; a scale of 2^118 or more in magnitude (memory that was never written may
// hold any) stands for NaN, as an infinite one does.
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
constexpr uint32_t kScaleNone = 0x7a80;          // bf16 bits of 2^118: the magnitude from which on a scale stands for NaN

// Every kernel here begins with this: the next kernel of the stream may be set up from now on
// (where it allows that), and the memory of the kernels before is complete.  For calls one after
// another on a stream it hides the setup: 8 heads on 700 keys 10.3 -> 8.1 us, as first built.
// A block may thus be on its SM while the kernels before it still write what it will read, so
// memory is not read-only for its lifetime: no load here may take the non-coherent path (no
// __ldg, no __restrict__).  What those kernels write (codes, scales, q, k, v, parts) is loaded past L1.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

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
    const int page = pg.table[at];
    return page >= 0 && page < pg.num_pages ? page : -1;
}

__device__ __forceinline__ int clamped(const int32_t* p, int b, int top) {
    if (p == nullptr) return top;
    const int v = p[b];
    return v < 0 ? 0 : (v > top ? top : v);
}

// ---------------------------------------------------------------- rows and what they see
// All G = H / H_kv query heads of a key/value head, times N_q queries, are the rows that meet
// its keys: row = head in group * N_q + query.
struct Rows {
    const int32_t* key_lens;
    const int32_t* q_lens;     // or NULL: N_q
    int N_q, R;                // R = G * N_q
    int causal;
    int window;                // < 0: none; at most 2^30, as keys are, so that positions stay within int
};

// Keys [lo, hi) that a row of a sequence with kl keys and ql queries sees (hi <= lo: none).
__device__ __forceinline__ void row_keys(const Rows& p, int kl, int ql, int row, int& lo, int& hi) {
    const int i = p.N_q == 1 ? 0 : row % p.N_q;
    const int at = kl - ql + i;
    lo = p.window >= 0 ? max(0, at - p.window) : 0;
    hi = row < p.R && i < ql ? (p.causal ? max(0, min(kl, at + 1)) : kl) : 0;
}

// What a block of rows of a sequence attends to.
struct Entry {
    int b;
    int r0, nr;            // first row and rows of the block
    int kl, ql;            // keys and queries of the sequence
    int lo, hi;            // keys some row of the block sees: [lo, hi), lo rounded down to a multiple of kTile
    int all_lo, all_hi;    // keys every row sees
    int units;             // of kUnit keys from lo, at least 1
};

template <int RB, int kTile, int kUnit>
__device__ __forceinline__ Entry entry_of_rows(const Rows& p, const Paging& pg, int b, int r0) {
    Entry x;
    x.b = b;
    x.r0 = r0;
    x.nr = min(RB, p.R - r0);
    x.kl = clamped(p.key_lens, b, pg.max_pages * pg.page_size);
    x.ql = clamped(p.q_lens, b, p.N_q);
    int i0 = 0, i1 = p.N_q - 1;              // the queries among the rows
    if (x.nr < p.N_q) {
        const int a = r0 % p.N_q, z = a + x.nr - 1;
        if (z < p.N_q) {
            i0 = a;
            i1 = z;
        }
    }
    const bool rows_without = i1 >= x.ql;
    i1 = min(i1, x.ql - 1);
    const int off = x.kl - x.ql;
    x.hi = i0 > i1 ? 0 : (p.causal ? max(0, min(x.kl, off + i1 + 1)) : x.kl);
    x.all_hi = rows_without ? 0 : (p.causal ? max(0, min(x.kl, off + i0 + 1)) : x.kl);
    x.lo = x.all_lo = 0;
    if (p.window >= 0) {
        x.lo = min(max(0, off + i0 - p.window), x.hi) & ~(kTile - 1);
        x.all_lo = max(0, off + i1 - p.window);
    }
    x.units = max(1, (x.hi - x.lo + kUnit - 1) / kUnit);
    return x;
}

// Of the kernel for many rows (fa_kv4_rows.cuh).
struct RowsParams {
    const uint8_t* k_codes;
    const uint16_t* k_scales;
    const uint8_t* v_codes;
    const uint16_t* v_scales;
    Paging pg;
    Rows rows;
    int H_kv;
    __nv_bfloat16* o;                // [B, H_kv, R, D]
    float* lse;                      // [B, H_kv, R]
    float scale_log2;
    unsigned long long wait_limit;
    int row_blocks;                  // of kBlockM rows
    int splits;                      // ranges of keys of a block of rows, one CTA each
    int split_inv;                   // ceil(2^16 / splits)
    float* part;                     // with splits > 1, per CTA: sums of P V [D/4][128 rows][4],
    float* part_ml;                  // and per row the max, the sum of rounded P and of P: [3][128]
};

// ---------------------------------------------------------------- weights
// Weights are 2^(score - ref - kShift), with ref the reference max of the row, which may lag by 8:
// at most 2^-8 (2^-7 where scores near 2^20 round the bound itself), so that sums of n values V stay
// below 2^127 while n |V| stays below 2^134 (2^14 keys of 2^120, or any number of 2^104), and at
// least 2^-126, which is 2^-110 of the largest
// (smaller ones count as zero; with a shift of 24 that would be 2^-102, which shows where all other
// keys of a row are so far below one whose value is 0).  At the other end of the format, where
// values are multiples of 2^-110, sums of 32 bits still tell 2^-149 apart, 2^-23 of that at a
// weight of 2^-16.  The shift cancels in O; the sum of the weights gets it back for the LSE.
constexpr float kShift = 16.f;
constexpr float kUnshift = 65536.f;          // 2^kShift
// A reference of about m that is exact with and without the shift added.
__device__ __forceinline__ float reference(float m) { return (m + kShift) - kShift; }
// Log-sum-exp of a row, from its reference and the sum of its weights.
__device__ __forceinline__ float lse_of(float ref, float sum) {
    return sum == 0.f ? -INFINITY : (ref + log2f(sum * kUnshift)) * 0.69314718055994531f;
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
// -24 s, exact for 5 significant bits, as 1024 s - 131/128 * 1024 s: from |s| = 2^118 on 1024 s is
// infinite and this, and so every code, NaN.  (With a plain -24 s a hidden scale of 2^123.4 or more
// would give codes of -inf, and 0 * inf NaN in the rows that do not see it.)
__device__ __forceinline__ uint32_t minus_24(uint32_t s2) {
    uint32_t t, r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t) : "r"(s2), "r"(0x44804480u));                  // 1024
    asm("fma.rn.bf16x2 %0, %1, %2, %1;" : "=r"(r) : "r"(t), "r"(0xBF83BF83u));               // -131/128
    return r;
}
// The same in one instruction, of scales below 2^118.
__device__ __forceinline__ uint32_t minus_24_of_a_number(uint32_t s2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(s2), "r"(0xC1C0C1C0u));
    return r;
}
// Whether a scale stands for NaN.
__device__ __forceinline__ bool no_scale(uint32_t s) { return (s & 0x7fffu) >= kScaleNone; }

// ---------------------------------------------------------------- writing the cache
// Both kernels below give a thread 8 channels of a token.  With many tokens a head, block
// (x, y) takes head x mod H_kv of sequence x / H_kv and steps through its tokens from block
// y, four a thread, so that eight loads are on their way at once: 2 x 32 x 8000 x 128 written
// and read back take 125 us (5.4 TB/s), with one token a thread 153, with two 128, with eight
// 138 (8 x 12 x 1024 x 64: 13.4, 14.5, 13.1, 16.4).  Where a head has less than a block's
// tokens, blocks take consecutive rows of all heads, one a thread (a decoding step's tokens,
// 24 x 8 x 1 x 128: 6.0 -> 4.4 us, as first built).
constexpr int kRowThreads = 256;
constexpr int kRowsPerThread = 4;
constexpr int kMaxRowBlocks = 65535;

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
    uint32_t rows;             // flat: B * H_kv * N
};

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One thread quantises 8 channels of a token; the four threads of a group share the extremes.
__device__ __forceinline__ void quantise8(uint4 x, uint32_t& word, uint32_t& scale) {
    const uint32_t xv[4] = {x.x, x.y, x.z, x.w};
    const uint32_t hi = max_nan_bf16x2(max_nan_bf16x2(xv[0], xv[1]), max_nan_bf16x2(xv[2], xv[3]));
    const uint32_t lo = min_nan_bf16x2(min_nan_bf16x2(xv[0], xv[1]), min_nan_bf16x2(xv[2], xv[3])) ^ 0x80008000u;
    // low half the largest value, high half the largest of the negated ones
    uint32_t e = max_nan_bf16x2(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    e = max_nan_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, 1));
    e = max_nan_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, 2));
    const bool positive = __uint_as_float(e << 16) >= __uint_as_float(e & 0xffff0000u);
    const uint32_t mag = (positive ? e : e >> 16) & 0x7fffu;     // of a NaN: above kMagLargest
    // RNE of the 8-bit significand to 5 bits (a carry raises the exponent), over 8, sign turned
    const uint32_t five = (mag + 3u + ((mag >> 3) & 1u)) & ~7u;
    scale = (five - (3u << 7)) | (positive ? 0x8000u : 0u);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__uint_as_float(scale << 16)));
    // rint(x / s), ties to even, without a division: x / s is k + 1/2 or at least 2^-9 away
    // from it (8-bit x, 5-bit s), so the product with an approximate 1 / s, rounded once to a
    // grid of 2^-11 (6144 + .), lands on the tie exactly when the quotient does.  Then
    // 1.5 * 2^23 + rint has the code less 8 in its lowest bits, and the sum of these times
    // 16^i, modulo 2^32, is the word, less a constant.
    constexpr uint32_t kMagic = 0x4B400000u;
    word = 0x88888888u - kMagic * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __uint_as_float((i & 1) ? (xv[i >> 1] & 0xffff0000u) : (xv[i >> 1] << 16));
        const float q = fminf(__fmaf_rn(f, inv, 6144.f), 6144.f + 7.f);    // |x / s| <= 8.25: only 7 clamps
        word += __float_as_uint(__fadd_rn(q, 12582912.f - 6144.f)) << (4 * i);
    }
    if (mag - kMagSmallest > kMagLargest - kMagSmallest) {
        scale = mag > kMagLargest ? kScaleNaN : 0u;
        word = 0x88888888u;
    }
}

// 4 D bytes read and 9 D / 8 written a token and head, with the arithmetic close behind: 2 x 32 x
// 8000 x 128 take 70 us, 52 at the copy rate, and the schedulers issue in 76 of 100 cycles
// (before the codes were summed as integers, and with 64-bit indexes, 83 us).
template <int D, bool kFlat>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const AppendParams p) {
    after_previous();
    constexpr int kEach = kFlat ? 1 : kRowsPerThread;
    constexpr int kLanes = D / 8;      // threads per row
    constexpr int kRows = kRowThreads / kLanes;
    const int sub = threadIdx.x % kLanes;
    int bh = (int)blockIdx.x, r = threadIdx.x / kLanes;
    bool valid = true;
    if (kFlat) {
        const uint32_t at = blockIdx.x * kRows + r;
        valid = at < p.rows;
        bh = valid ? (int)(at / (uint32_t)p.N) : 0;
        r = valid ? (int)(at - (uint32_t)bh * (uint32_t)p.N) : 0;
    }
    const int b = bh / p.H_kv, h = bh - b * p.H_kv;
    const int nl = clamped(p.new_lens, b, p.N);
    const int first = max(0, p.key_lens[b]) - nl;    // of the new tokens' positions
    const uint32_t top = (uint32_t)(p.pg.max_pages * p.pg.page_size);
    const uint4* const k = p.k + (long long)bh * p.N * kLanes + sub;
    const uint4* const v = p.v + (long long)bh * p.N * kLanes + sub;
    // (a flat block's threads make one step each, together: they share the scales by shuffles)
    for (int n0 = blockIdx.y * (kRows * kEach); kFlat ? n0 == 0 : n0 < nl; n0 += kFlat ? 1 : (int)gridDim.y * (kRows * kEach)) {
        uint4 kx[kEach], vx[kEach];
        uint32_t row[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int n = n0 + i * kRows + r, pos = first + n;
            row[i] = 0xffffffffu;
            kx[i] = vx[i] = make_uint4(0, 0, 0, 0);
            if (valid && n < nl && (uint32_t)pos < top) {
                kx[i] = __ldcg(k + (size_t)n * kLanes);
                vx[i] = __ldcg(v + (size_t)n * kLanes);
                int off;
                const int page = page_of(p.pg, b, page_div(p.pg, pos, off));
                if (page >= 0) row[i] = ((uint32_t)page * (uint32_t)p.H_kv + (uint32_t)h) * (uint32_t)p.pg.page_size + (uint32_t)off;
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            uint32_t kw, ks, vw, vs;
            quantise8(kx[i], kw, ks);
            quantise8(vx[i], vw, vs);
            if (row[i] == 0xffffffffu) continue;
            p.k_codes[(size_t)row[i] * kLanes + sub] = kw;
            p.v_codes[(size_t)row[i] * kLanes + sub] = vw;
            if ((sub & 3) == 0) {
                p.k_scales[(size_t)row[i] * (D / kGroup) + (sub >> 2)] = (uint16_t)ks;
                p.v_scales[(size_t)row[i] * (D / kGroup) + (sub >> 2)] = (uint16_t)vs;
            }
        }
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
    uint32_t rows;             // flat: B * H_kv * N
};

__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint32_t scale) {
    const uint32_t s2 = scale | (scale << 16), z2 = minus_24(s2);
    const uint32_t a = codes_to_bf16x2(0, w, s2, z2), b = codes_to_bf16x2(1, w, s2, z2);   // channels (0,4), (1,5)
    const uint32_t c = codes_to_bf16x2(2, w, s2, z2), d = codes_to_bf16x2(3, w, s2, z2);   // (2,6), (3,7)
    return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632),
                      __byte_perm(c, d, 0x7632));
}

// Bound by memory: 9 D / 8 bytes read and 4 D written a token and head (2 x 32 x 8000 x 128: 56
// us, 6.0 TB/s).
template <int D, bool kFlat>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const ReadParams p) {
    after_previous();
    constexpr int kEach = kFlat ? 1 : kRowsPerThread;
    constexpr int kLanes = D / 8;
    constexpr int kRows = kRowThreads / kLanes;
    const int sub = threadIdx.x % kLanes;
    int bh = (int)blockIdx.x, r = threadIdx.x / kLanes;
    bool valid = true;
    if (kFlat) {
        const uint32_t at = blockIdx.x * kRows + r;
        valid = at < p.rows;
        bh = valid ? (int)(at / (uint32_t)p.N) : 0;
        r = valid ? (int)(at - (uint32_t)bh * (uint32_t)p.N) : 0;
    }
    const int b = bh / p.H_kv, h = bh - b * p.H_kv;
    const int kl = clamped(p.key_lens, b, p.pg.max_pages * p.pg.page_size);
    const long long first = p.first != nullptr ? (long long)p.first[b] : 0;
    uint4* const k = p.k + (long long)bh * p.N * kLanes + sub;
    uint4* const v = p.v + (long long)bh * p.N * kLanes + sub;
    for (int n0 = blockIdx.y * (kRows * kEach); n0 < p.N && valid; n0 += kFlat ? p.N : (int)gridDim.y * (kRows * kEach)) {
        uint32_t kw[kEach], vw[kEach], ks[kEach], vs[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int n = n0 + i * kRows + r;
            const long long pos = first + n;
            kw[i] = vw[i] = 0x88888888u;
            ks[i] = vs[i] = 0;
            if (n < p.N && pos >= 0 && pos < kl) {
                int off;
                const int page = page_of(p.pg, b, page_div(p.pg, (int)pos, off));
                if (page >= 0) {
                    const uint32_t row = ((uint32_t)page * (uint32_t)p.H_kv + (uint32_t)h) * (uint32_t)p.pg.page_size + (uint32_t)off;
                    kw[i] = __ldcg(p.k_codes + (size_t)row * kLanes + sub);
                    vw[i] = __ldcg(p.v_codes + (size_t)row * kLanes + sub);
                    ks[i] = __ldcg(p.k_scales + (size_t)row * (D / kGroup) + (sub >> 2));
                    vs[i] = __ldcg(p.v_scales + (size_t)row * (D / kGroup) + (sub >> 2));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int n = n0 + i * kRows + r;
            if (n >= p.N) continue;
            k[(size_t)n * kLanes] = dequantise8(kw[i], ks[i]);
            v[(size_t)n * kLanes] = dequantise8(vw[i], vs[i]);
        }
    }
}

}  // namespace kv4
}  // namespace fa
