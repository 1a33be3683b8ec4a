// fa_kv4_attend.cuh -- attention over the 4-bit paged cache of fa_kv4_kernel.cuh, for few
// query rows per key/value head (decode, grouped heads, a few proposed tokens).
//
// All G = H / H_kv query heads of a key/value head, times N_q queries, are the rows that
// meet its keys: rows come in blocks of 8 * NB.  Per 16 keys a warp computes
//     S^T = K Q^T    (16 keys x 8 rows; m16n8k16, A = K dequantised in registers)
//     O^T += V^T P^T (16 channels x 8 rows per MMA; A = V^T dequantised in registers)
// so the dequantised operand is the 16-high A of the MMA and goes straight from the
// shared-memory bytes to the registers the MMA reads; no bf16 copy of the cache exists
// anywhere.  P^T is the accumulator of S^T with rows and columns exchanged, which is one
// movmatrix per 8 keys.  The order of channels along K is free in S (Q is permuted alike)
// and so is the order of channels along M in O, so each thread takes contiguous bytes.
//
// The cache streams through a per-warp ring of 16-key tiles filled with 16-byte cp.async
// copies (every wait is for the thread's own copies, so no barrier and nothing to time
// out).  The work of all sequences and heads is one line of 128-key units cut into equal
// shares, one per CTA: a long sequence is spread over many CTAs and many short ones share
// a CTA, whatever the lengths.  A (sequence, head, row block) that ends up in several CTAs
// is merged by the last of them to finish, from partial results in the workspace.
#pragma once

#include "fa_kv4_kernel.cuh"

namespace fa {
namespace kv4 {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                        // keys per warp and step
constexpr int kUnit = kTile * kWarps;            // keys per CTA and step
constexpr int kMaxEntries = 1024;                // (sequence, row block) pairs per launch

struct AttendParams {
    const __nv_bfloat16* q;    // [B, H_kv, R, D], R = G * N_q
    const uint8_t* k_codes;
    const uint16_t* k_scales;
    const uint8_t* v_codes;
    const uint16_t* v_scales;
    const int32_t* key_lens;
    const int32_t* q_lens;     // or NULL: N_q
    __nv_bfloat16* o;
    float* lse;
    Paging pg;
    int H_kv, N_q, R;
    int row_blocks;            // per sequence and head
    long long e0;              // first entry (sequence * row_blocks + row block) of this launch
    int E;                     // entries of this launch, <= kMaxEntries
    float scale_log2;          // scale * log2(e)
    int causal;
    int window;                // < 0: none
    float* part;               // per CTA two partial results: [2][RB][D] sums and [2][RB][4] (max, sums)
    float* part_ml;
    unsigned long long* words; // arrival words [E, H_kv]
    unsigned long long ticket; // not 0
};

template <int D, int NB>
struct Cfg {
    static constexpr int kRB = 8 * NB;                        // rows per block
    static constexpr int kRow = D / 2;                        // bytes of codes per token
    static constexpr int kSRow = D / kGroup * 2;              // bytes of scales per token
    static constexpr int kStageBytes = 2 * kTile * (kRow + kSRow);
    static constexpr int kStages = D == 128 ? 4 : 6;
    static constexpr int kKOff = 0;
    static constexpr int kVOff = kTile * kRow;
    static constexpr int kKSOff = 2 * kTile * kRow;
    static constexpr int kVSOff = kKSOff + kTile * kSRow;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kORow = D + 4;                       // padded fp32 row of the exchange
    static constexpr int kRedOff = kRingBytes;                // [kWarps][8][kORow]
    static constexpr int kRedBytes = kWarps * 8 * kORow * 4;
    static constexpr int kStatOff = kRedOff + kRedBytes;      // [kWarps][kRB] max, rounded sum, sum
    static constexpr int kStatBytes = 3 * kWarps * kRB * 4;
    static constexpr int kLimOff = kStatOff + kStatBytes;     // [kRB] first and one past the last visible key
    static constexpr int kQOff = kLimOff + 2 * kRB * 4;       // NB > 1: [NB][D/16][32] B fragments
    static constexpr int kQBytes = NB > 1 ? NB * (D / 16) * 32 * 8 : 0;
    static constexpr int kPreOff = kQOff + kQBytes;           // [E + 1] first unit of an entry
    static constexpr int kMiscOff = kPreOff + (kMaxEntries + 1) * 4;
    static constexpr int kSmemBytes = kMiscOff + 64;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
    if constexpr (W == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
    else if constexpr (W == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// Counts an arrival and tells whether it is the last of n.  The word holds
// (ticket << 16) | count; an arrival that finds another ticket (an earlier call, or what
// the workspace held) tries once to claim the word, and every add lands on a claimed
// word.  The last arrival clears it, so that a captured call, whose ticket is the same at
// each replay, starts anew.
__device__ __forceinline__ bool arrive_last(unsigned long long* word, unsigned long long ticket, int n) {
    const unsigned long long cur = atomicAdd(word, 0ull);
    if ((cur >> 16) != ticket) atomicCAS(word, cur, ticket << 16);
    const unsigned long long old = atomicAdd(word, 1ull);
    if ((int)(old & 0xffffull) + 1 != n) return false;
    atomicExch(word, 0ull);
    return true;
}

// What an entry (sequence, row block) attends to.
struct Entry {
    int b;
    int r0, nr;      // first row and rows of the block
    int kl, ql;      // keys and queries of the sequence
    int lo, hi;      // keys some row of the block sees: [lo, hi), lo a multiple of kTile
    int units;       // at least 1
};

template <int RB>
__device__ __forceinline__ Entry entry_of(const AttendParams& p, int e) {
    Entry x;
    const long long g = p.e0 + e;
    x.b = (int)(g / p.row_blocks);
    x.r0 = (int)(g - (long long)x.b * p.row_blocks) * RB;
    x.nr = min(RB, p.R - x.r0);
    x.kl = clamped(p.key_lens, x.b, p.pg.max_pages * p.pg.page_size);
    x.ql = clamped(p.q_lens, x.b, p.N_q);
    // the queries among the rows (row = head in group * N_q + query)
    int i0 = x.r0 % p.N_q, i1 = (x.r0 + x.nr - 1) % p.N_q;
    if (x.nr >= p.N_q || i1 < i0) {
        i0 = 0;
        i1 = p.N_q - 1;
    }
    i1 = min(i1, x.ql - 1);
    const long long off = (long long)x.kl - x.ql;
    long long lo = 0, hi = i0 > i1 ? 0 : x.kl;
    if (p.causal && off + i1 + 1 < hi) hi = off + i1 + 1;
    if (p.window >= 0 && off + i0 - p.window > 0) lo = off + i0 - p.window;
    if (hi < 0) hi = 0;
    if (lo > hi) lo = hi;
    x.lo = (int)lo & ~(kTile - 1);
    x.hi = (int)hi;
    x.units = max(1, (x.hi - x.lo + kUnit - 1) / kUnit);
    return x;
}

// Walks the units of the line: unit k of head h of entry e.
template <int RB>
struct Cursor {
    Entry x;
    int e, h, k;
    __device__ __forceinline__ void seek(const AttendParams& p, const int* pre, int u) {
        int a = 0, z = p.E;            // pre[a] <= u < pre[z]
        while (z - a > 1) {
            const int m = (a + z) >> 1;
            if (pre[m] <= u) a = m; else z = m;
        }
        e = a;
        x = entry_of<RB>(p, e);
        const int in = u - pre[a];
        h = in / x.units;
        k = in - h * x.units;
    }
    __device__ __forceinline__ void next(const AttendParams& p) {
        if (++k < x.units) return;
        k = 0;
        if (++h < p.H_kv) return;
        h = 0;
        if (++e < p.E) x = entry_of<RB>(p, e);
    }
};

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) attend_kernel(const AttendParams p) {
    using C = Cfg<D, NB>;
    constexpr int RB = C::kRB;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    float* const red = reinterpret_cast<float*>(smem + C::kRedOff);
    float* const st_max = reinterpret_cast<float*>(smem + C::kStatOff);      // [kWarps][RB]
    float* const st_sumr = st_max + kWarps * RB;
    float* const st_sum = st_sumr + kWarps * RB;
    int* const row_lo = reinterpret_cast<int*>(smem + C::kLimOff);
    int* const row_hi = row_lo + RB;
    int* const pre = reinterpret_cast<int*>(smem + C::kPreOff);
    int* const misc = reinterpret_cast<int*>(smem + C::kMiscOff);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;       // MMA fragment coordinates

    // ------------------------------------------------ the line of units and this CTA's share
    {
        const int per = (p.E + kThreads - 1) / kThreads;
        const int a = min(p.E, tid * per), z = min(p.E, a + per);
        int sum = 0;
        for (int e = a; e < z; ++e) sum += entry_of<RB>(p, e).units * p.H_kv;
        int inc = sum;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, sh);
            if (lane >= sh) inc += y;
        }
        if (lane == 31) misc[warp] = inc;
        __syncthreads();
        int at = inc - sum;
        for (int w = 0; w < warp; ++w) at += misc[w];
        for (int e = a; e < z; ++e) {
            pre[e] = at;
            at += entry_of<RB>(p, e).units * p.H_kv;
        }
        if (tid == kThreads - 1) pre[p.E] = at;
        __syncthreads();
    }
    const int total = pre[p.E];
    const int ctas = min((int)gridDim.x, total);
    if ((int)blockIdx.x >= ctas) return;
    auto share = [&](int c) { return (int)((long long)total * c / ctas); };
    const int u0 = share(blockIdx.x), u1 = share(blockIdx.x + 1);

    // ------------------------------------------------ loading
    const uint32_t ring = base + (uint32_t)(warp * C::kStages * C::kStageBytes);
    Cursor<RB> ld;
    ld.seek(p, pre, u0);
    uint32_t loaded = 0;     // one bit per tile, newest lowest: its keys are in the ring
    int ld_page = -1, ld_off = 0;
    // the page of the tile the cursor stands at, one step ahead of the copies that need it
    auto look_up = [&](int u) {
        ld_page = -1;
        const int pos = ld.x.lo + ld.k * kUnit + warp * kTile;
        if (u < u1 && pos < ld.x.hi) ld_page = page_of(p.pg, ld.x.b, page_div(p.pg, pos, ld_off));
    };
    auto issue = [&](int u) {        // copies the cursor's tile to its stage and moves on
        loaded = (loaded << 1) | (ld_page >= 0 ? 1u : 0u);
        if (ld_page >= 0) {
            const uint32_t st = ring + (uint32_t)((u - u0) % C::kStages * C::kStageBytes);
            const long long tok = ((long long)ld_page * p.H_kv + ld.h) * p.pg.page_size + ld_off;
            const int left = ld.x.kl - (ld.x.lo + ld.k * kUnit + warp * kTile);   // keys there are, > 0
            constexpr int kChunks = kTile * C::kRow / 16;            // 64 (D = 128) or 32
            constexpr int kPer = C::kRow / 16;                       // chunks of a token: 4 or 2
#pragma unroll
            for (int c = lane; c < kChunks; c += 32) {
                const int key = c / kPer, ch = c % kPer;
                // rows and chunks are placed so that the fragment loads below are free of
                // bank conflicts: the eight lanes (D = 128) or sixteen (D = 64) that one
                // shared-memory access serves hit different banks
                const int ks = D == 128 ? key ^ ((key >> 2) & 1) : key ^ (((key >> 2) & 1) << 1);
                const int vc = D == 128 ? ch ^ (((key >> 1) & 1) << 1) : ch;
                cp_async16(st + C::kKOff + ks * C::kRow + ch * 16, p.k_codes + tok * C::kRow + c * 16, 16);
                cp_async16(st + C::kVOff + key * C::kRow + vc * 16, p.v_codes + tok * C::kRow + c * 16, 16);
            }
            // scales; those behind the sequence's last key are zeroed, so that what an
            // unwritten row holds (a NaN, say) never meets the zero weights of masked keys
            constexpr int kSChunks = kTile * C::kSRow / 16;          // 8 or 4
            if (lane < 2 * kSChunks) {
                const int c = lane % kSChunks;
                const int n = max(0, min(16, left * C::kSRow - c * 16));
                const uint16_t* src = (lane < kSChunks ? p.k_scales : p.v_scales) + tok * (D / kGroup) + c * 8;
                cp_async16(st + (lane < kSChunks ? C::kKSOff : C::kVSOff) + c * 16, src, n);
            }
        }
        cp_async_commit();
        if (u + 1 < u1) ld.next(p);
        look_up(u + 1);
    };
    look_up(u0);
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) issue(u0 + s);

    // ------------------------------------------------ state of the block's rows
    constexpr int kKW = D / 32;      // words of a key's codes per thread (a quarter of the row)
    constexpr int kVW = D / 64;      // words of a key's codes per thread (an eighth of the row)
    constexpr int kMT = 4 * kVW;     // 16-channel tiles of O^T
    float acc[NB][kMT][4];
    float sumr[NB][4];               // sums of the rounded probabilities (every lane's copy is whole)
    float sum[NB][2];                // this lane's share of the sums, not rounded
    float ref[NB][2];                // reference max of rows 2t, 2t + 1 (log2 units), equal in all lanes of a t
    uint32_t qf[NB == 1 ? D / 16 : 1][2];
    const uint32_t qs = base + C::kQOff;

    auto load_q = [&](const Cursor<RB>& cu) {
        const __nv_bfloat16* q = p.q + ((long long)cu.x.b * p.H_kv + cu.h) * p.R * D + (long long)cu.x.r0 * D;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (NB > 1 && warp % NB != nb) continue;     // one warp per 8 rows fills the shared copy
            const int r = nb * 8 + g;
            const uint4* src = reinterpret_cast<const uint4*>(q + (long long)r * D + t * (D / 4));
#pragma unroll
            for (int w = 0; w < kKW; ++w) {
                const uint4 x = r < cu.x.nr ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                const uint32_t f[4] = {__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                       __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632)};
                if constexpr (NB == 1) {
                    qf[2 * w][0] = f[0];
                    qf[2 * w][1] = f[1];
                    qf[2 * w + 1][0] = f[2];
                    qf[2 * w + 1][1] = f[3];
                } else if (warp < NB) {
                    const uint32_t dst = qs + (uint32_t)(((nb * (D / 16) + 2 * w) * 32 + lane) * 8);
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(f[0]), "r"(f[1]) : "memory");
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + 256), "r"(f[2]), "r"(f[3]) : "memory");
                }
            }
        }
    };

    Cursor<RB> cu;
    cu.seek(p, pre, u0);
    int start = u0;                  // first unit of the current segment
    bool fresh = true;
    int all_lo = 0, all_hi = 0;      // keys every row of the block sees

    for (int u = u0; u < u1; ++u) {
        if (fresh) {
            fresh = false;
            start = u;
            load_q(cu);
            if (tid < RB) {
                const int i = (cu.x.r0 + tid) % p.N_q;
                const long long at = (long long)cu.x.kl - cu.x.ql + i;
                long long lo = 0, hi = (tid < cu.x.nr && i < cu.x.ql) ? cu.x.kl : 0;
                if (p.causal && at + 1 < hi) hi = at + 1;
                if (p.window >= 0 && at - p.window > 0) lo = at - p.window;
                row_lo[tid] = (int)min(lo, 0x7fffffffLL);
                row_hi[tid] = (int)max(hi, 0LL);
            }
            __syncthreads();
            all_lo = 0;
            all_hi = 0x7fffffff;
            for (int r = 0; r < cu.x.nr; ++r) {
                all_lo = max(all_lo, row_lo[r]);
                all_hi = min(all_hi, row_hi[r]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int m = 0; m < kMT; ++m)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[nb][m][c] = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) sumr[nb][c] = 0.f;
                sum[nb][0] = sum[nb][1] = 0.f;
                ref[nb][0] = ref[nb][1] = -INFINITY;
            }
        }
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        if ((loaded >> (C::kStages - 1)) & 1u) {
            const uint32_t st = ring + (uint32_t)((u - u0) % C::kStages * C::kStageBytes);
            const int pos = cu.x.lo + cu.k * kUnit + warp * kTile;
            // MMA row i of the tile (i < 8) is key i/2 + 4 (i mod 2), row 8 + i that key + 8
            const int key0 = (g >> 1) + 4 * (g & 1);
            // ---------------------------------------- scores
            float s[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
            {
                const int slot0 = D == 128 ? key0 ^ ((key0 >> 2) & 1) : key0 ^ (((key0 >> 2) & 1) << 1);
                uint32_t w0[kKW], w1[kKW];
                lds_words<kKW>(st + C::kKOff + slot0 * C::kRow + t * (C::kRow / 4), w0);
                lds_words<kKW>(st + C::kKOff + (slot0 + 8) * C::kRow + t * (C::kRow / 4), w1);
                const uint32_t sa = st + C::kKSOff + key0 * C::kSRow + (t * (D / 4) / kGroup) * 2;
                uint32_t s0 = lds_u16(sa), s1 = lds_u16(sa + 8 * C::kSRow);
                s0 |= s0 << 16;
                s1 |= s1 << 16;
                const uint32_t z0 = minus_24(s0), z1 = minus_24(s1);
#pragma unroll
                for (int w = 0; w < kKW; ++w) {
                    const uint32_t a0 = codes_to_bf16x2<0>(w0[w], s0, z0), a1 = codes_to_bf16x2<0>(w1[w], s1, z1);
                    const uint32_t a2 = codes_to_bf16x2<1>(w0[w], s0, z0), a3 = codes_to_bf16x2<1>(w1[w], s1, z1);
                    const uint32_t c0 = codes_to_bf16x2<2>(w0[w], s0, z0), c1 = codes_to_bf16x2<2>(w1[w], s1, z1);
                    const uint32_t c2 = codes_to_bf16x2<3>(w0[w], s0, z0), c3 = codes_to_bf16x2<3>(w1[w], s1, z1);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if constexpr (NB == 1) {
                            mma_bf16(s[0], a0, a1, a2, a3, qf[2 * w][0], qf[2 * w][1]);
                            mma_bf16(s[0], c0, c1, c2, c3, qf[2 * w + 1][0], qf[2 * w + 1][1]);
                        } else {
                            uint32_t b[2];
                            lds_words<2>(qs + (uint32_t)(((nb * (D / 16) + 2 * w) * 32 + lane) * 8), b);
                            mma_bf16(s[nb], a0, a1, a2, a3, b[0], b[1]);
                            lds_words<2>(qs + (uint32_t)(((nb * (D / 16) + 2 * w + 1) * 32 + lane) * 8), b);
                            mma_bf16(s[nb], c0, c1, c2, c3, b[0], b[1]);
                        }
                    }
                }
            }
            // ---------------------------------------- mask, reference max, probabilities
            const bool edge = pos < all_lo || pos + kTile > all_hi;
            if (edge) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int r = nb * 8 + 2 * t + (c & 1), key = pos + key0 + (c >> 1) * 8;
                        if (key < row_lo[r] || key >= row_hi[r]) s[nb][c] = -INFINITY;
                    }
            }
            // the reference moves only when some score exceeds it by more than 2^8: until
            // then probabilities stay below 2^8 and nothing needs to be rescaled
            bool grow = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                grow |= fmaxf(s[nb][0], s[nb][2]) * p.scale_log2 > ref[nb][0] + 8.f;
                grow |= fmaxf(s[nb][1], s[nb][3]) * p.scale_log2 > ref[nb][1] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = fmaxf(s[nb][c], s[nb][c + 2]) * p.scale_log2;
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        if (m > ref[nb][c]) {
                            const float f = ex2_approx(ref[nb][c] - m);   // 0 from a reference of -inf
                            ref[nb][c] = m;
                            sum[nb][c] *= f;
                            sumr[nb][c] *= f;
#pragma unroll
                            for (int mt = 0; mt < kMT; ++mt) {
                                acc[nb][mt][c] *= f;
                                acc[nb][mt][c + 2] *= f;
                            }
                        }
                    }
            }
            uint32_t pb[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                // a row that has seen no key yet has reference -inf: 2^(-inf - 0) = 0
                const float m0 = ref[nb][0] == -INFINITY ? 0.f : ref[nb][0];
                const float m1 = ref[nb][1] == -INFINITY ? 0.f : ref[nb][1];
                const float p0 = ex2_approx(fmaf(s[nb][0], p.scale_log2, -m0));
                const float p1 = ex2_approx(fmaf(s[nb][1], p.scale_log2, -m1));
                const float p2 = ex2_approx(fmaf(s[nb][2], p.scale_log2, -m0));
                const float p3 = ex2_approx(fmaf(s[nb][3], p.scale_log2, -m1));
                sum[nb][0] += p0 + p2;
                sum[nb][1] += p1 + p3;
                // P rounds to bf16 (2^-8) for the tensor cores; O is divided by the sum of
                // the rounded values, so a row that one key dominates stays exact
                pb[nb][0] = transpose8x8(pack_bf16x2(p0, p1));
                pb[nb][1] = transpose8x8(pack_bf16x2(p2, p3));
                mma_bf16(sumr[nb], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, pb[nb][0], pb[nb][1]);
            }
            // ---------------------------------------- O^T += V^T P^T
            {
                // MMA k index 2t is key t, 2t + 1 key t + 4, 2t + 8 and 2t + 9 those + 8
                uint32_t w[4][kVW], sv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = t + 4 * j;
                    const int byte = g * (C::kRow / 8);
                    const int ch = D == 128 ? (byte >> 4) ^ (((key >> 1) & 1) << 1) : byte >> 4;
                    lds_words<kVW>(st + C::kVOff + key * C::kRow + ch * 16 + (byte & 15), w[j]);
                    sv[j] = lds_u16(st + C::kVSOff + key * C::kSRow + (g * (D / 8) / kGroup) * 2);
                }
                const uint32_t sA = sv[0] | (sv[1] << 16), sB = sv[2] | (sv[3] << 16);
                bool poisoned = false;
                if (edge) {
                    // a NaN group meets zero weights in the rows that do not see its key:
                    // the tile is then taken row by row, with the hidden keys' scales zero
                    bool bad = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) bad |= (sv[j] & 0x7fffu) > 0x7f80u;
                    poisoned = __any_sync(0xffffffffu, bad);
                }
                if (!poisoned) {
                    const uint32_t zA = minus_24(sA), zB = minus_24(sB);
#pragma unroll
                    for (int vw = 0; vw < kVW; ++vw) {
                        const uint32_t la = __byte_perm(w[0][vw], w[1][vw], 0x5410);
                        const uint32_t ha = __byte_perm(w[0][vw], w[1][vw], 0x7632);
                        const uint32_t lb = __byte_perm(w[2][vw], w[3][vw], 0x5410);
                        const uint32_t hb = __byte_perm(w[2][vw], w[3][vw], 0x7632);
#define FA_KV4_PV(I)                                                                                       \
    {                                                                                                      \
        const uint32_t a0 = codes_to_bf16x2<I>(la, sA, zA), a1 = codes_to_bf16x2<I>(ha, sA, zA);           \
        const uint32_t a2 = codes_to_bf16x2<I>(lb, sB, zB), a3 = codes_to_bf16x2<I>(hb, sB, zB);           \
        _Pragma("unroll") for (int nb = 0; nb < NB; ++nb)                                                  \
            mma_bf16(acc[nb][4 * vw + I], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);                           \
    }
                        FA_KV4_PV(0)
                        FA_KV4_PV(1)
                        FA_KV4_PV(2)
                        FA_KV4_PV(3)
                    }
                } else {
                    for (int r = 0; r < RB; ++r) {
                        uint32_t sr[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = pos + t + 4 * j;
                            sr[j] = key >= row_lo[r] && key < row_hi[r] ? sv[j] : 0u;
                        }
                        const uint32_t sA = sr[0] | (sr[1] << 16), sB = sr[2] | (sr[3] << 16);
                        const uint32_t zA = minus_24(sA), zB = minus_24(sB);
                        const bool mine0 = (r & 7) == 2 * t, mine1 = (r & 7) == 2 * t + 1;
#pragma unroll
                        for (int vw = 0; vw < kVW; ++vw) {
                            const uint32_t la = __byte_perm(w[0][vw], w[1][vw], 0x5410);
                            const uint32_t ha = __byte_perm(w[0][vw], w[1][vw], 0x7632);
                            const uint32_t lb = __byte_perm(w[2][vw], w[3][vw], 0x5410);
                            const uint32_t hb = __byte_perm(w[2][vw], w[3][vw], 0x7632);
#define FA_KV4_PV_ROW(I)                                                                                   \
    {                                                                                                      \
        const uint32_t a0 = codes_to_bf16x2<I>(la, sA, zA), a1 = codes_to_bf16x2<I>(ha, sA, zA);           \
        const uint32_t a2 = codes_to_bf16x2<I>(lb, sB, zB), a3 = codes_to_bf16x2<I>(hb, sB, zB);           \
        _Pragma("unroll") for (int nb = 0; nb < NB; ++nb) {                                                \
            float one[4] = {0.f, 0.f, 0.f, 0.f};                                                           \
            mma_bf16(one, a0, a1, a2, a3, pb[nb][0], pb[nb][1]);                                           \
            if (nb == (r >> 3)) {                                                                          \
                if (mine0) acc[nb][4 * vw + I][0] += one[0], acc[nb][4 * vw + I][2] += one[2];             \
                if (mine1) acc[nb][4 * vw + I][1] += one[1], acc[nb][4 * vw + I][3] += one[3];             \
            }                                                                                              \
        }                                                                                                  \
    }
                            FA_KV4_PV_ROW(0)
                            FA_KV4_PV_ROW(1)
                            FA_KV4_PV_ROW(2)
                            FA_KV4_PV_ROW(3)
                        }
                    }
                }
            }
        }
        __syncwarp();                        // every lane has read the stage
        issue(u + C::kStages);

        const bool ends = cu.k + 1 == cu.x.units;
        if (!ends && u + 1 < u1) {
            cu.next(p);
            continue;
        }
        // ------------------------------------------------ the segment's rows: combine the warps
        const int nr = cu.x.nr;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = sum[nb][c];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    const int r = nb * 8 + 2 * t + c;
                    st_max[warp * RB + r] = ref[nb][c];
                    st_sumr[warp * RB + r] = sumr[nb][c];
                    st_sum[warp * RB + r] = l;
                }
            }
        __syncthreads();
        const int item_first = pre[cu.e] + cu.h * cu.x.units;       // the item's units on the line
        const bool whole = start == item_first && ends;
        const int slot = (int)blockIdx.x * 2 + (start == u0 ? 0 : 1);
        const long long row0 = ((long long)cu.x.b * p.H_kv + cu.h) * p.R + cu.x.r0;
        for (int nb = 0; nb < NB; ++nb) {
            if (nb * 8 >= nr) break;
            if (nb > 0) __syncthreads();     // the exchange buffer is free again
#pragma unroll
            for (int nc = 0; nc < NB; ++nc) {
                if (nc != nb) continue;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = 2 * t + c;
                    if (nb * 8 + r >= nr) continue;
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, st_max[w * RB + nb * 8 + r]);
                    const float f = ref[nc][c] == -INFINITY ? 0.f : ex2_approx(ref[nc][c] - m);
                    float* dst = red + (warp * 8 + r) * C::kORow + g * (D / 8);
#pragma unroll
                    for (int vw = 0; vw < kVW; ++vw) {
                        float4 lo4 = make_float4(acc[nc][4 * vw][c], acc[nc][4 * vw + 1][c], acc[nc][4 * vw + 2][c],
                                                 acc[nc][4 * vw + 3][c]);
                        float4 hi4 = make_float4(acc[nc][4 * vw][c + 2], acc[nc][4 * vw + 1][c + 2],
                                                 acc[nc][4 * vw + 2][c + 2], acc[nc][4 * vw + 3][c + 2]);
                        lo4.x *= f, lo4.y *= f, lo4.z *= f, lo4.w *= f;
                        hi4.x *= f, hi4.y *= f, hi4.z *= f, hi4.w *= f;
                        *reinterpret_cast<float4*>(dst + vw * 8) = lo4;
                        *reinterpret_cast<float4*>(dst + vw * 8 + 4) = hi4;
                    }
                }
            }
            __syncthreads();
            const int rows = min(8, nr - nb * 8);
            for (int it = tid; it < rows * (D / 4); it += kThreads) {
                const int r = it / (D / 4), c4 = it % (D / 4), rr = nb * 8 + r;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, st_max[w * RB + rr]);
                float lr = 0.f, l = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = st_max[w * RB + rr];
                    const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - m);
                    lr = fmaf(st_sumr[w * RB + rr], f, lr);
                    l = fmaf(st_sum[w * RB + rr], f, l);
                    const float4 x = *reinterpret_cast<const float4*>(red + (w * 8 + r) * C::kORow + 4 * c4);
                    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
                }
                if (whole) {
                    const float inv = l == 0.f ? 0.f : 1.f / lr;
                    uint2 pk;
                    pk.x = pack_bf16x2(a.x * inv, a.y * inv);
                    pk.y = pack_bf16x2(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + 4 * c4) = pk;
                    if (c4 == 0) p.lse[row0 + rr] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                } else {
                    *reinterpret_cast<float4*>(p.part + ((long long)slot * RB + rr) * D + 4 * c4) = a;
                    if (c4 == 0)
                        *reinterpret_cast<float4*>(p.part_ml + ((long long)slot * RB + rr) * 4) = make_float4(m, lr, l, 0.f);
                }
            }
        }
        if (!whole) {
            // ---------------------------------------- partial: the last CTA of the item merges
            // the CTA that holds unit x is the largest c with share(c) <= x
            auto holder = [&](int x) { return (int)((((long long)x + 1) * ctas - 1) / total); };
            const int cf = holder(item_first), cl = holder(item_first + cu.x.units - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0)
                misc[0] = arrive_last(p.words + (long long)cu.e * p.H_kv + cu.h, p.ticket, cl - cf + 1) ? 1 : 0;
            __syncthreads();
            if (misc[0]) {
                __threadfence();
                // a CTA whose share starts inside the item has it first, else last
                auto slot_of = [&](int c) { return (long long)(2 * c + (share(c) >= item_first ? 0 : 1)); };
                for (int it = tid; it < nr * (D / 4); it += kThreads) {
                    const int rr = it / (D / 4), c4 = it % (D / 4);
                    float m = -INFINITY;
#pragma unroll 8
                    for (int c = cf; c <= cl; ++c) m = fmaxf(m, __ldcg(p.part_ml + (slot_of(c) * RB + rr) * 4));
                    float lr = 0.f, l = 0.f;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = cf; c <= cl; ++c) {
                        const long long at = slot_of(c) * RB + rr;
                        const float4 ml = __ldcg(reinterpret_cast<const float4*>(p.part_ml + at * 4));
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part + at * D) + c4);
                        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                        lr = fmaf(ml.y, f, lr);
                        l = fmaf(ml.z, f, l);
                        a.x = fmaf(x.x, f, a.x);
                        a.y = fmaf(x.y, f, a.y);
                        a.z = fmaf(x.z, f, a.z);
                        a.w = fmaf(x.w, f, a.w);
                    }
                    const float inv = l == 0.f ? 0.f : 1.f / lr;
                    uint2 pk;
                    pk.x = pack_bf16x2(a.x * inv, a.y * inv);
                    pk.y = pack_bf16x2(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + 4 * c4) = pk;
                    if (c4 == 0) p.lse[row0 + rr] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                }
            }
        }
        __syncthreads();                     // statistics, exchange buffer and row limits are free again
        cu.next(p);
        fresh = true;
    }
    cp_async_wait<0>();
}

}  // namespace kv4
}  // namespace fa
