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

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;                        // keys per warp and step: two MMA tiles
constexpr int kUnit = kTile * kWarps;            // keys per CTA and step
constexpr int kMaxEntries = 512;                 // (sequence, row block) pairs per launch

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
    int b0, rb0;               // sequence and row block of this launch's first entry
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
    static constexpr int kCtasPerSm = NB == 1 ? 4 : 2;
    static constexpr int kRow = D / 2;                        // bytes of codes per token
    static constexpr int kSRow = D / kGroup * 2;              // bytes of scales per token
    static constexpr int kStageBytes = 2 * kTile * (kRow + kSRow);
    static constexpr int kStages = NB == 1 && D == 128 ? 2 : 4;
    static constexpr int kVOff = kTile * kRow;                // within a stage: K codes, V codes, K scales, V scales
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
    static_assert((kSmemBytes + 1024) * kCtasPerSm <= 233472, "shared memory of an SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// Arrivals of a call's CTAs at an item.  The word holds (ticket << 16) | count.  Before its
// arrival a CTA makes sure that the word carries this call's ticket: one that finds
// another (an earlier call, or what the workspace held) tries once to claim the word, and
// whoever fails found it claimed.  The last arrival clears it, so that a captured call,
// whose ticket is the same at each replay, starts anew.
__device__ __forceinline__ void arrive_claim(unsigned long long* word, unsigned long long ticket) {
    const unsigned long long cur = atomicAdd(word, 0ull);
    if ((cur >> 16) != ticket) atomicCAS(word, cur, ticket << 16);
}
__device__ __forceinline__ bool arrive_last(unsigned long long* word, int n) {
    const unsigned long long old = atomicAdd(word, 1ull);
    if ((int)(old & 0xffffull) + 1 != n) return false;
    atomicExch(word, 0ull);
    return true;
}

// What an entry (sequence, row block) attends to.
struct Entry {
    int b;
    int r0, nr;            // first row and rows of the block
    int kl, ql;            // keys and queries of the sequence
    int lo, hi;            // keys some row of the block sees: [lo, hi), lo rounded down to a multiple of kTile
    int all_lo, all_hi;    // keys every row sees
    int units;             // at least 1
};

template <int RB>
__device__ __forceinline__ Entry entry_of(const AttendParams& p, int e) {
    Entry x;
    int g = p.rb0 + e;
    x.b = p.b0;
    if (p.row_blocks == 1) {
        x.b += g;
        g = 0;
    } else {
        const int n = g / p.row_blocks;
        x.b += n;
        g -= n * p.row_blocks;
    }
    x.r0 = g * RB;
    x.nr = min(RB, p.R - x.r0);
    x.kl = clamped(p.key_lens, x.b, p.pg.max_pages * p.pg.page_size);
    x.ql = clamped(p.q_lens, x.b, p.N_q);
    // the queries among the rows (row = head in group * N_q + query)
    int i0 = 0, i1 = p.N_q - 1;
    if (x.nr < p.N_q) {
        const int a = x.r0 % p.N_q, z = a + x.nr - 1;
        if (z < p.N_q) {
            i0 = a;
            i1 = z;
        }
    }
    const bool rows_without = i1 >= x.ql;
    i1 = min(i1, x.ql - 1);
    const long long off = (long long)x.kl - x.ql;
    long long lo = 0, hi = i0 > i1 ? 0 : x.kl, all_lo = 0, all_hi = rows_without ? 0 : x.kl;
    if (p.causal) {
        hi = min(hi, off + i1 + 1);
        all_hi = min(all_hi, off + i0 + 1);
    }
    if (p.window >= 0) {
        lo = max(lo, off + i0 - p.window);
        all_lo = max(all_lo, off + i1 - p.window);
    }
    hi = max(hi, 0ll);
    lo = min(lo, hi);
    x.lo = (int)lo & ~(kTile - 1);
    x.hi = (int)hi;
    x.all_lo = (int)all_lo;
    x.all_hi = (int)max(all_hi, 0ll);
    x.units = max(1, (x.hi - x.lo + kUnit - 1) / kUnit);
    return x;
}

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, Cfg<D, NB>::kCtasPerSm) attend_kernel(const AttendParams p) {
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

    // ------------------------------------------------ the line of units
    {
        constexpr int kPer = kMaxEntries / kThreads;
        int n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n[i] = 0;
            if (i * kThreads < p.E) {            // thread's entries: tid * per .. + per - 1, per = ceil(E / kThreads)
                const int per = (p.E + kThreads - 1) / kThreads, e = tid * per + i;
                if (i < per && e < p.E) n[i] = entry_of<RB>(p, e).units * p.H_kv;
            }
            sum += n[i];
        }
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
        const int per = (p.E + kThreads - 1) / kThreads;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i < per && tid * per + i < p.E) pre[tid * per + i] = at;
            at += n[i];
        }
        if (tid == kThreads - 1) pre[p.E] = at;
        __syncthreads();
    }
    // this CTA's share: total units over the CTAs, the first total % ctas get one more
    const int total = pre[p.E];
    const int ctas = min((int)gridDim.x, total);
    if ((int)blockIdx.x >= ctas) return;
    const int each = total / ctas, more = total - each * ctas;
    auto share = [&](int c) { return each * c + min(c, more); };
    const int u0 = share(blockIdx.x), u1 = share(blockIdx.x + 1);

    // ------------------------------------------------ loading: a cursor ahead of the arithmetic
    int l_e, l_h, l_left;            // entry, head, units left in the item
    int l_units, l_lo, l_hi, l_b, l_pos;
    {
        int a = 0, z = p.E;          // pre[a] <= u0 < pre[z]
        while (z - a > 1) {
            const int m = (a + z) >> 1;
            if (pre[m] <= u0) a = m; else z = m;
        }
        l_e = a;
    }
    Entry x = entry_of<RB>(p, l_e);  // of the current segment
    int seg_h, seg_k;                // its head, and the first of its units in the item
    {
        const int in = u0 - pre[l_e];
        seg_h = in / x.units;
        seg_k = in - seg_h * x.units;
        l_h = seg_h;
        l_units = x.units;
        l_left = x.units - seg_k;
        l_lo = x.lo + warp * kTile;
        l_hi = x.hi;
        l_b = x.b;
        l_pos = l_lo + seg_k * kUnit;
    }
    int seg_e = l_e;
    int l_page[2], l_off[2];
    // pages of the cursor's tile, a step before the copies need them; a tile is two runs of
    // 16 keys, each inside one page
    auto look_up = [&](bool any) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l_page[i] = -1;
            l_off[i] = 0;
            const int pos = l_pos + 16 * i;
            if (any && pos < l_hi) l_page[i] = page_of(p.pg, l_b, page_div(p.pg, pos, l_off[i]));
        }
    };
    const uint32_t ring = base + (uint32_t)(warp * C::kStages * C::kStageBytes);
    // Rows and chunks of 16 bytes are placed so that the fragment loads below are free of
    // bank conflicts: the lanes that one shared-memory access serves hit different banks.
    constexpr int kPer = C::kRow / 16;            // chunks of a token's codes: 4 or 2
    uint32_t dst_k, dst_v, dst_s;                 // where this lane's chunks go within a stage
    const uint8_t *src_k, *src_v, *src_s;         // and where they come from, for row 0 of the cache
    {
        const int key = lane / kPer, ch = lane % kPer;
        const int ks = D == 128 ? key ^ ((key >> 2) & 1) : key ^ (((key >> 2) & 1) << 1);
        const int vc = D == 128 ? ch ^ (((key >> 1) & 1) << 1) : ch;
        dst_k = ks * C::kRow + ch * 16;
        dst_v = C::kVOff + key * C::kRow + vc * 16;
        src_k = p.k_codes + lane * 16;
        src_v = p.v_codes + lane * 16;
        constexpr int kSC = kTile * C::kSRow / 16;               // chunks of a tile's scales, per tensor: 16 or 8
        const int c = lane % kSC;
        dst_s = (lane < kSC ? C::kKSOff : C::kVSOff) + c * 16;
        src_s = reinterpret_cast<const uint8_t*>(lane < kSC ? p.k_scales : p.v_scales) + c % (kSC / 2) * 16;
    }
    const bool s_second = lane % (kTile * C::kSRow / 16) >= kTile * C::kSRow / 32;   // its scales are of the second run
    uint32_t loaded = 0;             // two bits per tile, newest lowest: which runs are in the ring
    uint32_t l_stage = 0;
    auto issue = [&](bool any, bool next) {      // copies the cursor's tile and moves the cursor on
        uint32_t row[2];
        loaded <<= 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            row[i] = ((uint32_t)l_page[i] * (uint32_t)p.H_kv + (uint32_t)l_h) * (uint32_t)p.pg.page_size + (uint32_t)l_off[i];
            if (l_page[i] >= 0) loaded |= 1u << i;
        }
        const uint32_t st = ring + l_stage * C::kStageBytes;
        if (any) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (l_page[i] >= 0) {
#pragma unroll
                    for (int j = 0; j < C::kRow / 32; ++j) {     // 16 keys: kRow / 32 chunks a lane
                        cp_async16(st + dst_k + i * 16 * C::kRow + j * 512, src_k + (size_t)row[i] * C::kRow + j * 512);
                        cp_async16(st + dst_v + i * 16 * C::kRow + j * 512, src_v + (size_t)row[i] * C::kRow + j * 512);
                    }
                }
            const int page = s_second ? l_page[1] : l_page[0];
            if (page >= 0 && lane < 2 * (kTile * C::kSRow / 16))
                cp_async16(st + dst_s, src_s + (size_t)(s_second ? row[1] : row[0]) * C::kSRow);
        }
        cp_async_commit();
        l_stage = l_stage + 1 == C::kStages ? 0 : l_stage + 1;
        if (next) {
            l_pos += kUnit;
            if (--l_left == 0) {                 // the next item: next head, or next entry
                if (++l_h == p.H_kv) {
                    l_h = 0;
                    const Entry y = entry_of<RB>(p, ++l_e);
                    l_units = y.units;
                    l_lo = y.lo + warp * kTile;
                    l_hi = y.hi;
                    l_b = y.b;
                }
                l_left = l_units;
                l_pos = l_lo;
            }
        }
        look_up(next);
    };
    look_up(true);
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) issue(u0 + s < u1, u0 + s + 1 < u1);

    // ------------------------------------------------ state of the block's rows
    constexpr int kKW = D / 32;      // words of a key's codes per thread (a quarter of the row)
    constexpr int kVW = D / 64;      // words of a key's codes per thread (an eighth of the row)
    constexpr int kMT = 4 * kVW;     // 16-channel tiles of O^T
    float acc[NB][kMT][4];
    float sumr[NB][4];               // sums of the rounded probabilities (every lane's copy is whole)
    float sum[NB][2];                // this lane's share of the sums, not rounded
    float ref[NB][2];                // reference max of rows 2t, 2t + 1 (log2 units), equal in all lanes of a t
    float top[NB][2];                // raw score above which the reference moves
    float neg[NB][2];                // -ref, or 0 while the row has seen no key
    uint32_t qf[NB == 1 ? D / 16 : 1][2];
    const uint32_t qs = base + C::kQOff;
    // MMA row i of a 16-key tile (i < 8) is key i/2 + 4 (i mod 2), row 8 + i that key + 8
    const int key0 = (g >> 1) + 4 * (g & 1);
    const uint32_t at_k = (uint32_t)((D == 128 ? key0 ^ ((key0 >> 2) & 1) : key0 ^ (((key0 >> 2) & 1) << 1)) * C::kRow +
                                     t * (C::kRow / 4));
    const uint32_t at_ks = C::kKSOff + (uint32_t)(key0 * C::kSRow + (t * (D / 4) / kGroup) * 2);
    // MMA k index 2t is key t, 2t + 1 key t + 4, 2t + 8 and 2t + 9 those + 8
    const int vb = g * (C::kRow / 8);
    const uint32_t at_v = C::kVOff + (uint32_t)(t * C::kRow + (D == 128 ? (vb >> 4) ^ (((t >> 1) & 1) << 1) : vb >> 4) * 16 + (vb & 15));
    const uint32_t at_vs = C::kVSOff + (uint32_t)(t * C::kSRow + (g * (D / 8) / kGroup) * 2);
    const float inv_scale = 1.f / p.scale_log2;

    uint32_t c_stage = 0;
    for (int u = u0; u < u1;) {
        // ============================================ a segment: units seg_k .. of an item
        const int n = min(x.units - seg_k, u1 - u);
        const int item_first = pre[seg_e] + seg_h * x.units;
        const bool whole = seg_k == 0 && n == x.units;
        unsigned long long* const word = p.words + (long long)seg_e * p.H_kv + seg_h;
        if (!whole && tid == 0) arrive_claim(word, p.ticket);
        {
            const __nv_bfloat16* q = p.q + (((long long)x.b * p.H_kv + seg_h) * p.R + x.r0) * D;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (NB > 1 && warp != nb % kWarps) continue;     // one warp per 8 rows fills the shared copy
                const int r = nb * 8 + g;
                const uint4* src = reinterpret_cast<const uint4*>(q + (long long)r * D + t * (D / 4));
#pragma unroll
                for (int w = 0; w < kKW; ++w) {
                    const uint4 y = r < x.nr ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                    const uint32_t f[4] = {__byte_perm(y.x, y.z, 0x5410), __byte_perm(y.x, y.z, 0x7632),
                                           __byte_perm(y.y, y.w, 0x5410), __byte_perm(y.y, y.w, 0x7632)};
                    if constexpr (NB == 1) {
                        qf[2 * w][0] = f[0];
                        qf[2 * w][1] = f[1];
                        qf[2 * w + 1][0] = f[2];
                        qf[2 * w + 1][1] = f[3];
                    } else {
                        const uint32_t dst = qs + (uint32_t)(((nb * (D / 16) + 2 * w) * 32 + lane) * 8);
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(f[0]), "r"(f[1]) : "memory");
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + 256), "r"(f[2]), "r"(f[3]) : "memory");
                    }
                }
            }
        }
        if (tid < RB) {
            const int i = p.N_q == 1 ? 0 : (x.r0 + tid) % p.N_q;
            const long long at = (long long)x.kl - x.ql + i;
            long long lo = 0, hi = (tid < x.nr && i < x.ql) ? x.kl : 0;
            if (p.causal) hi = min(hi, at + 1);
            if (p.window >= 0) lo = max(lo, at - p.window);
            row_lo[tid] = (int)min(lo, 0x7fffffffLL);
            row_hi[tid] = (int)max(hi, 0LL);
        }
        __syncthreads();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[nb][m][c] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) sumr[nb][c] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sum[nb][c] = neg[nb][c] = 0.f;
                ref[nb][c] = top[nb][c] = -INFINITY;
            }
        }
        int pos = x.lo + seg_k * kUnit + warp * kTile;
        for (int k = 0; k < n; ++k, ++u, pos += kUnit) {
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t have = (loaded >> (2 * (C::kStages - 1))) & 3u;
            const uint32_t st = ring + c_stage * C::kStageBytes;
            if (have != 0) {
                // ------------------------------------ scores of two 16-key tiles
                float s[2][NB][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) s[j][nb][0] = s[j][nb][1] = s[j][nb][2] = s[j][nb][3] = 0.f;
                    uint32_t w0[kKW], w1[kKW];
                    lds_words<kKW>(st + at_k + j * 16 * C::kRow, w0);
                    lds_words<kKW>(st + at_k + (j * 16 + 8) * C::kRow, w1);
                    uint32_t s0 = lds_u16(st + at_ks + j * 16 * C::kSRow), s1 = lds_u16(st + at_ks + (j * 16 + 8) * C::kSRow);
                    s0 = __byte_perm(s0, s0, 0x1010);
                    s1 = __byte_perm(s1, s1, 0x1010);
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
                                mma_bf16(s[j][0], a0, a1, a2, a3, qf[2 * w][0], qf[2 * w][1]);
                                mma_bf16(s[j][0], c0, c1, c2, c3, qf[2 * w + 1][0], qf[2 * w + 1][1]);
                            } else {
                                uint32_t b[2];
                                lds_words<2>(qs + (uint32_t)(((nb * (D / 16) + 2 * w) * 32 + lane) * 8), b);
                                mma_bf16(s[j][nb], a0, a1, a2, a3, b[0], b[1]);
                                lds_words<2>(qs + (uint32_t)(((nb * (D / 16) + 2 * w + 1) * 32 + lane) * 8), b);
                                mma_bf16(s[j][nb], c0, c1, c2, c3, b[0], b[1]);
                            }
                        }
                    }
                }
                // ------------------------------------ mask, reference max, probabilities
                const bool edge = pos < x.all_lo || pos + kTile > x.all_hi || have != 3;
                if (edge) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int r = nb * 8 + 2 * t + (c & 1), key = pos + 16 * j + key0 + (c >> 1) * 8;
                                if (key < row_lo[r] || key >= row_hi[r] || !((have >> j) & 1u)) s[j][nb][c] = -INFINITY;
                            }
                }
                // the reference moves only when some score exceeds it by more than 2^8: until
                // then probabilities stay below 2^8 and nothing needs to be rescaled
                bool grow = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        grow |= fmaxf(max3f(s[0][nb][c], s[0][nb][c + 2], s[1][nb][c]), s[1][nb][c + 2]) > top[nb][c];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float m = fmaxf(max3f(s[0][nb][c], s[0][nb][c + 2], s[1][nb][c]), s[1][nb][c + 2]) * p.scale_log2;
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            if (m > ref[nb][c]) {
                                const float f = ex2_approx(ref[nb][c] - m);   // 0 from a reference of -inf
                                ref[nb][c] = m;
                                neg[nb][c] = -m;
                                top[nb][c] = (m + 8.f) * inv_scale;
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
                uint32_t pb[2][NB][2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const float p0 = ex2_approx(fmaf(s[j][nb][0], p.scale_log2, neg[nb][0]));
                        const float p1 = ex2_approx(fmaf(s[j][nb][1], p.scale_log2, neg[nb][1]));
                        const float p2 = ex2_approx(fmaf(s[j][nb][2], p.scale_log2, neg[nb][0]));
                        const float p3 = ex2_approx(fmaf(s[j][nb][3], p.scale_log2, neg[nb][1]));
                        sum[nb][0] += p0 + p2;
                        sum[nb][1] += p1 + p3;
                        // P rounds to bf16 (2^-8) for the tensor cores; O is divided by the sum of
                        // the rounded values, so a row that one key dominates stays exact
                        pb[j][nb][0] = transpose8x8(pack_bf16x2(p0, p1));
                        pb[j][nb][1] = transpose8x8(pack_bf16x2(p2, p3));
                        mma_bf16(sumr[nb], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, pb[j][nb][0], pb[j][nb][1]);
                    }
                // ------------------------------------ O^T += V^T P^T
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w[4][kVW], sv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lds_words<kVW>(st + at_v + (j * 16 + 4 * i) * C::kRow, w[i]);
                        sv[i] = lds_u16(st + at_vs + (j * 16 + 4 * i) * C::kSRow);
                    }
                    bool poisoned = false;
                    if (edge) {
                        // what lies behind the last key, or was not loaded, counts as zero; a NaN
                        // group of another key meets zero weights in the rows that do not see
                        // it: the tile is then taken row by row, with the hidden keys' scales zero
                        bool bad = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (pos + 16 * j + t + 4 * i >= x.kl || !((have >> j) & 1u)) sv[i] = 0;
                            bad |= (sv[i] & 0x7fffu) > 0x7f80u;
                        }
                        poisoned = __any_sync(0xffffffffu, bad);
                    }
                    if (!poisoned) {
                        const uint32_t sA = __byte_perm(sv[0], sv[1], 0x5410), sB = __byte_perm(sv[2], sv[3], 0x5410);
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
            mma_bf16(acc[nb][4 * vw + I], a0, a1, a2, a3, pb[j][nb][0], pb[j][nb][1]);                     \
    }
                            FA_KV4_PV(0)
                            FA_KV4_PV(1)
                            FA_KV4_PV(2)
                            FA_KV4_PV(3)
#undef FA_KV4_PV
                        }
                    } else {
#pragma unroll 1
                        for (int r = 0; r < RB; ++r) {
                            uint32_t sr[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = pos + 16 * j + t + 4 * i;
                                sr[i] = key >= row_lo[r] && key < row_hi[r] ? sv[i] : 0u;
                            }
                            const uint32_t sA = __byte_perm(sr[0], sr[1], 0x5410), sB = __byte_perm(sr[2], sr[3], 0x5410);
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
            mma_bf16(one, a0, a1, a2, a3, pb[j][nb][0], pb[j][nb][1]);                                     \
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
#undef FA_KV4_PV_ROW
                            }
                        }
                    }
                }
            }
            __syncwarp();                        // every lane has read the stage
            c_stage = c_stage + 1 == C::kStages ? 0 : c_stage + 1;
            issue(u + C::kStages < u1, u + C::kStages + 1 < u1);
        }

        // -------------------------------------------- the segment's rows: combine the warps
        const int nr = x.nr;
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
        const int slot = (int)blockIdx.x * 2 + (u - n == u0 ? 0 : 1);
        const long long row0 = ((long long)x.b * p.H_kv + seg_h) * p.R + x.r0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (nb * 8 < nr) {
            if (nb > 0) __syncthreads();         // the exchange buffer is free again
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 2 * t + c;
                if (nb * 8 + r < nr) {
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, st_max[w * RB + nb * 8 + r]);
                    const float f = ref[nb][c] == -INFINITY ? 0.f : ex2_approx(ref[nb][c] - m);
                    float* dst = red + (warp * 8 + r) * C::kORow + g * (D / 8);
#pragma unroll
                    for (int vw = 0; vw < kVW; ++vw) {
                        *reinterpret_cast<float4*>(dst + vw * 8) =
                            make_float4(acc[nb][4 * vw][c] * f, acc[nb][4 * vw + 1][c] * f, acc[nb][4 * vw + 2][c] * f,
                                        acc[nb][4 * vw + 3][c] * f);
                        *reinterpret_cast<float4*>(dst + vw * 8 + 4) =
                            make_float4(acc[nb][4 * vw][c + 2] * f, acc[nb][4 * vw + 1][c + 2] * f,
                                        acc[nb][4 * vw + 2][c + 2] * f, acc[nb][4 * vw + 3][c + 2] * f);
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
                    const float4 y = *reinterpret_cast<const float4*>(red + (w * 8 + r) * C::kORow + 4 * c4);
                    a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
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
        }
        if (!whole) {
            // ---------------------------------------- partial: the last CTA of the item merges
            auto holder = [&](int v) {           // the CTA whose share has unit v
                const int big = more * (each + 1);
                return v < big ? v / (each + 1) : more + (v - big) / each;
            };
            const int cf = holder(item_first), cl = holder(item_first + x.units - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) misc[0] = arrive_last(word, cl - cf + 1) ? 1 : 0;
            __syncthreads();
            if (misc[0]) {
                __threadfence();
                // a CTA whose share starts inside the item has it first, else last: all but
                // the first CTA have it first
                const long long first = (long long)(2 * cf + (share(cf) >= item_first ? 0 : 1)) * RB;
                auto at = [&](int c) { return c == cf ? first : (long long)(2 * c) * RB; };
                // statistics of each row, a warp per row and a lane per CTA
                float* const fin = st_max;       // [RB] merged max, [RB] 1 / merged sum (the warps' own are used up)
                for (int rr = warp; rr < nr; rr += kWarps) {
                    float m = -INFINITY;
                    for (int c = cf + lane; c <= cl; c += 32) m = fmaxf(m, __ldcg(p.part_ml + (at(c) + rr) * 4));
#pragma unroll
                    for (int sh = 16; sh > 0; sh >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
                    float lr = 0.f, l = 0.f;
                    for (int c = cf + lane; c <= cl; c += 32) {
                        const float4 ml = __ldcg(reinterpret_cast<const float4*>(p.part_ml + (at(c) + rr) * 4));
                        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                        lr = fmaf(ml.y, f, lr);
                        l = fmaf(ml.z, f, l);
                    }
#pragma unroll
                    for (int sh = 16; sh > 0; sh >>= 1) {
                        lr += __shfl_xor_sync(0xffffffffu, lr, sh);
                        l += __shfl_xor_sync(0xffffffffu, l, sh);
                    }
                    if (lane == 0) {
                        fin[rr] = m;
                        fin[RB + rr] = l == 0.f ? 0.f : 1.f / lr;
                        p.lse[row0 + rr] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                    }
                }
                __syncthreads();
                // sums, 4 channels a thread; with few rows several threads share the CTAs of one
                const int items = nr * (D / 4);
                const int groups = items * 2 > kThreads ? 1 : kThreads / items;
                const bool in = groups == 1 || tid < items * groups;
                for (int it = in ? tid : items; it < items * groups; it += kThreads) {
                    const int gi = it / items, i = it - gi * items, rr = i / (D / 4), c4 = i % (D / 4);
                    const float m = fin[rr];
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = cf + gi; c <= cl; c += groups) {
                        const float mc = __ldcg(p.part_ml + (at(c) + rr) * 4);
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part + (at(c) + rr) * D) + c4);
                        const float f = mc == -INFINITY ? 0.f : ex2_approx(mc - m);
                        a.x = fmaf(y.x, f, a.x);
                        a.y = fmaf(y.y, f, a.y);
                        a.z = fmaf(y.z, f, a.z);
                        a.w = fmaf(y.w, f, a.w);
                    }
                    if (groups > 1) {
                        *reinterpret_cast<float4*>(red + it * 4) = a;
                    } else {
                        const float inv = fin[RB + rr];
                        uint2 pk;
                        pk.x = pack_bf16x2(a.x * inv, a.y * inv);
                        pk.y = pack_bf16x2(a.z * inv, a.w * inv);
                        *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + 4 * c4) = pk;
                    }
                }
                if (groups > 1) {
                    __syncthreads();
                    if (tid < items) {
                        const int rr = tid / (D / 4), c4 = tid % (D / 4);
                        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int gi = 0; gi < groups; ++gi) {
                            const float4 y = *reinterpret_cast<const float4*>(red + (gi * items + tid) * 4);
                            a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
                        }
                        const float inv = fin[RB + rr];
                        uint2 pk;
                        pk.x = pack_bf16x2(a.x * inv, a.y * inv);
                        pk.y = pack_bf16x2(a.z * inv, a.w * inv);
                        *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + 4 * c4) = pk;
                    }
                }
            }
        }
        __syncthreads();                         // statistics, exchange buffer and row limits are free again
        seg_k = 0;
        if (u < u1 && ++seg_h == p.H_kv) {
            seg_h = 0;
            x = entry_of<RB>(p, ++seg_e);
        }
    }
    cp_async_wait<0>();
}

}  // namespace kv4
}  // namespace fa
