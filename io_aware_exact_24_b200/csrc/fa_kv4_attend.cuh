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
// The cache streams through a per-warp ring of 32-key tiles filled with 16-byte cp.async
// copies (every wait is for the thread's own copies, so no barrier and nothing to time
// out).  The work of all sequences and heads is one line of 128-key units cut into equal
// shares, one per CTA: a long sequence is spread over many CTAs and many short ones share
// a CTA, whatever the lengths.  A (sequence, head, row block) that ends up in several CTAs
// is merged by the last of them to finish, from partial results in the workspace.
//
// What bounds it: a token and head is 144 bytes at d = 128, and at the rate at which memory
// delivers them an SM has to take in 44 codes a cycle.  Dequantising 8 of them is 12
// instructions of two issue cycles each, so the arithmetic, not the memory, is what a long
// cache waits for: 4 x 32 heads on 16384 keys of 128 channels take 75 us, 4.0 TB/s.  Of an
// earlier 74 the copies alone took 57 and the arithmetic alone 72; without the FMAs of the
// dequantisation it was 62, without all of it 48, without the MMAs 65.  Keeping 8, 12 or 16 warps
// to an SM (255, 168, 128 registers) made no difference.  A short call is a chain of latencies:
// lengths, page, codes, a tile (0.8 us alone), the exchange, the arrival and the merge, 8.4 us for
// 8 heads on 700 keys.
#pragma once

#include <type_traits>

#include "fa_kv4_kernel.cuh"

namespace fa {
namespace kv4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;                        // keys per warp and step: two MMA tiles
constexpr int kUnit = kTile * kWarps;            // keys per CTA and step
constexpr int kMaxEntries = 512;                 // (sequence, row block) pairs per launch
// Merging an item costs its last CTA 0.1 us for each part that a thread has to add, so where
// these can be more than kFlat, every kFan are merged by the last of theirs and then these sums
// (kGroups: 2 x 4 heads on 40000 keys, 222 parts, 48 -> 18.8 us; 8 x 4 on 8192, 55 parts, 17.4 ->
// 14.3).  Elsewhere it would cost 0.6 to 1.5 us a call.
constexpr int kFan = 16, kFlat = 36;
// Threads that share the parts of a row of an item of nr rows.
template <int D>
__host__ __device__ constexpr int row_groups(int nr) {
    return 2 * nr * (D / 4) > kThreads ? 1 : kThreads / (nr * (D / 4));
}

struct AttendParams {
    const __nv_bfloat16* q;    // [B, H_kv, R, D]
    const uint8_t* k_codes;
    const uint16_t* k_scales;
    const uint8_t* v_codes;
    const uint16_t* v_scales;
    __nv_bfloat16* o;
    float* lse;
    Paging pg;
    Rows rows;
    int H_kv;
    int row_blocks;            // per sequence and head
    int b0, rb0;               // sequence and row block of this launch's first entry
    int E;                     // entries of this launch, <= kMaxEntries
    float scale_log2;          // scale * log2(e)
    float* part;               // per CTA two partial results: [2][RB][D] sums and [2][RB][4] (max, sums)
    float* part_ml;
    unsigned long long* words; // arrival words [E, H_kv]
    unsigned long long* group_words;   // and one per partial result
    unsigned long long ticket; // not 0
};

template <int D, int NB>
struct Cfg {
    static constexpr int kRB = 8 * NB;                        // rows per block
    static constexpr int kCtasPerSm = NB == 1 ? 3 : 2;
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
    static constexpr int kQOff = kRedOff;                     // [NB][D/32][32] pairs of B fragments; in turn with the exchange
    static constexpr int kPreOff = kLimOff + 2 * kRB * 4;     // [E + 1] first unit of an entry
    static constexpr int kMiscOff = kPreOff + (kMaxEntries + 1) * 4;
    static constexpr int kSmemBytes = kMiscOff + 64;
    static_assert((kSmemBytes + 1024) * kCtasPerSm <= 233472, "shared memory of an SM");
};

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
// Plain loads, which the compiler may move between the barriers.
template <int W>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}
__device__ __forceinline__ uint32_t lds_u16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// Arrivals of a call's CTAs at an item.  The word holds (ticket << 16) | count, and 0 after
// a call.  At its segment's start a CTA tries to claim a 0 for this call's ticket; one that
// found something else there (not a call's word: what the workspace held at first) tries
// again from that value before it arrives, and whoever fails found the word claimed.  The
// last arrival clears it, so that a captured call, whose ticket is the same at each replay,
// starts anew.
__device__ __forceinline__ unsigned long long arrive_claim(unsigned long long* word, unsigned long long ticket) {
    return atomicCAS(word, 0ull, ticket << 16);
}
__device__ __forceinline__ bool arrive_last(unsigned long long* word, unsigned long long found, unsigned long long ticket,
                                            int n) {
    if (found != 0 && (found >> 16) != ticket) atomicCAS(word, found, ticket << 16);
    // releases this CTA's partial results (all its threads', after their barrier) and, for the
    // last one, acquires the others'
    unsigned long long old;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
    if ((int)(old & 0xffffull) + 1 != n) return false;
    atomicExch(word, 0ull);
    return true;
}

// Entry e of a launch: its sequence and row block.
template <int RB>
__device__ __forceinline__ Entry entry_of(const AttendParams& p, int e) {
    int g = p.rb0 + e, b = p.b0;
    if (p.row_blocks == 1) {
        b += g;
        g = 0;
    } else {
        const int n = g / p.row_blocks;
        b += n;
        g -= n * p.row_blocks;
    }
    return entry_of_rows<RB, kTile, kUnit>(p.rows, p.pg, b, g * RB);
}

template <int D, int NB, bool kOneRun, bool kGroups>
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

    after_previous();

    // ------------------------------------------------ the line of units
    Entry x;                         // of the current segment; first, of the thread's own entry
    const bool few = p.E <= 32;      // then every warp makes the line by itself, an entry per lane
    if (few) {
        x = entry_of<RB>(p, min(lane, p.E - 1));
        const int n = lane < p.E ? x.units * p.H_kv : 0;
        int inc = n;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, sh);
            if (lane >= sh) inc += y;
        }
        if (lane < p.E) pre[lane] = inc - n;     // (all warps the same)
        if (lane == 31) pre[p.E] = inc;
        __syncwarp();
    } else {
        constexpr int kPer = kMaxEntries / kThreads;
        const int per = (p.E + kThreads - 1) / kThreads;     // thread's entries: tid * per .. + per - 1
        int n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid * per + i;
            n[i] = i < per && e < p.E ? entry_of<RB>(p, e).units * p.H_kv : 0;
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
    if (few) {
        l_e = __popc(__ballot_sync(0xffffffffu, lane < p.E && pre[min(lane, p.E)] <= u0)) - 1;
        auto from = [&](int& v) { v = __shfl_sync(0xffffffffu, v, l_e); };
        from(x.b), from(x.r0), from(x.nr), from(x.kl), from(x.ql), from(x.lo), from(x.hi), from(x.all_lo), from(x.all_hi), from(x.units);
    } else {
        int a = 0, z = p.E;          // pre[a] <= u0 < pre[z]
        while (z - a > 1) {
            const int m = (a + z) >> 1;
            if (pre[m] <= u0) a = m; else z = m;
        }
        l_e = a;
        x = entry_of<RB>(p, l_e);
    }
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
    // A tile is kRuns runs of consecutive rows of the cache: one where page_size is a multiple
    // of 32, else two of 16 keys.  Each lane looks up the page of one of the warp's next 32
    // tiles of the item, a step before the first of them is copied.  A run that is not there
    // (past the last visible key, or no page) is not copied, and masked.
    constexpr int kRuns = kOneRun ? 1 : 2;
    int l_page[kRuns], l_off[kRuns];             // of the lane's tile; page -1: not there
    uint32_t l_row[kRuns];                       // and its first row in the cache
    int l_at = 0, l_u = u0;                      // the next tile's lane, and the unit of lane 0
    auto look_up = [&]() {
        l_u += l_at;
        l_at = 0;
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int pos = l_pos + lane * kUnit + 16 * i;
            l_page[i] = -1;
            if (pos < l_hi && l_u + lane < u1) {
                l_page[i] = page_of(p.pg, l_b, page_div(p.pg, pos, l_off[i]));
            }
        }
    };
    const uint32_t ring = (uint32_t)(warp * C::kStages * C::kStageBytes);
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
        src_s = reinterpret_cast<const uint8_t*>(lane < kSC ? p.k_scales : p.v_scales) + (kOneRun ? c : c % (kSC / 2)) * 16;
    }
    // the run of which this lane copies scales; none where there are fewer chunks than lanes
    const int s_run = lane >= 2 * (kTile * C::kSRow / 16) ? -1 : (kOneRun ? 0 : (lane % (kTile * C::kSRow / 16)) / (kTile * C::kSRow / 32));
    uint32_t loaded = 0;             // kRuns bits per tile, newest lowest: which runs are in the ring
    const uint32_t ring_end = ring + C::kStages * C::kStageBytes;
    auto issue = [&](uint32_t st) {              // copies the cursor's tile and moves on
        if (l_at == 0) {
#pragma unroll
            for (int i = 0; i < kRuns; ++i)
                l_row[i] = (uint32_t)l_page[i] < (uint32_t)p.pg.num_pages
                               ? ((uint32_t)l_page[i] * (uint32_t)p.H_kv + (uint32_t)l_h) * (uint32_t)p.pg.page_size + (uint32_t)l_off[i]
                               : 0xffffffffu;
        }
        uint32_t row[kRuns];
        bool there[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            row[i] = __shfl_sync(0xffffffffu, l_row[i], l_at);
            there[i] = row[i] != 0xffffffffu;    // the same for all lanes
            loaded = loaded * 2 + (there[i] ? 1u : 0u);
        }
#pragma unroll
        for (int i = 0; i < kRuns; ++i)
            if (there[i]) {
                const uint8_t* const k = src_k + (size_t)row[i] * C::kRow;
                const uint8_t* const v = src_v + (size_t)row[i] * C::kRow;
#pragma unroll
                for (int j = 0; j < 2 / kRuns * (C::kRow / 32); ++j) {   // 16 keys: kRow / 32 chunks a lane
                    cp_async16(base + st + dst_k + i * 16 * C::kRow + j * 512, k + j * 512);
                    cp_async16(base + st + dst_v + i * 16 * C::kRow + j * 512, v + j * 512);
                }
                if (s_run == i) cp_async16(base + st + dst_s, src_s + (size_t)row[i] * C::kSRow);
            }
        cp_async_commit();
        ++l_at;
        if (--l_left == 0) {                     // the next item: next head, or next entry
            l_left = 0x7fffffff;
            if (l_u + l_at < u1) {               // (behind the share nothing more is there)
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
            look_up();
        } else if (l_at == 32) {
            l_pos += 32 * kUnit;
            look_up();
        }
    };
    look_up();
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) issue(ring + s * C::kStageBytes);

    // ------------------------------------------------ state of the block's rows
    constexpr int kKW = D / 32;      // words of a key's codes per thread (a quarter of the row)
    constexpr int kVW = D / 64;      // words of a key's codes per thread (an eighth of the row)
    constexpr int kMT = 4 * kVW;     // 16-channel tiles of O^T
    float acc[NB][kMT][4];
    float sumr[NB][4];               // sums of the rounded probabilities (every lane's copy is whole)
    float2 sum[NB];                  // this lane's share of the sums, not rounded
    float ref[NB][2];                // reference max of rows 2t, 2t + 1 (log2 units), equal in all lanes of a t
    float top[NB][2];                // raw score above which the reference moves
    float2 neg[NB];                  // -ref - kShift, or 0 while the row has seen no key
    uint8_t* const qs = smem + C::kQOff + lane * 16;
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

    uint32_t st = ring;              // the stage of the tile to take next
    // A tile of 32 keys; kEdge: not every row of the block sees all of them.
    auto tile = [&](auto edge_tag, const int pos, const uint32_t have) {
        constexpr bool edge = decltype(edge_tag)::value;
        // which of its 16-key halves are in the ring, from the bits of its runs (the first run highest)
        auto half_there = [&](int j) { return kOneRun ? true : ((have >> (1 - j)) & 1u) != 0; };
        // ------------------------------------ scores of two 16-key tiles
        float s[2][NB][4];
        uint32_t w0[2][kKW], w1[2][kKW], s0[2], s1[2], z0[2], z1[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) s[j][nb][0] = s[j][nb][1] = s[j][nb][2] = s[j][nb][3] = 0.f;
            lds_words<kKW>(smem + st + at_k + j * 16 * C::kRow, w0[j]);
            lds_words<kKW>(smem + st + at_k + (j * 16 + 8) * C::kRow, w1[j]);
            s0[j] = lds_u16(smem + st + at_ks + j * 16 * C::kSRow);
            s1[j] = lds_u16(smem + st + at_ks + (j * 16 + 8) * C::kSRow);
            s0[j] = __byte_perm(s0[j], s0[j], 0x1010);
            s1[j] = __byte_perm(s1[j], s1[j], 0x1010);
            z0[j] = minus_24(s0[j]);
            z1[j] = minus_24(s1[j]);
        }
#pragma unroll
        for (int w = 0; w < kKW; ++w) {
            uint32_t b[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) lds_words<4>(qs + (nb * kKW + w) * 512, b[nb]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a0 = codes_to_bf16x2(0, w0[j][w], s0[j], z0[j]), a1 = codes_to_bf16x2(0, w1[j][w], s1[j], z1[j]);
                const uint32_t a2 = codes_to_bf16x2(1, w0[j][w], s0[j], z0[j]), a3 = codes_to_bf16x2(1, w1[j][w], s1[j], z1[j]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_bf16(s[j][nb], a0, a1, a2, a3, b[nb][0], b[nb][1]);
                const uint32_t c0 = codes_to_bf16x2(2, w0[j][w], s0[j], z0[j]), c1 = codes_to_bf16x2(2, w1[j][w], s1[j], z1[j]);
                const uint32_t c2 = codes_to_bf16x2(3, w0[j][w], s0[j], z0[j]), c3 = codes_to_bf16x2(3, w1[j][w], s1[j], z1[j]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_bf16(s[j][nb], c0, c1, c2, c3, b[nb][2], b[nb][3]);
            }
        }
        // ------------------------------------ mask, reference max, probabilities
        if (edge) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int r = nb * 8 + 2 * t + (c & 1), key = pos + 16 * j + key0 + (c >> 1) * 8;
                        if (key < row_lo[r] || key >= row_hi[r] || !half_there(j)) s[j][nb][c] = -INFINITY;
                    }
        }
        // the reference moves only when some score exceeds it by more than 2^8: until
        // then weights stay below 2^8 times the largest and nothing needs to be rescaled
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
                        m = reference(m);
                        const float f = ex2_approx(ref[nb][c] - m);   // 0 from a reference of -inf
                        ref[nb][c] = m;
                        (c == 0 ? neg[nb].x : neg[nb].y) = -(m + kShift);
                        top[nb][c] = (m + 8.f) * inv_scale;
                        (c == 0 ? sum[nb].x : sum[nb].y) *= f;
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
                const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
                float2 e0 = __ffma2_rn(make_float2(s[j][nb][0], s[j][nb][1]), scale2, neg[nb]);
                float2 e1 = __ffma2_rn(make_float2(s[j][nb][2], s[j][nb][3]), scale2, neg[nb]);
                e0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
                e1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
                sum[nb] = __fadd2_rn(sum[nb], __fadd2_rn(e0, e1));
                // P rounds to bf16 (2^-8) for the tensor cores; O is divided by the sum of
                // the rounded values, so a row that one key dominates stays exact
                pb[j][nb][0] = transpose8x8(pack_bf16x2(e0.x, e0.y));
                pb[j][nb][1] = transpose8x8(pack_bf16x2(e1.x, e1.y));
                mma_bf16(sumr[nb], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, pb[j][nb][0], pb[j][nb][1]);
            }
        // ------------------------------------ O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w[4][kVW], sv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lds_words<kVW>(smem + st + at_v + (j * 16 + 4 * i) * C::kRow, w[i]);
                sv[i] = lds_u16(smem + st + at_vs + (j * 16 + 4 * i) * C::kSRow);
            }
            bool poisoned = false;
            if (edge) {
                // what lies behind the last key, or was not loaded, counts as zero; a NaN
                // group of another key meets zero weights in the rows that do not see
                // it: the tile is then taken row by row, with the hidden keys' scales zero
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (pos + 16 * j + t + 4 * i >= x.kl || !half_there(j)) sv[i] = 0;
                    bad |= no_scale(sv[i]);
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
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = codes_to_bf16x2(i, la, sA, zA), a1 = codes_to_bf16x2(i, ha, sA, zA);
                        const uint32_t a2 = codes_to_bf16x2(i, lb, sB, zB), a3 = codes_to_bf16x2(i, hb, sB, zB);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_bf16(acc[nb][4 * vw + i], a0, a1, a2, a3, pb[j][nb][0], pb[j][nb][1]);
                    }
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
#pragma unroll
                    for (int vw = 0; vw < kVW; ++vw) {
                        const uint32_t la = __byte_perm(w[0][vw], w[1][vw], 0x5410);
                        const uint32_t ha = __byte_perm(w[0][vw], w[1][vw], 0x7632);
                        const uint32_t lb = __byte_perm(w[2][vw], w[3][vw], 0x5410);
                        const uint32_t hb = __byte_perm(w[2][vw], w[3][vw], 0x7632);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a0 = codes_to_bf16x2(i, la, sA, zA), a1 = codes_to_bf16x2(i, ha, sA, zA);
                            const uint32_t a2 = codes_to_bf16x2(i, lb, sB, zB), a3 = codes_to_bf16x2(i, hb, sB, zB);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float one[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_bf16(one, a0, a1, a2, a3, pb[j][nb][0], pb[j][nb][1]);
                                // (selected, not indexed by r: acc stays in registers)
                                const bool m0 = r == nb * 8 + 2 * t, m1 = r == nb * 8 + 2 * t + 1;
                                acc[nb][4 * vw + i][0] += m0 ? one[0] : 0.f;
                                acc[nb][4 * vw + i][1] += m1 ? one[1] : 0.f;
                                acc[nb][4 * vw + i][2] += m0 ? one[2] : 0.f;
                                acc[nb][4 * vw + i][3] += m1 ? one[3] : 0.f;
                            }
                        }
                    }
                }
            }
        }
    };

    // The CTAs [cf, cl] that share an item, and this one's group of them [gf, ge].
    struct Sharers {
        int cf, cl, gf, ge, first_slot;
        bool grouped;
        // a CTA whose share starts inside the item has it first, else last: all but cf have it first
        __device__ __forceinline__ int slot_of(int c) const { return c == cf ? first_slot : 2 * c; }
    };
    auto sharers = [&](int first, int units, int nr) {
        int ea = each;
        asm volatile("" : "+r"(ea));             // (worked out twice, not kept over the tiles)
        auto holder = [&](int v) {               // the CTA whose share has unit v
            const int big = more * (ea + 1);
            return v < big ? v / (ea + 1) : more + (v - big) / ea;
        };
        Sharers s;
        s.cf = holder(first);
        s.cl = holder(first + units - 1);
        s.gf = s.cf + ((int)blockIdx.x - s.cf) / kFan * kFan;
        s.ge = min(s.gf + kFan - 1, s.cl);
        s.first_slot = 2 * s.cf + (ea * s.cf + min(s.cf, more) >= first ? 0 : 1);
        s.grouped = kGroups && s.cl - s.cf >= kFlat * row_groups<D>(nr);
        return s;
    };
    for (int u = u0; u < u1;) {
        // ============================================ a segment: units seg_k .. of an item
        const int n = min(x.units - seg_k, u1 - u);
        const int item_first = pre[seg_e] + seg_h * x.units;
        const bool whole = seg_k == 0 && n == x.units;
        unsigned long long* const word = p.words + (long long)seg_e * p.H_kv + seg_h;
        unsigned long long found = 0, gfound = 0;
        if (!whole && tid == 0) found = arrive_claim(word, p.ticket);
        {
            // Q as B fragments, two k-steps of the MMA to 16 bytes, shared by the warps
            const __nv_bfloat16* q = p.q + (((long long)x.b * p.H_kv + seg_h) * p.rows.R + x.r0) * D;
            for (int i = warp; i < NB * kKW; i += kWarps) {
                const int r = i / kKW * 8 + g, w = i % kKW;
                const uint4 y = r < x.nr ? __ldcg(reinterpret_cast<const uint4*>(q + (long long)r * D + t * (D / 4)) + w)
                                         : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(qs + i * 512) =
                    make_uint4(__byte_perm(y.x, y.z, 0x5410), __byte_perm(y.x, y.z, 0x7632), __byte_perm(y.y, y.w, 0x5410),
                               __byte_perm(y.y, y.w, 0x7632));
            }
        }
        if (tid < RB) {
            int lo, hi;
            row_keys(p.rows, x.kl, x.ql, x.r0 + tid, lo, hi);
            row_lo[tid] = lo;
            row_hi[tid] = hi;
        }
        __syncthreads();
        if (kGroups && !whole && tid == 0) {
            const Sharers sh = sharers(item_first, x.units, x.nr);
            if (sh.grouped) gfound = arrive_claim(p.group_words + sh.slot_of(sh.gf), p.ticket);
        }
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
                ref[nb][c] = top[nb][c] = -INFINITY;
            }
            sum[nb] = neg[nb] = make_float2(0.f, 0.f);
        }
        int pos = x.lo + seg_k * kUnit + warp * kTile;
        const int full_hi = x.all_hi - kTile;
        for (int k = 0; k < n; ++k, ++u, pos += kUnit) {
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t have = (loaded >> (kRuns * (C::kStages - 1))) & ((1u << kRuns) - 1u);
            if (pos >= x.all_lo && pos <= full_hi && have == (1u << kRuns) - 1u)
                tile(std::false_type{}, pos, have);
            else if (have != 0)
                tile(std::true_type{}, pos, have);
            __syncwarp();                        // every lane has read the stage
            issue(st);
            st += C::kStageBytes;
            if (st == ring_end) st = ring;
        }

        // -------------------------------------------- the segment's rows: combine the warps
        const int nr = x.nr;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = c == 0 ? sum[nb].x : sum[nb].y;
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
        const long long row0 = ((long long)x.b * p.H_kv + seg_h) * p.rows.R + x.r0;
        auto combine = [&](auto block) {         // eight rows; a lambda, so that acc is indexed by constants
            constexpr int nb = decltype(block)::value;
            if (nb * 8 >= nr) return;
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
                    if (c4 == 0) p.lse[row0 + rr] = lse_of(m, l);
                } else {
                    *reinterpret_cast<float4*>(p.part + ((long long)slot * RB + rr) * D + 4 * c4) = a;
                    if (c4 == 0)
                        *reinterpret_cast<float4*>(p.part_ml + ((long long)slot * RB + rr) * 4) = make_float4(m, lr, l, 0.f);
                }
            }
        };
        combine(std::integral_constant<int, 0>{});
        if constexpr (NB > 1) combine(std::integral_constant<int, 1>{});
        if (!whole) {
            // ---------------------------------------- partial: the last CTA of the item merges
            const Sharers sh = sharers(item_first, x.units, nr);
            for (bool last_level = !kGroups || !sh.grouped;; last_level = true) {
                __syncthreads();
                // parts 0 .. c1: the CTAs from base on, or every kFan-th
                const int apart = kGroups && last_level && sh.grouped ? kFan : 1;
                const int base = last_level ? sh.cf : sh.gf, c1 = ((last_level ? sh.cl : sh.ge) - base) / apart;
                if (tid == 0)
                    misc[0] = arrive_last(last_level ? word : p.group_words + sh.slot_of(base), last_level ? found : gfound,
                                          p.ticket, c1 + 1);
                __syncthreads();
                if (!misc[0]) break;
                auto at = [&](int c) { return (long long)sh.slot_of(base + c * apart) * RB; };
                // sums, 4 channels a thread: of up to kEach rows, or, with few rows, of some of the
                // CTAs of one row.  kAhead * kEach loads at a time, the first of them on their way
                // while the rows' statistics are made.
                const int items = nr * (D / 4);
                const int groups = row_groups<D>(nr);
                constexpr int kEach = RB * (D / 4) / kThreads, kAhead = 4;
                static_assert(kEach * kThreads == RB * (D / 4), "rows of a block");
                float mc[kAhead][kEach];
                float4 y[kAhead][kEach];
                const bool one = groups == 1;    // one thread has all CTAs of a row
                const int gi = one ? 0 : tid / items, step = one ? kAhead : kAhead * kEach * groups;
                const int it0 = tid - gi * items, c40 = tid % (D / 4);
                auto row_of = [&](int e) { return one ? (it0 + e * kThreads) / (D / 4) : it0 / (D / 4); };
                auto fetch = [&](int c0) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            // (without branches, so that the loads go out together)
                            const int c = one ? c0 + i : c0 + (i * kEach + e) * groups;
                            const long long r = at(min(c, c1)) + min(row_of(e), nr - 1);
                            mc[i][e] = __ldcg(p.part_ml + r * 4);
                            y[i][e] = __ldcg(reinterpret_cast<const float4*>(p.part + r * D) + c40);
                            if (c > c1) mc[i][e] = -INFINITY;
                        }
                };
                float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);       // the warp's first row, a CTA per lane
                if (warp < nr && lane <= c1) ml = __ldcg(reinterpret_cast<const float4*>(p.part_ml + (at(lane) + warp) * 4));
                fetch(gi);
                // statistics of each row: a warp per row, a lane per CTA
                float* const fin = st_max;       // [RB] merged max, then 1 / merged sum, or both sums (the warps' own are used up)
                for (int rr = warp; rr < nr; rr += kWarps) {
                    float m = -INFINITY, lr = 0.f, l = 0.f;
                    for (int c = lane; c <= c1; c += 32) {
                        if (rr != warp || c != lane) ml = __ldcg(reinterpret_cast<const float4*>(p.part_ml + (at(c) + rr) * 4));
                        const float n = fmaxf(m, ml.x);
                        const float f = m == -INFINITY ? 0.f : ex2_approx(m - n);
                        const float h = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - n);
                        lr = fmaf(lr, f, ml.y * h);
                        l = fmaf(l, f, ml.z * h);
                        m = n;
                    }
                    float n = m;
#pragma unroll
                    for (int sh = 16; sh > 0; sh >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, sh));
                    const float f = m == -INFINITY ? 0.f : ex2_approx(m - n);
                    lr *= f;
                    l *= f;
#pragma unroll
                    for (int sh = 16; sh > 0; sh >>= 1) {
                        lr += __shfl_xor_sync(0xffffffffu, lr, sh);
                        l += __shfl_xor_sync(0xffffffffu, l, sh);
                    }
                    if (lane == 0) {
                        fin[rr] = n;
                        if (last_level) {
                            fin[RB + rr] = l == 0.f ? 0.f : 1.f / lr;
                            p.lse[row0 + rr] = lse_of(n, l);
                        } else {
                            fin[RB + rr] = lr;
                            fin[2 * RB + rr] = l;
                        }
                    }
                }
                __syncthreads();
                if (!last_level && tid < nr)     // into the first part's place, which all have read
                    *reinterpret_cast<float4*>(p.part_ml + (at(0) + tid) * 4) = make_float4(fin[tid], fin[RB + tid], fin[2 * RB + tid], 0.f);
                auto put = [&](int rr, int c4, const float4& a) {
                    if (!last_level) {
                        *reinterpret_cast<float4*>(p.part + (at(0) + rr) * D + 4 * c4) = a;
                        return;
                    }
                    const float inv = fin[RB + rr];
                    uint2 pk;
                    pk.x = pack_bf16x2(a.x * inv, a.y * inv);
                    pk.y = pack_bf16x2(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + 4 * c4) = pk;
                };
                float4 a[kEach];
#pragma unroll
                for (int e = 0; e < kEach; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = gi; c <= c1;) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const float m = fin[min(row_of(e), RB - 1)];
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const float f = mc[i][e] == -INFINITY ? 0.f : ex2_approx(mc[i][e] - m);
                            a[e].x = fmaf(y[i][e].x, f, a[e].x);
                            a[e].y = fmaf(y[i][e].y, f, a[e].y);
                            a[e].z = fmaf(y[i][e].z, f, a[e].z);
                            a[e].w = fmaf(y[i][e].w, f, a[e].w);
                        }
                    }
                    c += step;
                    if (c <= c1) fetch(c);
                }
                if (!one) {
#pragma unroll
                    for (int e = 1; e < kEach; ++e)
                        a[0].x += a[e].x, a[0].y += a[e].y, a[0].z += a[e].z, a[0].w += a[e].w;
                }
                if (one) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (it0 + e * kThreads < items) put(row_of(e), c40, a[e]);
                } else {
                    if (gi < groups) *reinterpret_cast<float4*>(red + tid * 4) = a[0];
                    __syncthreads();
                    if (tid < items) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int i = 0; i < groups; ++i) {
                            const float4 w = *reinterpret_cast<const float4*>(red + (i * items + tid) * 4);
                            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                        }
                        put(row_of(0), c40, v);
                    }
                }
                if (last_level) break;
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
