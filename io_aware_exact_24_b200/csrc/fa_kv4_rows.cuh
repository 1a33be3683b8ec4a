// fa_kv4_rows.cuh -- attention over the 4-bit paged cache for many query rows per key/value
// head (pieces of prompts), on the tcgen05 tensor cores.
//
// The rows of a key/value head (fa_kv4_kernel.cuh: Rows) come in blocks of 128, one CTA each.
// The kernel is the forward of fa_fwd_kernel.cuh (S = Q K^T and O += P V in TMEM, two softmax
// warps per lane quadrant, the reference max that moves by 2^8) with another source of K and
// V: four warps copy the codes of a 128-key tile to shared memory, one tile ahead, turn them
// into bf16 and store them to the swizzled tiles that the MMAs read.  The values are exact
// (fa_kv4_kernel.cuh), so the tensor cores multiply what a read-back cache would hold, and no
// bf16 copy of the cache passes through memory.
//
// The codes of a 32-bit word come out as channels (0,4) (1,5) (2,6) (3,7).  K is stored in
// that order, Q goes to TMEM in it, and of O, whose columns follow V's, the epilogue picks the
// columns back.
//
// Where the blocks are few, CTAs share one's keys in ranges and leave unnormalised sums in the
// workspace; join_kernel, a launch behind, adds them up.  It has a block for every 32 rows and 8
// channels, where the last CTA of a block of rows, alone, would take 0.1 us or more for each range.
//
// A NaN group of V would reach the rows that do not see its key as 0 * NaN: it is stored as
// zeros and noted in a mask per tile, and the softmax threads, which know what their row sees,
// make the group's channels NaN at the end.
//
// What bounds it: 2 x 32 heads (8 of keys), 512 queries, 8000 keys take 174 us, 746 TFLOP/s (137
// us at d = 64); the products alone are 78 us at the rate of a large one.  256 blocks are 1.73
// waves, so the SMs are idle for 14 % of it.  Else no unit is full (tensor pipe 43 % of the cycles, ALU 44,
// exponentials 42, issue 54): a tile takes a CTA 1.25 us, in which the makers turn 32768 codes
// into 64 KB of operands, the eight softmax warps take 128 x 128 scores, and each waits for the
// other, since shared memory and TMEM hold two tiles.  A short call is launch, setup, tiles,
// epilogue and join: 8 x 128 rows on 700 keys, 13.2 us.
#pragma once

#include <type_traits>

#include "fa_fwd_kernel.cuh"
#include "fa_kv4_kernel.cuh"

namespace fa {
namespace kv4 {

constexpr int kRowsThreads = 512;          // 8 softmax warps, 4 control warps, 4 that make K and V tiles
constexpr int kMakerWarp = 12;
constexpr int kMakers = 4;
// Registers per thread: 512 x 128 at launch; 2 x 128 x 184 + 128 x 48 + 128 x 96 are as many.
constexpr uint32_t kRegsRowsSoftmax = 184;
constexpr uint32_t kRegsRowsControl = 48;
constexpr uint32_t kRegsRowsMaker = 96;
// Tiles whose notes are kept.  A maker writes tile j's when the scores of tile j - stages are
// done, so the softmax warps have taken those of j - stages - 1 and j - stages - 2 out, one
// each, and are through with all tiles before.
constexpr int kNotes = 8;
static_assert(kNotes >= fa::Cfg<64>::kStagesK + 3 && kNotes >= fa::Cfg<128>::kStagesK + 3, "notes still to be read");

template <int D>
struct RowsCfg {
    using F = fa::Cfg<D>;
    // TMEM: the scores, two P buffers, O with its row sums (and 16 unused columns that the
    // rescale touches), and Q: as the A operand it would be read from shared memory once per
    // tile, whose bandwidth the tiles' making takes
    static constexpr int kPBufs = 2;
    __host__ __device__ static constexpr uint32_t col_p(int b) { return 128u + 64u * b; }
    static constexpr uint32_t kColO = 128u + 64u * kPBufs, kColL = kColO + D, kColQ = kColL + 32;
    static_assert(kColQ + D / 2 <= 512, "TMEM columns");
    // barriers: q_full, q_ready, then per ring full and empty, s_full[2], s_free, p_full, pv_done, drain
    static constexpr int kNumBars = 2 + 2 * F::kStages + 2 + 1 + 2 * kPBufs + 1;
    static constexpr int kBarOff = F::kBarOff;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;   // tmem base, abort flag
    static constexpr int kMrefOff = kMiscOff + 16;
    static constexpr int kEpiOff = kMrefOff + kGroups * kBlockM * 8;           // m, sum, NaN groups [2][row] each
    // notes of a tile: a word per maker warp (bits 0-1: its runs that are not there, bit 2: NaN
    // groups), then its 32 keys' NaN bits per group
    static constexpr int kNoteBytes = kMakers * 4 * (1 + D / kGroup);
    static constexpr int kNoteOff = kEpiOff + 3 * kGroups * kBlockM * 4;
    // staging of a maker warp: 16 bytes of K's codes and of V's per pass and lane, then its 32
    // keys' scales of K and of V
    static constexpr int kPass = D / kGroup;
    static constexpr int kStageOff = (kNoteOff + kNotes * kNoteBytes + 15) / 16 * 16;
    static constexpr int kStageV = kPass * 32 * 16;
    static constexpr int kStageS = 2 * kStageV;
    static constexpr int kStageWarp = kStageS + 2 * 32 * (D / kGroup) * 2;
    static constexpr int kSmemBytes = kStageOff + kMakers * kStageWarp + 1024;
    static_assert(kSmemBytes <= 232448 && kSmemBytes > 116 * 1024, "one CTA per SM");
};

// The pairs (0,1) (2,3) (4,5) (6,7) of 8 channels as (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ uint4 code_order(uint4 x) {
    return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                      __byte_perm(x.y, x.w, 0x7632));
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
template <int D, bool kOneRun>
__global__ void __launch_bounds__(kRowsThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o, const RowsParams p) {
    using F = fa::Cfg<D>;
    using C = RowsCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* const base_ptr = smem_raw + (base - raw_base);

    auto bar = [&](int i) { return base + C::kBarOff + 8u * (uint32_t)i; };
    const uint32_t bar_q_full = bar(0), bar_q_ready = bar(1);
    auto bar_full = [&](int r, int s) { return bar(2 + r * F::kStagesK + s); };
    auto bar_empty = [&](int r, int s) { return bar(2 + F::kStages + r * F::kStagesK + s); };
    auto bar_s_full = [&](int g) { return bar(2 + 2 * F::kStages + g); };
    const uint32_t bar_s_free = bar(4 + 2 * F::kStages);
    auto bar_p_full = [&](int b) { return bar(5 + 2 * F::kStages + b); };
    auto bar_pv_done = [&](int b) { return bar(5 + C::kPBufs + 2 * F::kStages + b); };
    const uint32_t bar_drain = bar(5 + 2 * C::kPBufs + 2 * F::kStages);
    volatile uint32_t* const part_at = reinterpret_cast<volatile uint32_t*>(base_ptr + C::kMiscOff + 8);
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + C::kMiscOff);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 4);
    const uint32_t mref_w = base + C::kMrefOff;
    float* const epi = reinterpret_cast<float*>(base_ptr + C::kEpiOff);
    const uint32_t q_tile = base + F::kQOff;
    auto ring_slot = [&](int r, int s) {
        return r == 0 ? base + F::kKOff + (uint32_t)(s * F::kTileBytes) : base + F::kVOff + (uint32_t)(s * F::kVSlotBytes);
    };
    auto note = [&](int j) { return reinterpret_cast<volatile uint32_t*>(base_ptr + C::kNoteOff + (j % kNotes) * C::kNoteBytes); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows that see more keys (causal: the later ones of a head) start first
    int back = (int)blockIdx.x, split = 0;
    if (p.splits > 1) {          // CTAs are few then: x * ceil(2^16 / splits) >> 16 is exact
        back = (int)((blockIdx.x * (uint32_t)p.split_inv) >> 16);
        split = (int)blockIdx.x - back * p.splits;
    }
    const int m0 = (p.row_blocks - 1 - back) * kBlockM;
    const int h = blockIdx.y, b = blockIdx.z;

    // ---- setup
    if (warp == kProducerWarp && lane == 0) {
        mbar_init(bar_q_full, 1);
        mbar_init(bar_q_ready, D / 16);          // one warp per lane quadrant and 32 columns
        for (int r = 0; r < 2; ++r)
            for (int s = 0; s < (r == 0 ? F::kStagesK : F::kStagesV); ++s) {
                mbar_init(bar_full(r, s), kMakers);
                mbar_init(bar_empty(r, s), 1);
            }
        mbar_init(bar_s_full(0), 1);
        mbar_init(bar_s_full(1), 1);
        mbar_init(bar_s_free, 4);
        for (int i = 0; i < C::kPBufs; ++i) {
            mbar_init(bar_p_full(i), 4);
            mbar_init(bar_pv_done(i), 1);
        }
        mbar_init(bar_drain, 2);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_o);
    }
    for (int i = threadIdx.x; i < kGroups * kBlockM; i += kRowsThreads) st_relaxed_shared_u64(mref_w + 8u * (uint32_t)i, ~0ull);
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(tmem_holder), kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    // the ones box of every V slot: the PV product's last columns sum the rounded P
    for (int i = threadIdx.x; i < F::kStagesV * (F::kBoxBytes / 16); i += kRowsThreads) {
        const uint32_t a = ring_slot(1, i / (F::kBoxBytes / 16)) + (uint32_t)F::kTileBytes + (uint32_t)(i % (F::kBoxBytes / 16)) * 16u;
        sts16(a, F::kOnesWord, F::kOnesWord, F::kOnesWord, F::kOnesWord);
    }
    fence_proxy_async_smem();
    after_previous();
    Entry x = entry_of_rows<kBlockM, 32, kBlockN>(p.rows, p.pg, b, m0);
    int n_kv = x.hi > x.lo ? x.units : 0;
    if (p.splits > 1) {
        const int t0 = (int)((uint32_t)n_kv * (uint32_t)split / (uint32_t)p.splits);
        n_kv = (int)((uint32_t)n_kv * (uint32_t)(split + 1) / (uint32_t)p.splits) - t0;
        x.lo += t0 * kBlockN;
    }
    if (threadIdx.x == 0) {      // (kept here: registers are short)
        part_at[0] = ((uint32_t)(b * p.H_kv + h) * (uint32_t)p.row_blocks + (uint32_t)(m0 / kBlockM)) * (uint32_t)p.splits + (uint32_t)split;
        part_at[1] = (uint32_t)m0;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp >= kMakerWarp) {
        setmaxnreg_dec<kRegsRowsMaker>();
        // =========================================================== K and V tiles
        // Warp w makes keys 32w .. 32w + 31 of each tile.  A lane takes one group of 32 channels
        // (a scale, 16 bytes of codes) of a key: 8 (d = 128) or 16 keys of the same group lie in
        // neighbouring lanes, which store to different banks.
        // The codes come through shared memory by cp.async, one tile ahead, each lane its own
        // bytes: a load to a register would have to land at every proxy fence.
        constexpr int kG = D / kGroup, kKeys = 32 / kG, kPass = C::kPass;
        static_assert(kPass * kKeys == 32, "a warp's keys");
        constexpr int kRuns = kOneRun ? 1 : 2;
        const int w = warp - kMakerWarp;
        const int key_l = lane % kKeys, grp = lane / kKeys;
        const uint32_t stage = base + (uint32_t)(C::kStageOff + w * C::kStageWarp);
        bool ok = true;
        // first rows of the warp's runs of tiles j0 .. j0 + 31, a tile per lane (~0: not there)
        uint32_t l_row[kRuns], row[kRuns];
        auto rows_of = [&](int j) {
            if ((j & 31) == 0) {
#pragma unroll
                for (int i = 0; i < kRuns; ++i) {
                    const int pos = x.lo + (j + lane) * kBlockN + w * 32 + 16 * i;
                    l_row[i] = 0xffffffffu;
                    if (pos < x.kl) {
                        int off;
                        const int page = page_of(p.pg, b, page_div(p.pg, pos, off));
                        if (page >= 0)
                            l_row[i] = ((uint32_t)page * (uint32_t)p.H_kv + (uint32_t)h) * (uint32_t)p.pg.page_size + (uint32_t)off;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kRuns; ++i) row[i] = __shfl_sync(0xffffffffu, l_row[i], j & 31);
        };
        // where this lane's chunks lie behind a run's first row
        constexpr int kRow = D / 2, kSRow = kG * 2, kRunPass = kPass / kRuns;
        const uint8_t* const src_k = p.k_codes + key_l * kRow + grp * 16;
        const uint8_t* const src_v = p.v_codes + key_l * kRow + grp * 16;
        constexpr int kSC = 32 * kSRow / 16;         // 16-byte chunks of the warp's scales, per tensor: 16 or 8
        const int s_chunk = lane % kSC, s_run = s_chunk / (kSC / kRuns);
        const uint8_t* const src_s = reinterpret_cast<const uint8_t*>(lane < kSC ? p.k_scales : p.v_scales) + s_chunk % (kSC / kRuns) * 16;
        auto copy_k = [&]() {            // K and both scales of the rows just looked up
            uint32_t s_row = row[0];
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                if (i == s_run) s_row = row[i];
                if (row[i] != 0xffffffffu) {
                    const uint8_t* const src = src_k + (size_t)row[i] * kRow;
#pragma unroll
                    for (int o = 0; o < kRunPass; ++o)
                        cp_async16(stage + (uint32_t)(((i * kRunPass + o) * 32 + lane) * 16), src + o * kKeys * kRow);
                }
            }
            if (s_row != 0xffffffffu && lane < 2 * kSC)
                cp_async16(stage + (uint32_t)(C::kStageS + lane * 16), src_s + (size_t)s_row * kSRow);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto copy_v = [&](const uint32_t (&vr)[kRuns]) {
#pragma unroll
            for (int i = 0; i < kRuns; ++i)
                if (vr[i] != 0xffffffffu) {
                    const uint8_t* const src = src_v + (size_t)vr[i] * kRow;
#pragma unroll
                    for (int o = 0; o < kRunPass; ++o)
                        cp_async16(stage + (uint32_t)(C::kStageV + ((i * kRunPass + o) * 32 + lane) * 16), src + o * kKeys * kRow);
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto lds2 = [](uint32_t a) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
            return (uint32_t)v;
        };
        const uint32_t at_s = stage + (uint32_t)(C::kStageS + key_l * kSRow + grp * 2);
        auto store = [&](auto is_k, uint32_t slot, int o, const uint4& c, uint32_t s) {
            // (V's scales that stand for NaN have been made zeros)
            const uint32_t s2 = __byte_perm(s, s, 0x1010), z2 = decltype(is_k)::value ? minus_24(s2) : minus_24_of_a_number(s2);
            const int key = w * 32 + o * kKeys + key_l;
            const uint32_t at = slot + (uint32_t)((grp >> 1) * F::kBoxBytes + key * 128);
            const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sts16(at + (uint32_t)(((((grp & 1) << 2) + i) ^ (key & 7)) << 4), codes_to_bf16x2(0, word[i], s2, z2),
                      codes_to_bf16x2(1, word[i], s2, z2), codes_to_bf16x2(2, word[i], s2, z2), codes_to_bf16x2(3, word[i], s2, z2));
        };
        // K tiles are made one ahead of V tiles: a V slot is free only when the tile two before has
        // been through the softmax, and the next scores should not wait for that.
        uint32_t v_row[kRuns];           // of the V tile to make next
        uint32_t v_sc[kPass];            // and its scales
        auto make_k = [&](int j) {       // makes K of the tile whose copies are complete, and starts the next one's
            const int sl = j % F::kStagesK;
            uint32_t gone = 0;           // runs that are not there
            uint4 cw[kPass];
            uint32_t sc[kPass];
            bool bad = false;
            const int left = x.kl - (x.lo + j * kBlockN + w * 32 + key_l);   // keys of the sequence from the lane's first on
            __syncwarp();                // the scales are other lanes' copies
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                v_row[i] = row[i];
                if (row[i] == 0xffffffffu) gone |= kOneRun ? 3u : 1u << i;
            }
            // a run that is not there gives whatever is in the staging: its scores are masked, and
            // its V, as that of rows behind the last key, which may hold anything, counts as zero
#pragma unroll
            for (int o = 0; o < kPass; ++o) {
                cw[o] = lds16(stage + (uint32_t)((o * 32 + lane) * 16));
                sc[o] = lds2(at_s + o * kKeys * kSRow);
                v_sc[o] = lds2(at_s + 32 * kSRow + o * kKeys * kSRow);
                if (o * kKeys >= left || row[o / kRunPass] == 0xffffffffu) v_sc[o] = 0;
                bad |= no_scale(v_sc[o]);
            }
            __syncwarp();
            if (j + 1 < n_kv) rows_of(j + 1);
            else
#pragma unroll
                for (int i = 0; i < kRuns; ++i) row[i] = 0xffffffffu;
            copy_k();
            if (!__all_sync(0xffffffffu, wait_bounded(bar_empty(0, sl), ((uint32_t)(j / F::kStagesK) & 1u) ^ 1u, abort_flag, p.wait_limit)))
                return false;
            // notes first: whoever sees this tile's scores sees them too
            const bool any_bad = __any_sync(0xffffffffu, bad);
            if (any_bad) {
                uint32_t word = 0;           // lane g's: the 32 keys' bits of group g
#pragma unroll
                for (int o = 0; o < kPass; ++o) {
                    const bool is = no_scale(v_sc[o]);
                    const uint32_t bal = __ballot_sync(0xffffffffu, is);
                    if (lane < kG) word |= ((bal >> (lane * kKeys)) & ((1u << kKeys) - 1u)) << (o * kKeys);
                    if (is) v_sc[o] = 0;
                }
                if (lane < kG) note(j)[kMakers + w * kG + lane] = word;
            }
            if (lane == 0) note(j)[w] = gone | (any_bad ? 4u : 0u);
#pragma unroll
            for (int o = 0; o < kPass; ++o) store(std::true_type{}, ring_slot(0, sl), o, cw[o], sc[o]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full(0, sl));
            return true;
        };
        if (n_kv > 0) {
            rows_of(0);
            copy_k();
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            ok = make_k(0);
            copy_v(v_row);
        }
        for (int j = 0; j < n_kv && ok; ++j) {
            const int sl = j % F::kStagesV;
            uint4 cw[kPass];
            uint32_t sc[kPass];
#pragma unroll
            for (int o = 0; o < kPass; ++o) sc[o] = v_sc[o];
            asm volatile("cp.async.wait_group 1;" ::: "memory");     // K of tile j + 1
            if (j + 1 < n_kv)
                ok = make_k(j + 1);
            else
                asm volatile("cp.async.commit_group;" ::: "memory");
            if (!ok) break;
            asm volatile("cp.async.wait_group 1;" ::: "memory");     // V of tile j
#pragma unroll
            for (int o = 0; o < kPass; ++o) cw[o] = lds16(stage + (uint32_t)(C::kStageV + (o * 32 + lane) * 16));
            if (j + 1 >= n_kv)
#pragma unroll
                for (int i = 0; i < kRuns; ++i) v_row[i] = 0xffffffffu;
            copy_v(v_row);
            ok = __all_sync(0xffffffffu, wait_bounded(bar_empty(1, sl), ((uint32_t)(j / F::kStagesV) & 1u) ^ 1u, abort_flag, p.wait_limit));
            if (!ok) break;
#pragma unroll
            for (int o = 0; o < kPass; ++o) store(std::false_type{}, ring_slot(1, sl), o, cw[o], sc[o]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full(1, sl));
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");   // nothing lands after the CTA's end
        __syncwarp();
    } else if (warp >= kProducerWarp) {
        setmaxnreg_dec<kRegsRowsControl>();
        if (warp == kProducerWarp) {
            if (lane == 0 && n_kv > 0) {
                mbar_arrive_expect_tx(bar_q_full, (uint32_t)F::kTileBytes);
                for (int bx = 0; bx < F::kBoxes; ++bx)
                    tma_load_4d(q_tile + bx * F::kBoxBytes, &tm_q, bar_q_full, bx * F::kBoxCols, (int)part_at[1], h, b, policy_evict_first());
                (void)wait_own_work(bar_q_full, 0);   // the copy has landed before the CTA can exit
            }
        } else if (warp == kMmaWarp || warp == kPvWarp) {
            // ======================================================= MMA issuers
            if (lane == 0 && n_kv > 0) {
                bool ok = true;
                if (warp == kMmaWarp) {
                    ok = wait_bounded(bar_q_ready, 0, abort_flag, p.wait_limit);
                    tc_fence_after();
                    for (int i = 0; i < n_kv && ok; ++i) {
                        if (i > 0) ok = wait_bounded(bar_s_free, (uint32_t)((i - 1) & 1), abort_flag, p.wait_limit);
                        const int sl = i % F::kStagesK;
                        if (ok) ok = wait_bounded(bar_full(0, sl), (uint32_t)((i / F::kStagesK) & 1), abort_flag, p.wait_limit);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t slot = ring_slot(0, sl);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t koff = (uint32_t)((kk / 4) * F::kBoxBytes + (kk % 4) * 32);
                            umma_ts(tmem + F::col_s(0), tmem + C::kColQ + (uint32_t)(kk * 8), smem_desc_sw128(slot + koff, 16, 1024),
                                    F::kIdescQK, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(bar_s_full(i & 1));
                        umma_commit(bar_empty(0, sl));
                    }
                } else {
                    for (int j = 0; j < n_kv && ok; ++j) {
                        const int pb = j % C::kPBufs, sl = j % F::kStagesV;
                        ok = wait_bounded(bar_p_full(pb), (uint32_t)((j / C::kPBufs) & 1), abort_flag, p.wait_limit);
                        if (ok) ok = wait_bounded(bar_full(1, sl), (uint32_t)((j / F::kStagesV) & 1), abort_flag, p.wait_limit);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t slot = ring_slot(1, sl);
#pragma unroll
                        for (int kk = 0; kk < kBlockN / 16; ++kk)
                            umma_ts(tmem + C::kColO, tmem + C::col_p(pb) + (uint32_t)(kk * 8),
                                    smem_desc_sw128(slot + (uint32_t)(kk * 16 * 128), F::kBoxBytes, 1024), F::kIdescPV,
                                    (j > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(bar_pv_done(pb));
                        umma_commit(bar_empty(1, sl));
                    }
                }
                // every MMA and commit has landed before TMEM is freed, after an abort too
                umma_commit(bar_drain);
                (void)wait_own_work(bar_drain, 0);
            }
        }
        __syncwarp();
    } else {
        setmaxnreg_inc<kRegsRowsSoftmax>();
        // =========================================================== softmax: one thread per row, tiles in turn
        const int qd = warp & 3, g = warp >> 2;
        const int r = qd * 32 + lane;
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        int lo, lim;
        row_keys(p.rows, x.kl, x.ql, m0 + r, lo, lim);
        const float c = p.scale_log2;
        float m_seen = -INFINITY, lu = 0.f;
        uint32_t nan_groups = 0;         // groups of V that a key this row sees holds as NaN
        constexpr uint32_t kNone = 1u << 31;
        if (lim <= lo) {                 // no row, or no key: nothing of it is kept, and it asks for no mask
            lo = 0, lim = 0x7fffffff;
            nan_groups = kNone;
        }
        bool ok = true;
        if (n_kv > 0 && 32 * g < D / 2) {
            // Q into TMEM, in the order of the codes: columns 32g .. 32g + 31 of this row
            ok = __all_sync(0xffffffffu, wait_bounded(bar_q_full, 0, abort_flag, p.wait_limit));
            if (ok) {
                uint32_t u[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = code_order(lds16(q_tile + (uint32_t)(g * F::kBoxBytes + r * 128 + ((i ^ (r & 7)) << 4))));
                    u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
                }
                tmem_st32(tmem + lane_off + C::kColQ + 32u * g, u);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_q_ready);
            }
        }
        for (int j = g; j < n_kv && ok; j += 2) {
            bool good = wait_bounded(bar_s_full(g), (uint32_t)((j >> 1) & 1), abort_flag, p.wait_limit);
            if (!__all_sync(0xffffffffu, good)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int kbase = x.lo + j * kBlockN;
            float s[kBlockN];
            {
                uint32_t u[kBlockN];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4)
                    tmem_ld32(tmem + lane_off + F::col_s(0) + 32u * q4, *reinterpret_cast<uint32_t(*)[32]>(&u[32 * q4]));
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < kBlockN; ++i) {
                    reg_after_wait(u[i]);
                    s[i] = __uint_as_float(u[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_s_free);
            uint32_t notes = 0;          // bits 2w, 2w + 1: runs of warp w that are not there
            uint32_t any_nan = 0;
#pragma unroll
            for (int w = 0; w < kMakers; ++w) {
                const uint32_t n = note(j)[w];
                notes |= (n & 3u) << (2 * w);
                any_nan |= n & 4u;
            }
            if (any_nan) {
                for (int w = 0; w < kMakers; ++w)
                    if (note(j)[w] & 4u)
                        for (int q = 0; q < D / kGroup; ++q) {
                            const uint32_t bits = note(j)[kMakers + w * (D / kGroup) + q];
                            for (int i = 0; i < 32; ++i) {
                                const int key = kbase + w * 32 + i;
                                if (((bits >> i) & 1u) && key >= lo && key < lim) nan_groups |= 1u << q;
                            }
                        }
            }
            if (__any_sync(0xffffffffu, kbase + kBlockN > lim || kbase < lo || notes != 0)) {
#pragma unroll
                for (int i = 0; i < kBlockN; ++i)
                    if (kbase + i >= lim || kbase + i < lo || ((notes >> (i / 16)) & 1u)) s[i] = -INFINITY;
            }
            const float mx = fmaxf(fmaxf(chunk_max32(s, 0), chunk_max32(s, 32)), fmaxf(chunk_max32(s, 64), chunk_max32(s, 96)));
            float m_prev = -INFINITY;
            if (j > 0) {
                good = wait_tagged_max(mref_w + 8u * (uint32_t)((g ^ 1) * kBlockM + r), (uint32_t)(j - 1), m_prev, abort_flag, p.wait_limit);
                if (!__all_sync(0xffffffffu, good)) {
                    ok = false;
                    break;
                }
            }
            const float t_max = mx * c;
            const float m_cur = (t_max > m_prev + kRescaleThreshold) ? reference(t_max) : m_prev;
            if (j + 1 < n_kv)
                st_relaxed_shared_u64(mref_w + 8u * (uint32_t)(g * kBlockM + r), ((unsigned long long)(uint32_t)j << 32) | __float_as_uint(m_cur));
            if (m_cur != m_seen) {
                lu *= ex2_approx(m_seen - m_cur);
                m_seen = m_cur;
            }
            const float mu = (m_cur == -INFINITY) ? 0.f : m_cur + kShift;
            const int pb = j % C::kPBufs;
            if (j >= C::kPBufs) {
                good = wait_bounded(bar_pv_done(pb), (uint32_t)(((j - C::kPBufs) / C::kPBufs) & 1), abort_flag, p.wait_limit);
                if (!__all_sync(0xffffffffu, good)) {
                    ok = false;
                    break;
                }
            }
            // P rounds to bf16 (2^-8) for the tensor cores; O is divided by the sum of the rounded
            // values.  (All on MUFU: the polynomial of the dense forward would lose a NaN.)
            float2 lu2 = make_float2(0.f, 0.f);
            const uint32_t taddr_p = tmem + lane_off + C::col_p(pb);
            exp_store_half<0, 0>(s, c, mu, taddr_p, lu2);
            exp_store_half<0, 1>(s, c, mu, taddr_p, lu2);
            lu += lu2.x + lu2.y;
            const float alpha = (m_cur != m_prev) ? ex2_approx(m_prev - m_cur) : 1.f;
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                good = wait_bounded(bar_pv_done((j - 1) % C::kPBufs), (uint32_t)(((j - 1) / C::kPBufs) & 1), abort_flag, p.wait_limit);
                if (!__all_sync(0xffffffffu, good)) {
                    tmem_wait_st();
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int q4 = 0; q4 < D / 32 + 1; ++q4) {   // O and its row-sum columns
                    const uint32_t ocol = tmem + lane_off + C::kColO + 32u * q4;
                    uint32_t u[32];
                    tmem_ld32(ocol, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        reg_after_wait(u[i]);
                        u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
                    }
                    tmem_st32(ocol, u);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p_full(pb));
        }

        // ---------------------------------------------------------- epilogue
        const bool have_o = n_kv > 0;
        bool good = ok;
        if (good && have_o) {
            // (the products' warps end here too when they gave up: then a tile is missing from O)
            good = __all_sync(0xffffffffu, wait_bounded(bar_drain, 0, abort_flag, p.wait_limit) && *abort_flag == 0);
            if (good) tc_fence_after();
        }
        const int row = (int)part_at[1] + r;
        epi[g * kBlockM + r] = m_seen;
        epi[(2 + g) * kBlockM + r] = lu;
        epi[(4 + g) * kBlockM + r] = __uint_as_float(nan_groups);
        good = !named_bar_or(kBarQuadBase + qd, 64, !good);
        nan_groups = __float_as_uint(epi[4 * kBlockM + r]) | __float_as_uint(epi[5 * kBlockM + r]);
        const bool none = nan_groups & kNone;
        const float m0w = epi[r], m1w = epi[kBlockM + r];
        const float m_fin = none ? -INFINITY : fmaxf(m0w, m1w);
        const float f0 = (m0w == m_fin) ? 1.f : ex2_approx(m0w - m_fin);
        const float f1 = (m1w == m_fin) ? 1.f : ex2_approx(m1w - m_fin);
        const float lu_row = none ? 0.f : epi[2 * kBlockM + r] * f0 + epi[3 * kBlockM + r] * f1;
        if (p.splits > 1) {
            // (a part that a wait gave up on has NaN for its sums, and so have the rows that it joins:
            // an answer that leaves keys out would look like any other)
            const size_t at = part_at[0];
            if (row < p.rows.R && g == 0) {
                float* const ml = p.part_ml + at * 3 * kBlockM + r;
                ml[0] = good ? m_fin : 0.f;
                ml[2 * kBlockM] = good ? lu_row : __int_as_float(0x7fc00000);
            }
            if (good && have_o) {
                uint32_t u[32];
                tmem_ld32(tmem + lane_off + C::kColL, u);
                tmem_wait_ld();
                reg_after_wait(u[0]);
                if (row < p.rows.R && g == 0) p.part_ml[(at * 3 + 1) * kBlockM + r] = __uint_as_float(u[0]);
#pragma unroll
                for (int q4 = 0; q4 < D / 64; ++q4) {
                    const int col0 = g * (D / 2) + 32 * q4;
                    const bool is_nan = (nan_groups >> (col0 / kGroup)) & 1u;
                    tmem_ld32(tmem + lane_off + C::kColO + (uint32_t)col0, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        reg_after_wait(u[i]);
                        if (is_nan) u[i] = 0x7fc00000u;
                    }
                    uint4* const dst = reinterpret_cast<uint4*>(p.part) + (at * (D / 4) + col0 / 4) * kBlockM + r;
                    if (row < p.rows.R)
#pragma unroll
                        for (int v4 = 0; v4 < 8; ++v4) {   // channels back in order
                            const int u0 = 8 * (v4 / 2) + v4 % 2;
                            dst[v4 * kBlockM] = make_uint4(u[u0], u[u0 + 2], u[u0 + 4], u[u0 + 6]);
                        }
                }
            } else if (row < p.rows.R && g == 0) {
                p.part_ml[(at * 3 + 1) * kBlockM + r] = good ? 0.f : __int_as_float(0x7fc00000);
            }
        } else if (good) {
            float l_row = 0.f;
            if (have_o) {
                uint32_t u[32];
                tmem_ld32(tmem + lane_off + C::kColL, u);
                tmem_wait_ld();
                reg_after_wait(u[0]);
                l_row = none ? 0.f : __uint_as_float(u[0]);
            }
            const float inv_row = l_row == 0.f ? 0.f : 1.f / l_row;
#pragma unroll
            for (int q4 = 0; q4 < D / 64; ++q4) {
                const int col0 = g * (D / 2) + 32 * q4;
                const float inv_l = !none && ((nan_groups >> (col0 / kGroup)) & 1u) ? __int_as_float(0x7fc00000) : inv_row;
                uint32_t u[32];
                if (have_o) {
                    tmem_ld32(tmem + lane_off + C::kColO + (uint32_t)col0, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        reg_after_wait(u[i]);
                        if (none) u[i] = 0u;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) u[i] = 0u;
                }
                auto two = [&](int a, int z) { return pack_bf16x2(__uint_as_float(u[a]) * inv_l, __uint_as_float(u[z]) * inv_l); };
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    // columns (0,4) (1,5) (2,6) (3,7) of 8 channels, back in order
                    const int cc = col0 / 8 + v4, u0 = 8 * v4;
                    sts16(q_tile + (uint32_t)((cc >> 3) * kSwizzleBoxBytes + r * 128 + (((cc & 7) ^ (r & 7)) << 4)),
                          two(u0, u0 + 2), two(u0 + 4, u0 + 6), two(u0 + 1, u0 + 3), two(u0 + 5, u0 + 7));
                }
            }
            if (g == 0 && row < p.rows.R)
                p.lse[((size_t)b * p.H_kv + h) * (size_t)p.rows.R + row] = lse_of(m_fin, lu_row);
        }
        fence_proxy_async_smem();
        const bool any_bad = named_bar_or(kBarSoftmaxAll, kSoftmaxWarps * 32, !good);
        if (!any_bad && threadIdx.x == 0 && p.splits == 1) {
            for (int bx = 0; bx < F::kOBoxes; ++bx) tma_store_4d(&tm_o, q_tile + bx * kSwizzleBoxBytes, bx * 64, (int)part_at[1], h, b);
            bulk_commit_group();
            bulk_wait_group_read0();
        }
        if (any_bad && p.splits == 1 && row < p.rows.R) {   // the whole block's rows, as above
            const size_t at = ((size_t)b * p.H_kv + h) * (size_t)p.rows.R + row;
            if (g == 0) p.lse[at] = __int_as_float(0x7fc00000);
            uint4* const dst = reinterpret_cast<uint4*>(p.o + at * D) + g * (D / 16);
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) dst[i] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the ranges of a block of rows.  Block (x, y, z): 32 rows and 8 channels of row block y
// of head z, a row per lane, the ranges dealt out to the warps.  The parts are in L2, so what
// counts is that all loads are on their way at once.
constexpr int kJoinWarps = 4;

struct JoinParams {
    const float4* part;
    const float* part_ml;
    __nv_bfloat16* o;
    float* lse;
    int R, splits;
};

struct Joined {
    float m = -INFINITY, l = 0.f, lu = 0.f;   // reference max, sums of rounded P and of P
    float acc[8] = {};
    // A part without a key the row sees counts nothing, whatever its sums hold.
    __device__ __forceinline__ void add(float m2, float l2, float lu2, const float (&v)[8]) {
        const bool none = m2 == -INFINITY && lu2 == 0.f;
        const float top = fmaxf(m, m2);
        const float a = m == top ? 1.f : ex2_approx(m - top), w = m2 == top ? 1.f : ex2_approx(m2 - top);
        m = top;
        l = l * a + (none ? 0.f : l2 * w);
        lu = lu * a + (none ? 0.f : lu2 * w);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * a + (none ? 0.f : v[i] * w);
    }
};

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const JoinParams p) {
    after_previous();
    __shared__ float other[kJoinWarps - 1][11][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c8 = blockIdx.x % (D / 8), r0 = (int)(blockIdx.x / (D / 8)) * 32;
    const int row = (int)blockIdx.y * kBlockM + r0 + lane;
    if (row - lane >= p.R) return;
    const int r = r0 + min(lane, p.R - 1 - (row - lane));   // behind the last row nothing was written
    const size_t at = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * p.splits;
    Joined x;
    constexpr int kEach = 4;
    for (int s0 = warp; s0 < p.splits; s0 += kJoinWarps * kEach) {
        float ml[kEach][3], v[kEach][8];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const size_t a = at + min(s0 + i * kJoinWarps, p.splits - 1);
#pragma unroll
            for (int k = 0; k < 3; ++k) ml[i][k] = __ldcg(p.part_ml + (a * 3 + k) * kBlockM + r);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 f = __ldcg(p.part + (a * (D / 4) + 2 * c8 + k) * kBlockM + r);
                v[i][4 * k] = f.x, v[i][4 * k + 1] = f.y, v[i][4 * k + 2] = f.z, v[i][4 * k + 3] = f.w;
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (s0 + i * kJoinWarps < p.splits) x.add(ml[i][0], ml[i][1], ml[i][2], v[i]);
    }
    if (warp > 0) {
        float(*const to)[32] = other[warp - 1];
        to[0][lane] = x.m, to[1][lane] = x.l, to[2][lane] = x.lu;
#pragma unroll
        for (int i = 0; i < 8; ++i) to[3 + i][lane] = x.acc[i];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < kJoinWarps - 1; ++w) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = other[w][3 + i][lane];
        x.add(other[w][0][lane], other[w][1][lane], other[w][2][lane], v);
    }
    if (row >= p.R) return;
    const size_t out = (size_t)blockIdx.z * p.R + row;
    const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
    uint4 y;
    y.x = pack_bf16x2(x.acc[0] * inv, x.acc[1] * inv), y.y = pack_bf16x2(x.acc[2] * inv, x.acc[3] * inv);
    y.z = pack_bf16x2(x.acc[4] * inv, x.acc[5] * inv), y.w = pack_bf16x2(x.acc[6] * inv, x.acc[7] * inv);
    *reinterpret_cast<uint4*>(p.o + out * D + 8 * c8) = y;
    if (c8 == 0) p.lse[out] = lse_of(x.m, x.lu);
}

}  // namespace kv4
}  // namespace fa
