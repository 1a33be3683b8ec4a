// fa_kv4.cu -- host side of the 4-bit paged key/value cache entry points (include/fa.h):
// argument checks (before any CUDA call), workspace layout and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "fa_kv4_attend.cuh"
#include "fa_kv4_kernel.cuh"
#include "fa_kv4_rule.h"

namespace {

using fa_internal::cuda_fail;
using fa_internal::launch_overlapped;
using fa_internal::ready_device;
namespace kv4 = fa::kv4;

constexpr int kMaxPositions = 1 << 30;   // max_pages * page_size: positions and tile numbers stay within int

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Checks that the three entry points share; *empty: nothing to do.
int validate(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
             const int32_t* block_table, const int32_t* key_lens, const int32_t* lens, int B, int H_kv, int N, int d,
             int num_pages, int page_size, int max_pages, bool* empty) {
    if (B < 0 || H_kv < 0 || N < 0 || num_pages < 0 || max_pages < 0 || page_size <= 0) return FA_ERR_INVALID_ARG;
    if (page_size % 16 != 0) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > kMaxPositions) return FA_ERR_UNSUPPORTED;
    // rows of one head's tokens are numbered in 32 bits (a cache of 2^32 rows is over 300 GB)
    if ((unsigned __int128)num_pages * H_kv * page_size >= ((unsigned __int128)1 << 32)) return FA_ERR_UNSUPPORTED;
    *empty = B == 0 || H_kv == 0 || N == 0;
    if (*empty) return FA_OK;
    if (B > 65535 || H_kv > 65535) return FA_ERR_UNSUPPORTED;
    if (key_lens == nullptr) return FA_ERR_INVALID_ARG;
    if (num_pages > 0 &&
        (k_codes == nullptr || k_scales == nullptr || v_codes == nullptr || v_scales == nullptr))
        return FA_ERR_INVALID_ARG;
    for (const void* p : {k_codes, k_scales, v_codes, v_scales})
        if (!aligned(p, 16)) return FA_ERR_MISALIGNED;
    for (const int32_t* p : {block_table, key_lens, lens})
        if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
    return FA_OK;
}

kv4::Paging paging(const int32_t* table, int num_pages, int page_size, int max_pages) {
    kv4::Paging pg;
    pg.table = table;
    pg.num_pages = num_pages;
    pg.page_size = page_size;
    pg.max_pages = max_pages;
    kv4::divisor((uint32_t)page_size, pg.magic, pg.shift);
    return pg;
}

// Launch of the kernels that write and read tokens (see kv4::kRowsPerThread); false if B * H_kv
// exceeds the launch limits, or N that of positions.
bool row_grid(int B, int H_kv, int N, int d, dim3* grid, bool* flat, uint32_t* rows) {
    const long long block = kv4::kRowThreads / (d / 8), per = block * kv4::kRowsPerThread, heads = (long long)B * H_kv;
    if (heads > 0x7fffffffLL || N > kMaxPositions) return false;
    *flat = N < per && heads * N <= 0x7fffffffLL;
    *rows = *flat ? (uint32_t)(heads * N) : 0;
    *grid = *flat ? dim3((unsigned)((heads * N + block - 1) / block))
                  : dim3((unsigned)heads, (unsigned)std::min<long long>((N + per - 1) / per, kv4::kMaxRowBlocks));
    return true;
}

// A 48-bit ticket other than 0 for each attention launch (see kv4::arrive_last).
unsigned long long next_ticket() {
    static std::atomic<unsigned long long> seq{
        (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull};
    unsigned long long t = 0;
    while (t == 0) t = (seq.fetch_add(1, std::memory_order_relaxed) + 1) & ((1ull << 48) - 1);
    return t;
}

using kv4::ctas_per_sm;
static_assert(ctas_per_sm(8) == kv4::Cfg<128, 1>::kCtasPerSm && ctas_per_sm(8) == kv4::Cfg<64, 1>::kCtasPerSm &&
                  ctas_per_sm(16) == kv4::Cfg<128, 2>::kCtasPerSm && ctas_per_sm(16) == kv4::Cfg<64, 2>::kCtasPerSm &&
                  kv4::kRuleUnit == kv4::kUnit && kv4::kRuleEntries == kv4::kMaxEntries,
              "the rule's kernels");

// Workspace of the attention: two partial results per CTA, then the arrival words.  The kernel
// for many rows keeps one partial result per CTA where it splits the keys.
struct Layout {
    size_t part, ml, words, group_words, rows_ml, total;
};
Layout layout(int B, int H, int H_kv, int N_q, int d, int num_sms, int rb) {
    const long long R = (long long)(H / H_kv) * N_q;
    const size_t slots = 2 * (size_t)num_sms * ctas_per_sm(rb);
    const long long entries = (R + rb - 1) / rb * B;
    Layout L{};
    L.part = 0;
    L.ml = round_up(slots * rb * d * 4);
    L.words = L.ml + round_up(slots * rb * 16);
    L.group_words = L.words + round_up((size_t)std::min<long long>(entries, kv4::kMaxEntries) * H_kv * 8);
    L.total = L.group_words + round_up(slots * 8);
    const int splits = R > 16 ? kv4::most_splits(R, (long long)B * H_kv, num_sms) : 1;
    if (splits > 1) {
        const size_t parts = (size_t)splits * B * H_kv * ((R + 127) / 128) * 128;   // rows
        L.rows_ml = round_up(parts * d * 4);
        L.total = std::max(L.total, L.rows_ml + round_up(parts * 12));
    }
    return L;
}

// Whatever the lengths that choose rb.
size_t workspace_size(int B, int H, int H_kv, int N_q, int d, int num_sms) {
    return std::max(layout(B, H, H_kv, N_q, d, num_sms, 8).total, layout(B, H, H_kv, N_q, d, num_sms, 16).total);
}

std::once_flag g_once[64];
int g_status[64];

template <int D, int NB, bool kGroups>
cudaError_t set_smem() {
    const int bytes = kv4::Cfg<D, NB>::kSmemBytes;
    const cudaError_t e =
        cudaFuncSetAttribute(kv4::attend_kernel<D, NB, false, kGroups>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kv4::attend_kernel<D, NB, true, kGroups>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
int prepare_attend(int dev) {
    std::call_once(g_once[dev], [&] {
        cudaError_t e = set_smem<64, 1, false>();
        if (e == cudaSuccess) e = set_smem<64, 1, true>();
        if (e == cudaSuccess) e = set_smem<64, 2, false>();
        if (e == cudaSuccess) e = set_smem<128, 1, false>();
        if (e == cudaSuccess) e = set_smem<128, 1, true>();
        if (e == cudaSuccess) e = set_smem<128, 2, false>();
        g_status[dev] = e == cudaSuccess ? FA_OK : cuda_fail("cudaFuncSetAttribute(MaxDynamicSharedMemorySize)", e);
    });
    return g_status[dev];
}

template <int D, int NB, bool kGroups>
cudaError_t launch_attend(const kv4::AttendParams& p, int num_sms, cudaStream_t s) {
    const int grid = num_sms * ctas_per_sm(8 * NB), smem = kv4::Cfg<D, NB>::kSmemBytes;
    return launch_overlapped(p.pg.page_size % kv4::kTile == 0 ? kv4::attend_kernel<D, NB, true, kGroups>
                                                              : kv4::attend_kernel<D, NB, false, kGroups>,
                             grid, kv4::kThreads, smem, s, p);
}
template <int D>
cudaError_t launch_attend(const kv4::AttendParams& p, int rb, bool groups, int num_sms, cudaStream_t s) {
    if (rb != 8) return launch_attend<D, 2, false>(p, num_sms, s);
    return groups ? launch_attend<D, 1, true>(p, num_sms, s) : launch_attend<D, 1, false>(p, num_sms, s);
}

// fa_fwd_kv4; with wait_limit > 0 only by the kernel for many rows, whose waits it bounds.
int fwd(const void* q, const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
        const int32_t* block_table, const int32_t* key_lens, const int32_t* q_lens, void* o, float* lse, int B,
        int H, int H_kv, int N_q, int d, int num_pages, int page_size, int max_pages, float scale, int causal,
        int window_left, void* workspace, size_t workspace_bytes, fa_stream_t stream,
        unsigned long long wait_limit) {
    bool empty = false;
    int st = validate(k_codes, k_scales, v_codes, v_scales, block_table, key_lens, q_lens, B, H_kv, N_q, d, num_pages,
                      page_size, max_pages, &empty);
    if (st != FA_OK) return st;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!std::isfinite(scale) || !(scale > 0.f) || !(scale_log2 > 0.f) || !std::isfinite(scale_log2))
        return FA_ERR_INVALID_ARG;
    if (H < 0 || (H_kv > 0 && H % H_kv != 0) || (H_kv == 0 && H != 0)) return FA_ERR_INVALID_ARG;
    if (empty || H == 0) return wait_limit > 0 ? FA_ERR_INVALID_ARG : FA_OK;
    if (H > 65535) return FA_ERR_UNSUPPORTED;
    const long long R = (long long)(H / H_kv) * N_q;
    const long long units = (long long)max_pages * page_size / kv4::kUnit + 2;   // most of one row block
    if (R > 0x3fffffffLL || units * H_kv > 0x3fffffffLL) return FA_ERR_UNSUPPORTED;
    if (q == nullptr || o == nullptr || lse == nullptr || workspace == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256)) return FA_ERR_MISALIGNED;
    int dev = -1, sms = 0;
    st = ready_device(&dev, &sms);
    if (st != FA_OK) sms = fa_internal::current_num_sms();
    if (workspace_bytes < workspace_size(B, H, H_kv, N_q, d, sms)) return FA_ERR_INVALID_ARG;
    if (st == FA_OK) st = prepare_attend(dev);
    if (st != FA_OK) return st;
    kv4::Rows rows{};
    rows.key_lens = key_lens;
    rows.q_lens = q_lens;
    rows.N_q = N_q;
    rows.R = (int)R;
    rows.causal = causal ? 1 : 0;
    rows.window = window_left < 0 ? -1 : std::min(window_left, kMaxPositions);
    const kv4::Paging pg = paging(block_table, num_pages, page_size, max_pages);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long room = (long long)max_pages * page_size;
    const kv4::Choice choice = kv4::choose(B, H_kv, R, N_q, d, room, rows.window, sms);
    const int rb = choice.rows_a_block;
    const long long keys = kv4::block_keys(room, rows.window, N_q, rb);
    const Layout L = layout(B, H, H_kv, N_q, d, sms, rb);
    if (wait_limit > 0 && !choice.many) return FA_ERR_INVALID_ARG;   // nothing would wait
    if (choice.many) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        kv4::RowsParams p{};
        p.k_codes = static_cast<const uint8_t*>(k_codes);
        p.k_scales = static_cast<const uint16_t*>(k_scales);
        p.v_codes = static_cast<const uint8_t*>(v_codes);
        p.v_scales = static_cast<const uint16_t*>(v_scales);
        p.pg = pg;
        p.rows = rows;
        p.H_kv = H_kv;
        p.o = static_cast<__nv_bfloat16*>(o);
        p.lse = lse;
        p.scale_log2 = scale_log2;
        p.splits = choice.splits;
        p.wait_limit = wait_limit;
        p.part = reinterpret_cast<float*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + L.rows_ml);
        return fa_internal::launch_kv4_rows(q, o, B, d, p, s);
    }
    kv4::AttendParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_codes = static_cast<const uint8_t*>(k_codes);
    p.k_scales = static_cast<const uint16_t*>(k_scales);
    p.v_codes = static_cast<const uint8_t*>(v_codes);
    p.v_scales = static_cast<const uint16_t*>(v_scales);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.pg = pg;
    p.H_kv = H_kv;
    p.rows = rows;
    p.row_blocks = (int)((R + rb - 1) / rb);
    p.scale_log2 = scale_log2;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part = reinterpret_cast<float*>(ws + L.part);
    p.part_ml = reinterpret_cast<float*>(ws + L.ml);
    p.words = reinterpret_cast<unsigned long long*>(ws + L.words);
    p.group_words = reinterpret_cast<unsigned long long*>(ws + L.group_words);
    const long long entries = (long long)B * p.row_blocks;
    // the line of units of one launch stays within int
    const long long chunk = std::min<long long>(kv4::kMaxEntries, std::max<long long>(1, 0x3fffffffLL / (units * H_kv)));
    for (long long e0 = 0; e0 < entries; e0 += chunk) {
        p.b0 = (int)(e0 / p.row_blocks);
        p.rb0 = (int)(e0 % p.row_blocks);
        p.E = (int)std::min(chunk, entries - e0);
        p.ticket = next_ticket();
        // parts of an item, if the sequences are alike
        const long long parts = std::min<long long>((keys + kv4::kUnit - 1) / kv4::kUnit, (long long)sms * ctas_per_sm(rb) / (p.E * H_kv));
        const int nr = (int)std::min<long long>(R, rb);
        const bool groups = parts > kv4::kFlat * (d == 64 ? kv4::row_groups<64>(nr) : kv4::row_groups<128>(nr));
        const cudaError_t e = d == 64 ? launch_attend<64>(p, rb, groups, sms, s) : launch_attend<128>(p, rb, groups, sms, s);
        if (e != cudaSuccess) return cuda_fail("kernel launch (4-bit cache attention)", e);
    }
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_kv4_append(const void* k, const void* v, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                  const int32_t* block_table, const int32_t* key_lens, const int32_t* new_lens, int B, int H_kv,
                  int N_new, int d, int num_pages, int page_size, int max_pages, fa_stream_t stream) {
    bool empty = false;
    int st = validate(k_codes, k_scales, v_codes, v_scales, block_table, key_lens, new_lens, B, H_kv, N_new, d,
                      num_pages, page_size, max_pages, &empty);
    if (st != FA_OK || empty) return st;
    if (k == nullptr || v == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16)) return FA_ERR_MISALIGNED;
    kv4::AppendParams p{};
    p.k = static_cast<const uint4*>(k);
    p.v = static_cast<const uint4*>(v);
    p.k_codes = static_cast<uint32_t*>(k_codes);
    p.k_scales = static_cast<uint16_t*>(k_scales);
    p.v_codes = static_cast<uint32_t*>(v_codes);
    p.v_scales = static_cast<uint16_t*>(v_scales);
    p.key_lens = key_lens;
    p.new_lens = new_lens;
    p.pg = paging(block_table, num_pages, page_size, max_pages);
    p.H_kv = H_kv;
    p.N = N_new;
    dim3 grid;
    bool flat = false;
    if (!row_grid(B, H_kv, N_new, d, &grid, &flat, &p.rows)) return FA_ERR_UNSUPPORTED;
    int dev = -1, sms = 0;
    st = ready_device(&dev, &sms);
    if (st != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto kernel = d == 64 ? (flat ? kv4::append_kernel<64, true> : kv4::append_kernel<64, false>)
                                : (flat ? kv4::append_kernel<128, true> : kv4::append_kernel<128, false>);
    const cudaError_t e = launch_overlapped(kernel, grid, kv4::kRowThreads, 0, s, p);
    return e == cudaSuccess ? FA_OK : cuda_fail("kernel launch (4-bit cache append)", e);
}

int fa_kv4_read(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                const int32_t* block_table, const int32_t* key_lens, const int32_t* first, void* k, void* v, int B,
                int H_kv, int N, int d, int num_pages, int page_size, int max_pages, fa_stream_t stream) {
    bool empty = false;
    int st = validate(k_codes, k_scales, v_codes, v_scales, block_table, key_lens, first, B, H_kv, N, d, num_pages,
                      page_size, max_pages, &empty);
    if (st != FA_OK || empty) return st;
    if (k == nullptr || v == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16)) return FA_ERR_MISALIGNED;
    kv4::ReadParams p{};
    p.k_codes = static_cast<const uint32_t*>(k_codes);
    p.k_scales = static_cast<const uint16_t*>(k_scales);
    p.v_codes = static_cast<const uint32_t*>(v_codes);
    p.v_scales = static_cast<const uint16_t*>(v_scales);
    p.key_lens = key_lens;
    p.first = first;
    p.k = static_cast<uint4*>(k);
    p.v = static_cast<uint4*>(v);
    p.pg = paging(block_table, num_pages, page_size, max_pages);
    p.H_kv = H_kv;
    p.N = N;
    dim3 grid;
    bool flat = false;
    if (!row_grid(B, H_kv, N, d, &grid, &flat, &p.rows)) return FA_ERR_UNSUPPORTED;
    int dev = -1, sms = 0;
    st = ready_device(&dev, &sms);
    if (st != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto kernel = d == 64 ? (flat ? kv4::read_kernel<64, true> : kv4::read_kernel<64, false>)
                                : (flat ? kv4::read_kernel<128, true> : kv4::read_kernel<128, false>);
    const cudaError_t e = launch_overlapped(kernel, grid, kv4::kRowThreads, 0, s, p);
    return e == cudaSuccess ? FA_OK : cuda_fail("kernel launch (4-bit cache read)", e);
}

size_t fa_fwd_kv4_workspace_size(int B, int H, int H_kv, int N_q, int d) {
    if (B <= 0 || H <= 0 || H_kv <= 0 || N_q <= 0 || H % H_kv != 0 || (d != 64 && d != 128)) return 0;
    if (B > 65535 || H > 65535) return 0;
    return workspace_size(B, H, H_kv, N_q, d, fa_internal::current_num_sms());
}

int fa_fwd_kv4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
               const int32_t* block_table, const int32_t* key_lens, const int32_t* q_lens, void* o, float* lse, int B,
               int H, int H_kv, int N_q, int d, int num_pages, int page_size, int max_pages, float scale, int causal,
               int window_left, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
    return fwd(q, k_codes, k_scales, v_codes, v_scales, block_table, key_lens, q_lens, o, lse, B, H, H_kv, N_q, d, num_pages,
               page_size, max_pages, scale, causal, window_left, workspace, workspace_bytes, stream, 0);
}

int fa_selftest_kv4_timeout(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                            const void* v_scales, const int32_t* block_table, const int32_t* key_lens,
                            const int32_t* q_lens, void* o, float* lse, int B, int H, int H_kv, int N_q, int d,
                            int num_pages, int page_size, int max_pages, float scale, int causal, int window_left,
                            void* workspace, size_t workspace_bytes, unsigned long long limit_cycles,
                            fa_stream_t stream) {
    if (limit_cycles < 1 || limit_cycles > (1ull << 32)) return FA_ERR_INVALID_ARG;
    const int st = fwd(q, k_codes, k_scales, v_codes, v_scales, block_table, key_lens, q_lens, o, lse, B, H, H_kv, N_q, d,
                       num_pages, page_size, max_pages, scale, causal, window_left, workspace, workspace_bytes, stream,
                       limit_cycles);
    return st != FA_OK ? st : fa_get_device_status(stream);
}

}  // extern "C"
