// fa_kv4_rule.h -- which kernel a call of the 4-bit cache attention takes: the one for few rows
// (fa_kv4_attend.cuh) with 8 or 16 rows a block, or the one for many rows (fa_kv4_rows.cuh) and
// with how many ranges of keys.  Plain arithmetic on the host.
//
// It knows the sizes of the call and the longest sequence that the page table has room for; the
// lengths are on the device, so a table much wider than its sequences can cost the better choice:
// with room for 65536 keys and 700 in use 16 rows of 8 heads take 13.8 us instead of 10.8.
// The constants, in us, are fitted to 3118 shapes that were measured with all three, for which of
// them is the quickest: 1 to 2048 heads of 64 and of 128 channels, 9 to 4096 rows, 1 to 131072
// keys, masks and windows, ragged lengths.  Over these, the choice takes 1.008 times the time of
// the quickest in the geometric mean and 1.38 at worst (16 rows or less are not given to the
// kernel for many).  Some of them, at 128 channels, in us by 8 rows, 16 rows, many:
//      8 x  8 heads,    16 keys,  20 rows     6.1     8.1     8.1
//      8 x  8 heads,    16 keys, 512 rows    40.3    42.6    17.0
//     64 x 32 heads,    16 keys,  20 rows    56.2    81.2   106.4
//     64 x 32 heads,    16 keys, 512 rows  1183.5  1326.0   441.9
//    100 x  1 heads,    60 keys,  24 rows     8.9    10.2     8.8
//    100 x  1 heads,    60 keys, 300 rows    95.8    65.7    22.3
//      1 x  8 heads,   700 keys,  20 rows    10.2    13.1    12.2
//      1 x  8 heads,   700 keys, 256 rows    19.3    16.6    14.3
//      8 x  8 heads,   700 keys,  20 rows    13.7    16.3    16.7
//      8 x  8 heads,   700 keys, 256 rows    68.2    54.4    17.1
//      1 x  8 heads, 32768 keys,  20 rows    37.6    38.3    30.9
//      8 x  8 heads,  4096 keys,  64 rows    78.0    56.6    34.4
#pragma once

#include <algorithm>

namespace fa {
namespace kv4 {

constexpr int kRuleUnit = 128;        // keys of a unit and of a tile
constexpr int kRuleEntries = 512;     // (sequence, row block) pairs of a launch of the kernel for few rows

// The kernel for few rows, with 8 or 16 rows a block.
struct FewCost {
    double start;                     // of the first launch
    double launch;                    // of each further one
    double unit, item;                // of an SM, for a unit and for a (sequence, head, row block)
    double merge, part;               // where an item is shared: once, and for each CTA that shares it
    int most_parts;                   // that cost it (beyond, with 8 rows, they are merged in two levels)
};
// The one for many rows.
struct ManyCost {
    double start;
    double join, join_block;          // of the second kernel, where keys are split, and of an SM for a block of rows
    double cta, tile;                 // of a wave of CTAs, and of a tile of each
};
constexpr FewCost kFew[2][2] = {{{4.2, 7.0, .36, .71, 4.3, .083, 60}, {6.0, 6.0, .50, 1.5, 5.3, .11, 1 << 30}},
                                {{4.1, 8.6, .59, .81, 5.0, .10, 60}, {7.4, 9.9, .85, 1.7, 4.3, .25, 1 << 30}}};   // [d = 128][16 rows]
constexpr ManyCost kMany[2] = {{.3, 1.0, 5.0, 6.0, 1.1}, {0., .75, 8.2, 7.1, 1.3}};

struct Choice {
    bool many;
    int rows_a_block;                 // of the kernel for few rows: 8 or 16
    int splits;                       // of the kernel for many rows: ranges of keys of a block of 128 rows
};

constexpr int ctas_per_sm(int rows_a_block) { return rows_a_block == 8 ? 3 : 2; }

// Keys that a block of rows meets at most: with a window, those of its queries and what the first
// of them is rounded down by.
inline long long block_keys(long long keys, int window, int N_q, int rows) {
    return window < 0 ? keys : std::min(keys, (long long)window + std::min(N_q, rows) + 31);
}

inline double few_us(const FewCost& c, int rows, int B, long long R, long long heads, long long keys, int num_sms) {
    const long long blocks = (R + rows - 1) / rows, each = std::max<long long>(1, (keys + kRuleUnit - 1) / kRuleUnit);
    const double items = (double)blocks * (double)heads;
    const double launches = (double)((blocks * B + kRuleEntries - 1) / kRuleEntries);
    const double parts = std::min((double)each, std::max(1., (double)num_sms * ctas_per_sm(rows) / items));
    return c.start + c.launch * (launches - 1) + (c.unit * (double)each + c.item) * items / num_sms +
           (each > 1 ? c.merge + c.part * std::min(parts, (double)c.most_parts) : 0.);
}

// Ranges of the keys of a block of 128 rows, where the blocks alone would leave half the SMs idle:
// at most as many as fill the SMs once, each with two tiles or more of the longest sequence there
// could be.  8 heads of 32768 keys, 128 rows: one CTA a block about 340 us, 18 of them 32; 1024
// rows, two CTAs, 173.
inline int most_splits(long long R, long long heads, int num_sms) {
    return (int)std::max<long long>(1, num_sms / ((R + 127) / 128 * heads));
}

inline double many_us(const ManyCost& c, long long R, long long heads, long long keys, int splits, int num_sms) {
    const long long blocks = (R + 127) / 128 * heads, tiles = std::max<long long>(1, (keys + kRuleUnit - 1) / kRuleUnit);
    const double waves = (double)((blocks * splits + num_sms - 1) / num_sms);
    return c.start + (splits > 1 ? c.join + c.join_block * (double)blocks / num_sms : 0.) +
           waves * (c.cta + c.tile * (double)((tiles + splits - 1) / splits));
}

// R = H / H_kv * N_q rows for each of B * H_kv heads; keys: the most that a sequence can have.
inline Choice choose(int B, int H_kv, long long R, int N_q, int d, long long keys, int window, int num_sms) {
    const long long heads = (long long)B * H_kv, keys128 = block_keys(keys, window, N_q, 128);
    Choice x{false, 8, 1};
    x.splits = (int)std::max<long long>(1, std::min<long long>(most_splits(R, heads, num_sms), keys128 / 256));
    if (R <= 8) return x;
    const FewCost* const f = kFew[d == 128];
    double best = few_us(f[0], 8, B, R, heads, block_keys(keys, window, N_q, 8), num_sms);
    const double us16 = few_us(f[1], 16, B, R, heads, block_keys(keys, window, N_q, 16), num_sms);
    if (us16 < best) {
        best = us16;
        x.rows_a_block = 16;
    }
    x.many = R > 16 && many_us(kMany[d == 128], R, heads, keys128, x.splits, num_sms) < best;
    return x;
}

}  // namespace kv4
}  // namespace fa
