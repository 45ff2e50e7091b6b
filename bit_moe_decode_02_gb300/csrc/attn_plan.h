// attn_plan.h -- which of the two attention kernels a call takes, and which groups of the
// prompt kernel are cut into parts.  Plain C++: it is worked out on the host, where lengths
// are not known but bounds of them, and a test runs it there.
#pragma once
#include "../../include/moe.h"

namespace moe {

// Groups of 256 rows of the prompt kernel: `whole` by a CTA each, `rest` more in up to `parts` parts each.
struct PromptCut {
    int whole, parts, rest;
};

namespace attn {

constexpr int kGroupRows = 256;           // of the prompt kernel's CTA
constexpr int kTileKeys = 128;            // of its tile
constexpr int kPartTiles = 4;             // a part of a group's keys has that many tiles at least

struct Call {
    int n_seqs, n_tokens, group, H;       // group: query heads of a kv head
    int D, blk, fmt;
    int table_stride, window;
};

// 4-bit items of eight rows: at most that many a sequence's kv head, on average.
inline bool narrow(const Call& c) { return c.fmt == MOE_KV_MXFP4 && (long long)c.n_tokens * c.group <= 8ll * c.n_seqs; }

// Pieces of `unit` keys that `rows` rows of one kv head see at most: what the table holds, or
// the window of their tokens wherever it begins.
inline long long pieces(const Call& c, long long rows, int unit)
{
    const long long held = ((long long)c.table_stride * c.blk + unit - 1) / unit;
    long long tokens = rows > 1 ? (rows - 1) / c.group + 2 : 1;
    if (c.window == 0)
        return held;
    tokens = tokens < c.n_tokens ? tokens : c.n_tokens;
    const long long seen = (c.window + tokens - 1 + unit - 2) / unit + 1;
    return seen < held ? seen : held;
}

// Which groups' keys are cut, and into how many parts: those that would be the last round of CTAs and leave SMs idle,
// one part an SM, for which the workspace has room, and none where the keys are too few.  (Up to two, in the fewest
// rounds, is slower more often than not: 8 sequences of 4,000 keys, 32 heads of 128 on 4, 80 and 216 rows 37 and 52 us
// for 30 and 44.)  The groups are an upper bound: what a batch's tokens make at most, however they lie in its sequences.
inline PromptCut prompt_cut(const Call& c, int num_sms)
{
    const long long seqs = c.n_seqs < c.n_tokens ? c.n_seqs : c.n_tokens;
    const long long groups = ((long long)c.n_tokens * c.group + (kGroupRows - 1) * seqs) / kGroupRows * c.H, rest = groups % num_sms;
    const long long most = pieces(c, kGroupRows, kTileKeys) / kPartTiles;
    long long parts = rest > 0 ? num_sms / rest : 1;
    parts = parts < most ? parts : most;
    if (parts <= 1)
        return PromptCut{(int)groups, 1, 0};
    return PromptCut{(int)(groups - rest), (int)parts, (int)rest};
}

// What a call is expected to take with each kernel, in ns.  Fitted to 15,400 calls of each: every
// format, block and head size; 16 to 80 heads on 1 to 16; 1 to 200 sequences of 50 to 20,000
// keys, whole and within windows, of one length and of several; 1 to 1,500 tokens each.  Over 3,000
// others the kernel that is taken is 0.6 % behind the better one on average, more than a tenth
// in one call of 38, mostly the decode kernel.
// Rows are the average of a sequence's kv head, keys the bound of `pieces`.

// Beside its start: a tile of 128 keys of an item, over all SMs, or for an item that is not cut
// on one; the join of an item over CTAs, less where a CTA has not a tile for every warp; an item
// more for every SM; a sequence's row tiles, which one thread walks.
inline double decode_ns(const Call& c, int num_sms)
{
    struct Cost {
        double start, tile, join, item, row;
    };
    static const Cost costs[2][3] = {{{6502, 460, 8455, 1265, 18}, {7233, 449, 8827, 1081, 16}, {6141, 268, 10126, 1299, 199}},
                                     {{7675, 614, 10922, 2143, 19}, {9014, 671, 13229, 2354, 16}, {7475, 412, 11032, 1228, 166}}};
    const bool mx = c.fmt == MOE_KV_MXFP4, eight = narrow(c);
    const Cost& k = costs[c.D == 128][eight ? 2 : mx];
    const long long rows = ((long long)c.n_tokens * c.group + c.n_seqs - 1) / c.n_seqs, of = eight ? 8 : 16;
    const double items = (double)c.n_seqs * c.H * ((rows + of - 1) / of);
    const double keys = (double)pieces(c, rows < of ? rows : of, c.blk) * c.blk, each = items * keys / num_sms;       // each: of an SM
    const int warps = eight ? 16 : mx ? 12 : 8;
    const bool cut = keys > 64 * warps;                       // over CTAs
    const double part = (each > c.blk ? each : c.blk) / (32 * warps);
    return k.start + k.tile / kTileKeys * (cut || each > keys ? each : keys) + (cut ? k.join * (part < 1 ? part : 1) : 0) + k.item * items / num_sms +
           k.row * rows;
}

// Beside its start: a tile of each round of CTAs, more where a group has more than 128 rows; a
// round more; the parts, and their join.
inline double prompt_ns(const Call& c, int num_sms)
{
    struct Cost {
        double start, tile, join, part, round;
    };
    static const Cost costs[2][2][2] = {{{{8138, 1147, 1296, 332, 6223}, {13135, 1419, 777, 337, 9764}},
                                         {{8560, 1321, 706, 363, 6330}, {13928, 1508, 0, 352, 10186}}},
                                        {{{10000, 1389, 1573, 352, 8060}, {18063, 1586, 1033, 327, 13407}},
                                         {{9864, 1538, 820, 356, 7581}, {18231, 1705, 325, 338, 13418}}}};
    const long long rows = ((long long)c.n_tokens * c.group + c.n_seqs - 1) / c.n_seqs;
    const Cost& k = costs[c.D == 128][c.fmt == MOE_KV_MXFP4][rows > 128];
    const long long groups = (long long)c.n_seqs * c.H * ((rows + kGroupRows - 1) / kGroupRows);
    const long long tiles = pieces(c, rows < kGroupRows ? rows : kGroupRows, kTileKeys);
    const PromptCut cut = prompt_cut(c, num_sms);
    const long long whole = groups < cut.whole ? groups : cut.whole, rounds = (whole + num_sms - 1) / num_sms;
    const bool rest = groups > whole;
    return k.start + k.tile * ((double)rounds * tiles + (rest ? (tiles + cut.parts - 1) / cut.parts : 0)) + k.round * (rounds + rest - 1) +
           (rest ? k.join + k.part * cut.parts : 0);
}

// The decode kernel where they are near one another: lengths that its runs of tiles happen to fit
// spare it half of the join.
inline bool takes_prompt_kernel(const Call& c, int num_sms) { return decode_ns(c, num_sms) > 1.0625 * prompt_ns(c, num_sms); }

}  // namespace attn
}  // namespace moe
