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

// What a call is expected to take with each kernel, in ns.  Fitted to 9,400 calls of each: E4M3
// and 4 bits; 64 heads of 64 on 8, 16 of 64 on 2, 32 of 128 on 4 and on 8; 1 to 64 sequences of
// 130 to 16,000 keys, whole and within windows of 128 to 1,024; 1 to 100 tokens each.  Over them,
// and over 1,500 others (INT8, other heads, blocks and lengths that differ), the kernel that is
// taken is 1 % behind the better one on average, more than a tenth in one call of 27, nearly
// always the decode kernel.
// Rows are the average of a sequence's kv head, keys the bound of `pieces`.

// Beside its start: a tile of 128 keys of an item, over all SMs, or for an item that is not cut
// on one; the join of an item over CTAs, less where a CTA has not a tile for every warp; an item
// more for every SM; a sequence's row tiles, which one thread walks.
inline double decode_ns(const Call& c, int num_sms)
{
    struct Cost {
        double start, tile, join, item, row;
    };
    static const Cost costs[2][3] = {{{6962, 500, 7913, 1039, 15}, {7154, 471, 8684, 1079, 15}, {7540, 303, 10010, 609, 29}},
                                     {{7760, 657, 10372, 1884, 16}, {8900, 704, 12961, 2259, 15}, {7685, 463, 10688, 779, 126}}};
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
    static const Cost costs[2][2][2] = {{{{8577, 1131, 499, 380, 6242}, {12855, 1426, 304, 385, 11201}},
                                         {{8817, 1295, 403, 378, 6481}, {13593, 1490, 0, 373, 11846}}},
                                        {{{10453, 1369, 949, 352, 8113}, {17991, 1599, 153, 339, 8113}},
                                         {{10106, 1516, 611, 343, 7693}, {17747, 1730, 8, 311, 7693}}}};
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
