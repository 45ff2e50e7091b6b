// linear_plan.h -- how a call of moe_linear is split over warps, CTAs and passes,
// and the shared memory of each pass.  Plain C++: it is worked out on the host, and a
// test runs it there over every size that a call may have.
#pragma once
#include "../../include/moe.h"

namespace moe {
namespace linear {

constexpr int kWarps = 16;
constexpr int kRows = 16;
constexpr int kCols = 256;                 // columns of a stage
constexpr int kCodeBytes = kRows * kCols / 2;
constexpr int kXBytes = 112 * 1024;        // most of x that a CTA keeps
constexpr int kSmem = 224 * 1024;
constexpr int kLeastStages = 2;            // of a warp's ring: one is loaded while one is read
constexpr int kMostStages = 6;
constexpr int kCluster = 4;                // CTAs that share their rows, where they do

// Bytes of one row's scales in a stage, and the aligned 4-byte words that may hold them.
constexpr int scale_bytes(int fmt, int group) { return fmt == MOE_FMT_MXFP4 ? kCols / 32 : 2 * kCols / group; }
constexpr int scale_words(int fmt, int group) { return scale_bytes(fmt, group) / 4 + 1; }

struct Size {
    int N, K, fmt, group;   // weights
    int M;                  // tokens
};

struct Plan {
    int tokens;     // of this pass
    int cs;         // CTAs of a cluster, which share all rows: each takes `steps` stages of columns
    int steps;
    int ks;         // warps of a CTA that share 16 rows
    int stages;
    int x_pitch;    // bytes of one token's x
    int off_sum, off_fac, off_red, off_join, off_ring;
    int stage_bytes;
    int smem() const { return off_ring + kWarps * stages * stage_bytes; }
};

// The shared memory of p's split; false: what is left does not hold the rings.
inline bool lay_out(Plan& p, const Size& a)
{
    const int K = p.steps * kCols < a.K ? p.steps * kCols : a.K, nt = p.tokens > 8 ? 2 : 1;
    // pitch of 64 mod 128 bytes: two tokens' 64-byte pieces cover all banks
    p.x_pitch = (2 * K + 63) / 128 * 128 + 64;
    int off = p.tokens * p.x_pitch;
    p.off_sum = off;
    if (a.fmt == MOE_FMT_INT4)
        off = (off + p.tokens * (K / a.group) * 4 + 15) & ~15;
    p.off_fac = off;
    off += 256;                       // factors, largest magnitudes
    p.off_red = off;
    off += kWarps * nt * 512;
    p.off_join = off;
    if (p.cs > 1)
        off += 2 * ((kWarps / p.ks + p.cs - 1) / p.cs) * p.cs * nt * 512;
    p.off_ring = (off + 127) / 128 * 128;
    p.stage_bytes = kCodeBytes + (kRows * scale_words(a.fmt, a.group) * 4 + 127) / 128 * 128;
    p.stages = (kSmem - p.off_ring) / (kWarps * p.stage_bytes);
    if (p.stages > kMostStages)
        p.stages = kMostStages;
    return p.stages >= kLeastStages;
}

// Tokens of a pass (as many as fit in shared memory, 16 at most), the split of the
// columns and the shared memory for `ctas` groups of cs CTAs; returns what all
// passes are expected to take, in ns.  A round (every team's next 16 rows) costs
// 900 per stage of the busiest warp, 400 more for a second tile of tokens, some 700
// for a join in the CTA and 1,400 for one in the cluster; x costs 33 per KB that a
// CTA takes in.  Fitted to 512..60,000 rows of 512..8,192 columns for 1, 8 and 16
// tokens, every split: the choice is within 1 % of the best one on average, 12 % at
// worst.  Beyond those sizes it is an extrapolation: a cluster's join buffer, large
// where ks is small, then leaves no room for some of the splits.
inline long long plan(Plan& best, const Size& a, int cs, int ctas)
{
    const int units = (a.N + kRows - 1) / kRows, steps = (a.K + kCols - 1) / kCols;
    Plan p{};
    p.cs = cs;
    p.steps = (steps + cs - 1) / cs;
    const int K = p.steps * kCols < a.K ? p.steps * kCols : a.K;
    const int most = kXBytes / (2 * K + 128) < 16 ? kXBytes / (2 * K + 128) : 16;
    for (p.tokens = a.M < most ? a.M : most; p.tokens > 0; --p.tokens) {
        long long least = -1;
        for (p.ks = 1; p.ks <= kWarps && p.ks <= p.steps; p.ks *= 2) {
            const long long teams = (long long)ctas * (kWarps / p.ks), rounds = (units + teams - 1) / teams;
            const int stages = (p.steps + p.ks - 1) / p.ks;
            const long long cost =
                rounds * (stages * (p.tokens <= 8 ? 900 : 1300) + (p.ks > 1 ? 700 + 33 * p.ks : 0) + (cs > 1 ? 1400 : 0));
            if ((least < 0 || cost < least) && lay_out(p, a)) {
                least = cost;
                best = p;
            }
        }
        if (least >= 0)
            return (a.M + p.tokens - 1) / p.tokens * (3500 + 33LL * p.tokens * K * 2 / 1024 + least);
    }
    best = Plan{};                    // (no size that moe_linear takes comes here)
    return 1LL << 62;
}

// The plan of a call's first pass: whole CTAs, or clusters that share the rows.
inline Plan choose(const Size& a, int num_sms, int clusters)
{
    Plan alone, shared;
    const long long cost = plan(alone, a, 1, num_sms);
    return clusters > 0 && a.K > kCols && plan(shared, a, kCluster, clusters) < cost ? shared : alone;
}

}  // namespace linear
}  // namespace moe
