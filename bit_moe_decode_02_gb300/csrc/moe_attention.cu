// moe_attention.cu -- attention over the 8-bit paged cache.
//
// out_i = sum_j e^{s_ij - m_i} v_j / (sum_j e^{s_ij - m_i} + e^{sink - m_i}),
// s_ij = scale q_i . k_j over the keys j that token i sees: its own position
// and before it, and with a window only the last `window` of them.
//
// decode_attn_kernel: one pass over the keys with a running maximum and sum.
// Bound by HBM: every visible code byte is read once for the (token, head)
// rows that share it, 16 at a time (an m16n8k16 MMA's rows).
//  - Work.  A tile is one cache block of one item (sequence, 16-row tile, kv
//    head); all tiles of the call, in order, are cut into equal contiguous runs,
//    one for each group of warps, whatever the lengths: the lengths are on the
//    device, so the cut is made there.  Runs that end inside an item leave
//    partial results, which are joined in a fixed order (results do not depend
//    on timing): within a CTA, then by the last CTA to arrive at an item's
//    counter.
//  - Loads.  A block's K and V codes of one head are contiguous: one bulk copy
//    per tile into the group's ring (192 KB in flight per SM), its scales with
//    an 8-byte cp.async on the same barrier.
//  - Operands.  Codes are exact in f16, so both products are f16 MMAs with fp32
//    sums.  The order of the summed index of an MMA is free: d for Q K^T and
//    the tokens for P V are taken so that a thread's operand bytes are
//    contiguous (16 of K, 8 of the transposed V) and the scores a thread holds
//    are exactly the probabilities that it feeds to the second product.
//  - Scales.  K's multiplies the scores.  V's enters the exponent: O is kept in
//    units of a reference scale, p' = 2^(s - m + log2(vs / ref) + 6), and changes
//    unit only when a block's scale leaves [ref / 2, 2 ref]; the running maximum
//    likewise moves only when a score passes it by 2^8.  So p' <= 2^15 in f16, and
//    what its subnormals lose of p is below 2^-31 a key: 2^20 keys lose less than the
//    output's rounding.
// Measured: 64 sequences of 12,000 tokens on average, 32 heads of 128 on 4 (INT8),
// 154 us, 5.35 TB/s of codes, 0.79 of a plain copy's rate.  Two warps a scheduler (230
// registers) are two chains of conversions and MMAs, which issue 0.4 instructions a
// cycle: that, not the loads in flight, is what is left.  One sequence of 4,300
// tokens, 64 heads of 64 on 8: 11.4 us, nearly all of it the way through: 1.9 us to
// find the tiles, 1.3 for the first loads, 0.9 for the tiles, a join in the CTA (1.1)
// and one over the CTAs (5); the same heads within a window of 128, 4 sequences: 7.0 us.
#include <cstdint>

#include "attn_device.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                 // rows of an item: (token, query head of the kv head) pairs
constexpr int kSub = 32;                  // tokens of a block that one warp takes

typedef long long i64;

// fp32 workspace: partial results of the groups' first and last items, then of the CTAs'.
constexpr int kMaxGroups = 8;
__host__ __device__ constexpr i64 slot_floats() { return kRows * 128 + 2 * kRows; }

struct Item {
    int b, c0, n, len;   // sequence
    int rt, h;           // row tile, kv head
    int jlo, jhi;        // its blocks
    int t0;              // its first tile
};

template <int BLK>
__device__ __forceinline__ void block_range(const AttnArgs& a, int n, int len, int rt, int& jlo, int& jhi)
{
    const int r0 = rt * kRows, r1 = min(r0 + kRows, n * a.group) - 1;
    const int p0 = len - n + r0 / a.group, p1 = len - n + r1 / a.group;
    jhi = p1 / BLK;
    jlo = a.window > 0 && p0 >= a.window ? (p0 - a.window + 1) / BLK : 0;
}

__device__ __forceinline__ int row_tiles(const AttnArgs& a, int n) { return (n * a.group + kRows - 1) / kRows; }

template <int BLK>
__device__ __forceinline__ i64 tiles_of(const AttnArgs& a, int b)
{
    int c0, n, len;
    if (!kv::sequence(a.c, b, c0, n, len)) {
        atomicExch(a.c.status, MOE_ERR_DEVICE_FAULT);
        return 0;
    }
    i64 t = 0;
#pragma unroll 1
    for (int rt = 0, nrt = row_tiles(a, n); rt < nrt; ++rt) {
        int lo, hi;
        block_range<BLK>(a, n, len, rt, lo, hi);
        t += hi - lo + 1;
    }
    return t * a.c.H;
}

// Sequence b's item that holds tile t >= pre[b].
template <int BLK>
__device__ __forceinline__ void item_in(const AttnArgs& a, const int* pre, int b, int t, Item& it)
{
    it.b = b;
    kv::sequence(a.c, b, it.c0, it.n, it.len);
    int at = pre[b];
#pragma unroll 1
    for (it.rt = 0;; ++it.rt) {
        block_range<BLK>(a, it.n, it.len, it.rt, it.jlo, it.jhi);
        const int here = (it.jhi - it.jlo + 1) * a.c.H;
        if (t < at + here)
            break;
        at += here;
    }
    const int nb = it.jhi - it.jlo + 1;
    it.h = (t - at) / nb;
    it.t0 = at + it.h * nb;
}

// The item that holds tile t, from the prefix sums of the sequences' tiles.
template <int BLK>
__device__ __forceinline__ void find_item(const AttnArgs& a, const int* pre, int t, Item& it)
{
    int lo = 0, hi = a.c.n_seqs;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    item_in<BLK>(a, pre, lo, t, it);
}

template <int BLK>
__device__ __forceinline__ void next_item(const AttnArgs& a, const int* pre, Item& it)
{
    it.t0 += it.jhi - it.jlo + 1;
    if (++it.h < a.c.H)
        return;
    it.h = 0;
    if (++it.rt < row_tiles(a, it.n)) {
        block_range<BLK>(a, it.n, it.len, it.rt, it.jlo, it.jhi);
        return;
    }
    int b = it.b + 1;
#pragma unroll 1
    while (pre[b + 1] <= it.t0)
        ++b;
    item_in<BLK>(a, pre, b, it.t0, it);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void group_sync(int id, int threads)
{
    if (threads == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Where row r of an item goes.
struct Place {
    int c0, r0, h;   // first token of the sequence in the batch, first row of the tile, kv head
    int nrows;
};
__device__ __forceinline__ void store_row4(const AttnArgs& a, const Place& p, int r, int col, float4 v, const Final& f)
{
    const int row = p.r0 + r, tok = p.c0 + row / a.group, hq = p.h * a.group + row % a.group;
    const i64 at = ((i64)tok * a.q_heads + hq) * a.c.D + col;
    uint2 o;
    o.x = tc::f2bf16_rne(v.x * f.mul) | (uint32_t)tc::f2bf16_rne(v.y * f.mul) << 16;
    o.y = tc::f2bf16_rne(v.z * f.mul) | (uint32_t)tc::f2bf16_rne(v.w * f.mul) << 16;
    *reinterpret_cast<uint2*>(a.out + at) = o;
    if (a.lse && col == 0)
        a.lse[(i64)tok * a.q_heads + hq] = f.lse;
}

// Partial results joined one after another.
struct Sum {
    float m = kNone, l = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
    __device__ __forceinline__ void add(float2 ml, float4 y)
    {
        const float mn = fmaxf(m, ml.x), w0 = ex2(m - mn), w1 = ex2(ml.x - mn);
        m = mn;
        l = l * w0 + ml.y * w1;
        v.x = v.x * w0 + y.x * w1, v.y = v.y * w0 + y.y * w1, v.z = v.z * w0 + y.z * w1, v.w = v.w * w0 + y.w * w1;
    }
    __device__ __forceinline__ void from_slot(const float* s, int D, int row, int col)
    {
        add(__ldcg(reinterpret_cast<const float2*>(s + kRows * D + 2 * row)), __ldcg(reinterpret_cast<const float4*>(s + row * D + col)));
    }
    __device__ __forceinline__ void to_slot(float* s, int D, int row, int col) const
    {
        __stcg(reinterpret_cast<float4*>(s + row * D + col), v);
        if (col == 0)
            __stcg(reinterpret_cast<float2*>(s + kRows * D + 2 * row), make_float2(m, l));
    }
};

// A group's part of an item that is left for the CTA to finish: its first one if
// that began in an earlier group's run (kSlot: joined over the group's warps, in
// the group's slot), and its last (kStage: the warps' results still lie in the
// stage that they read last).
enum { kSlot = 1, kStage = 2 };
struct Piece {
    int t0, t1;          // the item's tiles
    Place p;
    int where, stage;
};

template <int D, int FMT, int BLK>
struct Decode {
    static constexpr int GW = BLK / kSub;            // warps of a group
    static constexpr int NG = kWarps / GW;           // groups of a CTA
    static constexpr int STAGE = 2 * BLK * D;        // bytes of a tile
    static constexpr int NS = D == 64 ? 6 : 3;       // stages of a group's ring: 192 KB per CTA in all
    static constexpr int OFF_HDR = NG * NS * STAGE;                    // per stage: two scales, valid
    static constexpr int OFF_BAR = OFF_HDR + NG * NS * 16;
    static constexpr int OFF_ML = OFF_BAR + NG * NS * 16;              // full and empty barriers
    static constexpr int OFF_PIECE = OFF_ML + kWarps * kRows * 8;
    static constexpr int OFF_PRE = OFF_PIECE + NG * 2 * (int)sizeof(Piece);
    static constexpr int WHOLE = 2 * NG;             // items of at most so many tiles are not split over CTAs
    static constexpr int smem(int n_seqs) { return OFF_PRE + (n_seqs + 1) * 4; }
};

template <int D, int FMT, int BLK>
__global__ void __launch_bounds__(kThreads, 1) decode_attn_kernel(AttnArgs a, float* ws, unsigned* cnt)
{
    using C = Decode<D, FMT, BLK>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ i64 scan[kWarps];
    __shared__ int s_flag;
    int* pre = reinterpret_cast<int*>(sm + C::OFF_PRE);
    Piece* pieces = reinterpret_cast<Piece*>(sm + C::OFF_PIECE);
    float2* mls = reinterpret_cast<float2*>(sm + C::OFF_ML);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = warp / C::GW, sub = warp % C::GW;
    int* status = a.c.status;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR) + grp * C::NS * 2;
    uint64_t* empty = full + C::NS;
    if (sub == 0 && lane < C::NS) {
        tc::mbar_init(full + lane, 2);
        tc::mbar_init(empty + lane, C::GW);
    }
    if (tid < 2 * C::NG)
        pieces[tid].where = 0;

    // prefix sums of the sequences' tiles: up to four sequences a thread
    i64 all;
    {
        const int per = (a.c.n_seqs + kThreads - 1) / kThreads;
        i64 sum = 0;
#pragma unroll 1
        for (int i = 0; i < per; ++i)
            if (per * tid + i < a.c.n_seqs)
                sum += tiles_of<BLK>(a, per * tid + i);
        i64 incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const i64 x = __shfl_up_sync(~0u, incl, o);
            if (lane >= o)
                incl += x;
        }
        if (lane == 31)
            scan[warp] = incl;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncthreads();
        i64 at = incl - sum;
        all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            at += w < warp ? scan[w] : 0;
            all += scan[w];
        }
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int b = per * tid + i;
            if (b < a.c.n_seqs) {
                pre[b] = (int)at;
                if (per > 1)
                    at += tiles_of<BLK>(a, b);
            }
        }
        if (tid == 0)
            pre[a.c.n_seqs] = (int)all;
        __syncthreads();
    }
    if (all > 0x7fffffff) {                                   // more than 2^31 tiles of 4 KB at least
        if (tid == 0)
            atomicExch(status, MOE_ERR_DEVICE_FAULT);
        return;
    }
    const int N = (int)all, G = min((int)gridDim.x, N);       // CTAs with work
    if ((int)blockIdx.x >= G)
        return;
    // The CTA's run of tiles, its ends moved to the start of an item where that is
    // short: a join over CTAs costs more than two more tiles a group.  Lanes 0 and 1
    // look the ends' items up, the others that of the group's first tile should
    // neither end move; else all look again.
    const int each = N / G, more = N - each * G;              // CTA c begins with tile c each + min(c, more)
    int ct0 = blockIdx.x * each + min((int)blockIdx.x, more), ct1 = ct0 + each + ((int)blockIdx.x < more);
    int t_begin, t_end;
    auto share = [&]() {
        const int mine = (ct1 - ct0) / C::NG, left = (ct1 - ct0) % C::NG;
        t_begin = ct0 + grp * mine + min(grp, left);
        t_end = t_begin + mine + (grp < left);
    };
    share();
    Item it;
    int at = lane == 0 ? ct0 : lane == 1 ? ct1 : t_begin;
#pragma unroll 1
    for (bool again = false;; again = true) {
        find_item<BLK>(a, pre, min(at, N - 1), it);
        if (again)
            break;
        const int end = at < N && it.jhi - it.jlo + 1 <= C::WHOLE ? it.t0 : at, guess = t_begin;
        ct0 = __shfl_sync(~0u, end, 0);
        ct1 = __shfl_sync(~0u, end, 1);
        share();
        at = t_begin;
        if (at == guess)
            break;
    }
    if (ct0 == ct1)
        return;
    it.b = __shfl_sync(~0u, it.b, 2), it.c0 = __shfl_sync(~0u, it.c0, 2), it.n = __shfl_sync(~0u, it.n, 2);
    it.len = __shfl_sync(~0u, it.len, 2), it.rt = __shfl_sync(~0u, it.rt, 2), it.h = __shfl_sync(~0u, it.h, 2);
    it.jlo = __shfl_sync(~0u, it.jlo, 2), it.jhi = __shfl_sync(~0u, it.jhi, 2), it.t0 = __shfl_sync(~0u, it.t0, 2);
    const int gid = blockIdx.x * C::NG + grp;

    uint8_t* ring = sm + grp * C::NS * C::STAGE;
    float* hdr = reinterpret_cast<float*>(sm + C::OFF_HDR) + grp * C::NS * 4;
    const uint64_t pol = tc::l2_evict_first();
    float* slot = ws + (i64)(gridDim.x * 2 + gid) * slot_floats();                      // this group's

    // the tile stream: warp 0 of the group keeps its own place in it, NS - 1 tiles ahead
    Item pit{};
    int pt = t_begin, pj = 0, pid = 0, pst = 0, pround = 0;
    auto table_at = [&](const Item& it, int j) { return a.c.table[(i64)it.b * a.c.table_stride + j]; };
    auto produce = [&]() {
        const int st = pst;
        if (pround > 0)
            tc::mbar_wait(empty + st, (uint32_t)((pround - 1) & 1), status);
        if (++pst == C::NS) {
            pst = 0;
            ++pround;
        }
        const bool valid = pid >= 0 && pid < a.c.num_blocks;
        if (lane == 0) {
            float* hd = hdr + st * 4;
            hd[2] = valid ? 1.0f : 0.0f;
            if (valid) {
                const i64 at = ((i64)pid * a.c.H + pit.h) * 2;
                tc::mbar_expect_tx(full + st, C::STAGE);
                tc::bulk_copy_hint(ring + st * C::STAGE, a.c.codes + at * (BLK * D), C::STAGE, full + st, pol);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::su32(hd)), "l"(a.c.scales + at) : "memory");
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::su32(full + st)) : "memory");
            } else {
                atomicExch(status, MOE_ERR_DEVICE_FAULT);
                tc::mbar_arrive(full + st);
                tc::mbar_arrive(full + st);
            }
        }
        __syncwarp();
        if (++pt < t_end) {
            if (++pj > pit.jhi) {
                next_item<BLK>(a, pre, pit);
                pj = pit.jlo;
            }
            pid = table_at(pit, pj);     // used by the next call, a tile later
        }
    };

    // at first all of the ring, then the stage of the tile before
    auto fill = [&](int t) {
        if (sub == 0)
#pragma unroll 1
            while (pt < t_end && pt < t + C::NS)
                produce();
    };

    if (t_begin < t_end) {
        int j = it.jlo + t_begin - it.t0;
        if (sub == 0) {
            pit = it;
            pj = j;
            pid = table_at(it, j);
        }
        const int r = lane >> 2, c = lane & 3;
        int t = t_begin, cst = 0;
        uint32_t phase = 0;
        while (t < t_end) {
            // ---- an item, or the part of it in this group's run
            const int item_end = it.t0 + it.jhi - it.jlo + 1, seg_end = min(item_end, t_end);
            const int rows = min(kRows, it.n * a.group - it.rt * kRows);
            uint32_t qf[D / 16][4];
            float f[2];                  // score = sum * block's scale * f
            int plo[2], phi[2];          // first and last visible position of this thread's two rows
            uint32_t qw[2][D / 64][8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = it.rt * kRows + r + 8 * e, i = row / a.group;
                const bool in = r + 8 * e < rows;
                phi[e] = in ? it.len - it.n + i : -1;
                plo[e] = in && a.window > 0 ? phi[e] - a.window + 1 : 0;
                uint32_t (&w)[D / 64][8] = qw[e];
                if (in) {
                    const uint16_t* q = a.q + (i64)(it.c0 + i) * a.q_stride + (i64)(it.h * a.group + row % a.group) * D + 16 * c;
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch) {
                        const uint4 x = *reinterpret_cast<const uint4*>(q + 64 * ch), y = *reinterpret_cast<const uint4*>(q + 64 * ch + 8);
                        w[ch][0] = x.x, w[ch][1] = x.y, w[ch][2] = x.z, w[ch][3] = x.w;
                        w[ch][4] = y.x, w[ch][5] = y.y, w[ch][6] = y.z, w[ch][7] = y.w;
                    }
                } else {
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[ch][k] = 0;
                }
            }
            // the ring is filled while they are on their way
            fill(t);
            {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t big = 0;    // largest finite magnitude of the row
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            big = max(big, big_of(qw[e][ch][k]));
                    big = max(big, __shfl_xor_sync(~0u, big, 1));
                    big = max(big, __shfl_xor_sync(~0u, big, 2));
                    const RowScale rs = row_scale(big, a.scale);
                    f[e] = rs.f;
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            qf[ch * 4 + k / 2][(k & 1) * 2 + e] = scale_pair(qw[e][ch][k], rs);
                }
            }
            float o[D / 8][4], m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[i][k] = 0.0f;
            float ref = 0.0f, vmax = 0.0f;
            // positions that every row of the tile sees
            const int all_lo = a.window > 0 ? it.len - it.n + (it.rt * kRows + rows - 1) / a.group - a.window + 1 : 0;
            const int all_hi = it.len - it.n + it.rt * kRows / a.group;

            int st = 0;
            for (; t < seg_end; ++t, ++j) {
                fill(t);
                st = cst;
                tc::mbar_wait(full + st, phase, status);
                if (++cst == C::NS) {
                    cst = 0;
                    phase ^= 1;
                }
                const float4 hd = *reinterpret_cast<const float4*>(hdr + st * 4);
                const uint8_t* kt = ring + st * C::STAGE + sub * kSub * D;
                const uint8_t* vt = ring + st * C::STAGE + BLK * D + sub * kSub;
                const int p0 = j * BLK + sub * kSub;     // position of this warp's first token
                if (hd.z != 0.0f) {
                    float s[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            s[i][k] = 0.0f;
                    // token of column n of score tile i: 8 (n / 2) + 2 i + n % 2
                    const uint8_t* kp = kt + (8 * (r >> 1) + (r & 1)) * D + 16 * c;
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch) {
                        uint4 kw[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            kw[i] = *reinterpret_cast<const uint4*>(kp + 2 * i * D + 64 * ch);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t w = k == 0 ? kw[i].x : k == 1 ? kw[i].y : k == 2 ? kw[i].z : kw[i].w;
                                uint32_t b0, b1;
                                to_f16<FMT>(w, b0, b1);
                                mma16816(s[i], qf[ch * 4 + k], b0, b1);
                            }
                    }
                    const float cs[2] = {hd.x * f[0], hd.x * f[1]};
                    const bool whole = p0 >= all_lo && p0 + kSub - 1 <= all_hi;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            s[i][k] *= cs[k >> 1];
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int p = p0 + 8 * c + 2 * i + (k & 1), e = k >> 1;
                                if (p < plo[e] || p > phi[e])
                                    s[i][k] = -INFINITY;
                            }
                    }
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k >> 1] = fmaxf(mx[k >> 1], s[i][k]);
                    const float vs = hd.y;
                    const bool unit = !(vs <= 2.0f * ref && vs >= 0.5f * ref);
                    if (__any_sync(~0u, unit || mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
                        // a new maximum, or a new unit of O
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 1));
                            mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 2));
                            const float mn = fmaxf(m[e], mx[e]);
                            al[e] = ex2(m[e] - mn);
                            m[e] = mn;
                            l[e] *= al[e];
                        }
                        if (unit) {
                            vmax = fmaxf(vmax, vs);
                            const float now = new_unit(vs, vmax);
                            const float ch = ref / now;
                            ref = now;
                            al[0] *= ch;
                            al[1] *= ch;
                        }
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[i][0] *= al[0];
                            o[i][1] *= al[0];
                            o[i][2] *= al[1];
                            o[i][3] *= al[1];
                        }
                    }
                    const float ratio = fmaxf(vs / ref, 8.673617379884035e-19f);   // 2^-60
                    const float lr = __log2f(ratio) + kRoom, back = 1.0f / ratio;
                    const float mm[2] = {m[0] - lr, m[1] - lr};
                    float sum[2] = {0.0f, 0.0f};
                    uint32_t pf[2][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            p[k] = ex2(s[i][k] - mm[k >> 1]);
                            sum[k >> 1] += p[k];
                        }
                        pf[i >> 1][(i & 1) * 2] = pack_f16(p[0], p[1]);
                        pf[i >> 1][(i & 1) * 2 + 1] = pack_f16(p[2], p[3]);
                    }
                    l[0] += sum[0] * back;
                    l[1] += sum[1] * back;
                    const uint8_t* vp = vt + r * BLK + 8 * c;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint2 w = *reinterpret_cast<const uint2*>(vp + 8 * i * BLK);
                        uint32_t b0, b1;
                        to_f16<FMT>(w.x, b0, b1);
                        mma16816(o[i], pf[0], b0, b1);
                        to_f16<FMT>(w.y, b0, b1);
                        mma16816(o[i], pf[1], b0, b1);
                    }
                }
                if (t + 1 < seg_end) {
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive(empty + st);
                }
            }

            // ---- join the group's warps in the stage they have just read
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(~0u, l[e], 1);
                l[e] += __shfl_xor_sync(~0u, l[e], 2);
                if (c == 0)
                    mls[warp * kRows + r + 8 * e] = make_float2(m[e], l[e] * kUnroom);
            }
            group_sync(1 + grp, C::GW * 32);
            float* od = reinterpret_cast<float*>(ring + st * C::STAGE);
            const float unit = ref * kUnroom;
            // column group i of row x lies at i ^ (x % 8)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(od + (sub * kRows + r + 8 * e) * D + (i ^ r) * 8 + 2 * c) =
                        make_float2(o[i][2 * e] * unit, o[i][2 * e + 1] * unit);
            const Place place{it.c0, it.rt * kRows, it.h, rows};
            if (t == t_end) {
                // the group's last: finished with the CTA's others
                if (sub == 0 && lane == 0)
                    pieces[grp * 2 + 1] = Piece{it.t0, item_end, place, kStage, st};
                break;
            }
            group_sync(1 + grp, C::GW * 32);
            const bool done = it.t0 >= t_begin;
            for (int x = sub * 32 + lane; x < rows * (D / 4); x += C::GW * 32) {
                const int row = x / (D / 4), col = x % (D / 4) * 4;
                Sum sum;
#pragma unroll
                for (int w = 0; w < C::GW; ++w)
                    sum.add(mls[(grp * C::GW + w) * kRows + row],
                            *reinterpret_cast<const float4*>(od + (w * kRows + row) * D + ((col >> 3) ^ (row & 7)) * 8 + (col & 7)));
                if (done)
                    store_row4(a, place, row, col, sum.v, finish(sum.m, sum.l, a.sinks, it.h * a.group + (place.r0 + row) % a.group));
                else
                    sum.to_slot(slot, D, row, col);
            }
            if (!done && sub == 0 && lane == 0)
                pieces[grp * 2] = Piece{it.t0, item_end, place, kSlot, 0};
            tc::fence_proxy_async_smem();
            group_sync(1 + grp, C::GW * 32);
            if (lane == 0)
                tc::mbar_arrive(empty + st);
            next_item<BLK>(a, pre, it);
            j = it.jlo;
        }
    }

    // ---- finish the groups' pieces, in the order of their tiles
    __threadfence_block();
    __syncthreads();
    const float* gslots = ws + ((i64)gridDim.x * 2 + (i64)blockIdx.x * C::NG) * slot_floats();
    float* cslots = ws + (i64)blockIdx.x * 2 * slot_floats();
    int across = 0, cross[2] = {0, 0};
    // a piece a lane
    const Piece own = pieces[min(lane, 2 * C::NG - 1)];
    unsigned open = __ballot_sync(~0u, lane < 2 * C::NG && own.where);
    while (open) {
        const int first = __ffs(open) - 1, t0 = __shfl_sync(~0u, own.t0, first), t1 = __shfl_sync(~0u, own.t1, first);
        const Place place{__shfl_sync(~0u, own.p.c0, first), __shfl_sync(~0u, own.p.r0, first), __shfl_sync(~0u, own.p.h, first),
                          __shfl_sync(~0u, own.p.nrows, first)};
        // the item's pieces: the last ones of some groups, in their stages, and the first of
        // the next one, in its slot; or that alone
        const bool of_it = (open >> lane & 1) && own.t0 == t0;
        open &= ~__ballot_sync(~0u, of_it);
        const unsigned in_slot = __ballot_sync(~0u, of_it && own.where == kSlot);
        const int slot_at = in_slot ? (__ffs(in_slot) - 1) >> 1 : -1;
        // the warps whose results lie in their groups' stages, a lane each
        const int piece_of = (lane & (kWarps - 1)) / C::GW * 2 + 1, stage = __shfl_sync(~0u, own.stage, piece_of);
        const unsigned staged = __ballot_sync(~0u, of_it && own.where == kStage);
        const unsigned warps = __ballot_sync(~0u, lane < kWarps && (staged >> piece_of & 1));
        int ods[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            ods[w] = (w / C::GW * C::NS + __shfl_sync(~0u, stage, w)) * C::STAGE + w % C::GW * (kRows * D * 4);
        const bool done = t0 >= ct0 && t1 <= ct1;
        const int which = t0 < ct0 ? 0 : 1;
        for (int x = tid; x < place.nrows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), col = x % (D / 4) * 4, at = row * D + ((col >> 3) ^ (row & 7)) * 8 + (col & 7);
            Sum sum;
            if (slot_at >= 0)
                sum.from_slot(gslots + slot_at * slot_floats(), D, row, col);
            // all maxima first: the parts' weights then do not wait for one another
            float2 ml[kWarps];
            float M = sum.m;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = mls[w * kRows + row];
                if (!(warps >> w & 1))
                    ml[w] = make_float2(kNone, 0.0f);
                M = fmaxf(M, ml[w].x);
            }
            const float keep = ex2(sum.m - M);
            sum.m = M;
            sum.l *= keep;
            sum.v.x *= keep, sum.v.y *= keep, sum.v.z *= keep, sum.v.w *= keep;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (warps >> w & 1) {
                    const float4 y = *reinterpret_cast<const float4*>(sm + ods[w] + at * 4);
                    const float f = ex2(ml[w].x - M);
                    sum.l += ml[w].y * f;
                    sum.v.x += y.x * f, sum.v.y += y.y * f, sum.v.z += y.z * f, sum.v.w += y.w * f;
                }
            if (done)
                store_row4(a, place, row, col, sum.v, finish(sum.m, sum.l, a.sinks, place.h * a.group + (place.r0 + row) % a.group));
            else
                sum.to_slot(cslots + which * slot_floats(), D, row, col);
        }
        if (!done) {
            across |= 1 << which;
            cross[which] = first;
        }
    }

    // ---- items that span CTAs: the last one to arrive joins them all
    auto cta_of = [&](int t) {
        const int big = more * (each + 1);
        return t < big ? t / (each + 1) : more + (t - big) / each;
    };
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (!(across >> which & 1))
            continue;
        const Piece& p = pieces[cross[which]];
        const Place place = p.p;
        const int ca = cta_of(p.t0), cb = cta_of(p.t1 - 1);               // of its first and last tile
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            const unsigned old = atomicAdd(cnt + ca, 1u);
            s_flag = old == (unsigned)(cb - ca);
            if (s_flag)
                cnt[ca] = 0;
        }
        __syncthreads();
        if (!s_flag)
            continue;
        __threadfence();
        // maxima and sums of every part and row, then their weights, in the ring; every 4
        // columns' parts are summed by `split` threads, then those.  The first parts are
        // on their way while the weights are worked out
        const int K = cb - ca + 1, rows = place.nrows, n4 = rows * (D / 4), split = n4 <= kThreads / 2 ? kThreads / n4 : 1;
        float2* part = reinterpret_cast<float2*>(sm);                    // [K][kRows]; .x becomes the weight
        float2* total = part + gridDim.x * kRows;                        // [kRows]
        float4* acc = reinterpret_cast<float4*>(total + kRows);          // [kThreads]
        auto slot_of = [&](int k) { return ws + ((i64)(ca + k) * 2 + (k == 0)) * slot_floats(); };
        constexpr int AHEAD = 8;
        float4 y[AHEAD];
        auto load_parts = [&](int x, int k0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (x < n4 && k0 + i * split < K)
                    y[i] = __ldcg(reinterpret_cast<const float4*>(slot_of(k0 + i * split) + 4 * x));
        };
        const int from = split > 1 ? tid / n4 : 0, x_first = split > 1 ? (from < split ? tid % n4 : n4) : tid;
        load_parts(x_first, from);
        for (int i = tid; i < K * rows; i += kThreads)
            part[i / rows * kRows + i % rows] = __ldcg(reinterpret_cast<const float2*>(slot_of(i / rows) + kRows * D + 2 * (i % rows)));
        __syncthreads();
        // a warp takes a row, its lanes the parts
        for (int row = warp; row < rows; row += kWarps) {
            float M = kNone, L = 0.0f;
            for (int k = lane; k < K; k += 32)
                M = fmaxf(M, part[k * kRows + row].x);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
            for (int k = lane; k < K; k += 32) {
                const float2 ml = part[k * kRows + row];
                const float f = ex2(ml.x - M);
                L += ml.y * f;
                part[k * kRows + row].x = f;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                L += __shfl_xor_sync(~0u, L, o);
            if (lane == 0)
                total[row] = make_float2(M, L);
        }
        __syncthreads();
        for (int x0 = 0; x0 < n4; x0 += kThreads) {
            const int x = x0 + x_first, row = x / (D / 4), col = x % (D / 4) * 4;
            float4 v = make_float4(0, 0, 0, 0);
            if (x0)
                load_parts(x, from);
            if (x < n4)
                for (int k0 = from; k0 < K;) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
                        if (k0 + i * split < K) {
                            const float w = part[(k0 + i * split) * kRows + row].x;
                            v.x += y[i].x * w, v.y += y[i].y * w, v.z += y[i].z * w, v.w += y[i].w * w;
                        }
                    k0 += AHEAD * split;
                    load_parts(x, k0);
                }
            if (split > 1) {
                acc[tid] = v;
                __syncthreads();
                if (tid < n4)
                    for (int f = 1; f < split; ++f) {
                        const float4 y = acc[f * n4 + tid];
                        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                    }
            }
            if (x < n4 && from == 0)
                store_row4(a, place, row, col, v, finish(total[row].x, total[row].y, a.sinks, place.h * a.group + (place.r0 + row) % a.group));
        }
        __syncthreads();
    }
}

template <int D, int FMT, int BLK>
cudaError_t prepare_one()
{
    return cudaFuncSetAttribute(decode_attn_kernel<D, FMT, BLK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Decode<D, FMT, BLK>::smem(kMaxSeqs));
}

template <int D, int FMT>
cudaError_t prepare_blocks()
{
    cudaError_t e;
    if ((e = prepare_one<D, FMT, 32>()) != cudaSuccess || (e = prepare_one<D, FMT, 64>()) != cudaSuccess)
        return e;
    return prepare_one<D, FMT, 128>();
}

template <int D, int FMT, int BLK>
void launch_one(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    unsigned* cnt = reinterpret_cast<unsigned*>(a.ws);
    decode_attn_kernel<D, FMT, BLK><<<num_sms, kThreads, Decode<D, FMT, BLK>::smem(a.c.n_seqs), s>>>(
        a, reinterpret_cast<float*>(a.ws + kCounterBytes), cnt);
}

template <int D, int FMT>
void launch_blocks(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    if (a.c.blk == 32)
        launch_one<D, FMT, 32>(a, num_sms, s);
    else if (a.c.blk == 64)
        launch_one<D, FMT, 64>(a, num_sms, s);
    else
        launch_one<D, FMT, 128>(a, num_sms, s);
}

}  // namespace

size_t attention_workspace_bytes(int num_sms)
{
    return kCounterBytes + (size_t)num_sms * (2 + kMaxGroups) * slot_floats() * sizeof(float);
}

cudaError_t prepare_attention_kernels()
{
    cudaError_t e;
    if ((e = prepare_blocks<64, MOE_KV_E4M3>()) != cudaSuccess || (e = prepare_blocks<64, MOE_KV_INT8>()) != cudaSuccess ||
        (e = prepare_blocks<128, MOE_KV_E4M3>()) != cudaSuccess)
        return e;
    if ((e = prepare_blocks<128, MOE_KV_INT8>()) != cudaSuccess)
        return e;
    return prepare_prompt_kernels();
}

static cudaError_t launch_attention_decode(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    if (a.c.D == 64)
        a.c.fmt == MOE_KV_E4M3 ? launch_blocks<64, MOE_KV_E4M3>(a, num_sms, s) : launch_blocks<64, MOE_KV_INT8>(a, num_sms, s);
    else
        a.c.fmt == MOE_KV_E4M3 ? launch_blocks<128, MOE_KV_E4M3>(a, num_sms, s) : launch_blocks<128, MOE_KV_INT8>(a, num_sms, s);
    return cudaGetLastError();
}

cudaError_t launch_attention(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    // Against 128 keys the decode kernel spends 0.62 us of an SM on 16 rows (D = 64;
    // 0.86 for 128), spread over all SMs; the prompt kernel 1.45 us (2.2) on up to
    // 128 rows and 1.4 times that on 256, on one SM each.  The ratio is 2.3 to 2.6,
    // taken as 2.5.  Measured, decode / prompt kernel: 8 sequences of 4,000 keys, 64
    // heads of 64 on 8: 64 rows 48 / 68 us, 106 rows 74 / 73, 217 rows 133 / 88; one
    // such sequence, 432 rows: 57 / 81; 64 of them, 32 rows 140 / 180, 64 rows 263 / 182.
    // The lengths are on the device, so the rule sees their average alone.  The same heads, 63
    // single tokens and a prompt of 1,000 over 4,000 keys each: 267 us in one call, 80 + 117
    // in two; 255 and a prompt of 600 over 1,000 keys: 213 us, 88 + 27 in two.
    const long long rows = ((long long)a.c.n_tokens * a.group + a.c.n_seqs - 1) / a.c.n_seqs;     // of a sequence's kv head, on average
    const long long heads = (long long)a.c.n_seqs * a.c.H, waves = (heads * ((rows + 255) / 256) + num_sms - 1) / num_sms;
    const long long decode = 10 * heads * ((rows + 15) / 16), prompt = (rows > 128 ? 35 : 25) * waves * num_sms;
    return decode > prompt ? launch_attention_prompt(a, num_sms, s) : launch_attention_decode(a, num_sms, s);
}

}  // namespace moe
