// moe_attention.cu -- attention over the paged cache, in 8 or 4 bits.
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
//    counter.  A part is its keys' weighted sum over a power of two, half to all of their
//    mean, with its maximum and sum of weights: the weighted sum itself may pass fp32's
//    range where no value does.
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
// 145 us, 5.7 TB/s of codes, 0.83 of a plain copy's rate.  Two warps a scheduler (230
// registers) are two chains of conversions and MMAs, which issue 0.4 instructions a
// cycle: that, not the loads in flight, is what is left.  One sequence of 4,300
// tokens, 64 heads of 64 on 8: 11.8 us, nearly all of it the way through: 1.9 us to
// find the tiles, 1.3 for the first loads, 0.9 for the tiles, a join in the CTA (1.1)
// and one over the CTAs (5); the same heads within a window of 128, 4 sequences: 7.2 us.
// Lengths differ by more than their keys: of 700 to 9,000 tokens most take 14 to 18 us and
// one in four 10 to 12, by where the runs of tiles meet the items' ends.
// In 4 bits (mx_tile): the 64 sequences take 99 us, 4.4 TB/s (0.65 of a copy), bound by
// issue: 630 instructions for 32 keys and 8 rows at 0.55 a cycle, of which the conversions
// (one for two codes, at half rate) and products with scales are a third.  With items of 16
// rows, as in 8 bits, and 12 warps 149 us, with 8 warps 159; one sequence of 6,070 tokens
// 11.7 us, the same way through.
#include <algorithm>
#include <cstdint>

#include "attn_device.cuh"
#include "kv4_device.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kRows = 16;                 // rows of an item: (token, query head of the kv head) pairs
constexpr int kSub = 32;                  // tokens of a block that one warp takes

typedef long long i64;

// fp32 workspace: partial results of the groups' first and last items, then of the CTAs'.
constexpr int kMaxGroups = 16;
__host__ __device__ constexpr i64 slot_floats() { return kRows * 128 + 2 * kRows; }

struct Item {
    int b, c0, n, len;   // sequence
    int rt, h;           // row tile, kv head
    int jlo, jhi;        // its blocks
    int t0;              // its first tile
};

template <int BLK, int R>
__device__ __forceinline__ void block_range(const AttnArgs& a, int n, int len, int rt, int& jlo, int& jhi)
{
    const int r0 = rt * R, r1 = min(r0 + R, n * a.group) - 1;
    const int p0 = len - n + r0 / a.group, p1 = len - n + r1 / a.group;
    jhi = p1 / BLK;
    jlo = a.window > 0 && p0 >= a.window ? (p0 - a.window + 1) / BLK : 0;
}

template <int R>
__device__ __forceinline__ int row_tiles(const AttnArgs& a, int n) { return (n * a.group + R - 1) / R; }

template <int BLK, int R>
__device__ __forceinline__ i64 tiles_of(const AttnArgs& a, int b)
{
    int c0, n, len;
    if (!kv::sequence(a.c, b, c0, n, len)) {
        atomicExch(a.c.status, MOE_ERR_DEVICE_FAULT);
        return 0;
    }
    i64 t = 0;
#pragma unroll 1
    for (int rt = 0, nrt = row_tiles<R>(a, n); rt < nrt; ++rt) {
        int lo, hi;
        block_range<BLK, R>(a, n, len, rt, lo, hi);
        t += hi - lo + 1;
    }
    return t * a.c.H;
}

// Sequence b's item that holds tile t >= pre[b].
template <int BLK, int R>
__device__ __forceinline__ void item_in(const AttnArgs& a, const int* pre, int b, int t, Item& it)
{
    it.b = b;
    kv::sequence(a.c, b, it.c0, it.n, it.len);
    int at = pre[b];
#pragma unroll 1
    for (it.rt = 0;; ++it.rt) {
        block_range<BLK, R>(a, it.n, it.len, it.rt, it.jlo, it.jhi);
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
template <int BLK, int R>
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
    item_in<BLK, R>(a, pre, lo, t, it);
}

template <int BLK, int R>
__device__ __forceinline__ void next_item(const AttnArgs& a, const int* pre, Item& it)
{
    it.t0 += it.jhi - it.jlo + 1;
    if (++it.h < a.c.H)
        return;
    it.h = 0;
    if (++it.rt < row_tiles<R>(a, it.n)) {
        block_range<BLK, R>(a, it.n, it.len, it.rt, it.jlo, it.jhi);
        return;
    }
    int b = it.b + 1;
#pragma unroll 1
    while (pre[b + 1] <= it.t0)
        ++b;
    item_in<BLK, R>(a, pre, b, it.t0, it);
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

// A partial result: four columns of a row, as attn_device.cuh keeps them.
__device__ __forceinline__ void to_slot(float* s, int D, int row, int col, float m, float l, float4 v)
{
    __stcg(reinterpret_cast<float4*>(s + row * D + col), v);
    if (col == 0)
        __stcg(reinterpret_cast<float2*>(s + kRows * D + 2 * row), make_float2(m, l));
}

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

template <int D, int FMT, int BLK, int R>
struct Decode {
    static constexpr bool MX = FMT == MOE_KV_MXFP4;
    static constexpr int WARPS = R == 8 ? 16 : MX ? 12 : 8, THREADS = WARPS * 32;
    static constexpr int GW = BLK / kSub;            // warps of a group
    static constexpr int NG = WARPS / GW;            // groups of a CTA
    static constexpr int RECORD = MX ? kv4::record(BLK, D) : BLK * D;  // bytes of K or V of a block
    static constexpr int STAGE = 2 * RECORD;         // bytes of a tile
    // stages of a group's ring: 192 KB per CTA in all; MXFP4: 157 KB (139 for items of 8 rows), and 64
    // columns of the warps' O where an item ends within a run (in 8 bits, and at a run's end, they go
    // into the ring)
    static constexpr int NS = R == 8 ? (D == 64 ? 4 : 2) : D == 64 ? 6 : 3;
    static constexpr int OFF_O = NG * NS * STAGE;                      // [WARPS][R][64] fp32
    static constexpr int OFF_VS = OFF_O + (MX ? WARPS * R * 64 * 4 : 0);       // [WARPS][D / 32][kSub] f16
    static constexpr int OFF_HDR = OFF_VS + (MX ? WARPS * D * 2 : 0); // per stage: two scales, valid
    static constexpr int OFF_BAR = OFF_HDR + NG * NS * 16;
    static constexpr int OFF_ML = OFF_BAR + NG * NS * 16;              // full and empty barriers
    static constexpr int OFF_PIECE = OFF_ML + WARPS * kRows * 8;
    static constexpr int OFF_PRE = OFF_PIECE + NG * 2 * (int)sizeof(Piece);
    static constexpr int WHOLE = 2 * NG;             // items of at most so many tiles are not split over CTAs
    static constexpr int smem(int n_seqs) { return OFF_PRE + (n_seqs + 1) * 4; }
};

// One warp's 32 tokens of a block in 4 bits: scores, running maximum, P V.
//  - K.  A key's codes become f16 times 2^(13 + e_g - e), e_g a group's exponent and e the
//    key's largest: exact down to 2^-27, and no key's size touches another's.  Its score
//    is then multiplied by 2^e.
//  - V.  A group's scale goes into P, 2^(e - unit), unit the exponent that the 32 columns
//    of O are kept in.  Scales within [unit - 7, unit + 1] go as they are; where one is
//    not, the unit moves to the largest, and what is more than 2^7 below goes in passes of
//    its own, each with a unit of its own.
template <int D, int BLK, int R>
__device__ __forceinline__ void mx_tile(const uint8_t* stage, int sub, uint8_t* scratch, const uint32_t (&qf)[D / 16][R / 4], const float (&f)[2],
                                        float (&o)[D * R / 128][4], float (&m)[2], float (&l)[2], int& unit, int& vmax, int p0, const int (&plo)[2],
                                        const int (&phi)[2], bool whole, int any_lo, int any_hi)
{
    constexpr int REC = kv4::record(BLK, D), G = D / 32, W = D / 32;       // W: words of a thread's codes of a key
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const uint8_t* kt = stage + sub * (kSub * D / 2);
    const uint8_t* ks = stage + BLK * D / 2 + sub * D;
    const uint8_t* vt = stage + REC + sub * (kSub * D / 2);
    const uint8_t* vs = stage + REC + BLK * D / 2 + sub * D;

    // this thread's four keys' scales (key of score tile i: 8 (r / 2) + 2 i + r % 2), two and two
    const uint32_t kb = *reinterpret_cast<const uint32_t*>(ks + (r * G + (D == 128 ? c : c >> 1)) * 4);
    uint32_t e2[2] = {kb & 0x00ff00ffu, kb >> 8 & 0x00ff00ffu}, top[2], col[2][2];
    uint32_t ksc[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        top[h] = e2[h];
        if (D == 128)
            top[h] = max2(top[h], __shfl_xor_sync(~0u, top[h], 1));
        top[h] = max2(top[h], __shfl_xor_sync(~0u, top[h], 2));
        // f16 2^(13 + e_g - e): exponent field 28 - (e - e_g), 0 where that is 28 or more
        const uint32_t x = (0x001c001cu - min2(top[h] - e2[h], 0x001c001cu)) << 10;
        ksc[h] = __byte_perm(x, 0, 0x1010);
        ksc[h + 2] = __byte_perm(x, 0, 0x3232);
        if constexpr (R == 16) {
            col[h][0] = __shfl_sync(~0u, top[h], 8 * c);
            col[h][1] = __shfl_sync(~0u, top[h], 8 * c + 4);
        }
    }
    constexpr int OT = D * R / 128;
    // a key's or a pair of keys' codes of this thread; the keys' own exponents, and those of the
    // keys whose scores it holds: of 16 rows 8 c + 2 i + j, of 8 its own four
    uint32_t w[4][W];
    {
        const uint8_t* kp = kt + (8 * (r >> 1) + (r & 1)) * (D / 2) + (D / 8) * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(kp + i * D);
                w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(kp + i * D);
                w[i][0] = x.x, w[i][1] = x.y;
            }
        }
    }
    // P, as the second product's operand: of 16 rows pf[i / 2][i % 2 * 2 + e], of 8 pf[0][i], for the
    // keys 8 c + 2 i, 8 c + 2 i + 1
    uint32_t pf[2][4];
    if constexpr (R == 8) {
        // keys in the MMA's 16 rows, queries in its 8 columns
        float s[4][2];                   // key 8 (r / 2) + 2 i + r % 2 by rows 2 c, 2 c + 1
        {
            float d[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
#pragma unroll
            for (int ch = 0; ch < W; ++ch)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[4], y[4];
                    kv4::to_f16(w[2 * i][ch], x);
                    kv4::to_f16(w[2 * i + 1][ch], y);
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint32_t ka[4] = {mul_f16(x[k], ksc[2 * i]), mul_f16(y[k], ksc[2 * i + 1]), mul_f16(x[k + 1], ksc[2 * i]),
                                                mul_f16(y[k + 1], ksc[2 * i + 1])};
                        mma16816(d[i], ka, qf[2 * ch + k / 2][0], qf[2 * ch + k / 2][1]);
                    }
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t e = top[i & 1];                 // a byte in each half: the upper one leaves the float at the top
                const float k = kv4::scale_of(i < 2 ? e : e >> 16);
                s[i][0] = d[i / 2][i % 2 * 2] * (k * f[0]);
                s[i][1] = d[i / 2][i % 2 * 2 + 1] * (k * f[1]);
            }
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = p0 + 8 * (r >> 1) + 2 * i + (r & 1);
                    if (p < plo[e] || p > phi[e])
                        s[i][e] = -INFINITY;
                }
        }
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            mx[e] = fmaxf(fmaxf(s[0][e], s[1][e]), fmaxf(s[2][e], s[3][e]));
        if (__any_sync(~0u, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1)
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], k));
                const float mn = fmaxf(m[e], mx[e]);
                al[e] = ex2(m[e] - mn);
                m[e] = mn;
                l[e] *= al[e];
            }
#pragma unroll
            for (int i = 0; i < OT; ++i) {
                o[i][0] *= al[0];
                o[i][1] *= al[1];
                o[i][2] *= al[0];
                o[i][3] *= al[1];
            }
        }
        const float mm[2] = {m[0] - kRoom, m[1] - kRoom};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = ex2(s[i][0] - mm[0]), y = ex2(s[i][1] - mm[1]);
            l[0] += x;
            l[1] += y;
            // keys r by rows -> rows r by keys 2 c, 2 c + 1 of the eight, which are 8 c + 2 i and the next
            asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pf[0][i]) : "r"(pack_f16(x, y)));
            pf[1][i] = 0;
        }
    } else {
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
        {
#pragma unroll
            for (int ch = 0; ch < W; ++ch)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h[4];
                    kv4::to_f16(w[i][ch], h);
                    mma16816(s[i], qf[2 * ch], mul_f16(h[0], ksc[i]), mul_f16(h[1], ksc[i]));
                    mma16816(s[i], qf[2 * ch + 1], mul_f16(h[2], ksc[i]), mul_f16(h[3], ksc[i]));
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t e = col[i & 1][j];
                const float k = kv4::scale_of(i < 2 ? e : e >> 16);
                s[i][j] *= k * f[0];
                s[i][2 + j] *= k * f[1];
            }
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
        if (__any_sync(~0u, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
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
#pragma unroll
            for (int i = 0; i < OT; ++i) {
                o[i][0] *= al[0];
                o[i][1] *= al[0];
                o[i][2] *= al[1];
                o[i][3] *= al[1];
            }
        }
        {
            const float mm[2] = {m[0] - kRoom, m[1] - kRoom};
            float sum[2] = {0.0f, 0.0f};
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
            l[0] += sum[0];
            l[1] += sum[1];
        }
    }

    // V's scales: four tokens' bytes of one group a lane, those that no row sees left out
    uint32_t vb = D == 128 || lane < 16 ? *reinterpret_cast<const uint32_t*>(vs + 4 * lane) : 0u;
    if (!whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = p0 + 4 * (lane & 7) + k;
            if (p < any_lo || p > any_hi)
                vb &= ~(0xffu << 8 * k);
        }
    }
#pragma unroll 1
    for (;;) {
        uint32_t x[2] = {__byte_perm(vb, 0, 0x4140), __byte_perm(vb, 0, 0x4342)};
        uint32_t left = 0;
        {
            // each byte but 0 within [unit - 7, unit + 1]?
            const uint32_t lo = (uint32_t)max(unit - 8, 0) * 0x10001u, hi = (uint32_t)(unit + 1) * 0x10001u;
            uint32_t below;
            asm("add.u16x2 %0, %1, %2;" : "=r"(below) : "r"(x[0]), "r"(0xffffffffu));
            uint32_t y;
            asm("add.u16x2 %0, %1, %2;" : "=r"(y) : "r"(x[1]), "r"(0xffffffffu));
            const bool out = min2(min2(below, y), lo) != lo || max2(max2(x[0], x[1]), hi) != hi;
            const unsigned outs = __ballot_sync(~0u, out);
            if (outs) {
                uint32_t big = max2(x[0], x[1]);
                big = max(big & 0xffffu, big >> 16);
                big = max(big, __shfl_xor_sync(~0u, big, 1));
                big = max(big, __shfl_xor_sync(~0u, big, 2));
                big = max(big, __shfl_xor_sync(~0u, big, 4));
                vmax = max(vmax, (int)big);
                const int was = unit;
                const int least = max(vmax - 80, 16);
                if ((outs >> (lane & 24) & 0xffu) && big > 0)
                    unit = max((int)big, least);
                const float by = ex2((float)max(was - unit, -126));
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float ch = __shfl_sync(~0u, by, 8 * g);
#pragma unroll
                    for (int i = OT / G * g; i < OT / G * (g + 1); ++i) {
                        o[i][0] *= ch;
                        o[i][1] *= ch;
                        o[i][2] *= ch;
                        o[i][3] *= ch;
                    }
                }
                // what is further below goes in a later pass, or is nothing beside the largest
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int b = vb >> 8 * k & 0xff;
                    if (b < unit - 7) {
                        x[k >> 1] &= ~(0xffffu << 16 * (k & 1));
                        if (b >= least - 7)
                            left |= (uint32_t)b << 8 * k;
                    }
                }
            }
        }
        // 2^(e - unit) in f16: exponent field e - unit + 15, 0 for no scale
        const uint32_t base = (uint32_t)max(unit - 15, 0) * 0x10001u;      // unit >= 16, or no scale yet
        const uint32_t z0 = (max2(x[0], base) - base) << 10, z1 = (max2(x[1], base) - base) << 10;
        __syncwarp();
        if (D == 128 || lane < 16)
            *reinterpret_cast<uint2*>(scratch + 8 * lane) = make_uint2(z0, z1);
        __syncwarp();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint4 z = *reinterpret_cast<const uint4*>(scratch + g * (kSub * 2) + c * 16);
            const uint4 w = *reinterpret_cast<const uint4*>(vt + (g * 32 + lane) * 16);
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
            if constexpr (R == 8) {
                const uint32_t p[4] = {mul_f16(pf[0][0], z.x), mul_f16(pf[0][1], z.y), mul_f16(pf[0][2], z.z), mul_f16(pf[0][3], z.w)};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint32_t x[4], y[4];
                    kv4::to_f16(words[e], x);
                    kv4::to_f16(words[e + 1], y);
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint32_t va[4] = {x[k], y[k], x[k + 1], y[k + 1]};
                        mma16816(o[2 * g + e / 2], va, p[k], p[k + 1]);
                    }
                }
                continue;
            }
            const uint32_t pa[4] = {mul_f16(pf[0][0], z.x), mul_f16(pf[0][1], z.x), mul_f16(pf[0][2], z.y), mul_f16(pf[0][3], z.y)};
            const uint32_t pb[4] = {mul_f16(pf[1][0], z.z), mul_f16(pf[1][1], z.z), mul_f16(pf[1][2], z.w), mul_f16(pf[1][3], z.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h[4];
                kv4::to_f16(words[e], h);
                mma16816(o[4 * g + e], pa, h[0], h[1]);
                mma16816(o[4 * g + e], pb, h[2], h[3]);
            }
        }
        if (!__any_sync(~0u, left))
            break;
        vb = left;
    }
}

template <int D, int FMT, int BLK, int R>
__global__ void __launch_bounds__((Decode<D, FMT, BLK, R>::THREADS), 1) decode_attn_kernel(AttnArgs a, float* ws, unsigned* cnt)
{
    using C = Decode<D, FMT, BLK, R>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ i64 scan[Decode<D, FMT, BLK, R>::WARPS];
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
        const int per = (a.c.n_seqs + C::THREADS - 1) / C::THREADS;
        i64 sum = 0;
#pragma unroll 1
        for (int i = 0; i < per; ++i)
            if (per * tid + i < a.c.n_seqs)
                sum += tiles_of<BLK, R>(a, per * tid + i);
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
        for (int w = 0; w < C::WARPS; ++w) {
            at += w < warp ? scan[w] : 0;
            all += scan[w];
        }
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int b = per * tid + i;
            if (b < a.c.n_seqs) {
                pre[b] = (int)at;
                if (per > 1)
                    at += tiles_of<BLK, R>(a, b);
            }
        }
        if (tid == 0)
            pre[a.c.n_seqs] = (int)all;
        __syncthreads();
    }
    if (all > 0x7fffffff) {                                   // (a tile is 2,176 bytes at least)
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
        find_item<BLK, R>(a, pre, min(at, N - 1), it);
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
        if (pround > 0 && !tc::mbar_try_wait(empty + st, (uint32_t)((pround - 1) & 1)))
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
                tc::bulk_copy_hint(ring + st * C::STAGE, a.c.codes + at * C::RECORD, C::STAGE, full + st, pol);
                if constexpr (C::MX) {
                    tc::mbar_arrive(full + st);
                } else {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::su32(hd)), "l"(a.c.scales + at) : "memory");
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::su32(full + st)) : "memory");
                }
            } else {
                atomicExch(status, MOE_ERR_DEVICE_FAULT);
                tc::mbar_arrive(full + st);
                tc::mbar_arrive(full + st);
            }
        }
        __syncwarp();
        if (++pt < t_end) {
            if (++pj > pit.jhi) {
                next_item<BLK, R>(a, pre, pit);
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
            const int rows = min(R, it.n * a.group - it.rt * R);
            // this thread's two rows: r and r + 8 of 16, 2 c and 2 c + 1 of 8
            auto my_row = [&](int e) { return R == 8 ? 2 * c + e : r + 8 * e; };
            uint32_t qf[D / 16][R / 4];
            float f[2];                  // score = sum * block's scale * f
            int plo[2], phi[2];          // first and last visible position of the rows
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool in = my_row(e) < rows;
                phi[e] = in ? it.len - it.n + (it.rt * R + my_row(e)) / a.group : -1;
                plo[e] = in && a.window > 0 ? phi[e] - a.window + 1 : 0;
            }
            constexpr int QR = R / 8;    // rows whose queries this thread holds a part of: r (and r + 8)
            uint32_t qw[QR][D / 64][8];
#pragma unroll
            for (int e = 0; e < QR; ++e) {
                const int row = it.rt * R + r + 8 * e, i = row / a.group;
                uint32_t (&w)[D / 64][8] = qw[e];
                if (r + 8 * e < rows) {
                    // which of the d's a thread takes: those of its 16 bytes of K's codes
                    constexpr int mine = C::MX ? D / 4 : 16, step = C::MX ? 16 : 64;
                    const uint16_t* q = a.q + (i64)(it.c0 + i) * a.q_stride + (i64)(it.h * a.group + row % a.group) * D + mine * c;
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch) {
                        const uint4 x = *reinterpret_cast<const uint4*>(q + step * ch), y = *reinterpret_cast<const uint4*>(q + step * ch + 8);
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
                for (int e = 0; e < QR; ++e) {
                    uint32_t big = 0;    // largest finite magnitude of the row
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            big = max(big, big_of(qw[e][ch][k]));
                    big = max(big, __shfl_xor_sync(~0u, big, 1));
                    big = max(big, __shfl_xor_sync(~0u, big, 2));
                    const RowScale rs = row_scale(big, a.scale);
                    f[e] = C::MX ? rs.f * 0x1p-13f : rs.f;       // K's f16 operands are 2^13 up there
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            qf[ch * 4 + k / 2][(k & 1) * QR + e] = scale_pair(qw[e][ch][k], rs);
                }
                if constexpr (R == 8) {
                    const float mine = f[0];
                    f[0] = __shfl_sync(~0u, mine, 8 * c);
                    f[1] = __shfl_sync(~0u, mine, 8 * c + 4);
                }
            }
            constexpr int OT = D * R / 128;      // tiles of O: 16 rows by 8 columns, or 16 columns by 8 rows
            float o[OT][4], m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < OT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[i][k] = 0.0f;
            float ref = 0.0f, vmax = 0.0f;
            // MXFP4: the unit of O's 32 columns of group g, as a scale byte, and the largest byte seen:
            // in the lanes that look after g's bytes
            int unit4 = 0, vmax4 = 0;
            // positions that every row of the tile sees
            const int all_lo = a.window > 0 ? it.len - it.n + (it.rt * R + rows - 1) / a.group - a.window + 1 : 0;
            const int all_hi = it.len - it.n + it.rt * R / a.group;
            // and that any does
            const int any_lo = a.window > 0 ? all_hi - a.window + 1 : 0;
            const int any_hi = it.len - it.n + (it.rt * R + rows - 1) / a.group;

            int st = 0;
            for (; t < seg_end; ++t, ++j) {
                fill(t);
                st = cst;
                if (!tc::mbar_try_wait(full + st, phase))
                    tc::mbar_wait(full + st, phase, status);
                if (++cst == C::NS) {
                    cst = 0;
                    phase ^= 1;
                }
                const float4 hd = *reinterpret_cast<const float4*>(hdr + st * 4);
                const uint8_t* kt = ring + st * C::STAGE + sub * kSub * D;
                const uint8_t* vt = ring + st * C::STAGE + BLK * D + sub * kSub;
                const int p0 = j * BLK + sub * kSub;     // position of this warp's first token
                if constexpr (C::MX) {
                    if (hd.z != 0.0f)
                        mx_tile<D, BLK, R>(ring + st * C::STAGE, sub, reinterpret_cast<uint8_t*>(sm + C::OFF_VS) + warp * (D * 2), qf, f, o, m, l,
                                        unit4, vmax4, p0, plo, phi, p0 >= all_lo && p0 + kSub - 1 <= all_hi, any_lo, any_hi);
                } else if (hd.z != 0.0f) {
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
            float by[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (R == 8) {
                    l[e] += __shfl_xor_sync(~0u, l[e], 4);
                    l[e] += __shfl_xor_sync(~0u, l[e], 8);
                    l[e] += __shfl_xor_sync(~0u, l[e], 16);
                } else {
                    l[e] += __shfl_xor_sync(~0u, l[e], 1);
                    l[e] += __shfl_xor_sync(~0u, l[e], 2);
                }
                if ((R == 8 ? r : c) == 0)
                    mls[warp * kRows + my_row(e)] = make_float2(m[e], l[e] * kUnroom);
                by[e] = pow2_under(l[e]) * kDown;      // of O, whose probabilities are as far up as l's
            }
            group_sync(1 + grp, C::GW * 32);
            // MXFP4: at a run's end nothing of the ring is wanted any more, and it holds all of O; else 64
            // columns at a time go beside it
            constexpr int PART = C::MX ? 64 : D;
            const bool ends = t == t_end;
            float* od = reinterpret_cast<float*>(!C::MX ? ring + st * C::STAGE : ends ? ring : sm + C::OFF_O + grp * C::GW * (R * PART * 4));
            float unit[D / 32];
#pragma unroll
            for (int g = 0; g < D / 32; ++g)
                unit[g] = C::MX ? kv4::scale_of(__shfl_sync(~0u, unit4, 8 * g)) : ref;
            const Place place{it.c0, it.rt * R, it.h, rows};
            const bool done = it.t0 >= t_begin;
            // column group i of row x lies at i ^ (x % 8)
            auto put = [&](int i0, int i1, int width) {
                if constexpr (R == 8) {
#pragma unroll
                    for (int i = 0; i < OT; ++i)
                        if (2 * i >= i0 && 2 * i < i1)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int row = 2 * c + (k & 1);
                                od[(sub * R + row) * width + ((2 * i + (k >> 1) - i0) ^ row) * 8 + r] = o[i][k] * by[k & 1] * unit[i / 2];
                            }
                } else {
#pragma unroll
                    for (int i = 0; i < OT; ++i)
                        if (i >= i0 && i < i1)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                *reinterpret_cast<float2*>(od + (sub * R + r + 8 * e) * width + ((i - i0) ^ r) * 8 + 2 * c) =
                                    make_float2(o[i][2 * e] * by[e] * unit[i / 4], o[i][2 * e + 1] * by[e] * unit[i / 4]);
                }
            };
            if (ends) {
                put(0, D / 8, D);
                // the group's last: finished with the CTA's others
                if (sub == 0 && lane == 0)
                    pieces[grp * 2 + 1] = Piece{it.t0, item_end, place, kStage, st};
                break;
            }
#pragma unroll
            for (int p = 0; p < D / PART; ++p) {
                if (p > 0)
                    group_sync(1 + grp, C::GW * 32);
                put(p * (PART / 8), (p + 1) * (PART / 8), PART);
                group_sync(1 + grp, C::GW * 32);
                for (int x = sub * 32 + lane; x < rows * (PART / 4); x += C::GW * 32) {
                    const int row = x / (PART / 4), col = x % (PART / 4) * 4;
                    float M = kNone, l = 0.0f, f[C::GW];
#pragma unroll
                    for (int w = 0; w < C::GW; ++w)
                        M = fmaxf(M, mls[(grp * C::GW + w) * kRows + row].x);
#pragma unroll
                    for (int w = 0; w < C::GW; ++w) {
                        const float2 ml = mls[(grp * C::GW + w) * kRows + row];
                        const float x = ex2(ml.x - M);
                        l += ml.y * x;
                        f[w] = pow2_in(ml.y) * x;
                    }
                    const float whole = pow2_under(l);
                    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int w = 0; w < C::GW; ++w) {
                        const float4 y = *reinterpret_cast<const float4*>(od + (w * R + row) * PART + ((col >> 3) ^ (row & 7)) * 8 + (col & 7));
                        const float x = f[w] * whole;
                        v.x += y.x * x, v.y += y.y * x, v.z += y.z * x, v.w += y.w * x;
                    }
                    if (done)
                        store_row4(a, place, row, p * PART + col, v, finish_mean(M, l, a.sinks, it.h * a.group + (place.r0 + row) % a.group));
                    else
                        to_slot(slot, D, row, p * PART + col, M, l, v);
                }
            }
            if (!done && sub == 0 && lane == 0)
                pieces[grp * 2] = Piece{it.t0, item_end, place, kSlot, 0};
            tc::fence_proxy_async_smem();
            group_sync(1 + grp, C::GW * 32);
            if (lane == 0)
                tc::mbar_arrive(empty + st);
            next_item<BLK, R>(a, pre, it);
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
        const int piece_of = min(lane, C::WARPS - 1) / C::GW * 2 + 1, stage = __shfl_sync(~0u, own.stage, piece_of);
        const unsigned staged = __ballot_sync(~0u, of_it && own.where == kStage);
        const unsigned warps = __ballot_sync(~0u, lane < C::WARPS && (staged >> piece_of & 1));
        int ods[C::WARPS];
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w)
            ods[w] = (w / C::GW * C::NS + (C::MX ? 0 : __shfl_sync(~0u, stage, w))) * C::STAGE + w % C::GW * (R * D * 4);
        const bool done = t0 >= ct0 && t1 <= ct1;
        const int which = t0 < ct0 ? 0 : 1;
        for (int x = tid; x < place.nrows * (D / 4); x += C::THREADS) {
            const int row = x / (D / 4), col = x % (D / 4) * 4, at = row * D + ((col >> 3) ^ (row & 7)) * 8 + (col & 7);
            // all maxima and sums first: the parts' weights then do not wait for one another
            float2 ml[C::WARPS], first_ml = make_float2(kNone, 0.0f);
            float4 v = make_float4(0, 0, 0, 0);
            if (slot_at >= 0) {
                const float* s = gslots + slot_at * slot_floats();
                first_ml = __ldcg(reinterpret_cast<const float2*>(s + kRows * D + 2 * row));
                v = __ldcg(reinterpret_cast<const float4*>(s + row * D + col));
            }
            float M = first_ml.x;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) {
                ml[w] = mls[w * kRows + row];
                if (!(warps >> w & 1))
                    ml[w] = make_float2(kNone, 0.0f);
                M = fmaxf(M, ml[w].x);
            }
            // (l added up in pairs in ml[w].y, the weights in ml[w].x)
            first_ml.x = ex2(first_ml.x - M);
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) {
                const float x = ex2(ml[w].x - M);
                ml[w].x = pow2_in(ml[w].y) * x;
                ml[w].y *= x;
            }
#pragma unroll
            for (int s = 1; s < C::WARPS; s *= 2)
#pragma unroll
                for (int w = 0; w + s < C::WARPS; w += 2 * s)
                    ml[w].y += ml[w + s].y;
            const float l = first_ml.y * first_ml.x + ml[0].y, whole = pow2_under(l), keep = pow2_in(first_ml.y) * first_ml.x * whole;
            v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w)
                if (warps >> w & 1) {
                    const float4 y = *reinterpret_cast<const float4*>(sm + ods[w] + at * 4);
                    const float f = ml[w].x * whole;
                    v.x += y.x * f, v.y += y.y * f, v.z += y.z * f, v.w += y.w * f;
                }
            if (done)
                store_row4(a, place, row, col, v, finish_mean(M, l, a.sinks, place.h * a.group + (place.r0 + row) % a.group));
            else
                to_slot(cslots + which * slot_floats(), D, row, col, M, l, v);
        }
        if (!done) {
            across |= 1 << which;
            cross[which] = first;
        }
    }

    // ---- items that span CTAs: the last one to arrive joins them all.  A CTA arrives at both of its
    // items before it joins either: else the other's join, in another CTA, would wait for this one
    if (!across)
        return;
    auto cta_of = [&](int t) {
        const int big = more * (each + 1);
        return t < big ? t / (each + 1) : more + (t - big) / each;
    };
    int first_cta[2], last_cta[2];                                        // of the items' tiles
#pragma unroll
    for (int which = 0; which < 2; ++which)
        if (across >> which & 1) {
            const Piece& p = pieces[cross[which]];
            first_cta[which] = cta_of(p.t0);
            last_cta[which] = cta_of(p.t1 - 1);
        }
    __threadfence();
    __syncthreads();
    if (warp == 0) {
        bool last = false;
        if (lane < 2 && (across >> lane & 1)) {
            const int ca = lane ? first_cta[1] : first_cta[0], cb = lane ? last_cta[1] : last_cta[0];
            last = atomicAdd(cnt + ca, 1u) == (unsigned)(cb - ca);
            if (last)
                cnt[ca] = 0;
        }
        const unsigned both = __ballot_sync(~0u, last);
        if (lane == 0)
            s_flag = both;
    }
    __syncthreads();
    const int mine = s_flag;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (!(mine >> which & 1))
            continue;
        const Place place = pieces[which ? cross[1] : cross[0]].p;
        const int ca = which ? first_cta[1] : first_cta[0], cb = which ? last_cta[1] : last_cta[0];
        __threadfence();
        // maxima and sums of every part and row, then their weights, in the ring; every 4
        // columns' parts are summed by `split` threads, then those.  The first parts are
        // on their way while the weights are worked out
        const int K = cb - ca + 1, rows = place.nrows, n4 = rows * (D / 4), split = n4 <= C::THREADS / 2 ? C::THREADS / n4 : 1;
        float2* part = reinterpret_cast<float2*>(sm);                    // [K][kRows]; .x becomes the weight
        float2* total = part + gridDim.x * kRows;                        // [kRows]
        float4* acc = reinterpret_cast<float4*>(total + kRows);          // [C::THREADS]
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
        for (int i = tid; i < K * rows; i += C::THREADS)
            part[i / rows * kRows + i % rows] = __ldcg(reinterpret_cast<const float2*>(slot_of(i / rows) + kRows * D + 2 * (i % rows)));
        __syncthreads();
        // a warp takes a row, its lanes the parts
        for (int row = warp; row < rows; row += C::WARPS) {
            float M = kNone, L = 0.0f;
            for (int k = lane; k < K; k += 32)
                M = fmaxf(M, part[k * kRows + row].x);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
            for (int k = lane; k < K; k += 32) {
                const float2 ml = part[k * kRows + row];
                const float x = ex2(ml.x - M);
                L += ml.y * x;
                part[k * kRows + row].x = pow2_in(ml.y) * x;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                L += __shfl_xor_sync(~0u, L, o);
            if (lane == 0)
                total[row] = make_float2(M, L);
        }
        __syncthreads();
        for (int x0 = 0; x0 < n4; x0 += C::THREADS) {
            const int x = x0 + x_first, row = x / (D / 4), col = x % (D / 4) * 4;
            float4 v = make_float4(0, 0, 0, 0);
            if (x0)
                load_parts(x, from);
            if (x < n4) {
                const float whole = pow2_under(total[row].y);
                for (int k0 = from; k0 < K;) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
                        if (k0 + i * split < K) {
                            const float w = part[(k0 + i * split) * kRows + row].x * whole;
                            v.x += y[i].x * w, v.y += y[i].y * w, v.z += y[i].z * w, v.w += y[i].w * w;
                        }
                    k0 += AHEAD * split;
                    load_parts(x, k0);
                }
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
                store_row4(a, place, row, col, v, finish_mean(total[row].x, total[row].y, a.sinks, place.h * a.group + (place.r0 + row) % a.group));
        }
        __syncthreads();
    }
}

template <int D, int FMT, int BLK, int R>
cudaError_t prepare_one()
{
    return cudaFuncSetAttribute(decode_attn_kernel<D, FMT, BLK, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Decode<D, FMT, BLK, R>::smem(kMaxSeqs));
}

template <int D, int FMT, int R>
cudaError_t prepare_blocks()
{
    cudaError_t e;
    if ((e = prepare_one<D, FMT, 32, R>()) != cudaSuccess || (e = prepare_one<D, FMT, 64, R>()) != cudaSuccess)
        return e;
    return prepare_one<D, FMT, 128, R>();
}

template <int D, int FMT, int BLK, int R>
void launch_one(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    unsigned* cnt = reinterpret_cast<unsigned*>(a.ws);
    decode_attn_kernel<D, FMT, BLK, R><<<num_sms, Decode<D, FMT, BLK, R>::THREADS, Decode<D, FMT, BLK, R>::smem(a.c.n_seqs), s>>>(
        a, reinterpret_cast<float*>(a.ws + kCounterBytes), cnt);
}

template <int D, int FMT, int R>
void launch_blocks(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    if (a.c.blk == 32)
        launch_one<D, FMT, 32, R>(a, num_sms, s);
    else if (a.c.blk == 64)
        launch_one<D, FMT, 64, R>(a, num_sms, s);
    else
        launch_one<D, FMT, 128, R>(a, num_sms, s);
}

template <int D>
void launch_format(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    if (a.c.fmt == MOE_KV_E4M3)
        return launch_blocks<D, MOE_KV_E4M3, 16>(a, num_sms, s);
    if (a.c.fmt == MOE_KV_INT8)
        return launch_blocks<D, MOE_KV_INT8, 16>(a, num_sms, s);
    // Eight rows at most for a sequence's kv head, on average: queries in an MMA's columns, not its rows.
    // 64 sequences of 12,000 tokens, 32 heads of 128 on 4: 99 us, 149 in items of 16 rows; of 4,000 tokens, 64
    // heads of 64 on 8: 56 and 70; 8 of them with 16 rows: 25.5 and 23.2, with 64 rows 57 and 44.
    if (narrow(a.call()))
        return launch_blocks<D, MOE_KV_MXFP4, 8>(a, num_sms, s);
    launch_blocks<D, MOE_KV_MXFP4, 16>(a, num_sms, s);
}

}  // namespace

size_t attention_workspace_bytes(int num_sms)
{
    const size_t decode = kCounterBytes + (size_t)num_sms * (2 + kMaxGroups) * slot_floats() * sizeof(float);
    return std::max(decode, prompt_workspace_bytes(num_sms));
}

cudaError_t prepare_attention_kernels()
{
    cudaError_t e;
    if ((e = prepare_blocks<64, MOE_KV_E4M3, 16>()) != cudaSuccess || (e = prepare_blocks<64, MOE_KV_INT8, 16>()) != cudaSuccess ||
        (e = prepare_blocks<128, MOE_KV_E4M3, 16>()) != cudaSuccess || (e = prepare_blocks<128, MOE_KV_INT8, 16>()) != cudaSuccess)
        return e;
    if ((e = prepare_blocks<64, MOE_KV_MXFP4, 16>()) != cudaSuccess || (e = prepare_blocks<128, MOE_KV_MXFP4, 16>()) != cudaSuccess ||
        (e = prepare_blocks<64, MOE_KV_MXFP4, 8>()) != cudaSuccess || (e = prepare_blocks<128, MOE_KV_MXFP4, 8>()) != cudaSuccess)
        return e;
    return prepare_prompt_kernels();
}

static cudaError_t launch_attention_decode(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    if (a.c.D == 64)
        launch_format<64>(a, num_sms, s);
    else
        launch_format<128>(a, num_sms, s);
    return cudaGetLastError();
}

cudaError_t launch_attention(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    // By both kernels' expected times (attn_plan.h).  The decode kernel spreads 16 rows against 128 keys over all SMs; the
    // prompt kernel takes up to 256 rows on one SM each, or their keys in parts on several.  Measured, decode / prompt
    // kernel, 8 bits: 64 heads of 64 on 8, one sequence, 64 rows: of 600 keys 14.8 / 13.0 us, of 4,000 19.9 / 15.2, of
    // 16,000 29.4 / 24.4, within a window of 128 8.6 / 10.9; 8 sequences of 4,000 keys, 32 rows 30.0 / 28.6, 128 rows 75 / 45,
    // 216 rows 119 / 57; 32 heads of 128 on 4, one sequence, 64 rows: of 600 keys 14.2 / 16.5, of 4,000 24.9 / 18.5.
    // The lengths are on the device, so the rule sees the average tokens of a sequence, and of its keys what its row of the
    // table can hold or a window lets through: a table much wider than the keys in it counts as full.  64 heads of 64 on 8
    // in 8 bits, 63 single tokens and a prompt of 1,000 over 4,000 keys each: 236 us in one call, 72 + 103 in two; 255 and a
    // prompt of 600 over 1,000 keys: 199 us, 80 + 25 in two.
    return attn::takes_prompt_kernel(a.call(), num_sms) ? launch_attention_prompt(a, num_sms, s) : launch_attention_decode(a, num_sms, s);
}

}  // namespace moe
