// moe_linear.cu -- y = x W^T + b for a few tokens, W in 4 bits (MXFP4, or int4
// with group scales), in the caller's layout.
//
// Its floor is HBM's: K/2 bytes of codes a row, read once for up to 16 tokens.
//  - Operands.  m16n8k16 MMAs, 16 weight rows by 8 tokens, f16 with fp32 sums.  The
//    order of the summed index is free: a thread's operand of a 32-column block
//    is the 4 bytes of its eight consecutive columns.  E2M1 codes become f16
//    pairs by conversion, exactly.  An int4 code q is taken as the f16 subnormal
//    q 2^-24 that its bits are where they lie (q 2^-20 one nibble up, for which x
//    is a sixteenth): one logic operation a pair and a shift for every four.
//    The sum starts at -8 sum(x) 2^-24 of the group, so what is added up is (q - 8) x.
//  - Scales.  A group's sum is its own short chain of MMAs; the row's scale
//    multiplies it into the fp32 total.
//  - x is scaled per token by a power of two (largest magnitude into [2^13,
//    2^15)) and converted to f16 once per CTA: exact down to 2^-37 of it (int4:
//    2^-33 for the sixteenths).  A token's totals stay in its own units: MXFP4 takes
//    them into the weights' scales (1 to 2 % of the time), int4 multiplies at the end.
//  - Loads.  Each warp streams 16 rows by 256 columns a stage (2 KB, whole 128-byte
//    lines) through its own ring with 16-byte cp.async, XOR-swizzled so that the
//    operand reads have no bank conflicts; the caller's row pitch gives up to
//    eight-way ones.
//  - Split.  ks warps of a CTA share 16 rows, each with every ks-th stage of
//    columns, and add up through shared memory.  With many tokens of many columns
//    the largest part of a small call is every CTA's own pass over x; there a
//    cluster of four CTAs shares the rows, each with a quarter of the columns (and of
//    x), and adds up through distributed shared memory.  The launch picks both by the
//    expected time (plan(), linear_plan.h).
// Measured: 4 tokens, 151,936 rows of 2,048 columns (int4, groups of 64) 36 us, 4.6
// TB/s, 0.69 of a plain copy's rate: shared memory (0.67 busy) and issue slots (0.62)
// run beside the loads.  One token, 5,120 rows of 2,880 (MXFP4) 7.3 us, 7.9 MB: 1.4 us
// to start, 1.7 for x, 2.7 for the codes, 0.9 for the join.  13 tokens, 4,097 rows of
// 4,096: 9.5 us, with one CTA to the rows 12.6 (7.0 of them x).  More tokens of wide
// matrices (MXFP4) take passes, each of which reads all of W: 16,384 rows of 8,192, 16
// tokens in one, 37 us; 8,192 rows of 8,192, 8 tokens 18 us, 64 tokens in four 84;
// 5,120 rows of 13,824, 9 tokens 26 us, 16 tokens in two 47, 64 tokens in five 133.
#include <cstdint>

#include <cuda_fp16.h>

#include "linear_plan.h"
#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace linear;

constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4_part(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// max of each unsigned half
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight codes -> four f16 pairs: E2M1 in order; int4 as codes (0, 4) 2^-24,
// (1, 5) 2^-20, (2, 6) 2^-24, (3, 7) 2^-20.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4])
{
    if constexpr (FMT == MOE_FMT_MXFP4) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
    } else {
        h[0] = w & 0x000f000fu;
        h[1] = w & 0x00f000f0u;
        h[2] = w >> 8 & 0x000f000fu;
        h[3] = w >> 8 & 0x00f000f0u;
    }
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) { return __uint_as_float(lds32(a)); }
__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// E8M0 byte -> 2^(e - 127): 2^-127 for 0, NaN for 255.
__device__ __forceinline__ float e8m0(int e) { return __int_as_float(max(e << 23, 0x400000) + (e + 1 >> 8)); }
// Whether one of four bytes is 0 or 255.
__device__ __forceinline__ bool odd_byte(uint32_t w) { return __vcmpeq4(w, 0u) | __vcmpeq4(w, 0xffffffffu); }

// FMT, 32-column blocks of a group, 8-token tiles, whether a cluster's CTAs share rows.
template <int FMT, int SUBS, int NT, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(LinearArgs a, Plan p)
{
    constexpr int kGroup = 32 * SUBS, SB = scale_bytes(FMT, kGroup), SW = scale_words(FMT, kGroup);
    constexpr int PER = kCols / kGroup;         // groups of a stage
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int team = warp / p.ks, part = warp % p.ks, teams = kWarps / p.ks;
    uint32_t rank = 0;
    if (SHARED) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // waited for before the first remote store
    }
    // this CTA's columns, counted from the first of them
    const int step0 = SHARED ? rank * p.steps : 0, K = SHARED ? max(min(a.K - step0 * kCols, p.steps * kCols), 0) : a.K;
    const int nunits = (a.N + kRows - 1) / kRows, nsteps = (K + kCols - 1) / kCols;
    const int row_scale = FMT == MOE_FMT_MXFP4 ? a.K / 32 : 2 * (a.K / kGroup);   // bytes
    const uint32_t ring = tc::su32(sm + p.off_ring) + warp * p.stages * p.stage_bytes;
    const int half_k = a.K / 2;

    // this warp's stream: its stages of each of its team's units
    const int cs = SHARED ? kCluster : 1, nclusters = gridDim.x / cs, first = blockIdx.x / cs + team * nclusters, stride = nclusters * teams;
    int pu = first, ps = part;                                     // next to load
    uint32_t pst = ring;
    const uint32_t ring_end = ring + p.stages * p.stage_bytes;
    const int l3 = lane >> 3, ch = lane & 7;
    // rows l3, l3 + 4, l3 + 8, l3 + 12 of a stage, 16 bytes each
    const uint32_t d0 = l3 * 128 + ((ch ^ l3) << 4), d1 = (l3 + 4) * 128 + ((ch ^ l3 ^ 4) << 4);
    constexpr int kScaleCopies = (kRows * SW + 31) / 32;
    int soff[kScaleCopies];                                         // a scale word's row offset, its word in the low bits
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i) {
        const int k = lane + 32 * i;
        soff[i] = k < kRows * SW ? k / SW * row_scale + step0 * SB : -1;
    }
    const uint8_t *csrc = nullptr, *ssrc = nullptr;                 // the unit's codes (this lane's row) and scales
    int prows = 0;
    auto open_unit = [&]() {
        prows = min(a.N - pu * kRows, kRows);
        csrc = a.codes + (long long)pu * kRows * half_k + l3 * half_k + step0 * (kCols / 2) + ch * 16;
        ssrc = static_cast<const uint8_t*>(a.scales) + (long long)pu * kRows * row_scale;
    };
    auto load = [&]() {
        if (pu < nunits) {
            const uint8_t* src = csrc + ps * (kCols / 2);
            if (prows == kRows && (ps + 1) * kCols <= K) {
                cp16(pst + d0, src);
                cp16(pst + d1, src + 4 * half_k);
                cp16(pst + d0 + 1024, src + 8 * half_k);
                cp16(pst + d1 + 1024, src + 12 * half_k);
            } else if (ps * (kCols / 2) + ch * 16 < K / 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (l3 + 4 * i < prows)
                        cp16(pst + (i & 1 ? d1 : d0) + (i >> 1) * 1024, src + 4 * i * half_k);
            }
#pragma unroll
            for (int i = 0; i < kScaleCopies; ++i) {
                const int k = lane + 32 * i, at = (soff[i] + ps * SB & ~3) + 4 * (k % SW), end = prows * row_scale;
                if (soff[i] >= 0) {
                    if (at + 4 <= end)
                        cp4(pst + kCodeBytes + 4 * k, ssrc + at);
                    else if (at < end)
                        cp4_part(pst + kCodeBytes + 4 * k, ssrc + at, end - at);
                }
            }
            pst += p.stage_bytes;
            if (pst == ring_end)
                pst = ring;
            ps += p.ks;
            if (ps >= nsteps) {
                ps = part;
                pu += stride;
                open_unit();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (part >= nsteps)
        pu = nunits;                            // fewer stages than warps: nothing for this one
    open_unit();
    for (int i = 0; i < p.stages - 1; ++i)
        load();

    // x: f16, scaled per token, and (int4) each group's sum.  Pieces of 256 columns
    // of a token, dealt over the warps
    float2* fac = reinterpret_cast<float2*>(sm + p.off_fac);      // per token, what its totals are multiplied by
    uint32_t* bigs = reinterpret_cast<uint32_t*>(fac + 16);
    float* sums = reinterpret_cast<float*>(sm + p.off_sum);
    const int groups = K / kGroup, pieces = p.tokens * nsteps;
    const uint16_t* xsrc = a.x + step0 * kCols;
    if (tid < 16)
        bigs[tid] = 0;
    __syncthreads();
    // read once, eight pieces' loads at a time; bf16 waits where its f16 will lie
    for (int i0 = warp; i0 < pieces; i0 += 8 * kWarps) {
        uint4 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kWarps, m = i / nsteps, k = i % nsteps * 32 + lane;
            q[j] = make_uint4(0, 0, 0, 0);
            if (i < pieces && k < K / 8)
                q[j] = *reinterpret_cast<const uint4*>(xsrc + m * a.x_stride + 8 * k);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kWarps, m = i / nsteps, k = i % nsteps * 32 + lane;
            if (i >= pieces)
                break;
            const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
            uint32_t big = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                big = max_u16x2(big, w[e] & 0x7fff7fffu);
            big = max(big & 0xffffu, big >> 16);
            if (big >= 0x7f80u) {
                // NaN or infinity: the largest of the others
                big = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t u = w[e] & 0x7fffu, v = w[e] >> 16 & 0x7fffu;
                    big = max(big, max(u < 0x7f80u ? u : 0u, v < 0x7f80u ? v : 0u));
                }
            }
            if (k < K / 8)
                *reinterpret_cast<uint4*>(sm + m * p.x_pitch + k * 16) = q[j];
            big = __reduce_max_sync(~0u, big);
            if (lane == 0)
                atomicMax(bigs + m, big);
        }
    }
    __syncthreads();
    auto up_of = [&](int m) { return 14 + 127 - max((int)(bigs[m] >> 7), 1); };
    if (warp == kWarps - 1 && lane < p.tokens) {
        // MXFP4: 2^-up, which joins the weights' scales.  int4: 2^(24 - up) in two factors
        const int down = FMT == MOE_FMT_INT4 ? 24 - up_of(lane) : -up_of(lane), half = FMT == MOE_FMT_INT4 ? down / 2 : 0;
        fac[lane] = make_float2(ldexpf(1.0f, down - half), ldexpf(1.0f, half));
    }
    for (int i = warp; i < pieces; i += kWarps) {
        const int m = i / nsteps, k = i % nsteps * 32 + lane, up = up_of(m);
        // 2^up in two factors, the second 1 but for the smallest tokens
        const float u0 = __uint_as_float((uint32_t)(127 + min(up, 126)) << 23), u1 = __uint_as_float((uint32_t)(127 + max(up - 126, 0)) << 23);
        float sum = 0.0f;
        if (k < K / 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(sm + m * p.x_pitch + k * 16);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint4 o;
            uint32_t* ow = &o.x;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16) * u0;
            if (up > 126)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] *= u1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = FMT == MOE_FMT_INT4 && (e & 1) ? 0.0625f : 1.0f;
                const __half2 t = FMT == MOE_FMT_MXFP4 ? __floats2half2_rn(f[2 * e], f[2 * e + 1]) : __floats2half2_rn(f[e] * y, f[e + 4] * y);
                const float2 back = __half22float2(t);
                sum += (back.x + back.y) * (FMT == MOE_FMT_INT4 && (e & 1) ? 16.0f : 1.0f);
                ow[e] = *reinterpret_cast<const uint32_t*>(&t);
            }
            *reinterpret_cast<uint4*>(sm + m * p.x_pitch + k * 16) = o;
        }
        if constexpr (FMT == MOE_FMT_INT4) {
#pragma unroll
            for (int x = 1; x < 4 * SUBS; x <<= 1)
                sum += __shfl_xor_sync(~0u, sum, x);
            if (k < K / 8 && lane % (4 * SUBS) == 0)
                sums[m * groups + k / (4 * SUBS)] = sum * -4.76837158203125e-07f;    // -8 2^-24
        }
    }
    __syncthreads();

    // tokens that do not exist read the last one's operands; their columns are not stored
    uint32_t xp[NT], sp[NT][2], cp[8];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        xp[i] = tc::su32(sm) + min(8 * i + r, p.tokens - 1) * p.x_pitch + 16 * c;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            sp[i][k] = tc::su32(sums) + min(8 * i + 2 * c + k, p.tokens - 1) * groups * 4;
    }
#pragma unroll
    for (int b = 0; b < 8; ++b)
        cp[b] = r * 128 + ((b ^ r) << 4) + 4 * c;          // a 32-column block's codes in a stage
    // MXFP4: a token's totals are kept in its own units all along, whatever the others' size: weights' scales reach
    // from 2^-127 to 2^127, so that no unit for all tokens keeps every total in range
    float unit[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            unit[i][k] = FMT == MOE_FMT_MXFP4 ? fac[min(8 * i + 2 * c + k, p.tokens - 1)].x : 1.0f;
    uint32_t st = ring;
    const int a0r = r * row_scale & 3, a1r = (r + 8) * row_scale & 3;
    // the clusters' CTAs go through the same number of joins
    const int rounds = SHARED ? (nunits + stride - 1) / stride : first < nunits ? (nunits - first + stride - 1) / stride : 0;
    for (int round = 0, u = first; round < rounds; ++round, u += stride) {
        const int my_steps = u < nunits ? nsteps : 0;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[i][k] = 0.0f;
        for (int s = part; s < my_steps; s += p.ks) {
            load();
            // all groups but the youngest stages - 1 are complete
            if (p.stages == 6)
                asm volatile("cp.async.wait_group 5;" ::: "memory");
            else if (p.stages == 5)
                asm volatile("cp.async.wait_group 4;" ::: "memory");
            else if (p.stages == 4)
                asm volatile("cp.async.wait_group 3;" ::: "memory");
            else if (p.stages == 3)
                asm volatile("cp.async.wait_group 2;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const int at0 = a0r + (step0 + s) * SB, at1 = a1r + (step0 + s) * SB;   // (low two bits)
            const uint32_t s0 = st + kCodeBytes + r * SW * 4, s1 = s0 + 8 * SW * 4;
            uint32_t e0[2], e1[2];                          // MXFP4: the two rows' eight scales
            bool plain = true;
            if constexpr (FMT == MOE_FMT_MXFP4) {
                uint32_t v[3], y[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    v[k] = lds32(s0 + 4 * k);
                    y[k] = lds32(s1 + 4 * k);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    e0[k] = __funnelshift_r(v[k], v[k + 1], 8 * (at0 & 3));
                    e1[k] = __funnelshift_r(y[k], y[k + 1], 8 * (at1 & 3));
                }
                plain = !__any_sync(~0u, odd_byte(e0[0]) || odd_byte(e0[1]) || odd_byte(e1[0]) || odd_byte(e1[1]));
            }
            const int ng = min(PER, (K - s * kCols) / kGroup);
            auto one_group = [&](int g) {
                float part_sum[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float z0 = 0.0f, z1 = 0.0f;
                    if constexpr (FMT == MOE_FMT_INT4) {
                        z0 = lds_f32(sp[i][0] + (s * PER + g) * 4);
                        z1 = lds_f32(sp[i][1] + (s * PER + g) * 4);
                    }
                    part_sum[i][0] = part_sum[i][2] = z0;
                    part_sum[i][1] = part_sum[i][3] = z1;
                }
#pragma unroll
                for (int b = 0; b < SUBS; ++b) {
                    const int blk = g * SUBS + b;                   // 32-column block of the stage
                    uint32_t lo[4], hi[4];
                    decode8<FMT>(lds32(st + cp[blk]), lo);
                    decode8<FMT>(lds32(st + cp[blk] + 1024), hi);
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 x = lds128(xp[i] + s * (kCols * 2) + blk * 64);
                        mma16816(part_sum[i], a0, x.x, x.y);
                        mma16816(part_sum[i], a1, x.z, x.w);
                    }
                }
                float f0, f1;
                if constexpr (FMT == MOE_FMT_MXFP4) {
                    const uint32_t v = e0[g >> 2], y = e1[g >> 2];
                    if (plain) {
                        // the byte to bits 23..30
                        f0 = __uint_as_float(__byte_perm(v, 0, 0x0444 | (g & 3) << 12) >> 1);
                        f1 = __uint_as_float(__byte_perm(y, 0, 0x0444 | (g & 3) << 12) >> 1);
                    } else {
                        f0 = e8m0(v >> 8 * (g & 3) & 255);
                        f1 = e8m0(y >> 8 * (g & 3) & 255);
                    }
                } else {
                    f0 = __half2float(__ushort_as_half((unsigned short)lds_u16(s0 + (at0 & 3) + 2 * g)));
                    f1 = __half2float(__ushort_as_half((unsigned short)lds_u16(s1 + (at1 & 3) + 2 * g)));
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][0] += f0 * unit[i][0] * part_sum[i][0];
                    acc[i][1] += f0 * unit[i][1] * part_sum[i][1];
                    acc[i][2] += f1 * unit[i][0] * part_sum[i][2];
                    acc[i][3] += f1 * unit[i][1] * part_sum[i][3];
                }
            };
            if (ng == PER) {
#pragma unroll
                for (int g = 0; g < PER; ++g)
                    one_group(g);
            } else {
#pragma unroll
                for (int g = 0; g < PER - 1; ++g)
                    if (g < ng)
                        one_group(g);
            }
            __syncwarp();
            st += p.stage_bytes;
            if (st == ring_end)
                st = ring;
        }

        // add up the team's parts
        if (p.ks > 1) {
            float* red = reinterpret_cast<float*>(sm + p.off_red) + warp * (NT * 128);
            if (part > 0)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    *reinterpret_cast<float4*>(red + i * 128 + lane * 4) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(p.ks * 32) : "memory");
            if (part == 0)
                for (int w = 1; w < p.ks; ++w)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(red + w * (NT * 128) + i * 128 + lane * 4);
                        acc[i][0] += v.x, acc[i][1] += v.y, acc[i][2] += v.z, acc[i][3] += v.w;
                    }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(p.ks * 32) : "memory");
        }
        bool mine = part == 0 && u < nunits;
        if constexpr (FMT == MOE_FMT_INT4)
            if (part == 0)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // (a token that does not exist has any factor)
                        const float2 v = fac[min(8 * i + 2 * c + (k & 1), p.tokens - 1)];
                        acc[i][k] = acc[i][k] * v.x * v.y;
                    }
        if constexpr (SHARED) {
            // the cluster's parts of the columns: CTA `team % cs` adds up a team's rows.  Two
            // buffers in turn: a CTA is past its reads of one when it arrives for the other
            const uint32_t slots = (teams + cs - 1) / cs, buf = (round & 1) * slots + team / cs;
            const uint32_t join = tc::su32(sm + p.off_join) + buf * cs * (NT * 512) + lane * 16;
            if (round == 0) {
                // another CTA's shared memory may be written once that CTA has started
                __syncwarp();
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            }
            if (mine) {
                uint32_t at;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(join + rank * (NT * 512)), "r"(team % cs));
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(at + i * 512), "f"(acc[i][0]), "f"(acc[i][1]), "f"(acc[i][2]), "f"(acc[i][3]) : "memory");
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            mine = mine && team % cs == (int)rank;
            if (mine) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[i][k] = 0.0f;
                for (int w = 0; w < cs; ++w)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 v = lds128(join + w * (NT * 512) + i * 512);
                        acc[i][0] += __uint_as_float(v.x), acc[i][1] += __uint_as_float(v.y);
                        acc[i][2] += __uint_as_float(v.z), acc[i][3] += __uint_as_float(v.w);
                    }
            }
        }
        if (mine)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = u * kRows + r + (k >> 1) * 8;
                if (row >= a.N)
                    continue;
                const float bias = a.bias ? tc::bf16f(a.bias[row]) : 0.0f;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int m = 8 * i + 2 * c + (k & 1);
                    if (m >= p.tokens)
                        continue;
                    const float y = a.bias ? acc[i][k] + bias : acc[i][k];
                    const long long at = m * a.out_stride + row;
                    if (a.out_type == MOE_DT_BF16)
                        static_cast<uint16_t*>(a.out)[at] = tc::f2bf16_rne(y);
                    else
                        static_cast<float*>(a.out)[at] = y;
                }
            }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

typedef void (*Kernel)(LinearArgs, Plan);

template <int FMT, int SUBS>
Kernel pick(int nt, bool shared)
{
    if (shared)
        return nt == 1 ? linear_kernel<FMT, SUBS, 1, true> : linear_kernel<FMT, SUBS, 2, true>;
    return nt == 1 ? linear_kernel<FMT, SUBS, 1, false> : linear_kernel<FMT, SUBS, 2, false>;
}

Kernel kernel_for(int fmt, int group, int nt, bool shared)
{
    if (fmt == MOE_FMT_MXFP4)
        return pick<MOE_FMT_MXFP4, 1>(nt, shared);
    return group == 32 ? pick<MOE_FMT_INT4, 1>(nt, shared) : group == 64 ? pick<MOE_FMT_INT4, 2>(nt, shared)
         : group == 128 ? pick<MOE_FMT_INT4, 4>(nt, shared) : pick<MOE_FMT_INT4, 8>(nt, shared);
}

// Clusters that run at once, 0 where there are none.
int clusters_of(Kernel k)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = kCluster;
    cfg.blockDim = kThreads;
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace

cudaError_t prepare_linear_kernels(int* clusters)
{
    for (int nt = 1; nt <= 2; ++nt)
        for (int i = 0; i < 10; ++i) {
            const cudaError_t e = cudaFuncSetAttribute(kernel_for(i / 2 ? MOE_FMT_INT4 : MOE_FMT_MXFP4, 16 << i / 2, nt, i & 1),
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess)
                return e;
        }
    *clusters = clusters_of(kernel_for(MOE_FMT_MXFP4, 32, 2, true));
    return cudaSuccess;
}

cudaError_t launch_linear(const LinearArgs& args, int num_sms, int clusters, cudaStream_t s)
{
    LinearArgs a = args;
    const Plan first = choose({a.N, a.K, a.fmt, a.group, a.M}, num_sms, clusters);
    const bool clustered = first.cs > 1;
    const int most = first.tokens, units = (a.N + kRows - 1) / kRows, groups = clustered ? clusters : num_sms;
    if (most < 1)
        return cudaErrorInvalidConfiguration;
    for (int m0 = 0; m0 < args.M; m0 += most) {
        a.M = args.M - m0 < most ? args.M - m0 : most;
        Plan p;
        plan(p, {a.N, a.K, a.fmt, a.group, a.M}, first.cs, groups);
        if (p.stages < kLeastStages || p.tokens < a.M)       // the kernel waits for all but the youngest stage
            return cudaErrorInvalidConfiguration;
        const int grid = (units < groups ? units : groups) * p.cs;
        const int nt = p.tokens > 8 ? 2 : 1;
        a.x = args.x + m0 * args.x_stride;
        a.out = static_cast<uint8_t*>(args.out) + m0 * args.out_stride * (args.out_type == MOE_DT_BF16 ? 2 : 4);
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = p.cs;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.gridDim = grid;
        cfg.blockDim = kThreads;
        cfg.dynamicSmemBytes = p.smem();
        cfg.stream = s;
        cfg.attrs = at;
        cfg.numAttrs = p.cs > 1 ? 1 : 0;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel_for(a.fmt, a.group, nt, clustered), a, p);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace moe
