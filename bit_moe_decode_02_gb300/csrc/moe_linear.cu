// moe_linear.cu -- y = x W^T + b for a few tokens, W in 4 bits (MXFP4, or int4
// with group scales), in the caller's layout.
//
// Bound by HBM: K/2 bytes of codes a row, read once for up to 16 tokens.
//  - Operands.  m16n8k16 MMAs, 16 weight rows by 8 tokens, f16 with fp32 sums.  The
//    order of the summed index is free: a thread's operand of a 32-column block
//    is the 4 bytes of its eight consecutive columns.  E2M1 codes become f16
//    pairs by conversion, exactly.  An int4 code q becomes 16 + q (its bits under
//    an exponent: one shift and one logic operation a pair), and the sum starts
//    at -24 sum(x) of the group, so what is added up is (q - 8) x.
//  - Scales.  A group's sum is its own short chain of MMAs; the row's scale times
//    the token's factor multiplies it into the fp32 total.
//  - x is scaled per token by a power of two (largest magnitude into [2^13,
//    2^15)) and converted to f16 once per CTA: exact down to 2^-37 of it.
//  - Loads.  Each warp streams 16 rows by 256 columns a stage (2 KB, whole 128-byte
//    lines) through its own ring with 16-byte cp.async, XOR-swizzled so that the
//    operand reads have no bank conflicts; the caller's row pitch gives up to
//    eight-way ones.
//  - Split.  ks warps of a CTA share 16 rows, each with every ks-th stage of
//    columns, and add up through shared memory; the launch picks ks so that all
//    warps have the same number of stages as nearly as it goes.
#include <cstdint>

#include <cuda_fp16.h>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;
constexpr int kCols = 256;                 // columns of a stage
constexpr int kCodeBytes = kRows * kCols / 2;
constexpr int kXBytes = 112 * 1024;        // most of x that a CTA keeps: two stages a warp still fit
constexpr int kSmem = 224 * 1024;
constexpr int kMostStages = 6;

// Bytes of one row's scales in a stage, and the aligned 4-byte words that may hold them.
__host__ __device__ constexpr int scale_bytes(int fmt, int group) { return fmt == MOE_FMT_MXFP4 ? kCols / 32 : 2 * kCols / group; }
__host__ __device__ constexpr int scale_words(int fmt, int group) { return scale_bytes(fmt, group) / 4 + 1; }

struct Plan {
    int tokens;     // of this pass
    int ks;         // warps that share 16 rows
    int stages;
    int x_pitch;    // bytes of one token's x
    int off_sum, off_fac, off_red, off_ring;
    int stage_bytes;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::su32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(void* dst, const void* src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::su32(dst)), "l"(src), "r"(bytes) : "memory");
}

// Eight codes -> four f16 pairs: E2M1 in order; int4 as (i, i + 4), each 16 + q.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4])
{
    if constexpr (FMT == MOE_FMT_MXFP4) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
    } else {
        h[0] = (w << 6 & 0x03c003c0u) | 0x4c004c00u;
        h[1] = (w << 2 & 0x03c003c0u) | 0x4c004c00u;
        h[2] = (w >> 2 & 0x03c003c0u) | 0x4c004c00u;
        h[3] = (w >> 6 & 0x03c003c0u) | 0x4c004c00u;
    }
}

// FMT, 32-column blocks of a group, 8-token tiles.
template <int FMT, int SUBS, int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(LinearArgs a, Plan p)
{
    constexpr int kGroup = 32 * SUBS, SB = scale_bytes(FMT, kGroup), SW = scale_words(FMT, kGroup);
    constexpr int PER = kCols / kGroup;         // groups of a stage
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int team = warp / p.ks, part = warp % p.ks, teams = kWarps / p.ks;
    const int nunits = (a.N + kRows - 1) / kRows, nsteps = (a.K + kCols - 1) / kCols;
    const int row_scale = FMT == MOE_FMT_MXFP4 ? a.K / 32 : 2 * (a.K / kGroup);   // bytes
    uint8_t* ring = sm + p.off_ring + warp * p.stages * p.stage_bytes;
    const uint8_t* scales = static_cast<const uint8_t*>(a.scales);
    const long long scale_end = (long long)a.N * row_scale;

    // this warp's stream: its stages of each of its team's units
    const int stride = gridDim.x * teams;
    int pu = blockIdx.x + team * gridDim.x, ps = part, pslot = 0;   // next to load
    auto load = [&]() {
        if (pu < nunits && ps < nsteps) {
            uint8_t* st = ring + pslot * p.stage_bytes;
            const int row0 = pu * kRows;
            const uint8_t* src = a.codes + (long long)row0 * (a.K / 2) + ps * (kCols / 2);
            const int ch = lane & 7, left = a.K / 2 - ps * (kCols / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = (lane >> 3) + 4 * i;
                if (row0 + x < a.N && ch * 16 < left)
                    cp16(st + x * 128 + ((ch ^ (x & 7)) << 4), src + (long long)x * (a.K / 2) + ch * 16);
            }
            uint32_t* ss = reinterpret_cast<uint32_t*>(st + kCodeBytes);
#pragma unroll
            for (int i = 0; i < (kRows * SW + 31) / 32; ++i) {
                const int k = lane + 32 * i, x = k / SW, w = k % SW;
                const long long at = (((long long)(row0 + x) * row_scale + ps * SB) & ~3ll) + 4 * w;
                if (k < kRows * SW && row0 + x < a.N && at < scale_end)
                    cp4(ss + k, scales + at, (int)min(4ll, scale_end - at));
            }
            pslot = pslot + 1 == p.stages ? 0 : pslot + 1;
            ps += p.ks;
            if (ps >= nsteps) {
                ps = part;
                pu += stride;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (part >= nsteps)
        pu = nunits;                            // fewer stages than warps: nothing for this one
    for (int i = 0; i < p.stages - 1; ++i)
        load();

    // x: f16, scaled per token, and (int4) each group's sum
    float* fac = reinterpret_cast<float*>(sm + p.off_fac);
    float* sums = reinterpret_cast<float*>(sm + p.off_sum);
    const int groups = a.K / kGroup;
    for (int m = warp; m < p.tokens; m += kWarps) {
        const uint16_t* x = a.x + m * a.x_stride;
        uint32_t big = 0;
        for (int i = lane; i < a.K / 8; i += 32) {
            const uint4 q = *reinterpret_cast<const uint4*>(x + 8 * i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = w[k] & 0x7fffu, v = w[k] >> 16 & 0x7fffu;
                big = max(big, max(u < 0x7f80u ? u : 0u, v < 0x7f80u ? v : 0u));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            big = max(big, __shfl_xor_sync(~0u, big, o));
        const int up = 14 + 127 - max((int)(big >> 7), 1);
        const float u0 = __uint_as_float((uint32_t)(127 + up / 2) << 23), u1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
        if (lane == 0)
            fac[m] = ldexpf(1.0f, -up);
        for (int i0 = 0; i0 < a.K / 8; i0 += 32) {
            const int i = i0 + lane;
            uint4 o = make_uint4(0, 0, 0, 0);
            float sum = 0.0f;
            if (i < a.K / 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(x + 8 * i);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                __half h[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16) * u0 * u1;
                    h[k] = __float2half_rn(f);
                    sum += __half2float(h[k]);
                }
                uint32_t* ow = &o.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 t = FMT == MOE_FMT_MXFP4 ? __halves2half2(h[2 * k], h[2 * k + 1]) : __halves2half2(h[k], h[k + 4]);
                    ow[k] = *reinterpret_cast<const uint32_t*>(&t);
                }
                *reinterpret_cast<uint4*>(sm + m * p.x_pitch + i * 16) = o;
            }
            if constexpr (FMT == MOE_FMT_INT4) {
#pragma unroll
                for (int s = 1; s < 4 * SUBS; s <<= 1)
                    sum += __shfl_xor_sync(~0u, sum, s);
                if (i < a.K / 8 && lane % (4 * SUBS) == 0)
                    sums[m * groups + i / (4 * SUBS)] = -24.0f * sum;
            }
        }
    }
    __syncthreads();

    bool has[NT];                               // this thread's token of the operand exists
    float tf[NT][2];
    const uint8_t* xp[NT];
    const float* sp[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        has[i] = 8 * i + r < p.tokens;
        xp[i] = sm + (8 * i + r) * p.x_pitch + 16 * c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int m = 8 * i + 2 * c + k;
            tf[i][k] = m < p.tokens ? fac[m] : 0.0f;
            sp[i][k] = m < p.tokens ? sums + m * groups : nullptr;
        }
    }
    int slot = 0;
    for (int u = blockIdx.x + team * gridDim.x; u < nunits; u += stride) {
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[i][k] = 0.0f;
        for (int s = part; s < nsteps; s += p.ks) {
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
            const uint8_t* st = ring + slot * p.stage_bytes;
            slot = slot + 1 == p.stages ? 0 : slot + 1;
            const uint8_t* ss = st + kCodeBytes;
            const long long at0 = (long long)(u * kRows + r) * row_scale + s * SB, at1 = at0 + 8ll * row_scale;
            const uint8_t* s0 = ss + r * SW * 4 + (at0 & 3);
            const uint8_t* s1 = ss + (r + 8) * SW * 4 + (at1 & 3);
            const int ng = min(PER, (a.K - s * kCols) / kGroup);
            auto one_group = [&](int g) {
                float part_sum[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float z0 = 0.0f, z1 = 0.0f;
                    if constexpr (FMT == MOE_FMT_INT4) {
                        z0 = sp[i][0] ? sp[i][0][s * PER + g] : 0.0f;
                        z1 = sp[i][1] ? sp[i][1][s * PER + g] : 0.0f;
                    }
                    part_sum[i][0] = part_sum[i][2] = z0;
                    part_sum[i][1] = part_sum[i][3] = z1;
                }
#pragma unroll
                for (int b = 0; b < SUBS; ++b) {
                    const int blk = g * SUBS + b;                   // 32-column block of the stage
                    const int off = ((blk ^ r) << 4) + 4 * c;
                    uint32_t lo[4], hi[4];
                    decode8<FMT>(*reinterpret_cast<const uint32_t*>(st + r * 128 + off), lo);
                    decode8<FMT>(*reinterpret_cast<const uint32_t*>(st + (r + 8) * 128 + off), hi);
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (has[i])
                            x = *reinterpret_cast<const uint4*>(xp[i] + (s * (kCols / 32) + blk) * 64);
                        mma16816(part_sum[i], a0, x.x, x.y);
                        mma16816(part_sum[i], a1, x.z, x.w);
                    }
                }
                float f0, f1;
                if constexpr (FMT == MOE_FMT_MXFP4) {
                    // 2^(e - 127): 2^-127 for e = 0, NaN for e = 255
                    const int e0 = s0[g], e1 = s1[g];
                    f0 = __int_as_float(max(e0 << 23, 0x400000) + (e0 + 1 >> 8));
                    f1 = __int_as_float(max(e1 << 23, 0x400000) + (e1 + 1 >> 8));
                } else {
                    f0 = __half2float(*reinterpret_cast<const __half*>(s0 + 2 * g));
                    f1 = __half2float(*reinterpret_cast<const __half*>(s1 + 2 * g));
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][0] += f0 * (tf[i][0] * part_sum[i][0]);
                    acc[i][1] += f0 * (tf[i][1] * part_sum[i][1]);
                    acc[i][2] += f1 * (tf[i][0] * part_sum[i][2]);
                    acc[i][3] += f1 * (tf[i][1] * part_sum[i][3]);
                }
            };
            if (ng == PER) {
#pragma unroll
                for (int g = 0; g < PER; ++g)
                    one_group(g);
            } else {
                for (int g = 0; g < ng; ++g)
                    one_group(g);
            }
            __syncwarp();
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
        if (part == 0)
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
Kernel pick(int nt)
{
    return nt == 1 ? linear_kernel<FMT, SUBS, 1> : linear_kernel<FMT, SUBS, 2>;
}

Kernel kernel_for(int fmt, int group, int nt)
{
    if (fmt == MOE_FMT_MXFP4)
        return pick<MOE_FMT_MXFP4, 1>(nt);
    return group == 32 ? pick<MOE_FMT_INT4, 1>(nt) : group == 64 ? pick<MOE_FMT_INT4, 2>(nt)
         : group == 128 ? pick<MOE_FMT_INT4, 4>(nt) : pick<MOE_FMT_INT4, 8>(nt);
}

int align16(int v) { return (v + 15) & ~15; }

}  // namespace

cudaError_t prepare_linear_kernels()
{
    for (int nt = 1; nt <= 2; ++nt)
        for (int i = 0; i < 5; ++i) {
            const cudaError_t e = cudaFuncSetAttribute(kernel_for(i ? MOE_FMT_INT4 : MOE_FMT_MXFP4, 16 << i, nt),
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess)
                return e;
        }
    return cudaSuccess;
}

cudaError_t launch_linear(const LinearArgs& args, int num_sms, cudaStream_t s)
{
    // tokens in passes of at most 16, and of no more than fit in shared memory
    // (one launch for 16 tokens of up to 3,520 columns)
    LinearArgs a = args;
    const int most = kXBytes / (2 * a.K + 128) < 16 ? kXBytes / (2 * a.K + 128) : 16;
    for (int m0 = 0; m0 < args.M; m0 += most) {
        Plan p{};
        p.tokens = args.M - m0 < most ? args.M - m0 : most;
        const int nt = p.tokens > 8 ? 2 : 1;
        // pitch of 64 mod 128 bytes: two tokens' 64-byte pieces cover all banks
        p.x_pitch = (2 * a.K + 63) / 128 * 128 + 64;
        int off = p.tokens * p.x_pitch;
        p.off_sum = off;
        if (a.fmt == MOE_FMT_INT4)
            off = align16(off + p.tokens * (a.K / a.group) * 4);
        p.off_fac = off;
        off += 64;
        p.off_red = off;
        off += kWarps * nt * 512;
        p.off_ring = (off + 127) / 128 * 128;
        p.stage_bytes = kCodeBytes + (kRows * scale_words(a.fmt, a.group) * 4 + 127) / 128 * 128;
        p.stages = (kSmem - p.off_ring) / (kWarps * p.stage_bytes);
        if (p.stages > kMostStages)
            p.stages = kMostStages;
        // stages that the busiest warp goes through, for each split of the columns;
        // a finer one costs a join, so it has to save a tenth
        const int units = (a.N + kRows - 1) / kRows, steps = (a.K + kCols - 1) / kCols;
        long long best = -1;
        for (int ks = 1; ks <= kWarps && ks <= steps; ks *= 2) {
            const long long teams = (long long)num_sms * (kWarps / ks);
            const long long cost = (units + teams - 1) / teams * ((steps + ks - 1) / ks);
            if (best < 0 || 10 * cost <= 9 * best) {
                best = cost;
                p.ks = ks;
            }
        }
        const int grid = units < num_sms ? units : num_sms;
        a.x = args.x + m0 * args.x_stride;
        a.out = static_cast<uint8_t*>(args.out) + m0 * args.out_stride * (args.out_type == MOE_DT_BF16 ? 2 : 4);
        a.M = p.tokens;
        kernel_for(a.fmt, a.group, nt)<<<grid, kThreads, p.off_ring + kWarps * p.stages * p.stage_bytes, s>>>(a, p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace moe
