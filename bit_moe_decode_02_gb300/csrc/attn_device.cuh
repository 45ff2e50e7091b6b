// attn_device.cuh -- what the attention kernels over the cache share.
// Included by .cu files only.
#pragma once
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;         // running maximum of a row that has seen no key
constexpr float kSlack = 8.0f;            // log2 units that a score may pass the kept maximum by
// A probability p = e^(s - m) is 2^6 p in f16: at most 2^15 with the slack and a unit that is
// off by 2, so that 11 bits are kept down to 2^-20 of the kept maximum and none below 2^-31
constexpr float kRoom = 6.0f;
constexpr float kUnroom = 0.015625f;      // 2^-6

// Four code bytes -> two f16 pairs, exact.
template <int FMT>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    if constexpr (FMT == MOE_KV_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    } else {
        // v + 128 below f16's 1024: 0x64uu is 1024 + uu
        w ^= 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<uint32_t*>(&x);
        hi = *reinterpret_cast<uint32_t*>(&y);
    }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// largest and smallest of each half, unsigned; products of f16 pairs
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A query row's scaling: its largest finite magnitude (bf16 bits, sign off) to
// [2^13, 2^15) by a factor of 2^up, so that f16 holds the row exactly down to
// 2^-37 of it.
struct RowScale {
    float u0, u1;   // 2^up = u0 u1
    float f;        // score = (scaled sum) * block's scale * f, in log2 units
};
__device__ __forceinline__ RowScale row_scale(uint32_t big, float scale)
{
    const int up = 14 + 127 - max((int)(big >> 7), 1);
    RowScale r;
    r.u0 = __uint_as_float((uint32_t)(127 + up / 2) << 23);
    r.u1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
    if (scale < 0.0f)
        r.u0 = -r.u0;
    r.f = ldexpf(fabsf(scale) * kLog2e, -up);
    return r;
}
// Largest finite magnitude in a word of two bf16, as bits.
__device__ __forceinline__ uint32_t big_of(uint32_t w)
{
    const uint32_t x = w & 0x7fffu, y = w >> 16 & 0x7fffu;
    return max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u);
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, const RowScale& r)
{
    return pack_f16(__uint_as_float(w << 16) * r.u0 * r.u1, __uint_as_float(w & 0xffff0000u) * r.u0 * r.u1);
}

// The unit that O is kept in: it changes only when a block's V scale leaves
// [ref / 2, 2 ref], and stays within 2^80 of the largest seen (O is below 2^44: 2^15 of a
// probability, 2^9 of a code, 2^20 keys).
__device__ __forceinline__ float new_unit(float vs, float vmax)
{
    return fmaxf(fmaxf(vs, vmax * 8.271806125530277e-25f), 7.52316384526264e-37f);   // 2^-80, 2^-120
}

// One row's final value from its sums: the sink joins the denominator.  A row that
// sees nothing has l = 0; a NaN (of the query, or the sink) goes through.
struct Final {
    float mul, lse;
};
__device__ __forceinline__ Final finish(float m, float l, const float* sinks, int hq)
{
    float M = m;
    if (sinks) {
        const float ms = sinks[hq] * kLog2e;
        M = fmaxf(m, ms);
        l = l * ex2(m - M) + (ms == M ? 1.0f : ex2(ms - M));
    }
    Final f;
    f.mul = l == 0.0f ? 0.0f : ex2(m - M) / l;
    f.lse = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
    return f;
}

// What is left of a row's sums for a join with others': not the sums, which may pass fp32's
// range where the values do not, but half to all of their mean, the sums over the power of two
// in l (exact, and no division in the way), kDown below that (codes reach 2^9 above a scale;
// what it loses lies below 2^-137), with m and l.  l is 1 at least where there is a key.
constexpr float kDown = 2.44140625e-4f;   // 2^-12
__device__ __forceinline__ float pow2_in(float l) { return __uint_as_float(__float_as_uint(l) & 0x7f800000u); }
__device__ __forceinline__ float pow2_under(float l) { return __uint_as_float(0x7f000000u - (__float_as_uint(l) & 0x7f800000u)); }   // 1 / pow2_in
// A row's result from such a mean of all its keys.
__device__ __forceinline__ Final finish_mean(float m, float l, const float* sinks, int hq)
{
    Final f = finish(m, l, sinks, hq);
    f.mul *= pow2_in(l) * (1.0f / kDown);
    return f;
}

}  // namespace attn
}  // namespace moe
