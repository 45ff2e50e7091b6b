// kv_device.cuh -- device helpers of the paged cache: which block a work item is,
// and block scales and codes in 8 bits.  Included by .cu files only.
#pragma once
#include <cuda_fp16.h>

#include "ops_internal.h"

namespace moe {
namespace kv {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100, the smallest magnitude a scale is made for

// One sequence's part of a batch: tokens [c0, c0 + n) of the batch are its
// positions [len - n, len).  false: the metadata does not describe that.
__device__ __forceinline__ bool sequence(const KvView& c, int b, int& c0, int& n, int& len)
{
    c0 = c.cu[b];
    const int c1 = c.cu[b + 1];
    len = c.len[b];
    n = c1 - c0;
    return c0 >= 0 && c1 >= c0 && c1 <= c.n_tokens && len >= n && len <= (long long)c.table_stride * c.blk;
}

// The idx-th cache block that the batch's tokens touch, counted over the
// sequences in order; one warp (all lanes) computes it.  Every sequence's
// blocks (len - n) / blk .. (len - 1) / blk.  false: there is no such block.
struct Touched {
    int b, c0, n, len;   // sequence
    int j;               // block of the sequence
};
__device__ __forceinline__ bool find_touched(const KvView& c, int idx, Touched& t)
{
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < c.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int c0 = 0, n = 0, len = 0, cnt = 0;
        if (b < c.n_seqs) {
            if (!sequence(c, b, c0, n, len)) {
                atomicExch(c.status, MOE_ERR_DEVICE_FAULT);
                n = 0;
            }
            if (n > 0)
                cnt = (len - 1) / c.blk - (len - n) / c.blk + 1;
        }
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, incl, o);
            if (lane >= o)
                incl += v;
        }
        const unsigned hit = __ballot_sync(~0u, idx < base + incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            t.b = b0 + src;
            t.c0 = __shfl_sync(~0u, c0, src);
            t.n = __shfl_sync(~0u, n, src);
            t.len = __shfl_sync(~0u, len, src);
            t.j = (t.len - t.n) / c.blk + idx - (base + __shfl_sync(~0u, incl - cnt, src));
            return true;
        }
        base += __shfl_sync(~0u, incl, 31);
    }
    return false;
}

// Physical block of block j of sequence b, or -1 (and the status word) where
// the table holds none.
__device__ __forceinline__ int physical(const KvView& c, int b, int j)
{
    const int id = c.table[(long long)b * c.table_stride + j];
    if (id < 0 || id >= c.num_blocks) {
        atomicExch(c.status, MOE_ERR_DEVICE_FAULT);
        return -1;
    }
    return id;
}

// The scale of a block whose largest finite magnitude is amax.  INT8:
// amax / 127.  E4M3: the smallest power of two with amax <= 448 * scale, so
// that dividing by it is exact and nothing saturates.
template <int FMT>
__device__ __forceinline__ float block_scale(float amax)
{
    const float a = fmaxf(amax, kTiny);
    if constexpr (FMT == MOE_KV_INT8)
        return __fdiv_rn(a, 127.0f);
    const uint32_t u = __float_as_uint(a);
    return __uint_as_float(((u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u)) << 23);   // 448 = 1.75 * 2^8
}

// Four values, already divided by their scale, -> four code bytes, each value
// rounded once to nearest even, saturating; NaN gives 0.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    a = a == a ? a : 0.0f;
    b = b == b ? b : 0.0f;
    c = c == c ? c : 0.0f;
    d = d == d ? d : 0.0f;
    if constexpr (FMT == MOE_KV_INT8) {
        const int i0 = __float2int_rn(fminf(fmaxf(a, -127.0f), 127.0f)), i1 = __float2int_rn(fminf(fmaxf(b, -127.0f), 127.0f));
        const int i2 = __float2int_rn(fminf(fmaxf(c, -127.0f), 127.0f)), i3 = __float2int_rn(fminf(fmaxf(d, -127.0f), 127.0f));
        return __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
    }
    uint32_t r = 0;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Four code bytes -> their values in units of the scale (exact).
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4])
{
    if constexpr (FMT == MOE_KV_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (float)(int8_t)(w >> (8 * i));
        return;
    }
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 p = __half22float2(*reinterpret_cast<__half2*>(&lo)), q = __half22float2(*reinterpret_cast<__half2*>(&hi));
    v[0] = p.x;
    v[1] = p.y;
    v[2] = q.x;
    v[3] = q.y;
}

// Two values -> bf16, nearest even, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace kv
}  // namespace moe
