// kv4_device.cuh -- device helpers of the 4-bit paged cache.  Included by .cu files only.
//
// A block of one head holds a record for K and one for V: E2M1 codes, then an E8M0 byte
// for each token's groups of 32 values along the head (0: a group of zeros).  Both lie
// as the lanes of an attention warp take them, 32 tokens ("sub") at a time:
//   K codes  [blk][D/2], the even d in the low nibble;
//   K scales [sub][2 (t/8) + t%2][group][(t/2) % 4], t the token of the sub;
//   V codes  [sub][group][d%8][t/8][(d/8) % 4] words of the eight tokens from 8 (t/8), the
//            first in the low nibble;
//   V scales [sub][group][t].
#pragma once
#include <cuda_fp16.h>

#include "kv_device.cuh"

namespace moe {
namespace kv4 {

// Bytes of a record.
__host__ __device__ constexpr int record(int blk, int D) { return blk * D / 32 * 17; }

template <int D>
__host__ __device__ constexpr int k_scale_at(int t, int g)
{
    return t / 32 * D + ((2 * (t % 32 / 8) + t % 2) * (D / 32) + g) * 4 + t / 2 % 4;
}
template <int D>
__host__ __device__ constexpr int v_scale_at(int t, int g)
{
    return (t / 32 * (D / 32) + g) * 32 + t % 32;
}
// Word of V's tokens 8 t8 .. 8 t8 + 7 and d = 32 g + 8 e + r.
template <int D>
__host__ __device__ constexpr int v_word_at(int t8, int g, int e, int r)
{
    return ((t8 / 4 * (D / 32) + g) * 8 + r) * 16 + t8 % 4 * 4 + e;
}

// Eight codes -> four f16 pairs, exact.
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// The scale byte of a group whose largest finite magnitude (bf16 bits) is `big`: the
// smallest 2^e with big <= 6 * 2^e, plus 127; 0 below 2^-100.
__device__ __forceinline__ uint32_t scale_byte(uint32_t big)
{
    // 6 = 1.5 * 2^2; 2^-100 is 0x0d80 in bf16
    return big < 0x0d80u ? 0u : (big >> 7) - 2 + ((big & 0x7fu) > 0x40u);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 x 8 nibbles, transposed: nibble j of word i <-> nibble i of word j.
__device__ __forceinline__ void transpose(uint32_t (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t x = w[i], y = w[i + 1];
        w[i] = (x & 0x0f0f0f0fu) | (y << 4 & 0xf0f0f0f0u);
        w[i + 1] = (x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (!(i & 2)) {
            const uint32_t x = w[i], y = w[i + 2];
            w[i] = __byte_perm(x, y, 0x6240);
            w[i + 2] = __byte_perm(x, y, 0x7351);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i], y = w[i + 4];
        w[i] = __byte_perm(x, y, 0x5410);
        w[i + 4] = __byte_perm(x, y, 0x7632);
    }
}

}  // namespace kv4
}  // namespace moe
