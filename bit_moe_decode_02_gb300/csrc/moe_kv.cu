// moe_kv.cu -- an 8-bit paged key/value cache: tokens quantised as they are
// written, and read back.
//
// A cache block holds `blk` tokens of one head: K codes [blk][D], then V codes
// [D][blk], each with one fp32 scale.  V lies transposed because the attention
// multiplies it along the tokens: four consecutive bytes along the summed
// dimension are one thread's matrix operand for K (along D) and for V (along
// the tokens) alike, so neither needs a transpose when it is read, once for
// every token generated, while a token is written only once.
#include <cstdint>

#include "kv_device.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kWriteThreads = 128;

// max of each half, unsigned: of magnitudes' bits, NaN and infinities above all others
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four values of a block without NaN or infinity -> codes.  INT8: adding 1.5 *
// 2^23 rounds to an integer, nearest even, in the sum's low bits.
template <int FMT>
__device__ __forceinline__ uint32_t encode4_finite(float a, float b, float c, float d)
{
    if constexpr (FMT == MOE_KV_INT8) {
        const float m = 12582912.0f;
        const uint32_t x = __byte_perm(__float_as_uint(__fadd_rn(a, m)), __float_as_uint(__fadd_rn(b, m)), 0x0040);
        const uint32_t y = __byte_perm(__float_as_uint(__fadd_rn(c, m)), __float_as_uint(__fadd_rn(d, m)), 0x0040);
        return __byte_perm(x, y, 0x5410);
    }
    uint32_t r = 0;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One CTA per (touched block, head, K or V): the largest finite magnitude of
// the block's new tokens sets the scale (never below the block's old one if it
// holds earlier tokens, whose codes are rounded again where it grew), then
// every new value is divided by it and rounded once.
// 6 prompts of 2,700 tokens on average, 4 heads of 128 (48 MB, 2 bytes in and 1 out per
// value), take 14.5 us, 3.3 TB/s, half of a plain copy's rate: waiting for loads, not
// HBM, bounds it (DRAM at 0.26 of its peak, the codes stay in L2; 10 of a warp's cycles
// per instruction wait for global memory).  A thread's values go out four loads at a
// time, behind the chain of metadata reads.  It issues on 0.56 of the cycles beside, so
// blocks without NaN or infinity skip their handling.  One token for each of 4
// sequences is bound by latency, 2.8 us: sequence, block number, scale and values are
// read one after another.  Every CTA looks its sequence up 32 at a time, so many
// sequences cost their square: one token each of 64, 256 and 1,024 sequences (8 heads
// of 64) take 4.2, 14.5 and 121 us.
template <int FMT, int D, int blk>
__global__ void __launch_bounds__(kWriteThreads)
kv_write_kernel(KvView c, const uint16_t* __restrict__ ksrc, const uint16_t* __restrict__ vsrc, long long kstride,
                long long vstride)
{
    extern __shared__ uint32_t tile[];   // [blk][D/2 + 1] words of two bf16
    __shared__ uint32_t red[kWriteThreads / 32];
    const int h = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
    kv::Touched t;
    if (!kv::find_touched(c, blockIdx.x, t))
        return;
    const int id = kv::physical(c, t.b, t.j);
    if (id < 0)
        return;
    const int start = t.len - t.n - t.j * blk;                 // offset of the sequence's first new token
    const int lo = start > 0 ? start : 0, hi = min(t.len - t.j * blk, blk);
    const uint16_t* src = which ? vsrc : ksrc;
    const long long stride = which ? vstride : kstride;
    src += (long long)(t.c0 - start + lo) * stride + (long long)h * D;
    constexpr int pitch = D / 2 + 1, vec = D / 8;
    float* sp = c.scales + ((long long)id * c.H + h) * 2 + which;
    const bool fresh = lo == 0;
    const float old = fresh ? 0.0f : *sp;

    uint32_t big = 0;
#pragma unroll 4
    for (int i = tid; i < (hi - lo) * vec; i += kWriteThreads) {
        const int r = i / vec, x = i % vec;
        const uint4 q = *reinterpret_cast<const uint4*>(src + r * stride + x * 8);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            big = max_u16x2(big, w[e] & 0x7fff7fffu);
            tile[(lo + r) * pitch + x * 4 + e] = w[e];
        }
    }
    auto block_max = [&](uint32_t v) {
        v = max(v & 0xffffu, v >> 16);
        v = __reduce_max_sync(~0u, v);
        __syncthreads();
        if ((tid & 31) == 0)
            red[tid >> 5] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWriteThreads / 32; ++i)
            v = max(v, red[i]);
        return v;
    };
    big = block_max(big);
    const bool finite = big < 0x7f80u;
    if (!finite) {
        // NaN or infinity among the values: the largest of the others
        big = 0;
        for (int i = tid; i < (hi - lo) * (D / 2); i += kWriteThreads) {
            const uint32_t w = tile[(lo + i / (D / 2)) * pitch + i % (D / 2)], x = w & 0x7fffu, y = w >> 16 & 0x7fffu;
            big = max(big, max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u));
        }
        big = block_max(big);
    }

    float scale = kv::block_scale<FMT>(__uint_as_float(big << 16)), ratio = 0.0f;
    const bool grown = !fresh && scale > old;
    if (!fresh && !grown)
        scale = old;
    const float inv = __fdiv_rn(1.0f, scale);
    if (grown)
        ratio = __fmul_rn(old, inv);
    if (tid == 0 && (fresh || grown))                          // after block_max: every thread has read the old scale
        *sp = scale;
    auto again = [&](uint32_t w) {
        float v[4];
        kv::decode4<FMT>(w, v);
        return kv::encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
    };
    auto encode = [&](float x, float y, float z, float w) {
        x = __fmul_rn(x, inv), y = __fmul_rn(y, inv), z = __fmul_rn(z, inv), w = __fmul_rn(w, inv);
        return finite ? encode4_finite<FMT>(x, y, z, w) : kv::encode4<FMT>(x, y, z, w);
    };

    uint8_t* dst = c.codes + (((long long)id * c.H + h) * 2 + which) * ((long long)blk * D);
    const int first = fresh || grown ? 0 : lo, last = fresh ? blk : hi;   // tokens whose codes change
    if (which == 0) {
        for (int i = tid; i < (last - first) * vec; i += kWriteThreads) {
            const int r = first + i / vec, x = i % vec;
            uint2* p = reinterpret_cast<uint2*>(dst + r * D + x * 8);
            uint2 o = make_uint2(0, 0);
            if (r < lo) {
                const uint2 was = *p;
                o = make_uint2(again(was.x), again(was.y));
            } else if (r < hi) {
                const uint32_t* w = tile + r * pitch + x * 4;
                o.x = encode(lo_bf16(w[0]), hi_bf16(w[0]), lo_bf16(w[1]), hi_bf16(w[1]));
                o.y = encode(lo_bf16(w[2]), hi_bf16(w[2]), lo_bf16(w[3]), hi_bf16(w[3]));
            }
            *p = o;
        }
    } else {
        // 16 tokens of two d's at a time: the bytes of tokens that keep their
        // codes are read and written back as they were
        const int g0 = first / 16, gs = (last + 15) / 16 - g0;
        for (int i = tid; i < (D / 2) * gs; i += kWriteThreads) {
            const int d2 = i / gs, g = g0 + i % gs;
            const uint32_t* w = tile + g * 16 * pitch + d2;
            uint4* p = reinterpret_cast<uint4*>(dst + 2 * d2 * blk + g * 16);
            uint4* q = reinterpret_cast<uint4*>(dst + (2 * d2 + 1) * blk + g * 16);
            uint32_t o[4], u[4];
            if (g * 16 >= lo && g * 16 + 16 <= hi) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w0 = w[4 * e * pitch], w1 = w[(4 * e + 1) * pitch], w2 = w[(4 * e + 2) * pitch], w3 = w[(4 * e + 3) * pitch];
                    o[e] = encode(lo_bf16(w0), lo_bf16(w1), lo_bf16(w2), lo_bf16(w3));
                    u[e] = encode(hi_bf16(w0), hi_bf16(w1), hi_bf16(w2), hi_bf16(w3));
                }
            } else {
                const uint4 zero = make_uint4(0, 0, 0, 0), was = fresh ? zero : *p, wat = fresh ? zero : *q;
                o[0] = was.x, o[1] = was.y, o[2] = was.z, o[3] = was.w;
                u[0] = wat.x, u[1] = wat.y, u[2] = wat.z, u[3] = wat.w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t0 = g * 16 + 4 * e;
                    if (t0 < lo && grown) {
                        const uint32_t m = t0 + 4 <= lo ? ~0u : (1u << 8 * (lo - t0)) - 1;
                        o[e] = (o[e] & ~m) | (again(o[e]) & m);
                        u[e] = (u[e] & ~m) | (again(u[e]) & m);
                    }
                    if (t0 + 4 > lo && t0 < hi) {
                        uint32_t v[4], m = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool in = t0 + k >= lo && t0 + k < hi;
                            v[k] = in ? w[(4 * e + k) * pitch] : 0u;
                            m |= in ? 0xffu << 8 * k : 0u;
                        }
                        o[e] = (o[e] & ~m) | (encode(lo_bf16(v[0]), lo_bf16(v[1]), lo_bf16(v[2]), lo_bf16(v[3])) & m);
                        u[e] = (u[e] & ~m) | (encode(hi_bf16(v[0]), hi_bf16(v[1]), hi_bf16(v[2]), hi_bf16(v[3])) & m);
                    }
                }
            }
            *p = make_uint4(o[0], o[1], o[2], o[3]);
            *q = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

constexpr int kReadThreads = 256;

// One CTA per (touched block, head): codes times the scale, rounded to bf16
// once.  V comes back through 4 x 4 byte transposes in registers.  Bound by HBM:
// 1 byte in and 2 out per value; all of a thread's loads, K's and V's, are out
// before the first is used.
template <int FMT, int D, int blk>
__global__ void __launch_bounds__(kReadThreads)
kv_read_kernel(KvView c, uint16_t* __restrict__ kdst, uint16_t* __restrict__ vdst, long long kstride, long long vstride)
{
    extern __shared__ uint32_t tile[];   // V: [D][blk/4] words
    const int h = blockIdx.y, tid = threadIdx.x;
    kv::Touched t;
    if (!kv::find_touched(c, blockIdx.x, t))
        return;
    const int id = kv::physical(c, t.b, t.j);
    if (id < 0)
        return;
    const int start = t.len - t.n - t.j * blk;
    const int lo = start > 0 ? start : 0, hi = min(t.len - t.j * blk, blk);
    const float2 scale = *reinterpret_cast<const float2*>(c.scales + ((long long)id * c.H + h) * 2);
    const uint8_t* ksrc = c.codes + ((long long)id * c.H + h) * 2 * ((long long)blk * D);
    const uint8_t* vsrc = ksrc + blk * D;
    kdst += (long long)(t.c0 - start) * kstride + (long long)h * D;   // row of the block's token 0
    vdst += (long long)(t.c0 - start) * vstride + (long long)h * D;

    // 16 codes at a time: of K's row (token) i / (D / 16), of V's row (d) i / (blk / 16)
    constexpr int kPer = (blk * D / 16 + kReadThreads - 1) / kReadThreads, kv16 = D / 16, vv16 = blk / 16;
    uint4 kw[kPer], vw[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kReadThreads;
        const bool in = i < blk * D / 16;
        kw[j] = vw[j] = make_uint4(0, 0, 0, 0);
        if (in && i / kv16 >= lo && i / kv16 < hi)
            kw[j] = *reinterpret_cast<const uint4*>(ksrc + i * 16);
        if (in && i % vv16 * 16 + 16 > lo && i % vv16 * 16 < hi)
            vw[j] = *reinterpret_cast<const uint4*>(vsrc + i * 16);
    }
    // word w of row d lies at w ^ (d / 4): the four rows of a transpose are
    // read by 32 lanes with few bank conflicts
    constexpr int wpr = blk / 4;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kReadThreads;
        if (i >= blk * D / 16)
            continue;
        const int d = i / vv16, w = i % vv16 * 4, x = d >> 2 & (wpr - 1);
        uint32_t* row = tile + d * wpr;
        row[w ^ x] = vw[j].x;
        row[(w + 1) ^ x] = vw[j].y;
        row[(w + 2) ^ x] = vw[j].z;
        row[(w + 3) ^ x] = vw[j].w;
    }
    auto pair = [&](uint32_t w, float s) {
        float v[4];
        kv::decode4<FMT>(w, v);
        return make_uint2(kv::bf16x2(v[0] * s, v[1] * s), kv::bf16x2(v[2] * s, v[3] * s));
    };
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kReadThreads, r = i / kv16;
        if (i >= blk * D / 16 || r < lo || r >= hi)
            continue;
        const uint2 p = pair(kw[j].x, scale.x), q = pair(kw[j].y, scale.x), x = pair(kw[j].z, scale.x), y = pair(kw[j].w, scale.x);
        uint4* o = reinterpret_cast<uint4*>(kdst + r * kstride + i % kv16 * 16);
        o[0] = make_uint4(p.x, p.y, q.x, q.y);
        o[1] = make_uint4(x.x, x.y, y.x, y.y);
    }
    __syncthreads();
    constexpr int dq = D / 4;
    const int q0 = lo / 4, nq = (hi + 3) / 4 - q0;
    for (int i = tid; i < dq * nq; i += kReadThreads) {
        const int d4 = i % dq, q = q0 + i / dq;
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = tile[(4 * d4 + e) * wpr + (q ^ (d4 & (wpr - 1)))];
        const uint32_t a = __byte_perm(r[0], r[1], 0x5140), b = __byte_perm(r[2], r[3], 0x5140);
        const uint32_t e = __byte_perm(r[0], r[1], 0x7362), f = __byte_perm(r[2], r[3], 0x7362);
        const uint32_t col[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(e, f, 0x5410),
                                 __byte_perm(e, f, 0x7632)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int tok = 4 * q + k;
            if (tok >= lo && tok < hi)
                *reinterpret_cast<uint2*>(vdst + tok * vstride + d4 * 4) = pair(col[k], scale.y);
        }
    }
}

// CTAs along a grid's x: an upper bound on the blocks that a batch touches (a sequence
// with n >= 1 new tokens touches at most (n - 1) / blk + 2, and no more than n), and one
// more.  A CTA that finds its block stops at its sequence; the last one finds none, so
// that it checks all sequences, or as many as end in one whose metadata is wrong.
unsigned touched_grid(const KvView& c)
{
    const long long most = (long long)c.n_tokens / c.blk + 2ll * c.n_seqs;
    return (unsigned)(most < c.n_tokens ? most : c.n_tokens) + 1;
}

typedef void (*WriteKernel)(KvView, const uint16_t*, const uint16_t*, long long, long long);
typedef void (*ReadKernel)(KvView, uint16_t*, uint16_t*, long long, long long);

template <int FMT, int D, int BLK>
struct Kernels {
    static WriteKernel get(const uint16_t*) { return kv_write_kernel<FMT, D, BLK>; }
    static ReadKernel get(uint16_t*) { return kv_read_kernel<FMT, D, BLK>; }
};
template <int FMT, int D, class P>
auto by_block(int blk, P tag)
{
    return blk == 32 ? Kernels<FMT, D, 32>::get(tag) : blk == 64 ? Kernels<FMT, D, 64>::get(tag) : Kernels<FMT, D, 128>::get(tag);
}
// The kernel of a cache's format, head size and block; the tag's type says write or read.
template <class P>
auto kernel_of(const KvView& c, P tag)
{
    if (c.fmt == MOE_KV_E4M3)
        return c.D == 64 ? by_block<MOE_KV_E4M3, 64>(c.blk, tag) : by_block<MOE_KV_E4M3, 128>(c.blk, tag);
    return c.D == 64 ? by_block<MOE_KV_INT8, 64>(c.blk, tag) : by_block<MOE_KV_INT8, 128>(c.blk, tag);
}

}  // namespace

cudaError_t launch_kv_write(const KvView& c, const uint16_t* k, const uint16_t* v, long long k_stride,
                            long long v_stride, cudaStream_t s)
{
    const dim3 grid(touched_grid(c), c.H, 2);
    const size_t smem = (size_t)c.blk * (c.D / 2 + 1) * 4;
    kernel_of(c, k)<<<grid, kWriteThreads, smem, s>>>(c, k, v, k_stride, v_stride);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, long long k_stride, long long v_stride,
                           cudaStream_t s)
{
    const dim3 grid(touched_grid(c), c.H);
    const size_t smem = (size_t)c.blk * c.D;
    kernel_of(c, k)<<<grid, kReadThreads, smem, s>>>(c, k, v, k_stride, v_stride);
    return cudaGetLastError();
}

}  // namespace moe
