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

// One CTA per (touched block, head, K or V): the largest finite magnitude of
// the block's new tokens sets the scale (never below the block's old one if it
// holds earlier tokens, whose codes are rounded again where it grew), then
// every new value is divided by it and rounded once.
// Memory-bound: 2 bytes in and 1 out per value.
template <int FMT, int D, int blk>
__global__ void __launch_bounds__(kWriteThreads)
kv_write_kernel(KvView c, const uint16_t* __restrict__ ksrc, const uint16_t* __restrict__ vsrc, long long kstride,
                long long vstride)
{
    extern __shared__ uint32_t tile[];   // [blk][D/2 + 1] words of two bf16
    __shared__ float red[kWriteThreads / 32];
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

    float amax = 0.0f;
    for (int i = tid; i < (hi - lo) * vec; i += kWriteThreads) {
        const int r = i / vec, x = i % vec;
        const uint4 q = *reinterpret_cast<const uint4*>(src + r * stride + x * 8);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t m0 = w[e] << 16 & 0x7fff0000u, m1 = w[e] & 0x7fff0000u;
            if (m0 < 0x7f800000u)
                amax = fmaxf(amax, __uint_as_float(m0));
            if (m1 < 0x7f800000u)
                amax = fmaxf(amax, __uint_as_float(m1));
            tile[(lo + r) * pitch + x * 4 + e] = w[e];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if ((tid & 31) == 0)
        red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWriteThreads / 32; ++i)
        amax = fmaxf(amax, red[i]);

    float* sp = c.scales + ((long long)id * c.H + h) * 2 + which;
    const bool fresh = lo == 0;
    float scale = kv::block_scale<FMT>(amax), ratio = 0.0f;
    const float old = fresh ? 0.0f : *sp;
    const bool grown = !fresh && scale > old;
    if (!fresh && !grown)
        scale = old;
    const float inv = __fdiv_rn(1.0f, scale);
    if (grown)
        ratio = old * inv;
    __syncthreads();                                           // every thread has read the old scale
    if (tid == 0 && (fresh || grown))
        *sp = scale;

    uint8_t* dst = c.codes + (((long long)id * c.H + h) * 2 + which) * ((long long)blk * D);
    const int first = fresh || grown ? 0 : lo, last = fresh ? blk : hi;   // tokens whose codes change
    if (which == 0) {
        for (int i = tid; i < (last - first) * vec; i += kWriteThreads) {
            const int r = first + i / vec, x = i % vec;
            uint2* p = reinterpret_cast<uint2*>(dst + r * D + x * 8);
            uint2 o = make_uint2(0, 0);
            if (r < lo) {
                const uint2 was = *p;
                float v[4], u[4];
                kv::decode4<FMT>(was.x, v);
                kv::decode4<FMT>(was.y, u);
                o.x = kv::encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
                o.y = kv::encode4<FMT>(u[0] * ratio, u[1] * ratio, u[2] * ratio, u[3] * ratio);
            } else if (r < hi) {
                const uint32_t* w = tile + r * pitch + x * 4;
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[2 * e] = __uint_as_float(w[e] << 16) * inv;
                    v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * inv;
                }
                o.x = kv::encode4<FMT>(v[0], v[1], v[2], v[3]);
                o.y = kv::encode4<FMT>(v[4], v[5], v[6], v[7]);
            }
            *p = o;
        }
    } else {
        // 16 tokens of one d at a time: the bytes of tokens that keep their
        // codes are read and written back as they were
        const int g0 = first / 16, gs = (last + 15) / 16 - g0;
        const uint16_t* t16 = reinterpret_cast<const uint16_t*>(tile);
        for (int i = tid; i < D * gs; i += kWriteThreads) {
            const int d = i / gs, g = g0 + i % gs;
            uint4* p = reinterpret_cast<uint4*>(dst + d * blk + g * 16);
            const bool keep = !fresh && (g * 16 < lo || g * 16 + 16 > hi);
            const uint4 was = keep ? *p : make_uint4(0, 0, 0, 0);
            const uint32_t wa[4] = {was.x, was.y, was.z, was.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t0 = g * 16 + 4 * e;
                uint32_t w = wa[e];
                if (t0 < lo && grown) {
                    float v[4];
                    kv::decode4<FMT>(w, v);
                    const uint32_t again = kv::encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
                    const uint32_t m = t0 + 4 <= lo ? ~0u : (1u << 8 * (lo - t0)) - 1;
                    w = (w & ~m) | (again & m);
                }
                if (t0 + 4 > lo && t0 < hi) {
                    float v[4];
                    uint32_t m = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int tok = t0 + b;
                        v[b] = 0.0f;
                        if (tok >= lo && tok < hi) {
                            v[b] = tc::bf16f(t16[tok * 2 * pitch + d]) * inv;
                            m |= 0xffu << 8 * b;
                        }
                    }
                    w = (w & ~m) | (kv::encode4<FMT>(v[0], v[1], v[2], v[3]) & m);
                }
                o[e] = w;
            }
            *p = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

constexpr int kReadThreads = 128;

// One CTA per (touched block, head, K or V): codes times the scale, rounded
// to bf16 once.  V comes back through 4 x 4 byte transposes in registers.
template <int FMT, int D, int blk>
__global__ void __launch_bounds__(kReadThreads)
kv_read_kernel(KvView c, uint16_t* __restrict__ kdst, uint16_t* __restrict__ vdst, long long kstride, long long vstride)
{
    extern __shared__ uint32_t tile[];   // V: [D][blk/4] words
    const int h = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
    kv::Touched t;
    if (!kv::find_touched(c, blockIdx.x, t))
        return;
    const int id = kv::physical(c, t.b, t.j);
    if (id < 0)
        return;
    const int start = t.len - t.n - t.j * blk;
    const int lo = start > 0 ? start : 0, hi = min(t.len - t.j * blk, blk);
    const float scale = c.scales[((long long)id * c.H + h) * 2 + which];
    const uint8_t* src = c.codes + (((long long)id * c.H + h) * 2 + which) * ((long long)blk * D);
    uint16_t* dst = which ? vdst : kdst;
    const long long stride = which ? vstride : kstride;
    dst += (long long)(t.c0 - start) * stride + (long long)h * D;   // row of the block's token 0
    if (which == 0) {
        constexpr int vec = D / 8;
        for (int i = tid; i < (hi - lo) * vec; i += kReadThreads) {
            const int r = lo + i / vec, x = i % vec;
            const uint2 w = *reinterpret_cast<const uint2*>(src + r * D + x * 8);
            float v[4], u[4];
            kv::decode4<FMT>(w.x, v);
            kv::decode4<FMT>(w.y, u);
            uint4 o;
            o.x = kv::bf16x2(v[0] * scale, v[1] * scale);
            o.y = kv::bf16x2(v[2] * scale, v[3] * scale);
            o.z = kv::bf16x2(u[0] * scale, u[1] * scale);
            o.w = kv::bf16x2(u[2] * scale, u[3] * scale);
            *reinterpret_cast<uint4*>(dst + r * stride + x * 8) = o;
        }
        return;
    }
    // word w of row d lies at w ^ (d / 4): the four rows of a transpose are
    // read by 32 lanes with few bank conflicts
    constexpr int wpr = blk / 4;
    for (int i = tid; i < D * wpr; i += kReadThreads) {
        const int d = i / wpr, w = i % wpr;
        tile[d * wpr + (w ^ (d >> 2 & (wpr - 1)))] = reinterpret_cast<const uint32_t*>(src)[i];
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
            if (tok < lo || tok >= hi)
                continue;
            float v[4];
            kv::decode4<FMT>(col[k], v);
            uint2 o;
            o.x = kv::bf16x2(v[0] * scale, v[1] * scale);
            o.y = kv::bf16x2(v[2] * scale, v[3] * scale);
            *reinterpret_cast<uint2*>(dst + tok * stride + d4 * 4) = o;
        }
    }
}

// Upper bound on the blocks that a batch touches: a sequence with n >= 1 new
// tokens touches at most (n - 1) / blk + 2, and no more than n.
int touched_bound(const KvView& c)
{
    const long long most = (long long)c.n_tokens / c.blk + 2ll * c.n_seqs;
    return (int)(most < c.n_tokens ? most : c.n_tokens);
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
    const dim3 grid(touched_bound(c), c.H, 2);
    const size_t smem = (size_t)c.blk * (c.D / 2 + 1) * 4;
    kernel_of(c, k)<<<grid, kWriteThreads, smem, s>>>(c, k, v, k_stride, v_stride);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, long long k_stride, long long v_stride,
                           cudaStream_t s)
{
    const dim3 grid(touched_bound(c), c.H, 2);
    const size_t smem = (size_t)c.blk * c.D;
    kernel_of(c, k)<<<grid, kReadThreads, smem, s>>>(c, k, v, k_stride, v_stride);
    return cudaGetLastError();
}

}  // namespace moe
