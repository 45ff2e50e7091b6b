// moe_kv4.cu -- the 4-bit paged key/value cache: tokens quantised as they are written,
// and read back.
//
// A group of 32 values of one token and head has a power-of-two scale of its own, so a
// token's codes depend on nothing but its values: no block is quantised again as it
// grows.  V lies transposed (kv4_device.cuh); 8 x 8 nibbles are turned in registers.
// Measured: 6 prompts of 2,700 tokens on average, 4 heads of 128 (34 MB in, 9 MB out),
// written and read back 21.6 us: the write about 11, waiting for loads (sequence -> block
// -> values) behind 0.55 of the issue slots, the read about 10.  One token for each of 5
// sequences 4.3 and 2.6 us; of 64, 256 and 1,024 sequences (8 heads of 64) 4.8, 5.4 and
// 13.1 us, since a CTA finds its sequence with one load a thread.
#include <cstdint>
#include <type_traits>

#include "kv4_device.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;                 // units of 16 values of K, and of V, of a thread whose loads are out at once

// The idx-th block that a batch's tokens touch: by each warp for itself, or of more than 32
// sequences by the whole CTA, four sequences a thread at most.
struct Found {
    kv::Touched t;
    int warps[kThreads / 32];
    int hit;
};
__device__ __forceinline__ bool find(const KvView& c, int idx, Found& f, kv::Touched& t)
{
    const int tid = threadIdx.x, lane = tid & 31, per = (c.n_seqs + kThreads - 1) / kThreads;
    if (c.n_seqs <= 32)
        return kv::find_touched(c, idx, t);
    auto blocks = [&](int b, int& c0, int& n, int& len) {
        if (!kv::sequence(c, b, c0, n, len)) {
            atomicExch(c.status, MOE_ERR_DEVICE_FAULT);
            n = 0;
        }
        return n > 0 ? (len - 1) / c.blk - (len - n) / c.blk + 1 : 0;
    };
    int sum = 0, c0, n, len;
#pragma unroll 1
    for (int i = 0; i < per; ++i)
        if (per * tid + i < c.n_seqs)
            sum += blocks(per * tid + i, c0, n, len);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        f.warps[tid >> 5] = incl;
    if (tid == 0)
        f.hit = 0;
    __syncthreads();
    for (int w = 0; w < tid >> 5; ++w)
        incl += f.warps[w];
    if (idx < incl && idx >= incl - sum) {
        int at = incl - sum;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int b = per * tid + i, cnt = b < c.n_seqs ? blocks(b, c0, n, len) : 0;
            if (idx < at + cnt) {
                f.t = kv::Touched{b, c0, n, len, (len - n) / c.blk + idx - at};
                f.hit = 1;
                break;
            }
            at += cnt;
        }
    }
    __syncthreads();
    t = f.t;
    return f.hit;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t finite_bits(uint32_t w)
{
    const uint32_t x = w & 0x7fffu, y = w >> 16 & 0x7fffu;
    return max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u);
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two bf16 times a power of two, exact but below 2^-126.
__device__ __forceinline__ uint32_t mul_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Eight values -> eight codes, each rounded once to nearest even, saturating.
__device__ __forceinline__ uint32_t to_codes(const uint32_t (&w)[4])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(lo_bf16(w[0])), "f"(hi_bf16(w[0])), "f"(lo_bf16(w[1])), "f"(hi_bf16(w[1])), "f"(lo_bf16(w[2])), "f"(hi_bf16(w[2])),
          "f"(lo_bf16(w[3])), "f"(hi_bf16(w[3])));
    return r;
}

// Half of a group's 32 values, the others in the lane beside it -> sixteen codes, and the
// group's scale byte.
__device__ __forceinline__ uint2 encode16(const uint4& p, const uint4& q, uint32_t& byte)
{
    uint32_t w[2][4] = {{p.x, p.y, p.z, p.w}, {q.x, q.y, q.z, q.w}};
    // largest magnitude of each half of the words, as bits: NaN and infinities above all others
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            m = max2(m, w[h][e] & 0x7fff7fffu);
    m = max2(m, __shfl_xor_sync(~0u, m, 1));
    uint32_t big = max(m & 0xffffu, m >> 16);
    if (__any_sync(~0u, big >= 0x7f80u)) {
        // NaN or infinity among the warp's values: the largest of the others; NaN becomes 0
        m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                m = max(m, finite_bits(w[h][e]));
                w[h][e] &= ((w[h][e] & 0x7fffu) > 0x7f80u ? 0u : 0xffffu) | ((w[h][e] & 0x7fff0000u) > 0x7f800000u ? 0u : 0xffff0000u);
            }
        big = max(m, __shfl_xor_sync(~0u, m, 1));
    }
    byte = kv4::scale_byte(big);
    const uint32_t inv = ((254u - byte) << 7) * 0x10001u;      // 2^-e
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[h][e] = mul_bf16(w[h][e], inv);
    return byte ? make_uint2(to_codes(w[0]), to_codes(w[1])) : make_uint2(0, 0);
}

// One CTA per (touched block, some heads): heads, as many as fit the buffer, at a time.
template <int D, int blk>
__global__ void __launch_bounds__(kThreads, 4)
kv4_write_kernel(KvView c, const uint16_t* __restrict__ ksrc, const uint16_t* __restrict__ vsrc, long long kstride, long long vstride,
                 int heads_per_cta)
{
    __shared__ __align__(8) uint32_t codes[blk * (D / 8)];     // V as written by token: [head][token][D / 8] words
    __shared__ Found found;
    constexpr int W = D / 8, U = D / 16, REC = kv4::record(blk, D);     // words and units of a token's head
    const int tid = threadIdx.x;
    kv::Touched t;
    if (!find(c, blockIdx.x, found, t))
        return;
    const int id = kv::physical(c, t.b, t.j);
    if (id < 0)
        return;
    const int start = t.len - t.n - t.j * blk;                 // offset of the sequence's first new token
    const int lo = start > 0 ? start : 0, hi = min(t.len - t.j * blk, blk), n = hi - lo;
    const bool fresh = lo == 0;
    const long long row0 = t.c0 - start + lo;
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, c.H), batch = blk / n;
    for (int hb = h0; hb < h1; hb += batch) {
        const int nh = min(batch, h1 - hb), units = nh * n * U;
        uint8_t* rec = c.codes + ((long long)id * c.H + hb) * 2 * REC;
        // row i of a head's `per`
        auto split = [&](int i, int per, int& h, int& r) {
            h = nh == 1 ? 0 : i / per;
            r = i - h * per;
        };
        for (int i0 = tid; i0 - tid < units; i0 += kAhead * kThreads) {
            uint4 k[kAhead][2], v[kAhead][2];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + e * kThreads, x = i % U;
                int h, r;
                split(i / U, n, h, r);
                k[e][0] = k[e][1] = v[e][0] = v[e][1] = make_uint4(0, 0, 0, 0);
                if (i < units) {
                    const long long col = (long long)(hb + h) * D + x * 16;
                    const uint4* kp = reinterpret_cast<const uint4*>(ksrc + (row0 + r) * kstride + col);
                    const uint4* vp = reinterpret_cast<const uint4*>(vsrc + (row0 + r) * vstride + col);
                    k[e][0] = kp[0], k[e][1] = kp[1];
                    v[e][0] = vp[0], v[e][1] = vp[1];
                }
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + e * kThreads, x = i % U;
                if (i0 - tid + e * kThreads >= units)
                    break;
                uint32_t kb, vb;
                const uint2 kc = encode16(k[e][0], k[e][1], kb), vc = encode16(v[e][0], v[e][1], vb);
                if (i >= units)
                    continue;
                int h, r;
                split(i / U, n, h, r);
                const int tok = lo + r;
                uint8_t* kr = rec + (long long)h * 2 * REC;
                reinterpret_cast<uint2*>(kr)[tok * U + x] = kc;
                reinterpret_cast<uint2*>(codes)[i] = vc;
                // a lane of the group's two writes K's scale, the other V's
                const int g = x / 2;
                if (x % 2 == 0)
                    kr[blk * D / 2 + kv4::k_scale_at<D>(tok, g)] = (uint8_t)kb;
                else
                    kr[REC + blk * D / 2 + kv4::v_scale_at<D>(tok, g)] = (uint8_t)vb;
            }
        }
        __syncthreads();
        // V: eight tokens by eight d's; words that hold other tokens too are merged
        const int t8lo = lo / 8, nt8 = (fresh ? blk / 8 : (hi + 7) / 8) - t8lo, pieces = nh * nt8 * W;
        for (int i = tid; i < pieces; i += kThreads) {
            const int x = i % W;
            int h, t8;
            split(i / W, nt8, h, t8);
            t8 += t8lo;
            uint32_t w[8], keep = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int tok = t8 * 8 + k;
                const bool in = tok >= lo && tok < hi;
                w[k] = in ? codes[(h * n + tok - lo) * W + x] : 0u;
                keep |= in || fresh ? 0u : 0xfu << 4 * k;
            }
            kv4::transpose(w);
            uint32_t* vr = reinterpret_cast<uint32_t*>(rec + ((long long)h * 2 + 1) * REC);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                uint32_t* p = vr + kv4::v_word_at<D>(t8, x / 4, x % 4, r);
                *p = keep ? (w[r] & ~keep) | (*p & keep) : w[r];
            }
        }
        if (fresh && hi < blk) {
            // unwritten tokens of a block whose first token came
            for (int i = tid; i < nh * (blk - hi) * W; i += kThreads) {
                const int x = i % W;
                int h, r;
                split(i / W, blk - hi, h, r);
                const int tok = hi + r;
                uint8_t* kr = rec + (long long)h * 2 * REC;
                reinterpret_cast<uint32_t*>(kr)[tok * W + x] = 0u;
                if (x % 4 == 0) {
                    kr[blk * D / 2 + kv4::k_scale_at<D>(tok, x / 4)] = 0;
                    kr[REC + blk * D / 2 + kv4::v_scale_at<D>(tok, x / 4)] = 0;
                }
            }
        }
        __syncthreads();
    }
}

// Eight codes -> eight bf16, times the scale, rounded once.
__device__ __forceinline__ uint4 decode8(uint32_t w, float s)
{
    uint32_t h[4], o[4];
    kv4::to_f16(w, h);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        o[e] = kv::bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// One CTA per (touched block, head): V's nibbles are turned back into shared memory, then
// both go out by token.
template <int D, int blk>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(KvView c, uint16_t* __restrict__ kdst, uint16_t* __restrict__ vdst, long long kstride, long long vstride, int heads_per_cta)
{
    __shared__ uint32_t codes[blk * (D / 8 + 1)];
    __shared__ Found found;
    constexpr int W = D / 8, REC = kv4::record(blk, D);
    const int tid = threadIdx.x;
    kv::Touched t;
    if (!find(c, blockIdx.x, found, t))
        return;
    const int id = kv::physical(c, t.b, t.j);
    if (id < 0)
        return;
    const int start = t.len - t.n - t.j * blk;
    const int lo = start > 0 ? start : 0, hi = min(t.len - t.j * blk, blk), n = hi - lo;
    const long long row0 = t.c0 - start + lo;
    const int t8lo = lo / 8, nt8 = (hi + 7) / 8 - t8lo, h1 = min((int)(blockIdx.y + 1) * heads_per_cta, c.H);
    for (int h = blockIdx.y * heads_per_cta; h < h1; ++h) {
        const uint8_t* kr = c.codes + ((long long)id * c.H + h) * 2 * REC;
        const uint8_t* vr = kr + REC;
        // all of a thread's words of K, and its share of V's, are on their way before the first is used
        constexpr int kK = (blk * W + kThreads - 1) / kThreads, kV = (blk / 8 * W + kThreads - 1) / kThreads;
        uint32_t kw[kK], vw[kV][8];
        uint8_t kb[kK], vb[kK];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int i = tid + j * kThreads, x = i % W, t8 = t8lo + i / W;
            if (i < nt8 * W)
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    vw[j][r] = reinterpret_cast<const uint32_t*>(vr)[kv4::v_word_at<D>(t8, x / 4, x % 4, r)];
        }
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            const int i = tid + j * kThreads, x = i % W, tok = lo + i / W;
            if (i < n * W) {
                kw[j] = reinterpret_cast<const uint32_t*>(kr)[tok * W + x];
                kb[j] = kr[blk * D / 2 + kv4::k_scale_at<D>(tok, x / 4)];
                vb[j] = vr[blk * D / 2 + kv4::v_scale_at<D>(tok, x / 4)];
            }
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int i = tid + j * kThreads, x = i % W, t8 = t8lo + i / W;
            if (i < nt8 * W) {
                kv4::transpose(vw[j]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    codes[(t8 * 8 + k) * (W + 1) + x] = vw[j][k];
            }
        }
        uint16_t* const kd = kdst + row0 * kstride + (long long)h * D;
        uint16_t* const vd = vdst + row0 * vstride + (long long)h * D;
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            const int i = tid + j * kThreads, x = i % W, r = i / W;
            if (i < n * W)
                *reinterpret_cast<uint4*>(kd + r * kstride + x * 8) = decode8(kw[j], kv4::scale_of(kb[j]));
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            const int i = tid + j * kThreads, x = i % W, r = i / W;
            if (i < n * W)
                *reinterpret_cast<uint4*>(vd + r * vstride + x * 8) = decode8(codes[(lo + r) * (W + 1) + x], kv4::scale_of(vb[j]));
        }
        __syncthreads();                                       // before the next head's V
    }
}

// As for the 8-bit cache: an upper bound on the blocks that a batch touches, and one more,
// whose CTA finds none and so checks every sequence.
unsigned touched_grid(const KvView& c)
{
    const long long most = (long long)c.n_tokens / c.blk + 2ll * c.n_seqs;
    return (unsigned)(most < c.n_tokens ? most : c.n_tokens) + 1;
}

// Heads of a CTA: finding the block costs as much as a third of a head's work, so several
// as long as every SM has three CTAs.
int heads_for(const KvView& c, int num_sms)
{
    int heads = 1;
    while (2 * heads <= c.H && (long long)touched_grid(c) * (c.H / (2 * heads)) >= 3 * num_sms)
        heads *= 2;
    return heads;
}

template <class F>
void by_size(const KvView& c, F f)
{
    auto block = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (c.blk == 32)
            f(d, std::integral_constant<int, 32>());
        else if (c.blk == 64)
            f(d, std::integral_constant<int, 64>());
        else
            f(d, std::integral_constant<int, 128>());
        (void)D;
    };
    if (c.D == 64)
        block(std::integral_constant<int, 64>());
    else
        block(std::integral_constant<int, 128>());
}

}  // namespace

cudaError_t launch_kv4_write(const KvView& c, const uint16_t* k, const uint16_t* v, long long k_stride, long long v_stride, cudaStream_t s)
{
    // single tokens: as many heads a CTA as fill it
    const int tokens = (c.n_tokens + c.n_seqs - 1) / c.n_seqs, fit = kThreads / (c.D / 16) / tokens;
    const int heads = fit < 1 ? 1 : fit < c.H ? fit : c.H;
    const dim3 grid(touched_grid(c), (c.H + heads - 1) / heads);
    by_size(c, [&](auto d, auto b) {
        kv4_write_kernel<decltype(d)::value, decltype(b)::value><<<grid, kThreads, 0, s>>>(c, k, v, k_stride, v_stride, heads);
    });
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const KvView& c, uint16_t* k, uint16_t* v, long long k_stride, long long v_stride, int num_sms, cudaStream_t s)
{
    const int heads = heads_for(c, num_sms);
    const dim3 grid(touched_grid(c), (c.H + heads - 1) / heads);
    by_size(c, [&](auto d, auto b) {
        kv4_read_kernel<decltype(d)::value, decltype(b)::value><<<grid, kThreads, 0, s>>>(c, k, v, k_stride, v_stride, heads);
    });
    return cudaGetLastError();
}

}  // namespace moe
