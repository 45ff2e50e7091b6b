// moe_rope.cu -- rotary positions of queries and keys.
//
// Pair i of a head turns by the angle pos * f_i: (u, v) -> (u cos - v sin, v cos + u sin).
// The angle is kept as a fraction of a turn: f_i / 2 pi as a 64-bit fraction, times the
// position, modulo 2^64, which wraps exactly; its top bits, as a signed number of half
// turns, are what sincospif takes.  fp32 angles would be off by pos * 2^-24 radians.
//
// Bound by HBM for prompts (each value read and written once), by latency for a few
// tokens.  A CTA takes a token: cosines and sines once for each pair, through shared
// memory, while the first heads' values are on their way; then 16 bytes of each half of a
// pair at a time, over all heads of queries and keys.  Measured: 11,363 tokens of 36 heads
// of 128, 96 of them turned in adjacent pairs, bf16 in and out (209 MB): 32.8 us, 6.4 TB/s,
// 0.94 of a plain copy; 7 tokens of 72 heads of 64: 2.0 us, the chain position -> angle ->
// cosine -> product of one launch.
#include <cstdint>

#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;                 // heads of a thread whose loads go out together
constexpr int kStage = 12288;             // bytes of heads that the staged kernel takes at once

template <class T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& w, float (&x)[8])
    {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(v[e] << 16);
            x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8])
    {
        return make_uint4(kv::bf16x2(x[0], x[1]), kv::bf16x2(x[2], x[3]), kv::bf16x2(x[4], x[5]), kv::bf16x2(x[6], x[7]));
    }
    struct __align__(4) Two {
        uint16_t x, y;
    };
    static __device__ __forceinline__ float one(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t round(float x) { return (uint16_t)kv::bf16x2(x, 0.0f); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& w, float (&x)[4])
    {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    typedef float2 Two;
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ float round(float x) { return x; }
};

__device__ __forceinline__ void turn(float2 cs, float u, float v, float& a, float& b)
{
    a = u * cs.x - v * cs.y;
    b = v * cs.x + u * cs.y;
}

// Where a token's heads are.
template <class T>
struct Heads {
    const T *qi, *ki;
    T *qo, *ko;
    int q_heads, D;
    __device__ __forceinline__ explicit Heads(const RopeArgs& a, long long t) : q_heads(a.q_heads), D(a.D)
    {
        qi = static_cast<const T*>(a.q) + t * a.q_stride;
        ki = static_cast<const T*>(a.k) + t * a.k_stride - (long long)a.q_heads * a.D;
        qo = static_cast<T*>(a.q_out) + t * a.q_out_stride;
        ko = static_cast<T*>(a.k_out) + t * a.k_out_stride - (long long)a.q_heads * a.D;
    }
    __device__ __forceinline__ const uint4* in(int h) const { return reinterpret_cast<const uint4*>((h < q_heads ? qi : ki) + h * D); }
    __device__ __forceinline__ uint4* out(int h) const { return reinterpret_cast<uint4*>((h < q_heads ? qo : ko) + h * D); }
};

// Cosines and sines of a token's pairs, times mscale.
__device__ __forceinline__ void make_table(const RopeArgs& a, int pos, float2* table)
{
    for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) {
        const long long phase = (long long)(a.turns[i] * (unsigned long long)pos);
        float s, c;
        sincospif((float)phase * 0x1p-63f, &s, &c);            // 2^63: half a turn
        table[i] = make_float2(c * a.mscale, s * a.mscale);
    }
}

// rot_dim in whole vectors of 16 bytes (HALF: each half).  A head's units are its pairs'
// vectors and then, where the rest of the head has to be copied, its.  A thread keeps its
// unit of the head, with its cosines and sines, and walks over the heads.
template <class T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a)
{
    using V = Vec<T>;
    constexpr int P = HALF ? V::N : V::N / 2;                  // pairs of a unit
    extern __shared__ __align__(16) uint8_t smem[];
    float2* table = reinterpret_cast<float2*>(smem);           // [rot / 2]
    const int tid = threadIdx.x, turning = a.rot / 2 / P, per_head = turning + (a.copy_rest ? (a.D - a.rot) / V::N : 0);
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, a.q_heads + a.k_heads);
    const Heads<T> heads(a, blockIdx.x);
    const int row = tid / per_head, step = kThreads / per_head, at = tid - row * per_head;     // at most 128 units
    const int first = row < step ? h0 + row : h1;
    const bool pair = at < turning;
    const int from = pair ? at : at - turning + a.rot / V::N;  // the unit's first vector
    uint4 x[kAhead], y[kAhead];
    auto load = [&](int h) {                                   // kAhead heads from h on
#pragma unroll
        for (int e = 0; e < kAhead; ++e, h += step)
            if (h < h1) {
                x[e] = heads.in(h)[from];
                if (HALF && pair)
                    y[e] = heads.in(h)[at + turning];
            }
    };
    const int pos = a.position[blockIdx.x];
    load(first);
    if (pos < 0)
        return;
    make_table(a, pos, table);
    __syncthreads();
    float2 cs[P];
    if (pair)
#pragma unroll
        for (int k = 0; k < P; ++k)
            cs[k] = table[at * P + k];
    for (int h = first; h < h1;) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e, h += step) {
            if (h >= h1)
                continue;
            uint4* p = heads.out(h);
            if (!pair) {
                p[from] = x[e];
                continue;
            }
            float v[V::N], w[V::N];
            V::get(x[e], v);
            if constexpr (HALF) {
                V::get(y[e], w);
#pragma unroll
                for (int k = 0; k < V::N; ++k)
                    turn(cs[k], v[k], w[k], v[k], w[k]);
                p[at] = V::put(v);
                p[at + turning] = V::put(w);
            } else {
#pragma unroll
                for (int k = 0; k < V::N / 2; ++k)
                    turn(cs[k], v[2 * k], v[2 * k + 1], w[2 * k], w[2 * k + 1]);
                p[at] = V::put(w);
            }
        }
        load(h);
    }
}

// Any rot_dim: whole heads through shared memory, where pairs lie as they may.
template <class T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_staged_kernel(RopeArgs a)
{
    using V = Vec<T>;
    extern __shared__ __align__(16) uint8_t smem[];
    T* stage = reinterpret_cast<T*>(smem);                     // [heads_per_pass][D]
    float2* table = reinterpret_cast<float2*>(smem + kStage);  // [rot / 2]
    const int tid = threadIdx.x, np = a.rot / 2, vecs = a.D / V::N;        // at most 128 vectors
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, a.q_heads + a.k_heads);
    const Heads<T> heads(a, blockIdx.x);
    const int row = tid / vecs, step = kThreads / vecs, at = tid - row * vecs;
    const int prow = tid / np, pstep = np < kThreads ? kThreads / np : 1, pat = np < kThreads ? tid - prow * np : tid;
    const int pos = a.position[blockIdx.x];
    if (pos < 0)
        return;
    const int most = kStage / (a.D * (int)sizeof(T));
    for (int hb = h0; hb < h1; hb += most) {
        const int n = min(most, h1 - hb);
        for (int r = row < step ? row : n; r < n;) {
            uint4 x[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (r + e * step < n)
                    x[e] = heads.in(hb + r + e * step)[at];
#pragma unroll
            for (int e = 0; e < kAhead; ++e, r += step)
                if (r < n)
                    reinterpret_cast<uint4*>(stage)[r * vecs + at] = x[e];
        }
        if (hb == h0)
            make_table(a, pos, table);
        __syncthreads();
        for (int p = pat; p < np; p += kThreads) {
            const float2 cs = table[p];
            for (int r = np < kThreads ? (prow < pstep ? prow : n) : 0; r < n; r += pstep) {
                T* u = stage + r * a.D + (HALF ? p : 2 * p);
                float v, w;
                if constexpr (HALF) {
                    turn(cs, V::one(u[0]), V::one(u[np]), v, w);
                    u[0] = V::round(v);
                    u[np] = V::round(w);
                } else {
                    typename V::Two* q = reinterpret_cast<typename V::Two*>(u);
                    turn(cs, V::one(q->x), V::one(q->y), v, w);
                    *q = typename V::Two{V::round(v), V::round(w)};
                }
            }
        }
        __syncthreads();
        for (int r = row < step ? row : n; r < n; r += step)
            heads.out(hb + r)[at] = reinterpret_cast<uint4*>(stage)[r * vecs + at];
        __syncthreads();
    }
}

typedef void (*Kernel)(RopeArgs);
template <class T>
Kernel pick(bool half, bool vec)
{
    return half ? (vec ? rope_kernel<T, true> : rope_staged_kernel<T, true>) : (vec ? rope_kernel<T, false> : rope_staged_kernel<T, false>);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int num_sms, cudaStream_t s)
{
    const bool half = a.layout == MOE_ROPE_HALF;
    const int n = a.type == MOE_DT_BF16 ? 8 : 4, step = half ? 2 * n : n;
    // whole vectors, or through shared memory: 35 and 40 us for 12,333 tokens of 36 heads of 128 in bf16
    const bool vec = a.rot % step == 0;                        // then the rest of the head is whole vectors too
    const int heads = a.q_heads + a.k_heads, np = a.rot / 2;
    // few tokens: their heads over several CTAs, a unit or two a thread
    const int units = vec ? (half ? np / n : 2 * np / n) + (a.copy_rest ? (a.D - a.rot) / n : 0) : a.D / n;
    const int fit = kThreads / units;
    a.heads_per_cta = a.n_tokens < 4 * num_sms && fit < heads ? fit : heads;
    const dim3 grid(a.n_tokens, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
    const Kernel k = a.type == MOE_DT_BF16 ? pick<uint16_t>(half, vec) : pick<float>(half, vec);
    k<<<grid, kThreads, np * sizeof(float2) + (vec ? 0 : kStage), s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
