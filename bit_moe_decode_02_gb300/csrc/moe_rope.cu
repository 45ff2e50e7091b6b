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
// pair at a time, over all heads of queries and keys.
#include <cstdint>

#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;                 // heads of a thread whose loads go out together

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

// VEC: 16 bytes at a time; else a pair (or a value of the rest) at a time.  A head's
// units are its pairs' and then, where the rest of the head has to be copied, its.  A
// thread keeps its unit of the head, with its cosines and sines, and walks over the heads.
template <class T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a)
{
    using V = Vec<T>;
    constexpr int P = VEC ? (HALF ? V::N : V::N / 2) : 1;      // pairs of a unit
    extern __shared__ __align__(16) float2 table[];            // [rot / 2]
    const int tid = threadIdx.x, np = a.rot / 2;
    const long long t = blockIdx.x;
    const int turning = np / P, rest = a.copy_rest ? (a.D - a.rot) / (VEC ? V::N : 1) : 0, per_head = turning + rest;
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, a.q_heads + a.k_heads);
    const int wide = min(per_head, kThreads), step = kThreads / wide;      // heads at a time
    const T* const qi = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* const ki = static_cast<const T*>(a.k) + t * a.k_stride - (long long)a.q_heads * a.D;
    T* const qo = static_cast<T*>(a.q_out) + t * a.q_out_stride;
    T* const ko = static_cast<T*>(a.k_out) + t * a.k_out_stride - (long long)a.q_heads * a.D;
    const int row = tid / wide, first = row < step ? h0 + row : h1;
    int at = tid - row * wide;

    uint4 x[kAhead], y[kAhead];                                // what was read (VEC)
    float xs[kAhead], ys[kAhead];
    auto load = [&](int h) {                                   // kAhead heads from h on
#pragma unroll
        for (int e = 0; e < kAhead; ++e, h += step) {
            if (h >= h1)
                continue;
            const T* p = (h < a.q_heads ? qi : ki) + h * a.D;
            const bool pair = at < turning;
            if constexpr (VEC) {
                const uint4* q = reinterpret_cast<const uint4*>(p);
                x[e] = q[pair ? at : at - turning + a.rot / V::N];
                if (HALF && pair)
                    y[e] = q[at + turning];
            } else if (!pair) {
                xs[e] = V::one(p[at - turning + a.rot]);
            } else if constexpr (HALF) {
                xs[e] = V::one(p[at]);
                ys[e] = V::one(p[at + np]);
            } else {
                const typename V::Two w = reinterpret_cast<const typename V::Two*>(p)[at];
                xs[e] = V::one(w.x);
                ys[e] = V::one(w.y);
            }
        }
    };
    const int pos = a.position[t];
    load(first);
    if (pos < 0)
        return;
    for (int i = tid; i < np; i += kThreads) {
        const long long phase = (long long)(a.turns[i] * (unsigned long long)pos);
        float s, c;
        sincospif((float)phase * 0x1p-63f, &s, &c);            // 2^63: half a turn
        table[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    for (;;) {
        float2 cs[P];
        if (at < turning)
#pragma unroll
            for (int k = 0; k < P; ++k)
                cs[k] = table[at * P + k];
        for (int h = first; h < h1;) {
#pragma unroll
            for (int e = 0; e < kAhead; ++e, h += step) {
                if (h >= h1)
                    continue;
                T* out = (h < a.q_heads ? qo : ko) + h * a.D;
                if constexpr (VEC) {
                    uint4* p = reinterpret_cast<uint4*>(out);
                    if (at >= turning) {
                        p[at - turning + a.rot / V::N] = x[e];
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
                } else {
                    if (at >= turning) {
                        out[at - turning + a.rot] = V::round(xs[e]);
                        continue;
                    }
                    float v, w;
                    turn(cs[0], xs[e], ys[e], v, w);
                    if constexpr (HALF) {
                        out[at] = V::round(v);
                        out[at + np] = V::round(w);
                    } else {
                        reinterpret_cast<typename V::Two*>(out)[at] = typename V::Two{V::round(v), V::round(w)};
                    }
                }
            }
            load(h);
        }
        // heads of more units than the CTA has threads: their next ones
        at += kThreads;
        if (at >= per_head || per_head <= kThreads)
            break;
        load(first);
    }
}

typedef void (*Kernel)(RopeArgs);
template <class T>
Kernel pick(bool half, bool vec)
{
    return half ? (vec ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                : (vec ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int num_sms, cudaStream_t s)
{
    const bool half = a.layout == MOE_ROPE_HALF;
    const int n = a.type == MOE_DT_BF16 ? 8 : 4, step = half ? 2 * n : n;
    const bool vec = a.rot % step == 0;                        // then the rest of the head is whole vectors too
    const int heads = a.q_heads + a.k_heads, np = a.rot / 2;
    // few tokens: their heads over several CTAs, a unit or two a thread
    const int per_head = (vec ? (half ? np / n : 2 * np / n) : np) + (a.copy_rest ? (a.D - a.rot) / (vec ? n : 1) : 0);
    const int fit = kThreads / per_head < 1 ? 1 : kThreads / per_head;
    a.heads_per_cta = a.n_tokens < 4 * num_sms && fit < heads ? fit : heads;
    const dim3 grid(a.n_tokens, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
    const Kernel k = a.type == MOE_DT_BF16 ? pick<uint16_t>(half, vec) : pick<float>(half, vec);
    k<<<grid, kThreads, (size_t)np * sizeof(float2), s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
