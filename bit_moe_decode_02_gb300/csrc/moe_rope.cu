// moe_rope.cu -- rotary positions of queries and keys.
//
// Pair i of a head turns by the angle pos * f_i: (u, v) -> (u cos - v sin, v cos + u sin).
// The angle is kept as a fraction of a turn: f_i / 2 pi as a 64-bit fraction, times the
// position, modulo 2^64, which wraps exactly; its top bits, as a signed number of half
// turns, are what sincospif takes.  fp32 angles would be off by pos * 2^-24 radians.
//
// Bound by HBM for prompts (each value read and written once), by latency for a few
// tokens.  A CTA takes some tokens: cosines and sines once for each (token, pair), in
// shared memory, then 16 bytes of each half of a pair at a time, over all heads of
// queries and keys.
#include <cstdint>

#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;             // of a CTA
constexpr int kAhead = 4;                 // units of a thread whose loads go out together

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
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ float round(float x) { return x; }
};

__device__ __forceinline__ void turn(float2 cs, float u, float v, float& a, float& b)
{
    a = u * cs.x - v * cs.y;
    b = v * cs.x + u * cs.y;
}

// VEC: 16 bytes at a time; else a pair (or a value of the rest) at a time.  A head's
// units are its pairs' and then, where the rest of the head has to be copied, its.
template <class T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a)
{
    using V = Vec<T>;
    constexpr int P = VEC ? (HALF ? V::N : V::N / 2) : 1;      // pairs of a unit
    extern __shared__ float2 table[];                          // [tokens][rot / 2]
    __shared__ int s_pos[kMaxTokens];
    const int tid = threadIdx.x, np = a.rot / 2, t0 = blockIdx.x * a.per_cta, nt = min(a.per_cta, a.n_tokens - t0);
    const int turning = np / P, rest = a.copy_rest ? (a.D - a.rot) / (VEC ? V::N : 1) : 0, per_head = turning + rest;
    const int heads = a.q_heads + a.k_heads, h0 = blockIdx.y * a.heads_per_cta, nh = min(a.heads_per_cta, heads - h0);
    const int units = nt * nh * per_head;

    struct Unit {
        const T* in;
        T* out;
        int t, at;       // token of the CTA (-1: none), unit of the head
    };
    auto unit = [&](int i) {
        Unit u;
        u.t = -1;
        if (i >= units)
            return u;
        const int head = i / per_head, h = h0 + head % nh;
        u.at = i - head * per_head;
        u.t = head / nh;
        const long long t = t0 + u.t;
        if (h < a.q_heads) {
            u.in = static_cast<const T*>(a.q) + t * a.q_stride + (long long)h * a.D;
            u.out = static_cast<T*>(a.q_out) + t * a.q_out_stride + (long long)h * a.D;
        } else {
            u.in = static_cast<const T*>(a.k) + t * a.k_stride + (long long)(h - a.q_heads) * a.D;
            u.out = static_cast<T*>(a.k_out) + t * a.k_out_stride + (long long)(h - a.q_heads) * a.D;
        }
        return u;
    };
    Unit u[kAhead];
    uint4 x[kAhead], y[kAhead];                                // VEC: what was read
    float xs[kAhead], ys[kAhead];
    auto load = [&](int i0) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            u[e] = unit(i0 + e * kThreads);
            if (u[e].t < 0)
                continue;
            const int at = u[e].at;
            if constexpr (VEC) {
                const uint4* p = reinterpret_cast<const uint4*>(u[e].in);
                const bool pair = at < turning;
                x[e] = p[pair ? at : at - turning + a.rot / V::N];
                if (HALF && pair)
                    y[e] = p[at + turning];
            } else {
                const bool pair = at < turning;
                xs[e] = V::one(u[e].in[pair ? (HALF ? at : 2 * at) : at - turning + a.rot]);
                if (pair)
                    ys[e] = V::one(u[e].in[HALF ? at + np : 2 * at + 1]);
            }
        }
    };
    load(tid);
    if (tid < nt)
        s_pos[tid] = a.position[t0 + tid];
    __syncthreads();
    for (int i = tid; i < nt * np; i += kThreads) {
        const int t = i / np, p = i - t * np;
        const long long phase = (long long)(a.turns[p] * (unsigned long long)(long long)s_pos[t]);
        float s, c;
        sincospif((float)phase * 0x1p-63f, &s, &c);            // 2^63: half a turn
        table[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    for (int i0 = tid; i0 < units; i0 += kAhead * kThreads) {
        if (i0 != tid)
            load(i0);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (u[e].t < 0 || s_pos[u[e].t] < 0)
                continue;
            const int at = u[e].at;
            const float2* cs = table + u[e].t * np + at * P;
            if constexpr (VEC) {
                uint4* p = reinterpret_cast<uint4*>(u[e].out);
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
                    u[e].out[at - turning + a.rot] = V::round(xs[e]);
                    continue;
                }
                float v, w;
                turn(cs[0], xs[e], ys[e], v, w);
                u[e].out[HALF ? at : 2 * at] = V::round(v);
                u[e].out[HALF ? at + np : 2 * at + 1] = V::round(w);
            }
        }
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
    a.per_cta = kThreads / np < 1 ? 1 : kThreads / np > kMaxTokens ? kMaxTokens : kThreads / np;
    // few tokens: one a CTA, and their heads over several, a unit a thread
    if (a.n_tokens < 2 * num_sms * a.per_cta)
        a.per_cta = 1;
    a.heads_per_cta = heads;
    if (a.n_tokens < 2 * num_sms) {
        const int per_head = vec ? (half ? np / n : 2 * np / n) : np;
        const int fit = kThreads / per_head < 1 ? 1 : kThreads / per_head;
        a.heads_per_cta = fit < heads ? fit : heads;
    }
    const dim3 grid((a.n_tokens + a.per_cta - 1) / a.per_cta, (heads + a.heads_per_cta - 1) / a.heads_per_cta);
    const Kernel k = a.type == MOE_DT_BF16 ? pick<uint16_t>(half, vec) : pick<float>(half, vec);
    k<<<grid, kThreads, (size_t)a.per_cta * np * sizeof(float2), s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
