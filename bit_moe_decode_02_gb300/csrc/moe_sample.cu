// moe_sample.cu -- the next token of each row of logits, by temperature, top-k,
// top-p and min-p from a given random number.
//
// Every weight w_i = e^{z_i}, z_i = (l_i - max l) / T <= 0, is rounded to a
// multiple of 2^-31, so sums of weights are integers: exact, and the same in
// every order.  The kept set is a prefix of the order "larger logit first, then
// lower index", found by its last member: a key (the logit's order-preserving
// bits) and how many of the tokens that share that key are in.
#include <cstdint>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
typedef unsigned long long u64;

// Larger float, larger key; NaN below everything, as -inf.
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (f != f)
        f = -INFINITY;
    if (f == 0.0f)
        f = 0.0f;   // -0 and +0 are the same logit
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float exponent_of(float l, float top, float inv_t)
{
    return l == top ? 0.0f : l == -INFINITY || top == INFINITY ? -INFINITY : (l - top) * inv_t;
}
__device__ __forceinline__ uint32_t weight_of(float z) { return __float2uint_rn(expf(z) * 2147483648.0f); }

__device__ __forceinline__ float load_logit(const SampleArgs& a, int row, int i)
{
    return a.logits_type == MOE_DT_BF16
               ? tc::bf16f(static_cast<const uint16_t*>(a.logits)[row * a.stride + i])
               : static_cast<const float*>(a.logits)[row * a.stride + i];
}

template <class T, class Op>
__device__ __forceinline__ T block_all(T v, Op op, T* red)
{
    for (int o = 16; o; o >>= 1)
        v = op(v, __shfl_xor_sync(~0u, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i)
        v = op(v, red[i]);
    return v;
}

// One CTA per row; every search is a bisection with a pass over the row.
__global__ void __launch_bounds__(kThreads) sample_simple_kernel(SampleArgs a)
{
    __shared__ u64 red[kThreads / 32];
    const int row = blockIdx.x, tid = threadIdx.x, V = a.V;
    auto add = [](u64 x, u64 y) { return x + y; };
    auto mx = [](u64 x, u64 y) { return x > y ? x : y; };
    u64 best = 0;
    for (int i = tid; i < V; i += kThreads)
        best = max(best, (u64)order_key(load_logit(a, row, i)) << 32 | (u64)(0xffffffffu - i));
    best = block_all(best, mx, red);
    const float top = key_value((uint32_t)(best >> 32)), T = a.p.temperature ? a.p.temperature[row] : 1.0f;
    if (!(T > 0.0f) || top == -INFINITY) {
        if (tid == 0) {
            a.token[row] = (int)(0xffffffffu - (uint32_t)best);
            if (a.logprob)
                a.logprob[row] = top == -INFINITY ? -INFINITY : 0.0f;
        }
        return;
    }
    const float inv_t = __fdiv_rn(1.0f, fmaxf(T, 1e-30f));
    // sums over the tokens whose key is at least `key`: how many, and their weights
    auto count_ge = [&](u64 key) {
        u64 n = 0;
        for (int i = tid; i < V; i += kThreads)
            n += (u64)order_key(load_logit(a, row, i)) >= key;
        return block_all(n, add, red);
    };
    auto weight_ge = [&](u64 key) {
        u64 n = 0;
        for (int i = tid; i < V; i += kThreads) {
            const float l = load_logit(a, row, i);
            if ((u64)order_key(l) >= key)
                n += weight_of(exponent_of(key_value(order_key(l)), top, inv_t));
        }
        return block_all(n, add, red);
    };
    u64 key = 0, ties = (u64)V;   // kept: keys above `key`, and the first `ties` tokens that have it
    const int k = a.p.top_k ? a.p.top_k[row] : 0;
    if (k > 0 && k < V) {
        u64 lo = 0, hi = 1ull << 32;   // count_ge(lo) >= k > count_ge(hi)
        while (hi - lo > 1) {
            const u64 mid = (lo + hi) / 2;
            if (count_ge(mid) >= (u64)k)
                lo = mid;
            else
                hi = mid;
        }
        key = lo;
        ties = k - count_ge(lo + 1);
    }
    const float p = a.p.top_p ? a.p.top_p[row] : 1.0f;
    auto tie_weight = [&](u64 kk) { return (u64)weight_of(exponent_of(key_value((uint32_t)kk), top, inv_t)); };
    u64 total = weight_ge(key + 1);
    {
        const u64 n = min(ties, count_ge(key) - count_ge(key + 1));
        total += n * tie_weight(key);
    }
    if (p < 1.0f) {
        u64 need = (u64)ceil((double)p * (double)total);
        if (!(p > 0.0f) || need < 1)
            need = 1;
        u64 lo = key, hi = 1ull << 32;
        if (weight_ge(key + 1) >= need) {
            // the last member's key is above `key`
            lo = key + 1;
            while (hi - lo > 1) {
                const u64 mid = (lo + hi) / 2;
                if (weight_ge(mid) >= need)
                    lo = mid;
                else
                    hi = mid;
            }
            key = lo;
            ties = (u64)V;
        }
        const u64 above = weight_ge(key + 1), w = tie_weight(key);
        const u64 t = w ? (need - above + w - 1) / w : ties;
        ties = min(ties, t);
    }
    const float q = a.p.min_p ? a.p.min_p[row] : 0.0f;
    const double least = (double)fminf(fmaxf(q, 0.0f), 1.0f) * 2147483648.0;
    auto pass = [&](int i, u64 tie_rank) -> u64 {
        const float l = load_logit(a, row, i);
        const uint32_t ok = order_key(l);
        if (ok < key || (ok == key && tie_rank >= ties))
            return 0;
        const u64 w = weight_of(exponent_of(key_value(ok), top, inv_t));
        return (double)w >= least ? w : 0;
    };
    // each thread a run of indexes, so that ranks and running sums follow the index
    const int per = (V + kThreads - 1) / kThreads, i0 = min(tid * per, V), i1 = min(i0 + per, V);
    __shared__ u64 pre[kThreads];
    u64 n = 0;
    for (int i = i0; i < i1; ++i)
        n += order_key(load_logit(a, row, i)) == key;
    __syncthreads();
    pre[tid] = n;
    __syncthreads();
    u64 rank = 0;
    for (int i = 0; i < tid; ++i)
        rank += pre[i];
    const u64 rank0 = rank;
    u64 sum = 0;
    for (int i = i0; i < i1; ++i) {
        sum += pass(i, rank);
        rank += order_key(load_logit(a, row, i)) == key;
    }
    __syncthreads();
    pre[tid] = sum;
    __syncthreads();
    u64 before = 0, all = 0;
    for (int i = 0; i < kThreads; ++i) {
        if (i < tid)
            before += pre[i];
        all += pre[i];
    }
    const float u = a.p.u[row];
    const double target = (u > 0.0f ? fmin((double)u, 1.0 - 5.9604644775390625e-08) : 0.0) * (double)all;
    if ((double)before <= target && (double)(before + sum) > target) {
        rank = rank0;
        u64 cum = before;
        for (int i = i0; i < i1; ++i) {
            cum += pass(i, rank);
            if ((double)cum > target) {
                a.token[row] = i;
                if (a.logprob)
                    a.logprob[row] = exponent_of(key_value(order_key(load_logit(a, row, i))), top, inv_t) -
                                     logf((float)all * 4.656612873077393e-10f);
                break;
            }
            rank += order_key(load_logit(a, row, i)) == key;
        }
    }
}

}  // namespace

cudaError_t prepare_sample_kernels() { return cudaSuccess; }

cudaError_t launch_sample(const SampleArgs& a, int, cudaStream_t s)
{
    sample_simple_kernel<<<a.M, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
