// moe_sample.cu -- the next token of each row of logits, by temperature, top-k,
// top-p and min-p from a given random number.
//
// Every weight w_i = e^{z_i}, z_i = (l_i - max l) / T <= 0, is rounded to a
// multiple of 2^-31, so sums of weights are integers: exact, and the same in
// every order (the histograms below add with atomics).  The kept set is a prefix
// of the order "larger logit first, then lower index".
//
// One cluster of CTAs per row, each with a contiguous part of the vocabulary.
//  1. The largest logit (one read from HBM; later passes find the row in L1 / L2).
//  2. With top-k or top-p: how many tokens there are in each 1/256 of z.  z is a
//     monotone function of the logit, so bins are runs of the order: top-k ends in a
//     bin that the counts name, top-p in one of the few that the counts times the bins'
//     middle weights leave open.
//  3. One pass adds up the weights before and between those bins (per warp, in the
//     vocabulary's order) and gathers the bins' own tokens in one CTA, which picks
//     the last member of the kept set from them.  Where all tokens that may be kept
//     are in the list (top-k of some hundreds, peaked rows), that CTA orders it and draws.
//  4. Else the warp in whose part the target lies walks it.
// Rows whose bins hold more than 4,096 tokens (thousands of equal logits, high
// temperatures) find the last member by histograms of counts and weights that
// narrow a bin down to one key (the logit's order-preserving bits), and how many of
// the tokens that share the key are in; those take a few more passes.
// What bounds it: rows are read three times, from L2 after the first (5 to 12 us a pass
// for 64 rows of 151,643, the last one's exponentials the longest); between passes a
// cluster barrier (0.7 us), the bins' sums over the cluster and their prefix sums (5
// us), and one CTA's choice of the last member (3 to 5 us).  Measured, one row of 32,000
// and 64 rows of 151,643 fp32 logits, others in each call: largest logit only 4.8 and
// 10.3 us, no filter 10 and 22, top-k 50 16 and 32, top-p 0.9 23 and 44, all filters
// mixed 20 and 57.
#include <cooperative_groups.h>
#include <cstdint>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCluster = 8;
constexpr int kMostVectors = 32 * 32 * kWarps;   // 16-byte vectors of a CTA's part: 32 rows of 32 a warp
constexpr int kBins = 768;                 // of 1/32 of z: weights are 0 from z = -22.2 on
constexpr int kFine = 5760;               // of 1/256 of z
constexpr int kFinePer = (kFine + kThreads - 1) / kThreads;
constexpr int kSort = kThreads;            // tokens that one CTA orders, one a thread
constexpr int kEach = 4;
constexpr int kList = kEach * kThreads;    // tokens that the cut's last member is picked from
typedef unsigned long long u64;

// Larger float, larger key; NaN below everything, as -inf; -0 as +0.
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (f != f)
        f = -INFINITY;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

constexpr uint32_t kFineBits = 0x4b000000u;   // 2^23 as a float

struct Row {
    float top, inv_t;
    // -inf and NaN logits: -inf or NaN, of weight 0 and in no bin
    __device__ __forceinline__ float z(float l) const { return l == top ? 0.0f : __fmul_rn(__fsub_rn(l, top), inv_t); }
    __device__ __forceinline__ static uint32_t weight(float z) { return __float2uint_rn(expf(z) * 2147483648.0f); }
    // 1/256 of z that a finite logit lies nearest to; beyond kFine for -inf and NaN.
    // Adding 2^23 rounds to an integer in the low bits
    __device__ __forceinline__ uint32_t fine_bits(float l) const
    {
        return __float_as_uint(__fmaf_rn(__fsub_rn(top, l), inv_t * 256.0f, 8388608.0f));
    }
    // z where the largest logit is finite: the same bits, from the difference that fine() takes
    __device__ __forceinline__ float z_finite(float l) const { return -__fmul_rn(__fsub_rn(top, l), inv_t); }
    __device__ __forceinline__ static float fine_middle(int b) { return (float)b * (-1.0f / 256.0f); }
    __device__ __forceinline__ static int bin(float z) { return z > -(float)kBins / 32.0f ? (int)(z * -32.0f) : kBins - 1; }
};

struct Shared {
    u64 best[kMostCluster];                // largest (key, lowest index) of each CTA
    u64 red[kWarps], red2[kWarps];
    union {
        uint32_t fine[kFinePer * kThreads];          // this CTA's counts; then the row's, as prefix sums
        struct {
            uint32_t cnt[kBins], w0[kBins], w1[kBins], w2[kBins];   // this CTA's histogram: counts, and sums of the
                                           // weights' bits 0..10, 11..21, 22..31 (none can pass 32 bits)
            uint32_t tcnt[kBins];          // the row's, inclusive prefix sums
            u64 tw[kBins];
        };
    };
    uint32_t share[kFinePer * kThreads / 2];   // the row's counts in this CTA's share of the bins (two CTAs or more)
    u64 list[kList];                       // the first CTA's: gathered tokens, as key and complement of the index
    u64 warp_sum[kWarps], part_sum[kMostCluster], part_raw[kMostCluster], part_mid[kMostCluster];
    u64 row_sum[kWarps];
    uint4 left_range[kWarps];
    uint32_t warp_ties[kWarps], part_ties[kMostCluster], row_ties[kWarps];
    uint32_t nlist;
    int found, kbin, pbin[2];
    float sq[kWarps];
    u64 about, last, said;                 // said: what one thread computes for all
};

template <class T>
__device__ __forceinline__ T warp_scan(T v)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(~0u, v, o);
        if ((int)(threadIdx.x & 31) >= o)
            v += x;
    }
    return v;
}

// Inclusive prefix sums over the CTA's threads, of two values at once; the totals stay
// in red[kWarps - 1] and red2[kWarps - 1].
__device__ __forceinline__ void block_scan2(u64& v, u64& w, u64* red, u64* red2)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(~0u, v, o), y = __shfl_up_sync(~0u, w, o);
        v += lane >= o ? x : 0;
        w += lane >= o ? y : 0;
    }
    if (lane == 31) {
        red[warp] = v;
        red2[warp] = w;
    }
    __syncthreads();
    if (warp < 2) {
        u64* r = warp ? red2 : red;
        r[lane] = warp_scan(r[lane]);
    }
    __syncthreads();
    if (warp) {
        v += red[warp - 1];
        w += red2[warp - 1];
    }
}

// Inclusive prefix sums over the CTA's threads.
__device__ __forceinline__ u64 block_scan(u64 v, u64* red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_scan(v);
    if (lane == 31)
        red[warp] = v;
    __syncthreads();
    if (warp == 0)
        red[lane] = warp_scan(red[lane]);
    __syncthreads();
    if (warp)
        v += red[warp - 1];
    __syncthreads();
    return v;
}

// Bitonic sort of the values of the first n threads (one each, n a power of two from
// 32 on), ascending or descending; for those threads alone.
__device__ __forceinline__ u64 sort_first(u64 v, int n, bool descending, u64* buf)
{
    const int tid = threadIdx.x;
    auto sync = [n]() { asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory"); };
    for (int k = 2; k <= n; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            u64 o;
            if (j >= 32) {
                sync();
                buf[tid] = v;
                sync();
                o = buf[tid ^ j];
            } else {
                o = __shfl_xor_sync(~0u, v, j);
            }
            const bool lower = (tid & j) == 0, up = ((tid & k) == 0) != descending;
            if (lower == up ? o < v : o > v)
                v = o;
        }
    return v;
}

// The vector at p whose first element is number i0 of a row of V: only the row's
// own elements are read.
template <bool BF16>
__device__ __noinline__ uint4 load_end(const uint8_t* p, int i0, int V)
{
    constexpr int VEC = BF16 ? 8 : 4;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        if (i0 + e >= 0 && i0 + e < V) {
            if (BF16)
                w[e >> 1] = __byte_perm(w[e >> 1], reinterpret_cast<const uint16_t*>(p)[e], e & 1 ? 0x5410 : 0x3254);
            else
                w[e] = reinterpret_cast<const uint32_t*>(p)[e];
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
struct Part {
    // The warp's vectors of 16 bytes of the row; vector v holds elements v * VEC - lead ..
    static constexpr int VEC = BF16 ? 8 : 4;
    const uint8_t* base;      // 16-byte aligned
    int lead, V, v0, v1;

    // Vector v; -inf, which has no weight, where there is no element.
    __device__ __forceinline__ uint4 load(int v) const
    {
        const int i0 = v * VEC - lead;
        if (v < v1 && i0 >= 0 && i0 + VEC <= V)
            return __ldg(reinterpret_cast<const uint4*>(base + (long long)v * 16));
        return load_end<BF16>(base + (long long)v * 16, v < v1 ? i0 : V, V);
    }
    // f(values, index of the first) of vector v
    template <class F>
    __device__ __forceinline__ void take(int v, uint4 q, F f) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float l[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            l[e] = BF16 ? __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16) : __uint_as_float(w[e]);
        f(l, v * VEC - lead);
    }
    template <class F>
    __device__ __forceinline__ void visit(int v, F f) const { take(v, load(v), f); }
    // all of the warp's elements, U vectors a lane at a time.  U = 1 keeps the code of
    // a pass small: it runs once, and a short call's time is that of fetching
    // instructions; the next vector is on its way meanwhile
    template <int U, class F>
    __device__ __forceinline__ void each(F f) const
    {
        const int first = v0 + (threadIdx.x & 31);
        if constexpr (U > 1) {
#pragma unroll 1
            for (int v = first; v < v1; v += 32 * U) {
                uint4 q[U];
#pragma unroll
                for (int k = 0; k < U; ++k)
                    q[k] = load(v + 32 * k);
#pragma unroll
                for (int k = 0; k < U; ++k)
                    take(v + 32 * k, q[k], f);
            }
        } else {
            uint4 q = load(first), r = load(first + 32);
#pragma unroll 1
            for (int v = first; v < v1; v += 32) {
                const uint4 now = q;
                q = r;
                if (v + 64 < v1)
                    r = load(v + 64);
                take(v, now, f);
            }
        }
    }
};

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__device__ __forceinline__ u64 block_sum(u64 v, u64* red)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(red[threadIdx.x & 31]);
}

// Of the list's n entries that are `member`s, largest first: the one at which the
// running sum of f reaches `target` (which all of them together reach).  Rounds of
// 1,024 equal digits of the range that is left, till few are: of the keys, and
// once one key is left of the indexes.
template <class In, class F>
__device__ __forceinline__ u64 select_last(int n, In member, F f, u64 target, Shared& sh)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t *lo = sh.fine, *hi = sh.fine + kThreads;
    bool by_low = false;                      // the key is found: what is left has it
    uint32_t key = 0, from = 0, to = ~0u;     // what is left: keys, or low words, from .. to
    auto left = [&](u64 e) {
        const uint32_t x = (uint32_t)(e >> 32), word = by_low ? (uint32_t)e : x;
        return word >= from && word <= to && (!by_low || x == key) && member(e);
    };
#pragma unroll 1
    while (true) {
        uint32_t ka = ~0u, kb = 0, la = ~0u, lb = 0, count = 0;
#pragma unroll 1
        for (int i = tid; i < n; i += kThreads) {
            const u64 e = sh.list[i];
            if (left(e)) {
                ka = min(ka, (uint32_t)(e >> 32));
                kb = max(kb, (uint32_t)(e >> 32));
                la = min(la, (uint32_t)e);
                lb = max(lb, (uint32_t)e);
                ++count;
            }
        }
        auto reduce = [&]() {
            ka = __reduce_min_sync(~0u, ka);
            kb = __reduce_max_sync(~0u, kb);
            la = __reduce_min_sync(~0u, la);
            lb = __reduce_max_sync(~0u, lb);
            count = __reduce_add_sync(~0u, count);
        };
        reduce();
        __syncthreads();
        if (lane == 0) {
            sh.left_range[warp] = make_uint4(ka, kb, la, lb);
            sh.warp_ties[warp] = count;
        }
        lo[tid] = hi[tid] = 0;
        if (tid == 0)
            sh.nlist = 0;
        __syncthreads();
        {
            const uint4 x = sh.left_range[lane];
            ka = x.x, kb = x.y, la = x.z, lb = x.w;
            count = sh.warp_ties[lane];
        }
        reduce();
        if (count <= 64)
            break;
        if (ka == kb && !by_low) {
            by_low = true;
            key = ka;
        }
        const uint32_t a = by_low ? la : ka, b = by_low ? lb : kb;
        from = a;
        to = b;
        const int s = max(0, 22 - __clz((int)(b - a)));          // the range in 10 bits; larger words first
#pragma unroll 1
        for (int i = tid; i < n; i += kThreads) {
            const u64 e = sh.list[i];
            if (left(e)) {
                const uint32_t d = (b - (by_low ? (uint32_t)e : (uint32_t)(e >> 32))) >> s;
                const u64 w = f(e);
                atomicAdd(lo + d, (uint32_t)w & 0xffffu);
                atomicAdd(hi + d, (uint32_t)(w >> 16));
            }
        }
        __syncthreads();
        const u64 own = lo[tid] + ((u64)hi[tid] << 16), run = block_scan(own, sh.red);
        if (run >= target && run - own < target) {
            sh.found = tid;
            sh.last = run - own;
        }
        __syncthreads();
        const uint32_t d = (uint32_t)sh.found << s;
        target -= sh.last;
        to = b - d;
        from = max(a, b - min(d + ((1u << s) - 1), b));
        __syncthreads();
    }
    // the few: what is before each is added up by 16 threads
    u64* few = reinterpret_cast<u64*>(sh.fine);
    u64* few_f = few + 64;
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
        const u64 e = sh.list[i];
        if (left(e)) {
            const uint32_t at = atomicAdd(&sh.nlist, 1u);
            few[at] = e;
            few_f[at] = f(e);
        }
    }
    __syncthreads();
    {
        static_assert(kThreads == 64 * 16, "16 threads for each of the few");
        const uint32_t i = tid >> 4, m = sh.nlist;
        const u64 e = few[i];
        u64 run = 0;
#pragma unroll
        for (uint32_t j = tid & 15; j < 64; j += 16)
            run += j < m && few[j] >= e ? few_f[j] : 0;
#pragma unroll
        for (int o = 8; o; o >>= 1)
            run += __shfl_xor_sync(~0u, run, o);
        if (i < m && run >= target && run - few_f[i] < target)
            sh.last = e;
    }
    __syncthreads();
    const u64 r = sh.last;
    __syncthreads();
    return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t dynamic[];
    Shared& sh = *reinterpret_cast<Shared*>(dynamic);
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();                     // waited for before the first access to another CTA's memory
    constexpr int VEC = Part<BF16>::VEC;
    const int c = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / c, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    Part<BF16> part;
    int per;                                 // vectors of a warp
    {
        const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (long long)row * a.stride * (BF16 ? 2 : 4);
        part.lead = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (BF16 ? 2 : 4);
        part.base = p - part.lead * (BF16 ? 2 : 4);
        part.V = a.V;
        const int nv = (a.V + part.lead + part.VEC - 1) / part.VEC;
        per = ((nv + c * kWarps - 1) / (c * kWarps) + 31) / 32 * 32;
        part.v0 = min((rank * kWarps + warp) * per, nv);
        part.v1 = min(part.v0 + per, nv);
    }

    const float T = a.p.temperature ? a.p.temperature[row] : 1.0f;
    const int k = a.p.top_k ? a.p.top_k[row] : 0;
    const float tp = a.p.top_p ? a.p.top_p[row] : 1.0f, mp = a.p.min_p ? a.p.min_p[row] : 0.0f, uu = a.p.u[row];
    const bool by_p = tp < 1.0f;

    // ---- 1. the largest logit, lowest index first
    u64 best;
    {
        float m = -INFINITY;
        int at = 0;                          // a row of -inf (or NaN): index 0
        part.template each<BF16 ? 2 : 4>([&](const float (&l)[VEC], int i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (l[e] > m) {
                    m = l[e];
                    at = i + e;
                }
        });
        best = (u64)order_key(m) << 32 | (0xffffffffu - (uint32_t)at);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 x = __shfl_xor_sync(~0u, best, o);
        best = x > best ? x : best;
    }
    if (lane == 0)
        sh.red[warp] = best;
    for (int i = tid; i < kFinePer * kThreads; i += kThreads)
        sh.fine[i] = 0;
    if (tid == 0) {
        sh.nlist = 0;
        sh.kbin = sh.pbin[0] = sh.pbin[1] = kFine;
        sh.last = 0;
    }
    __syncthreads();
    if (warp == 0) {
        best = sh.red[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const u64 x = __shfl_xor_sync(~0u, best, o);
            best = x > best ? x : best;
        }
    }
    cl.barrier_wait();
    if (warp == 0 && lane < c)
        *cl.map_shared_rank(&sh.best[rank], lane) = best;
    cl.sync();
    best = sh.best[0];
    for (int i = 1; i < c; ++i)
        best = sh.best[i] > best ? sh.best[i] : best;

    Row r;
    r.top = key_value((uint32_t)(best >> 32));
    if (!(T > 0.0f) || r.top == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.token[row] = (int)(0xffffffffu - (uint32_t)best);
            if (a.logprob)
                a.logprob[row] = r.top == -INFINITY ? -INFINITY : 0.0f;
        }
        return;
    }
    r.inv_t = __fdiv_rn(1.0f, fmaxf(T, 1e-30f));
    // w >= min_p * 2^31 in integers (the fp32 product is exact)
    const uint32_t least = (uint32_t)ceilf(fminf(fmaxf(mp, 0.0f), 1.0f) * 2147483648.0f);
    // fp64 is slow here: one thread computes such a product for all, and sums are
    // compared as integers (cum >= x as cum >= ceil(x), cum > x as cum > floor(x))
    auto need_of = [&](u64 total) {
        const double need = ceil((double)tp * (double)total);
        return need >= 1.0 ? (u64)need : 1ull;
    };
    auto target_of = [&](u64 total) {
        return (u64)((uu > 0.0f ? fmin((double)uu, 1.0 - 5.9604644775390625e-08) : 0.0) * (double)total);
    };
    auto one_for_all = [&](auto f, u64 x) {
        if (tid == 0)
            sh.said = f(x);
        __syncthreads();
        const u64 v = sh.said;
        __syncthreads();
        return v;
    };
    auto answer = [&](int i, float l, u64 total) {
        a.token[row] = i;
        if (a.logprob)
            a.logprob[row] = r.z(l) - logf((float)total * 4.656612873077393e-10f);
    };

    // the kept set: all tokens if `all`; else, as key and complement of the index,
    // those from `last` on; else (last == 0) larger keys than `key` and the first
    // `ties` tokens that have it
    bool all = true;
    u64 last = 0;
    uint32_t key = 0, ties = 0;
    if ((k > 0 && k < a.V) || by_p) {
        // ---- 2. counts in 1/256 of z
        part.template each<2>([&](const float (&l)[VEC], int) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const uint32_t b = r.fine_bits(l[e]);
                if (b < kFineBits + kFine)
                    atomicAdd(&sh.fine[b - kFineBits], 1u);
            }
        });
        const int tps = (kThreads + c - 1) / c;              // threads whose bins one CTA adds up
        if (c > 1) {
            // every CTA adds up its share of the bins, then takes all shares
            cl.sync();
            for (int b = tid; b < tps * kFinePer && rank * tps * kFinePer + b < kFine; b += kThreads) {
                uint32_t n = 0;
#pragma unroll 4
                for (int i = 0; i < c; ++i)
                    n += cl.map_shared_rank(&sh, i)->fine[rank * tps * kFinePer + b];
                sh.share[b] = n;
            }
            cl.sync();
            for (int b = tid; b < kFine; b += kThreads) {
                const int from = b / (tps * kFinePer);
                sh.fine[b] = cl.map_shared_rank(&sh, from)->share[b - from * tps * kFinePer];
            }
        }
        __syncthreads();
        uint32_t n[kFinePer], nsum = 0;
        u64 w[kFinePer], wsum = 0;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < kFinePer; ++j)
            n[j] = tid * kFinePer + j < kFine ? sh.fine[tid * kFinePer + j] : 0;
#pragma unroll
        for (int j = 0; j < kFinePer; ++j) {
            const uint32_t x = Row::weight(Row::fine_middle(tid * kFinePer + j));
            const float y = (float)n[j] * (float)x;
            w[j] = n[j] * (u64)x;
            nsum += n[j];
            wsum += w[j];
            sq += y * y;
        }
        if (by_p) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sq += __shfl_xor_sync(~0u, sq, o);
            if (lane == 0)
                sh.sq[warp] = sq;
        }
        u64 nb = nsum, wb = wsum;
        block_scan2(nb, wb, sh.red, sh.red2);
        nb -= nsum;
        wb -= wsum;
        const bool by_k = k > 0 && (u64)k < sh.red[kWarps - 1];
        u64 about = sh.red2[kWarps - 1];     // weight of what top-k leaves, but for the bins' width
        if (by_k) {
            u64 x = nb, y = wb;
#pragma unroll
            for (int j = 0; j < kFinePer; ++j) {
                if (x < (u64)k && x + n[j] >= (u64)k) {
                    sh.kbin = tid * kFinePer + j;
                    sh.about = y + ((u64)k - x) * Row::weight(Row::fine_middle(tid * kFinePer + j));
                }
                x += n[j];
                y += w[j];
            }
            __syncthreads();
            about = sh.about;
        }
        if (by_p) {
            // a bin's tokens may lie anywhere in it: its weight is off by up to 2^-9, 2^-9.8
            // in the mean square.  Four times what that makes of independent bins
            sq = 0.0f;
            for (int i = 0; i < kWarps; ++i)
                sq += sh.sq[i];
            const float share_p = fmaxf(tp, 0.0f) * (float)about, off = 0.0046f * sqrtf(sq) + 1e-5f * (float)about;
            const u64 t0 = (u64)fmaxf(share_p - off, 1.0f), t1 = (u64)fmaxf(share_p + off, 1.0f);
            u64 y = wb;
#pragma unroll
            for (int j = 0; j < kFinePer; ++j) {
                if (y < t0 && y + w[j] >= t0)
                    sh.pbin[0] = tid * kFinePer + j;
                if (y < t1 && y + w[j] >= t1)
                    sh.pbin[1] = tid * kFinePer + j;
                y += w[j];
            }
        }
        {
            uint32_t x = (uint32_t)nb;
#pragma unroll
            for (int j = 0; j < kFinePer; ++j) {
                x += n[j];
                sh.fine[tid * kFinePer + j] = x;   // no other CTA reads them any more
            }
        }
        __syncthreads();
        auto through = [&](int b) -> uint32_t { return b < 0 ? 0u : sh.fine[min(b, kFine - 1)]; };
        const int kb = sh.kbin;
        // the bands to gather: bins p0 .. p1, and kb if it is apart from them
        int p0 = by_p ? min(sh.pbin[0], kb) : kb;
        const int p1 = by_p ? min(sh.pbin[1], kb) : kb;
        const bool apart = by_k && p1 < kb;
        const uint32_t n_k = apart ? through(kb) - through(kb - 1) : 0;
        const bool alone = through(p1) + n_k <= kSort;       // the list takes all that may be kept, in order
        if (alone)
            p0 = 0;
        const uint32_t before = through(p0 - 1), n_p = through(p1) - before, n_list = n_p + n_k, before_k = through(kb - 1);
        const bool odd = r.top == INFINITY;                  // only infinities have weight, and none of them a bin
        all = !by_k && !by_p && !odd;                        // fewer tokens than k have weight
        const bool mixed = by_k && by_p && !apart && !alone;  // top-k ends where top-p does: needs the order
        if (!all && !odd && n_list <= (mixed ? kSort : kList)) {
            // ---- 3. weights before and between the bands; their tokens into the first CTA's list
            const bool sums = !alone || (by_p && (!by_k || apart));
            u64 kept = 0, raw = 0, mid = 0;
            auto gather = [&](float l, int i) {
                const uint32_t at = atomicAdd(cl.map_shared_rank(&sh.nlist, 0), 1u);
                *cl.map_shared_rank(&sh.list[at], 0) = (u64)order_key(l) << 32 | (0xffffffffu - (uint32_t)i);
            };
            // bands q0 .. q0 + qn and qa; bins from `end` on are beyond top-k
            const uint32_t q0 = kFineBits + p0, qn = min(p1, kFine - 1) - p0, qa = apart ? kFineBits + kb : ~0u, end = by_k ? kFineBits + kb + 1 : ~0u;
            const bool floor = least > 0;
            if (sums) {
                u64 tot = 0;
                part.template each<BF16 ? 1 : 2>([&](const float (&l)[VEC], int i) {
                    uint32_t x[VEC], b[VEC];
                    bool hit = false;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        b[e] = r.fine_bits(l[e]);
                        x[e] = Row::weight(r.z_finite(l[e]));
                        x[e] = b[e] < end ? x[e] : 0;
                        hit = hit || b[e] - q0 <= qn || b[e] == qa;
                    }
#pragma unroll
                    for (int e = 0; e < VEC; e += 2)
                        tot += (u64)x[e] + x[e + 1];
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        x[e] = b[e] < q0 ? x[e] : 0;
#pragma unroll
                    for (int e = 0; e < VEC; e += 2)
                        raw += (u64)x[e] + x[e + 1];
                    if (floor)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            kept += x[e] >= least ? x[e] : 0;
                    if (hit)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (b[e] - q0 <= qn || b[e] == qa)
                                gather(l[e], i + e);
                });
                mid = tot - raw;                             // the bands' own weights are taken off below
                if (!floor)
                    kept = raw;
            } else {
                part.template each<2>([&](const float (&l)[VEC], int i) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const uint32_t b = r.fine_bits(l[e]);
                        if (b - q0 <= qn || b == qa)
                            gather(l[e], i + e);
                    }
                });
            }
            if (sums) {
                kept = warp_sum(kept);
                raw = warp_sum(raw);
                mid = warp_sum(mid);
                if (lane == 0) {
                    sh.warp_sum[warp] = kept;
                    sh.red[warp] = raw;
                    sh.red2[warp] = mid;
                }
                __syncthreads();
                if (warp == 0) {
                    raw = warp_sum(sh.red[lane]);
                    mid = warp_sum(sh.red2[lane]);
                    if (lane == 0) {
                        *cl.map_shared_rank(&sh.part_raw[rank], 0) = raw;
                        *cl.map_shared_rank(&sh.part_mid[rank], 0) = mid;
                    }
                }
            }
            cl.sync();
            bool found = true;
            if (rank == 0) {
                raw = mid = 0;
                if (sums)
                    for (int i = 0; i < c; ++i) {
                        raw += sh.part_raw[i];
                        mid += sh.part_mid[i];
                    }
                int n2 = 32;
                while (n2 < (int)n_list)
                    n2 <<= 1;
                u64 e = tid < (int)n_list ? sh.list[tid] : 0, x = 0;
                bool in = false;
                const bool few = n_list <= kThreads / 4;
                if (sums) {
                    // the gathered tokens' weights were added to what lies between the bands
                    u64 w = 0;
                    for (int i = tid; i < (int)n_list; i += kThreads)
                        w += Row::weight(r.z(key_value((uint32_t)(sh.list[i] >> 32))));
                    w = warp_sum(w);
                    if (lane == 0)
                        sh.red[warp] = w;
                    __syncthreads();
                    mid -= warp_sum(sh.red[lane]);
                    __syncthreads();
                }
                if (!alone && !mixed) {
                    // only the last member is wanted: no order is needed
                    auto in_first = [&](u64 v) { return r.fine_bits(key_value((uint32_t)(v >> 32))) - q0 <= qn; };
                    auto weigh = [&](u64 v) -> u64 { return Row::weight(r.z(key_value((uint32_t)(v >> 32)))); };
                    auto one = [](u64) -> u64 { return 1; };
                    u64 cut_at;
                    if (by_p) {
                        u64 in_band = 0, beyond = 0, lk = ~0ull;
                        if (apart)
                            lk = select_last((int)n_list, [&](u64 v) { return !in_first(v); }, one, (u64)k - before_k, sh);
                        for (int i = tid; i < (int)n_list; i += kThreads) {
                            const u64 v = sh.list[i];
                            if (in_first(v))
                                in_band += weigh(v);
                            else if (v >= lk)
                                beyond += weigh(v);
                        }
                        in_band = block_sum(in_band, sh.red);
                        if (apart)
                            beyond = block_sum(beyond, sh.red);
                        const u64 need = one_for_all(need_of, raw + in_band + mid + beyond);
                        found = raw < need && raw + in_band >= need;     // the share is reached within the band
                        cut_at = found ? select_last((int)n_list, in_first, weigh, need - raw, sh) : ~0ull;
                    } else {
                        cut_at = select_last((int)n_list, in_first, one, (u64)k - before, sh);
                    }
                    if (tid == 0)
                        sh.last = ~cut_at;
                    __syncthreads();
                } else {
                    if (few) {
                        // each place in the order by counting what is before it, four threads an entry
                        const int i = tid >> 2;
                        e = i < (int)n_list ? sh.list[i] : 0;
                        int place = 0;
                        for (int j = tid & 3; j < (int)n_list; j += 4)
                            place += sh.list[j] > e;
                        place += __shfl_xor_sync(~0u, place, 1);
                        place += __shfl_xor_sync(~0u, place, 2);
                        __syncthreads();
                        if (i < (int)n_list && (tid & 3) == 0)
                            sh.list[place] = e;
                        __syncthreads();
                        e = tid < (int)n_list ? sh.list[tid] : 0;
                    } else {
                        __syncthreads();
                        if (tid < n2)
                            e = sort_first(e, n2, true, sh.list);
                    }
                    // this thread's place in the order, and its weight if top-k takes it
                    const uint32_t at = tid < (int)n_p ? before + tid : before_k + (tid - n_p);
                    if (tid < (int)n_list && (!by_k || at < (uint32_t)k))
                        x = Row::weight(r.z(key_value((uint32_t)(e >> 32))));
                    in = x != 0;
                    if (by_p) {
                        const u64 own = tid < (int)n_p ? x : 0;
                        u64 cum = own, rest = x - own;
                        block_scan2(cum, rest, sh.red, sh.red2);
                        const u64 in_band = sh.red[kWarps - 1];
                        const u64 need = one_for_all(need_of, raw + in_band + mid + sh.red2[kWarps - 1]);
                        in = in && tid < (int)n_p && raw + cum - own < need;
                        found = raw < need && raw + in_band >= need;
                    }
                    __syncthreads();
                    if (!few && tid < n2)
                        sh.list[tid] = e;
                    if (in)
                        atomicMax(&sh.last, ~e);                      // the last one has the largest complement
                    __syncthreads();
                }
                if (alone && found) {
                    if (!in || x < least)
                        x = 0;
                    // by index, the kept ones first
                    u64 by_index = x ? (u64)(0xffffffffu - (uint32_t)e) << 32 | x : ~0ull << 32, run = 0, total = 0;
                    if (few) {
                        if (tid < (int)n_list)
                            sh.list[tid] = by_index;
                        __syncthreads();
                        by_index = tid >> 2 < (int)n_list ? sh.list[tid >> 2] : 0;
                        for (int j = tid & 3; j < (int)n_list; j += 4) {
                            const u64 y = sh.list[j], add = y & 0xffffffffu;
                            total += add;
                            run += y <= by_index ? add : 0;
                        }
#pragma unroll
                        for (int o = 1; o <= 2; o <<= 1) {
                            total += __shfl_xor_sync(~0u, total, o);
                            run += __shfl_xor_sync(~0u, run, o);
                        }
                        x = tid & 3 ? 0 : by_index & 0xffffffffu;
                    } else {
                        if (tid < n2)
                            by_index = sort_first(by_index, n2, false, sh.list);
                        x = tid < n2 ? by_index & 0xffffffffu : 0;
                        run = block_scan(x, sh.red);
                        total = sh.red[kWarps - 1];
                    }
                    const u64 target = one_for_all(target_of, total);
                    if (x && run > target && run - x <= target) {
                        const int i = (int)(by_index >> 32);
                        answer(i, BF16 ? tc::bf16f(static_cast<const uint16_t*>(a.logits)[row * a.stride + i])
                                       : static_cast<const float*>(a.logits)[row * a.stride + i], total);
                    }
                }
                last = ~sh.last;                     // (select_last left other things there before)
                __syncthreads();
                if (tid < c)
                    *cl.map_shared_rank(&sh.last, tid) = found ? last : 0;
            }
            cl.sync();
            last = sh.last;
            if (alone && last)
                return;
            if (last) {
                // the list's kept tokens join their warps' sums
                const Shared* s0 = cl.map_shared_rank(&sh, 0);
                for (int i = tid; i < (int)n_list; i += kThreads) {
                    const u64 e = s0->list[i];
                    const uint32_t x = Row::weight(r.z(key_value((uint32_t)(e >> 32))));
                    const int g = ((int)(0xffffffffu - (uint32_t)e) + part.lead) / part.VEC / per;
                    if (e >= last && x >= least && g / kWarps == rank)
                        atomicAdd(&sh.warp_sum[g % kWarps], (u64)x);
                }
                if (tid < kWarps)
                    sh.warp_ties[tid] = 0;
            }
        }
        if (!all && !last) {
            // ---- many tokens in a bin: narrow it by its keys, first for k, then for p
            // the row's histogram from the CTAs', as prefix sums
            auto join = [&]() {
                cl.sync();
                u64 w = 0, n = 0;
                if (tid < kBins)
                    for (int i = 0; i < c; ++i) {
                        const Shared* s = cl.map_shared_rank(&sh, i);
                        w += (u64)s->w0[tid] + ((u64)s->w1[tid] << 11) + ((u64)s->w2[tid] << 22);
                        n += s->cnt[tid];
                    }
                block_scan2(w, n, sh.red, sh.red2);
                if (tid < kBins) {
                    sh.tw[tid] = w;
                    sh.tcnt[tid] = (uint32_t)n;
                }
                __syncthreads();
            };
            auto clear = [&]() {
                cl.sync();
                for (int i = tid; i < kBins; i += kThreads)
                    sh.cnt[i] = sh.w0[i] = sh.w1[i] = sh.w2[i] = 0;
                __syncthreads();
            };
            auto add = [&](int b, uint32_t w) {
                atomicAdd(&sh.cnt[b], 1u);
                atomicAdd(&sh.w0[b], w & 0x7ffu);
                atomicAdd(&sh.w1[b], w >> 11 & 0x7ffu);
                atomicAdd(&sh.w2[b], w >> 22);
            };
            // first prefix sum that reaches `need`
            auto first_of = [&](bool weights, u64 need) {
                if (tid < kBins) {
                    const u64 x = weights ? sh.tw[tid] : sh.tcnt[tid], before = tid ? (weights ? sh.tw[tid - 1] : sh.tcnt[tid - 1]) : 0;
                    if (x >= need && before < need)
                        sh.found = tid;
                }
                __syncthreads();
                const int b = sh.found;
                __syncthreads();
                return b;
            };
            // smallest key whose bin is at most b
            auto lowest_key = [&](int b) {
                uint32_t lo = 0, hi = (uint32_t)(best >> 32);       // hi is in bin 0
                while (lo < hi) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    const float z = r.z(key_value(mid));
                    if (z == z && Row::bin(z) <= b)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                return lo;
            };
            clear();
            part.template each<1>([&](const float (&l)[VEC], int) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float z = r.z(l[e]);
                    const uint32_t w = Row::weight(z);
                    if (w)
                        add(Row::bin(z), w);
                }
            });
            join();
            const u64 keep_w = tid < kBins ? sh.tw[tid] : 0;
            const uint32_t keep_n = tid < kBins ? sh.tcnt[tid] : 0;
            u64 total = sh.tw[kBins - 1];
            const bool cut_k = k > 0 && (uint32_t)k < sh.tcnt[kBins - 1];
            all = !cut_k && !by_p;
            for (int what = 0; what < 2; ++what) {
                const bool weights = what == 1;
                if (weights ? !by_p : !cut_k)
                    continue;
                __syncthreads();
                if (tid < kBins) {
                    sh.tw[tid] = keep_w;
                    sh.tcnt[tid] = keep_n;
                }
                __syncthreads();
                const u64 need = weights ? one_for_all(need_of, total) : (u64)k;
                const int b = first_of(weights, need);
                u64 wab = b ? sh.tw[b - 1] : 0, nab = b ? sh.tcnt[b - 1] : 0;      // weight and count above the range
                uint32_t lo = lowest_key(b);
                u64 range = (b ? (u64)lowest_key(b - 1) : (best >> 32) + 1) - lo;  // keys lo .. lo + range - 1
                while (true) {
                    const uint32_t width = (uint32_t)((range + kBins - 1) / kBins);
                    clear();
                    part.template each<1>([&](const float (&l)[VEC], int) {
#pragma unroll 1
                        for (int e = 0; e < VEC; ++e) {
                            const uint32_t kk = order_key(l[e]);
                            if (kk < lo || kk - lo >= range)
                                continue;
                            const uint32_t w = Row::weight(r.z(l[e]));
                            if (w)
                                add(kBins - 1 - (int)((kk - lo) / width), w);   // larger keys first
                        }
                    });
                    join();
                    u64 rest = need - (weights ? wab : nab);
                    const int s = first_of(weights, rest);
                    const u64 w0 = s ? sh.tw[s - 1] : 0, n0 = s ? sh.tcnt[s - 1] : 0;
                    const uint32_t here = sh.tcnt[s] - (uint32_t)n0;
                    wab += w0;
                    nab += n0;
                    rest -= weights ? w0 : n0;
                    const uint32_t from = (uint32_t)(kBins - 1 - s) * width;
                    lo += from;
                    range = range - from < width ? range - from : width;
                    if (range == 1) {
                        const u64 w = Row::weight(r.z(key_value(lo)));
                        key = lo;
                        ties = weights ? (uint32_t)((rest + w - 1) / w) : (uint32_t)rest;
                        ties = min(ties, here);
                        total = wab + ties * w;
                        break;
                    }
                }
            }
        }
    }

    // ---- 4. kept weights in the vocabulary's order
    const bool cut = !all && !last;
    if (!last) {
        u64 sum = 0;
        uint32_t eq = 0;
        if (cut)
            part.template each<1>([&](const float (&l)[VEC], int) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const uint32_t w = Row::weight(r.z(l[e])), kk = order_key(l[e]);
                    eq += kk == key;
                    sum += w >= least && kk > key ? w : 0;
                }
            });
        else
            part.template each<BF16 ? 1 : 2>([&](const float (&l)[VEC], int) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const uint32_t w = Row::weight(r.z(l[e]));
                    sum += w >= least ? w : 0;
                }
            });
        sum = warp_sum(sum);
        eq = __reduce_add_sync(~0u, eq);
        if (lane == 0) {
            sh.warp_sum[warp] = sum;
            sh.warp_ties[warp] = eq;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const u64 s = warp_sum(sh.warp_sum[lane]);
        const uint32_t n = __reduce_add_sync(~0u, sh.warp_ties[lane]);
        if (lane < c) {
            *cl.map_shared_rank(&sh.part_sum[rank], lane) = s;
            *cl.map_shared_rank(&sh.part_ties[rank], lane) = n;
        }
    }
    cl.sync();
    u64 wtie = 0;
    if (cut) {
        wtie = Row::weight(r.z(key_value(key)));
        wtie = wtie >= least ? wtie : 0;
    }
    u64 total = 0, cum = 0;
    uint32_t seen = 0, tie0 = 0;                 // ties so far, and before this CTA
    for (int i = 0; i < c; ++i) {
        if (i == rank) {
            cum = total;
            tie0 = seen;
        }
        total += sh.part_sum[i] + min(sh.part_ties[i], ties - min(ties, seen)) * wtie;
        seen += sh.part_ties[i];
    }
    const u64 target = one_for_all(target_of, total);
    // the warp in whose vectors the target lies (a lane for each warp)
    const uint32_t wt = sh.warp_ties[lane], wts = warp_scan(wt) - wt + tie0;
    const u64 ws = sh.warp_sum[lane] + min(wt, ties - min(ties, wts)) * wtie, wss = warp_scan(ws) + cum;
    const unsigned hit = __ballot_sync(~0u, wss > target && wss - ws <= target);
    if (!hit)
        return;
    const int tw = __ffs(hit) - 1;
    cum = __shfl_sync(~0u, wss - ws, tw);
    seen = __shfl_sync(~0u, wts, tw);
    Part<BF16> seg = part;
    seg.v0 = (rank * kWarps + tw) * per;
    seg.v1 = min(seg.v0 + per, (a.V + part.lead + part.VEC - 1) / part.VEC);
    // its rows of 32 vectors (at most 32: kMostVectors), one a warp
    uint32_t w[Part<BF16>::VEC], vl = 0, nl = 0;
    float val[Part<BF16>::VEC];
    u64 s = 0;
    auto row_of = [&](int x) {
        vl = nl = 0;
        s = 0;
        seg.visit(seg.v0 + 32 * x + lane, [&](const float (&l)[VEC], int i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const uint32_t kk = order_key(l[e]);
                const bool tie = cut && kk == key;
                const bool in = all || (last ? ((u64)kk << 32 | (0xffffffffu - (uint32_t)(i + e))) >= last : kk > key);
                const uint32_t y = in ? Row::weight(r.z(l[e])) : 0;
                nl += tie;
                vl |= (uint32_t)tie << e;
                w[e] = y >= least ? y : 0;
                val[e] = l[e];
                s += w[e];
            }
        });
    };
    row_of(warp);
    {
        const u64 rs = warp_sum(s);
        const uint32_t rt = __reduce_add_sync(~0u, nl);
        if (lane == 0) {
            sh.row_sum[warp] = rs;
            sh.row_ties[warp] = rt;
        }
    }
    __syncthreads();
    const uint32_t rt = sh.row_ties[lane], rts = warp_scan(rt) - rt + seen;
    const u64 rs = sh.row_sum[lane] + min(rt, ties - min(ties, rts)) * wtie, rss = warp_scan(rs) + cum;
    const int trow = __ffs(__ballot_sync(~0u, rss > target && rss - rs <= target)) - 1;
    if (warp != trow)
        return;
    cum = __shfl_sync(~0u, rss - rs, trow);
    seen = __shfl_sync(~0u, rts, trow);
    uint32_t rk = seen + warp_scan(nl) - nl;     // ties before this lane's
#pragma unroll
    for (int e = 0; e < Part<BF16>::VEC; ++e)
        if ((vl >> e & 1) && rk++ < ties) {
            w[e] = (uint32_t)wtie;
            s += wtie;
        }
    u64 at = cum + warp_scan(s) - s;
    if (at <= target && at + s > target) {
#pragma unroll
        for (int e = 0; e < Part<BF16>::VEC; ++e) {
            if (at <= target && at + w[e] > target)
                answer((seg.v0 + 32 * warp + lane) * Part<BF16>::VEC - part.lead + e, val[e], total);
            at += w[e];
        }
    }
}

}  // namespace

cudaError_t prepare_sample_kernels()
{
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    return e != cudaSuccess ? e : cudaFuncSetAttribute(sample_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
}

cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s)
{
    // CTAs a row: as few as take it; more while every row keeps its own SMs and a
    // CTA at least 2,048 tokens
    const int vectors = a.V / (a.logits_type == MOE_DT_BF16 ? 8 : 4) + 2;
    // (clusters of 8 find room beside one another on half of the SMs only: 16 rows of
    // 8 CTAs took twice the time of 16 rows of 4)
    int c = 1;
    while (c < kMostCluster && (vectors > c * kMostVectors ||
                                ((c < 4 ? 2ll : 4ll) * c * a.M <= num_sms && a.V >= 2 * c * 2048)))
        c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.M * c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return a.logits_type == MOE_DT_BF16 ? cudaLaunchKernelEx(&cfg, sample_kernel<true>, a)
                                        : cudaLaunchKernelEx(&cfg, sample_kernel<false>, a);
}

}  // namespace moe
