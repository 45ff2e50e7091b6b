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
//  2. With top-k or top-p: a histogram, in 1/32 steps of z, of counts and weights;
//     its prefix sums name the bin in which the kept set ends.  z is a monotone
//     function of the logit, so bins are runs of the order.  Tokens of weight 0
//     cannot be drawn and are left out.
//  3. If the bins up to that one hold at most 1,024 tokens (top-k up to some
//     hundreds, peaked rows), they are gathered and sorted in one CTA, which ends
//     the row.  Else the bin is narrowed by histograms of its keys until the last
//     member's key (the logit's order-preserving bits) is known, and how many of
//     the tokens that share it are in.
//  4. Sums of kept weights per CTA and warp, in the vocabulary's order; the warp in
//     whose part the target lies walks it.
#include <cooperative_groups.h>
#include <cstdint>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCluster = 16;
constexpr int kMostPart = 65536;           // tokens of a CTA: a bin's sum of 16-bit halves fits 32 bits
constexpr int kSlackPart = 32 * 32 * 8;    // a CTA's part may be this much above an equal share
constexpr int kBins = 768;                 // of 1/32 of z: weights are 0 from z = -22.2 on
constexpr int kList = kThreads;
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

struct Row {
    float top, inv_t;
    __device__ __forceinline__ float z(float l) const
    {
        return l == top ? 0.0f : !(l > -INFINITY) || top == INFINITY ? -INFINITY : __fmul_rn(__fsub_rn(l, top), inv_t);
    }
    __device__ __forceinline__ static uint32_t weight(float z) { return __float2uint_rn(expf(z) * 2147483648.0f); }
    __device__ __forceinline__ static int bin(float z) { return z > -(float)kBins / 32.0f ? (int)(z * -32.0f) : kBins - 1; }
};

struct Shared {
    u64 best[kMostCluster];                // largest (key, lowest index) of each CTA
    u64 red[kWarps];
    uint32_t cnt[kBins], lo[kBins], hi[kBins];       // this CTA's histogram: counts, halves of weights
    uint32_t tcnt[kBins];                  // the row's, inclusive prefix sums
    u64 tw[kBins];
    u64 list[kList];
    u64 part_sum[kMostCluster], warp_sum[kWarps];
    uint32_t part_ties[kMostCluster], warp_ties[kWarps];
    uint32_t nlist;
    int found;
    uint32_t found_key;
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

// Bitonic sort of the CTA's values (one a thread, n a power of two from 32 on),
// ascending or descending.
__device__ __forceinline__ u64 block_sort(u64 v, int n, bool descending, u64* buf)
{
    const int tid = threadIdx.x;
    for (int k = 2; k <= n; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            u64 o;
            if (j >= 32) {
                __syncthreads();
                if (tid < n)
                    buf[tid] = v;
                __syncthreads();
                o = tid < n ? buf[tid ^ j] : v;
            } else {
                o = __shfl_xor_sync(~0u, v, j);
            }
            const bool lower = (tid & j) == 0, up = ((tid & k) == 0) != descending;
            if (lower == up ? o < v : o > v)
                v = o;
        }
    return v;
}

template <bool BF16>
struct Part {
    // The warp's vectors of 16 bytes of the row; vector v holds elements v * VEC - lead ..
    static constexpr int VEC = BF16 ? 8 : 4;
    const uint8_t* base;      // 16-byte aligned
    int lead, V, v0, v1;

    // f(value, index) for each element of vector v (index -1: no element)
    template <class F>
    __device__ __forceinline__ void visit(int v, F f) const
    {
        const int i0 = v * VEC - lead;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (v < v1) {
            if (i0 >= 0 && i0 + VEC <= V) {
                q = *reinterpret_cast<const uint4*>(base + (long long)v * 16);
            } else {
                // the row's ends: only its own elements are read
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i0 + e >= 0 && i0 + e < V) {
                        if (BF16)
                            w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(base + (long long)v * 16)[e] << 16 * (e & 1);
                        else
                            w[e] = reinterpret_cast<const uint32_t*>(base + (long long)v * 16)[e];
                    }
                q = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float x = BF16 ? __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16) : __uint_as_float(w[e]);
            const int i = i0 + e;
            f(x, v < v1 && i >= 0 && i < V ? i : -1);
        }
    }
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
        const int lane = threadIdx.x & 31;
#pragma unroll 4
        for (int v = v0 + lane; v < v1; v += 32)
            visit(v, f);
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int c = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / c, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    cl.barrier_arrive();                     // waited for before the first access to another CTA's memory
    Part<BF16> part;
    {
        const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (long long)row * a.stride * (BF16 ? 2 : 4);
        part.lead = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (BF16 ? 2 : 4);
        part.base = p - part.lead * (BF16 ? 2 : 4);
        part.V = a.V;
        const int nv = (a.V + part.lead + part.VEC - 1) / part.VEC, per = ((nv + c * kWarps - 1) / (c * kWarps) + 31) / 32 * 32;
        part.v0 = min((rank * kWarps + warp) * per, nv);
        part.v1 = min(part.v0 + per, nv);
    }

    // ---- 1. the largest logit, lowest index first
    u64 best = 0;
    part.each([&](float l, int i) {
        if (i >= 0) {
            const u64 k = (u64)order_key(l) << 32 | (0xffffffffu - (uint32_t)i);
            best = k > best ? k : best;
        }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 x = __shfl_xor_sync(~0u, best, o);
        best = x > best ? x : best;
    }
    if (lane == 0)
        sh.red[warp] = best;
    for (int i = tid; i < kBins; i += kThreads)
        sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
    if (tid == 0)
        sh.nlist = 0;
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
    const float T = a.p.temperature ? a.p.temperature[row] : 1.0f;
    if (!(T > 0.0f) || r.top == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.token[row] = (int)(0xffffffffu - (uint32_t)best);
            if (a.logprob)
                a.logprob[row] = r.top == -INFINITY ? -INFINITY : 0.0f;
        }
        return;
    }
    r.inv_t = __fdiv_rn(1.0f, fmaxf(T, 1e-30f));
    int k = a.p.top_k ? a.p.top_k[row] : 0;
    const float tp = a.p.top_p ? a.p.top_p[row] : 1.0f, mp = a.p.min_p ? a.p.min_p[row] : 0.0f, uu = a.p.u[row];
    const bool by_p = tp < 1.0f;
    const double least = (double)fminf(fmaxf(mp, 0.0f), 1.0f) * 2147483648.0;
    const double u = uu > 0.0f ? fmin((double)uu, 1.0 - 5.9604644775390625e-08) : 0.0;
    auto need_of = [&](u64 total) {
        const double need = ceil((double)tp * (double)total);
        return need >= 1.0 ? (u64)need : 1ull;
    };
    auto answer = [&](int i, float l, u64 total) {
        a.token[row] = i;
        if (a.logprob)
            a.logprob[row] = r.z(l) - logf((float)total * 4.656612873077393e-10f);
    };

    uint32_t key = 0;                        // the kept set: larger keys, and the first `ties` tokens with this one
    uint32_t ties = 0xffffffffu;
    if ((k > 0 && k < a.V) || by_p) {
        // the row's histogram from the CTAs', as prefix sums
        auto join = [&](int bins) {
            cl.sync();
            u64 w = 0, n = 0;
            if (tid < bins) {
                uint32_t lo[kMostCluster], hi[kMostCluster], cn[kMostCluster];
#pragma unroll
                for (int i = 0; i < kMostCluster; ++i) {
                    lo[i] = hi[i] = cn[i] = 0;
                    if (i < c) {
                        const Shared* s = cl.map_shared_rank(&sh, i);
                        lo[i] = s->lo[tid];
                        hi[i] = s->hi[tid];
                        cn[i] = s->cnt[tid];
                    }
                }
#pragma unroll
                for (int i = 0; i < kMostCluster; ++i) {
                    w += (u64)lo[i] + ((u64)hi[i] << 16);
                    n += cn[i];
                }
            }
            w = block_scan(w, sh.red);
            n = block_scan(n, sh.red);
            if (tid < bins) {
                sh.tw[tid] = w;
                sh.tcnt[tid] = (uint32_t)n;
            }
            __syncthreads();
        };
        auto add = [&](int b, uint32_t w) {
            atomicAdd(&sh.cnt[b], 1u);
            atomicAdd(&sh.lo[b], w & 0xffffu);
            atomicAdd(&sh.hi[b], w >> 16);
        };
        // first of `bins` prefix sums that reaches `need`
        auto first_of = [&](bool weights, u64 need, int bins) {
            if (tid < bins) {
                const u64 x = weights ? sh.tw[tid] : sh.tcnt[tid], before = tid ? (weights ? sh.tw[tid - 1] : sh.tcnt[tid - 1]) : 0;
                if (x >= need && before < need)
                    sh.found = tid;
            }
            __syncthreads();
            const int b = sh.found;
            __syncthreads();
            return b;
        };

        // ---- 2. histogram of z
        part.each([&](float l, int i) {
            if (i < 0)
                return;
            const float z = r.z(l != l ? -INFINITY : l);
            const uint32_t w = Row::weight(z);
            if (w)
                add(Row::bin(z), w);
        });
        join(kBins);
        const uint32_t all = sh.tcnt[kBins - 1];
        const bool by_k = k > 0 && (uint32_t)k < all;
        int bin = kBins - 1;
        if (by_k)
            bin = first_of(false, k, kBins);
        else if (by_p)
            bin = first_of(true, need_of(sh.tw[kBins - 1]), kBins);
        const uint32_t n = sh.tcnt[bin];
        if (n <= kList) {
            // ---- 3a. few tokens: one CTA sorts them
            part.each([&](float l, int i) {
                if (i < 0)
                    return;
                const float z = r.z(l != l ? -INFINITY : l);
                if (Row::bin(z) <= bin && Row::weight(z)) {
                    const uint32_t at = atomicAdd(cl.map_shared_rank(&sh.nlist, 0), 1u);
                    *cl.map_shared_rank(&sh.list[at], 0) = (u64)order_key(l) << 32 | (0xffffffffu - (uint32_t)i);
                }
            });
            cl.sync();
            if (rank)
                return;
            int n2 = 32;
            while (n2 < (int)n)
                n2 <<= 1;
            u64 e = tid < (int)n ? sh.list[tid] : 0;
            __syncthreads();
            e = block_sort(e, n2, true, sh.list);
            u64 w = tid < (int)n && (!by_k || tid < k) ? Row::weight(r.z(key_value((uint32_t)(e >> 32)))) : 0;
            u64 cum = block_scan(w, sh.red);
            if (by_p) {
                // of all tokens that top-k leaves: with it, they are in the list
                const u64 total = by_k ? sh.red[kWarps - 1] : sh.tw[kBins - 1];
                if (cum - w >= need_of(total))
                    w = 0;
            }
            if ((double)w < least)
                w = 0;
            // by index: the kept ones first
            u64 by_index = w ? (u64)(0xffffffffu - (uint32_t)e) << 32 | w : ~0ull << 32;
            __syncthreads();
            by_index = block_sort(by_index, n2, false, sh.list);
            w = tid < n2 ? by_index & 0xffffffffu : 0;
            cum = block_scan(w, sh.red);
            const u64 total = sh.red[kWarps - 1];
            const double target = u * (double)total;
            if (w && (double)cum > target && (double)(cum - w) <= target) {
                const int i = (int)(by_index >> 32);
                const float l = BF16 ? tc::bf16f(static_cast<const uint16_t*>(a.logits)[row * a.stride + i])
                                     : static_cast<const float*>(a.logits)[row * a.stride + i];
                answer(i, l, total);
            }
            return;
        }

        // ---- 3b. narrow the bin by its keys, first for k, then for p
        // smallest key whose bin is at most b
        auto lowest_key = [&](int b) {
            uint32_t lo = 0, hi = (uint32_t)(best >> 32);       // hi is in bin 0
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                const float f = key_value(mid);
                if (f == f && f > -INFINITY && Row::bin(r.z(f)) <= b)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            return lo;
        };
        u64 total = sh.tw[kBins - 1];
        for (int what = 0; what < 2; ++what) {
            const bool weights = what == 1;
            if (weights ? !by_p : !by_k)
                continue;
            const u64 need = weights ? need_of(total) : (u64)k;
            const int b = first_of(weights, need, kBins);
            u64 wab = b ? sh.tw[b - 1] : 0, nab = b ? sh.tcnt[b - 1] : 0;      // weight and count above the range
            uint32_t lo = lowest_key(b);
            u64 range = (b ? (u64)lowest_key(b - 1) : (best >> 32) + 1) - lo;  // keys lo .. lo + range - 1
            // the z histogram is needed again for p
            const u64 keep_w = tid < kBins ? sh.tw[tid] : 0;
            const uint32_t keep_n = tid < kBins ? sh.tcnt[tid] : 0;
            u64 rest;
            while (true) {
                const u64 width = (range + kBins - 1) / kBins;
                cl.sync();
                for (int i = tid; i < kBins; i += kThreads)
                    sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
                __syncthreads();
                part.each([&](float l, int i) {
                    if (i < 0)
                        return;
                    const uint32_t kk = order_key(l);
                    if (kk < lo || kk - lo >= range)
                        return;
                    const uint32_t w = Row::weight(r.z(key_value(kk)));
                    if (w)
                        add(kBins - 1 - (int)((kk - lo) / (uint32_t)width), w);  // larger keys first
                });
                join(kBins);
                rest = need - (weights ? wab : nab);
                const int s = first_of(weights, rest, kBins);
                const u64 w0 = s ? sh.tw[s - 1] : 0, n0 = s ? sh.tcnt[s - 1] : 0;
                const uint32_t here = sh.tcnt[s] - (uint32_t)n0;
                wab += w0;
                nab += n0;
                rest -= weights ? w0 : n0;
                const uint32_t from = (uint32_t)(kBins - 1 - s) * (uint32_t)width;
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
            __syncthreads();
            if (tid < kBins) {
                sh.tw[tid] = keep_w;
                sh.tcnt[tid] = keep_n;
            }
            __syncthreads();
        }
    }

    // ---- 4. kept weights in the vocabulary's order
    u64 sum = 0;
    uint32_t eq = 0;
    const bool cut = ties != 0xffffffffu;
    auto kept = [&](float l) -> uint32_t {       // weight of a token above the cut
        const uint32_t w = Row::weight(r.z(l));
        return (double)w >= least ? w : 0;
    };
    part.each([&](float l, int i) {
        if (i < 0)
            return;
        const uint32_t kk = order_key(l);
        if (cut && kk <= key)
            eq += kk == key;
        else
            sum += kept(key_value(kk));
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        eq += __shfl_xor_sync(~0u, eq, o);
    }
    if (lane == 0) {
        sh.warp_sum[warp] = sum;
        sh.warp_ties[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        u64 s = sh.warp_sum[lane];
        uint32_t n = sh.warp_ties[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(~0u, s, o);
            n += __shfl_xor_sync(~0u, n, o);
        }
        if (lane < c) {
            *cl.map_shared_rank(&sh.part_sum[rank], lane) = s;
            *cl.map_shared_rank(&sh.part_ties[rank], lane) = n;
        }
    }
    cl.sync();
    const u64 wtie = cut ? kept(key_value(key)) : 0;
    u64 total = 0, before = 0;
    uint32_t tie0 = 0, seen = 0;                 // ties before this CTA, and so far
    for (int i = 0; i < c; ++i) {
        const uint32_t in = min(sh.part_ties[i], ties - min(ties, seen));
        if (i == rank) {
            before = total;
            tie0 = seen;
        }
        total += sh.part_sum[i] + in * wtie;
        seen += sh.part_ties[i];
    }
    const double target = u * (double)total;
    // the warp that holds the target
    u64 cum = before;
    seen = tie0;
    for (int w = 0; w < warp; ++w) {
        cum += sh.warp_sum[w] + min(sh.warp_ties[w], ties - min(ties, seen)) * wtie;
        seen += sh.warp_ties[w];
    }
    const u64 own = sh.warp_sum[warp] + min(sh.warp_ties[warp], ties - min(ties, seen)) * wtie;
    if ((double)cum > target || !((double)(cum + own) > target))
        return;
    for (int v = part.v0; v < part.v1; v += 32) {
        uint32_t w[Part<BF16>::VEC], vl = 0, nl = 0;
        float val[Part<BF16>::VEC];
        int idx[Part<BF16>::VEC], j = 0;
        u64 s = 0;
        part.visit(v + lane, [&](float l, int i) {
            const uint32_t kk = order_key(l);
            const bool tie = i >= 0 && cut && kk == key;
            nl += tie;
            vl |= (uint32_t)tie << j;
            w[j] = i < 0 || (cut && kk <= key) ? 0 : kept(key_value(kk));
            val[j] = key_value(kk);
            idx[j] = i;
            s += w[j++];
        });
        const uint32_t ti = warp_scan(nl), tn = __shfl_sync(~0u, ti, 31);
        uint32_t rk = seen + ti - nl;            // ties before this lane's
        if (vl)
#pragma unroll
            for (int e = 0; e < Part<BF16>::VEC; ++e)
                if (vl >> e & 1) {
                    if (rk++ < ties) {
                        w[e] = (uint32_t)wtie;
                        s += wtie;
                    }
                }
        const u64 si = warp_scan(s), sn = __shfl_sync(~0u, si, 31);
        u64 at = cum + si - s;
        if ((double)at <= target && (double)(at + s) > target) {
#pragma unroll
            for (int e = 0; e < Part<BF16>::VEC; ++e) {
                if ((double)at <= target && (double)(at + w[e]) > target)
                    answer(idx[e], val[e], total);
                at += w[e];
            }
        }
        cum += sn;
        seen += tn;
        if ((double)cum > target)
            break;
    }
}

}  // namespace

cudaError_t prepare_sample_kernels()
{
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(sample_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s)
{
    // CTAs a row: as many as leave every row its own SMs, up to 8 (a cluster of 16
    // may find no room), each with at least 2,048 tokens; and no more tokens a CTA
    // than its histogram takes (16 only above 458,752 tokens)
    int c = 1;
    while ((c < 8 && 2ll * c * a.M <= num_sms && a.V >= 2 * c * 2048) ||
           (c < kMostCluster && a.V > c * (kMostPart - kSlackPart)))
        c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.M * c);
    cfg.blockDim = dim3(kThreads);
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
