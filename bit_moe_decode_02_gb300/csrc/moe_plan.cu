// moe_plan.cu -- block tables, positions and slots of a step, from the requests' lengths.
//
// Three running sums over at most 1,024 sequences (new tokens, new blocks, blocks that
// come back), which every CTA makes for itself in shared memory; after that each
// token, new block and returned block is an element of its own, found by a search in
// those sums.  Bound by latency: lengths -> sums -> search -> table or ring -> slot.
#include <cstdint>

#include "ops_internal.h"

namespace moe {
namespace {

typedef long long i64;

constexpr int kThreads = 1024;            // a sequence each; 256 where those are enough
constexpr int kAhead = 4;                 // tokens that a thread looks up together
static_assert(kThreads == kMaxSeqs, "a thread a sequence");

// Tokens and taken blocks of a sequence are held to what cannot fit in any call before they
// are summed, so that 1,024 of them stay within 31 bits; what comes back saturates.
struct Sums {
    int tokens, taken;
    unsigned back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b)
{
    const unsigned back = a.back + b.back;
    return {a.tokens + b.tokens, a.taken + b.taken, back < a.back ? ~0u : back};
}

// Sums over all threads up to and with each; the whole CTA calls it.
__device__ __forceinline__ Sums scan(Sums v, Sums* warps, Sums& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
    auto up = [&](const Sums& x, int o) {
        return Sums{__shfl_up_sync(~0u, x.tokens, o), __shfl_up_sync(~0u, x.taken, o), __shfl_up_sync(~0u, x.back, o)};
    };
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums x = up(v, o);
        if (lane >= o)
            v = v + x;
    }
    if (lane == 31)
        warps[warp] = v;
    __syncthreads();
    Sums w = lane < n ? warps[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums x = up(w, o);
        if (lane >= o)
            w = w + x;
    }
    auto at = [&](int src) {
        return Sums{__shfl_sync(~0u, w.tokens, src), __shfl_sync(~0u, w.taken, src), __shfl_sync(~0u, w.back, src)};
    };
    all = at(n - 1);
    if (warp > 0)
        v = at(warp - 1) + v;
    return v;
}

// The sequences that elements i belong to: the last b < n with sum[b] <= i.
template <int N>
__device__ __forceinline__ void owners(const int* sum, int n, const int (&i)[N], int (&b)[N])
{
#pragma unroll
    for (int k = 0; k < N; ++k)
        b[k] = 0;
#pragma unroll 1
    for (int step = 1 << (31 - __clz(n)); step; step >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (b[k] + step < n && sum[b[k] + step] <= i[k])
                b[k] += step;
}

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(PlanArgs a, unsigned* cnt)
{
    __shared__ int s_cu[kMaxSeqs + 1], s_taken[kMaxSeqs + 1], s_back[kMaxSeqs + 1], s_had[kMaxSeqs];
    __shared__ Sums s_warps[32];
    __shared__ int s_last;
    const int b = threadIdx.x, n = a.n_seqs, log = a.log_block, blk = 1 << log;
    int want = 0, had = 0;
    if (b < n) {
        want = a.n_new[b];
        had = a.kv_len[b];
    }
    const int head = a.state[0], count = a.state[1];
    const bool pool = head >= 0 && head < a.ring_size && count >= 0 && count <= a.ring_size;
    const i64 room = (i64)a.table_stride * blk;
    const bool good = pool && had >= 0 && want >= -1 && (i64)had + (want > 0 ? want : 0) <= (room < 0x7fffffffll ? room : 0x7fffffffll);
    auto blocks_of = [&](int len) { return (int)(((unsigned)len + blk - 1) >> log); };
    const int blocks = blocks_of(had);
    Sums mine{0, 0, 0}, all;
    if (good && b < n) {
        mine.tokens = want > 0 ? min(want, a.n_tokens + 1) : 0;
        mine.taken = want > 0 ? blocks_of(had + mine.tokens) - blocks : 0;
        mine.back = want < 0 ? blocks : 0;
    }
    if (!good && threadIdx.x < n)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
    Sums incl = scan(mine, s_warps, all);
    // the first sequence whose blocks or tokens do not fit, and all after it, get none
    const bool fits = pool && incl.taken <= count && incl.tokens <= a.n_tokens;
    const bool come_back = pool && all.back <= (unsigned)(a.ring_size - count);      // else some block is free and held
    if (!come_back && pool && threadIdx.x == 0)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
    const int served = __syncthreads_count(b < n && fits);
    if (b < n && fits) {
        s_cu[b + 1] = incl.tokens;
        s_taken[b + 1] = incl.taken;
    }
    if (b < n) {
        s_back[b + 1] = come_back ? (int)incl.back : 0;
        s_had[b] = had;
    }
    if (b == 0)
        s_cu[0] = s_taken[0] = s_back[0] = 0;
    __syncthreads();
    const int tokens = s_cu[served], taken = s_taken[served], back = s_back[n];
    if (b < n && !fits) {
        s_cu[b + 1] = tokens;
        s_taken[b + 1] = taken;
    }
    __syncthreads();

    const int step = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
    auto ring_at = [&](i64 k) {                                // the k-th free block
        i64 at = head + k;
        at -= at >= a.ring_size ? a.ring_size : 0;
        return a.ring[at];
    };
    auto held = [&](int q) { return blocks_of(s_had[q]); };
    bool fault = false;
    for (int t0 = first; t0 < a.n_tokens; t0 += kAhead * step) {
        int t[kAhead], q[kAhead], pos[kAhead], id[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            t[e] = t0 + e * step;                              // below 2^20 + 4 * 152 * 1024
        owners(s_cu, n, t, q);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const bool in = t[e] < tokens;
            pos[e] = in ? s_had[q[e]] + t[e] - s_cu[q[e]] : -1;
            id[e] = 0;
            if (in && a.slot) {
                const int j = pos[e] >> log, h = held(q[e]);
                id[e] = j < h ? a.table[(i64)q[e] * a.table_stride + j] : ring_at((i64)s_taken[q[e]] + j - h);
            }
            q[e] = in ? q[e] : -1;
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (t[e] >= a.n_tokens)
                break;
            const bool known = id[e] >= 0 && id[e] < a.ring_size;
            fault |= !known;
            if (a.seq)
                a.seq[t[e]] = q[e];
            if (a.position)
                a.position[t[e]] = pos[e];
            if (a.slot)
                a.slot[t[e]] = known && pos[e] >= 0 ? ((i64)id[e] << log) + (pos[e] & (blk - 1)) : -1;
        }
    }
    for (int k = first; k < taken; k += step) {
        const int at_k[1] = {k};
        int q[1];
        owners(s_taken, n, at_k, q);
        const int id = ring_at(k);
        fault |= id < 0 || id >= a.ring_size;
        a.table[(i64)q[0] * a.table_stride + held(q[0]) + k - s_taken[q[0]]] = id;
    }
    for (int k = first; k < back; k += step) {
        const int at_k[1] = {k};
        int q[1];
        owners(s_back, n, at_k, q);
        const int id = a.table[(i64)q[0] * a.table_stride + k - s_back[q[0]]];
        fault |= id < 0 || id >= a.ring_size;
        i64 at = (i64)head + count + k;
        at -= at >= a.ring_size ? a.ring_size : 0;
        a.ring[at] = id;
    }
    if (fault)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);

    // lengths and the ring's state, once every CTA has read them where they are updated in place
    if (cnt) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            s_last = atomicAdd(cnt, 1u) == gridDim.x - 1;
            if (s_last)
                *cnt = 0;
        }
        __syncthreads();
        if (!s_last)
            return;
    } else if (blockIdx.x) {
        return;
    }
    if (b < n) {
        a.cu[b + 1] = s_cu[b + 1];
        a.kv_len_out[b] = good && want < 0 && come_back ? 0 : had + (s_cu[b + 1] - s_cu[b]);
    }
    if (b == 0) {
        a.cu[0] = 0;
        i64 at = (i64)head + taken;
        at -= pool && at >= a.ring_size ? a.ring_size : 0;
        a.state_out[0] = (int)at;
        a.state_out[1] = count - taken + back;
        if (a.admitted)
            a.admitted[0] = served;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, int num_sms, unsigned* cnt, cudaStream_t s)
{
    // elements at most: a token each, and a block each that is taken or comes back
    const i64 held = (i64)a.n_seqs * a.table_stride, most = a.n_tokens + (held < a.ring_size ? held : a.ring_size);
    // one CTA of 256 threads, or of 1,024 each: many threads make the sums slower
    const int threads = a.n_seqs <= 256 && most <= 2048 ? 256 : kThreads;
    const i64 ctas = (most + 2 * threads - 1) / (2 * threads);
    const int grid = threads < kThreads ? 1 : (int)(ctas < num_sms ? ctas : num_sms);
    const bool in_place = a.kv_len_out == a.kv_len || a.state_out == a.state;
    plan_kernel<<<grid, threads, 0, s>>>(a, grid > 1 && in_place ? cnt : nullptr);
    return cudaGetLastError();
}

}  // namespace moe
