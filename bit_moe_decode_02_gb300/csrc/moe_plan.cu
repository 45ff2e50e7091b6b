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

constexpr int kThreads = 1024;            // a sequence each
static_assert(kThreads == kMaxSeqs, "a thread a sequence");

struct Sums {
    i64 tokens, taken, back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) { return {a.tokens + b.tokens, a.taken + b.taken, a.back + b.back}; }

// Sums over all threads up to and with each; the whole CTA calls it.
__device__ __forceinline__ Sums scan(Sums v, Sums* warps, Sums& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
    auto up = [&](Sums x, int o) {
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
        v = v + at(warp - 1);
    __syncthreads();                                           // warps may be written again
    return v;
}

// The sequence that element i belongs to: the last b with sum[b] <= i.
__device__ __forceinline__ int owner(const int* sum, int n, int i)
{
    int lo = 0, hi = n;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(PlanArgs a, unsigned* cnt)
{
    __shared__ int s_cu[kMaxSeqs + 1], s_taken[kMaxSeqs + 1], s_back[kMaxSeqs + 1], s_had[kMaxSeqs];
    __shared__ Sums s_warps[32];
    __shared__ int s_last;
    const int b = threadIdx.x, blk = a.block, n = a.n_seqs;
    int want = 0, had = 0;
    if (b < n) {
        want = a.n_new[b];
        had = a.kv_len[b];
    }
    const int head = a.state[0], count = a.state[1];
    const bool pool = head >= 0 && head < a.ring_size && count >= 0 && count <= a.ring_size;
    const i64 room = (i64)a.table_stride * blk;
    const bool good = pool && had >= 0 && want >= -1 && (i64)had + (want > 0 ? want : 0) <= (room < 0x7fffffffll ? room : 0x7fffffffll);
    const int blocks = (int)(((i64)had + blk - 1) / blk);
    Sums mine{0, 0, 0}, all;
    if (good && b < n) {
        mine.tokens = want > 0 ? want : 0;
        mine.taken = want > 0 ? ((i64)had + want + blk - 1) / blk - blocks : 0;
        mine.back = want < 0 ? blocks : 0;
    }
    if (!good && threadIdx.x < n)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
    Sums incl = scan(mine, s_warps, all);
    // the first sequence whose blocks or tokens do not fit, and all after it, get none
    const bool fits = pool && incl.taken <= count && incl.tokens <= a.n_tokens;
    const bool come_back = pool && count + all.back <= a.ring_size;      // else some block is free and held
    if (!come_back && pool && threadIdx.x == 0)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
    const int served = __syncthreads_count(b < n && fits);
    const Sums before{incl.tokens - mine.tokens, incl.taken - mine.taken, incl.back - mine.back};
    if (b < n && fits) {
        s_cu[b + 1] = (int)incl.tokens;
        s_taken[b + 1] = (int)incl.taken;
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
    auto held = [&](int q) { return (int)(((i64)s_had[q] + blk - 1) / blk); };
    bool fault = false;
    for (int t = first; t < a.n_tokens; t += step) {
        int q = -1, pos = -1;
        i64 slot = -1;
        if (t < tokens) {
            q = owner(s_cu, n, t);
            pos = s_had[q] + t - s_cu[q];
            if (a.slot) {
                const int j = pos / blk, h = held(q);
                const int id = j < h ? a.table[(i64)q * a.table_stride + j] : ring_at((i64)s_taken[q] + j - h);
                if (id >= 0 && id < a.ring_size)
                    slot = (i64)id * blk + (pos - j * blk);
                else
                    fault = true;
            }
        }
        if (a.seq)
            a.seq[t] = q;
        if (a.position)
            a.position[t] = pos;
        if (a.slot)
            a.slot[t] = slot;
    }
    for (int k = first; k < taken; k += step) {
        const int q = owner(s_taken, n, k), id = ring_at(k);
        fault |= id < 0 || id >= a.ring_size;
        a.table[(i64)q * a.table_stride + held(q) + k - s_taken[q]] = id;
    }
    for (int k = first; k < back; k += step) {
        const int q = owner(s_back, n, k), id = a.table[(i64)q * a.table_stride + k - s_back[q]];
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
    const i64 ctas = (most + 2 * kThreads - 1) / (2 * kThreads);
    const int grid = (int)(ctas < num_sms ? ctas : num_sms);
    const bool in_place = a.kv_len_out == a.kv_len || a.state_out == a.state;
    plan_kernel<<<grid, kThreads, 0, s>>>(a, grid > 1 && in_place ? cnt : nullptr);
    return cudaGetLastError();
}

}  // namespace moe
