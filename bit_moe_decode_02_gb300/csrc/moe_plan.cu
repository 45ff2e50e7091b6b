// moe_plan.cu -- block tables, positions and slots of a step, from the requests' lengths.
//
// Three running sums over at most 1,024 sequences (new tokens, new blocks, blocks that
// come back), which every CTA makes for itself in shared memory; after that each
// token, new block and returned block is an element of its own, found by a search in
// those sums (a warp's 128 tokens by one).  Bound by latency: lengths -> sums -> search
// -> table or ring -> slot.  Measured: 61 sequences of a step 3.3 us; 1,000 requests whose
// prompts make 510,000 tokens (10 MB out) 8.3 us, of which the sums, which 608 CTAs make
// each for itself, are half the instructions (on 304 CTAs 8.9 us, on 152 11.6).
#include <cstdint>

#include "ops_internal.h"

namespace moe {
namespace {

typedef long long i64;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = kMaxSeqs / kThreads; // sequences of a thread
constexpr int kAhead = 4;                 // tokens that a thread takes together

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

// Sums over all threads before each; the whole CTA calls it.
__device__ __forceinline__ Sums scan(const Sums& mine, Sums* warps, Sums& all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums x{__shfl_up_sync(~0u, v.tokens, o), __shfl_up_sync(~0u, v.taken, o), __shfl_up_sync(~0u, v.back, o)};
        if (lane >= o)
            v = v + x;
    }
    if (lane == 31)
        warps[warp] = v;
    const Sums up{__shfl_up_sync(~0u, v.tokens, 1), __shfl_up_sync(~0u, v.taken, 1), __shfl_up_sync(~0u, v.back, 1)};
    __syncthreads();
    Sums before{0, 0, 0};
    all = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp)
            before = all;
        all = all + warps[w];
    }
    return lane ? before + up : before;
}

// The sequence that element i belongs to: the last b < n with sum[b] <= i.
__device__ __forceinline__ int owner(const int* sum, int n, int i)
{
    int b = 0;
#pragma unroll 1
    for (int step = 1 << (31 - __clz(n)); step; step >>= 1)
        if (b + step < n && sum[b + step] <= i)
            b += step;
    return b;
}
// The same for a whole warp's one element: 32 sums at a time.
__device__ __forceinline__ int owner_of_warp(const int* sum, int n, int i)
{
    const int lane = threadIdx.x & 31, at = lane * 32;
    const int first = 32 * (__popc(__ballot_sync(~0u, at < n && sum[at] <= i)) - 1);
    return first + __popc(__ballot_sync(~0u, first + lane < n && sum[first + lane] <= i)) - 1;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a, unsigned* cnt)
{
    __shared__ int s_cu[kMaxSeqs + 1], s_taken[kMaxSeqs + 1], s_back[kMaxSeqs + 1], s_had[kMaxSeqs];
    __shared__ Sums s_warps[kWarps];
    __shared__ int s_last;
    const int tid = threadIdx.x, n = a.n_seqs, log = a.log_block, blk = 1 << log;
    const int per = (n + kThreads - 1) / kThreads, b0 = tid * per;
    int want[kPer], had[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = i < per && b0 + i < n;
        want[i] = in ? a.n_new[b0 + i] : 0;
        had[i] = in ? a.kv_len[b0 + i] : 0;
    }
    const int head = a.state[0], count = a.state[1];
    const bool pool = head >= 0 && head < a.ring_size && count >= 0 && count <= a.ring_size;
    const i64 held_most = (i64)a.table_stride << log;
    const i64 room = held_most < 0x7fffffffll ? held_most : 0x7fffffffll;
    auto blocks_of = [&](int len) { return (int)(((unsigned)len + blk - 1) >> log); };
    Sums each[kPer], mine{0, 0, 0}, all;
    unsigned good = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        each[i] = Sums{0, 0, 0};
        if (pool && had[i] >= 0 && want[i] >= -1 && (i64)had[i] + (want[i] > 0 ? want[i] : 0) <= room) {
            good |= 1u << i;
            const int blocks = blocks_of(had[i]), tokens = want[i] > 0 ? min(want[i], a.n_tokens + 1) : 0;
            each[i] = Sums{tokens, tokens > 0 ? blocks_of(had[i] + tokens) - blocks : 0, want[i] < 0 ? (unsigned)blocks : 0u};
        } else if (i < per && b0 + i < n) {
            atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
        }
        mine = mine + each[i];
    }
    Sums sum = scan(mine, s_warps, all);
    const bool come_back = pool && all.back <= (unsigned)(a.ring_size - count);      // else some block is free and held
    if (!come_back && pool && tid == 0)
        atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
    // the first sequence whose blocks or tokens do not fit, and all after it, get none
    int mine_served = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= per || b0 + i >= n)
            break;
        sum = sum + each[i];
        if (pool && sum.taken <= count && sum.tokens <= a.n_tokens) {
            ++mine_served;
            s_cu[b0 + i + 1] = sum.tokens;
            s_taken[b0 + i + 1] = sum.taken;
        }
        s_back[b0 + i + 1] = come_back ? (int)sum.back : 0;
        s_had[b0 + i] = had[i];
    }
    if (tid == 0) {
        s_cu[0] = s_taken[0] = s_back[0] = 0;
        s_last = 0;
    }
    __syncthreads();
    if (mine_served)
        atomicAdd(&s_last, mine_served);
    __syncthreads();
    const int served = s_last, tokens = s_cu[served], taken = s_taken[served], back = s_back[n];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < per && b0 + i < n && b0 + i >= served) {
            s_cu[b0 + i + 1] = tokens;
            s_taken[b0 + i + 1] = taken;
        }
    __syncthreads();

    const int lane = tid & 31;
    auto ring_at = [&](i64 k) {                                // the k-th free block
        i64 at = head + k;
        at -= at >= a.ring_size ? a.ring_size : 0;
        return a.ring[at];
    };
    auto held = [&](int q) { return blocks_of(s_had[q]); };
    bool fault = false;
    // a warp takes 32 new blocks, 32 that come back, or 128 tokens in a row, most often of one sequence
    const int chunk = 32 * kAhead, taken_at = (taken + 31) / 32, back_at = taken_at + (back + 31) / 32;
    const int units = back_at + (a.n_tokens + chunk - 1) / chunk;
    for (int u = blockIdx.x * kWarps + (tid >> 5); u < units; u += gridDim.x * kWarps) {
        if (u < taken_at) {
            const int k = u * 32 + lane;
            if (k < taken) {
                const int id = ring_at(k), q = owner(s_taken, n, k);
                fault |= id < 0 || id >= a.ring_size;
                a.table[(i64)q * a.table_stride + held(q) + k - s_taken[q]] = id;
            }
        } else if (u < back_at) {
            const int k = (u - taken_at) * 32 + lane;
            if (k < back) {
                const int q = owner(s_back, n, k), id = a.table[(i64)q * a.table_stride + k - s_back[q]];
                fault |= id < 0 || id >= a.ring_size;
                i64 at = (i64)head + count + k;
                at -= at >= a.ring_size ? a.ring_size : 0;
                a.ring[at] = id;
            }
        } else {
            const int t0 = (u - back_at) * chunk, q0 = owner_of_warp(s_cu, n, t0);
            int q[kAhead], pos[kAhead], id[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int t = t0 + 32 * e + lane;
                q[e] = pos[e] = -1;
                id[e] = 0;
                if (t < tokens) {
                    q[e] = q0;
                    if (t >= s_cu[q0 + 1])
                        q[e] = owner(s_cu, n, t);
                    pos[e] = s_had[q[e]] + t - s_cu[q[e]];
                    if (a.slot) {
                        const int j = pos[e] >> log, h = held(q[e]);
                        id[e] = j < h ? a.table[(i64)q[e] * a.table_stride + j] : ring_at((i64)s_taken[q[e]] + j - h);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int t = t0 + 32 * e + lane;
                if (t >= a.n_tokens)
                    break;
                const bool known = id[e] >= 0 && id[e] < a.ring_size;
                fault |= !known;
                if (a.seq)
                    a.seq[t] = q[e];
                if (a.position)
                    a.position[t] = pos[e];
                if (a.slot)
                    a.slot[t] = known && pos[e] >= 0 ? ((i64)id[e] << log) + (pos[e] & (blk - 1)) : -1;
            }
        }
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
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = b0 + i;
        if (i >= per || b >= n)
            break;
        a.cu[b + 1] = s_cu[b + 1];
        a.kv_len_out[b] = (good >> i & 1) && want[i] < 0 && come_back ? 0 : had[i] + (s_cu[b + 1] - s_cu[b]);
    }
    if (tid == 0) {
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
    // a warp's units at most: 128 tokens, or 32 blocks that are taken or come back
    const i64 held = (i64)a.n_seqs * a.table_stride, blocks = held < a.ring_size ? held : a.ring_size;
    const i64 ctas = (a.n_tokens / (32 * kAhead) + blocks / 32 + 3 + kWarps - 1) / kWarps;
    const int grid = (int)(ctas < 4 * num_sms ? ctas : 4 * num_sms);
    const bool in_place = a.kv_len_out == a.kv_len || a.state_out == a.state;
    plan_kernel<<<grid, kThreads, 0, s>>>(a, grid > 1 && in_place ? cnt : nullptr);
    return cudaGetLastError();
}

}  // namespace moe
