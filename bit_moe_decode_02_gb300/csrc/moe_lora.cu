// moe_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
// out[m] = y[m] + s_a B_a (A_a x[m]), a the adapter of token m.  The adapters' weights
// are read once for every group of up to eight tokens that share one: a group is the
// eight columns of an m16n8k16 MMA (bf16, fp32 sums), 16 rows of A or B its rows, and
// the order of the summed index is free, so a lane's operands are 16 contiguous bytes.
// Two launches: the first leaves h = A x in fp32 in the workspace, in parts where the
// columns are split over CTAs; the second adds the parts up in their order, splits h
// into three bf16 terms (24 bits) and multiplies by B.  The second starts while the
// first runs and has its first weights on their way when it waits for h.
// Bound by HBM where every token has an adapter of its own: 64 of rank 64, 8,192 x 8,192
// (139 MB), 29 us, 4.8 TB/s: the second kernel streams at 6.5 TB/s, the first at 5, which
// more bytes in flight (4 chunks a buffer 28.6 to 29.5 us, three CTAs an SM 33) do not
// change; the start, the wait between the two and the parts take 3 us.  One token, rank 16,
// 5,120 x 2,880: 4.9 us, nearly all of it two chains of index -> weights -> sums.
#include <cstdint>

#include "kv_device.cuh"
#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

typedef long long i64;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxM = 64;                 // tokens of a call
constexpr int kGroup = 8;                 // tokens of a group
constexpr int kMaxParts = 16;             // of h, over the columns

// Tokens by adapter: groups of at most eight, in the order of their first tokens.  Every
// warp finds them for itself, two tokens a lane.
struct Groups {
    int mine[2];                          // adapters of tokens lane and lane + 32, -1: none
    unsigned heads[2];                    // the first tokens of the groups
    int n;
};
__device__ __forceinline__ Groups find_groups(const LoraArgs& a)
{
    const int lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1;
    Groups g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = lane + 32 * h;
        g.mine[h] = m < a.M ? a.index[m] : -1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (g.mine[h] >= a.n_adapters)
            atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
        if (g.mine[h] < 0 || g.mine[h] >= a.n_adapters)
            g.mine[h] = -1;
    }
    int before = __popc(__match_any_sync(~0u, g.mine[0]) & below);       // tokens before this one with its adapter
    g.heads[0] = __ballot_sync(~0u, g.mine[0] >= 0 && before % kGroup == 0);
    g.heads[1] = 0;
    if (a.M > 32) {
        before = __popc(__match_any_sync(~0u, g.mine[1]) & below);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            before += __shfl_sync(~0u, g.mine[0], i) == g.mine[1];
        g.heads[1] = __ballot_sync(~0u, g.mine[1] >= 0 && before % kGroup == 0);
    }
    g.n = __popc(g.heads[0]) + __popc(g.heads[1]);
    return g;
}
__device__ __forceinline__ int adapter_of(const Groups& g, int m) { return __shfl_sync(~0u, m < 32 ? g.mine[0] : g.mine[1], m & 31); }

// One group: its adapter, and its tokens (-1: none).
struct Group {
    int adapter, member[kGroup];
};
__device__ __forceinline__ Group group_at(const Groups& g, int i)
{
    const int lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1;
    const bool lo = (g.heads[0] >> lane & 1) && __popc(g.heads[0] & below) == i;
    const bool hi = (g.heads[1] >> lane & 1) && __popc(g.heads[0]) + __popc(g.heads[1] & below) == i;
    const unsigned in_lo = __ballot_sync(~0u, lo), in_hi = __ballot_sync(~0u, hi);
    const int head = in_lo ? __ffs(in_lo) - 1 : __ffs(in_hi) + 31;
    Group x;
    x.adapter = adapter_of(g, head);
    unsigned long long m = (unsigned long long)__ballot_sync(~0u, g.mine[1] == x.adapter) << 32 | __ballot_sync(~0u, g.mine[0] == x.adapter);
    m &= ~0ull << head;
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
        x.member[k] = __ffsll((long long)m) - 1;
        m &= m - 1;
    }
    return x;
}
// Member k of this lane's choice.
__device__ __forceinline__ int member_of(const Group& x, int k)
{
    int m = x.member[0];
#pragma unroll
    for (int i = 1; i < kGroup; ++i)
        m = k == i ? x.member[i] : m;
    return m;
}

// Parts of h, over the columns: as many (of 256 columns at least) as let the CTAs of the
// first kernel end together.  A lane for each number, every warp for itself.
__device__ __forceinline__ int parts_of(const LoraArgs& a, int groups)
{
    const int p = (threadIdx.x & 31) + 1, items = groups * ((a.rank + 15) / 16), most = min(kMaxParts, (a.cols + 255) / 256);
    // rounds of a CTA in 1/256 of an item, and what a round costs beside its loads
    const int rounds = (items * p + a.ctas - 1) / a.ctas, cost = rounds * (256 / p + 8);
    const unsigned best = __reduce_min_sync(~0u, p <= most ? (unsigned)cost << 5 | (unsigned)(p - 1) : ~0u);
    return (int)(best & 31) + 1;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 of the summed index: lane c of a row has 8c .. 8c + 7 of it
__device__ __forceinline__ void mma32(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& x)
{
    mma(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
    mma(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

__device__ __forceinline__ uint4 ldg(const uint16_t* p, bool in)
{
    return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// h[part][token][rank] = A x over a part of the columns
__global__ void __launch_bounds__(kThreads, 2) lora_a_kernel(LoraArgs a)
{
    __shared__ float red[kWarps][16 * kGroup];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Groups g = find_groups(a);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int rts = (a.rank + 15) / 16, parts = parts_of(a, g.n), items = g.n * rts * parts;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int part = item % parts, rt = item / parts % rts, grp = item / parts / rts;
        const Group group = group_at(g, grp);
        const int adapter = group.adapter, token = member_of(group, r);
        // chunks of 32 columns in equal runs for the parts; the warps take U of them in turn, so that the
        // CTA reads its rows in long pieces
        constexpr int U = 3;
        const int chunks = (a.cols + 31) / 32;
        const int k0 = ((int)((i64)chunks * part / parts) + warp * U) * 32, k1 = min((int)((i64)chunks * (part + 1) / parts) * 32, a.cols);
        const bool lo_in = rt * 16 + r < a.rank, hi_in = rt * 16 + r + 8 < a.rank;
        const uint16_t* lo = a.a + ((i64)adapter * a.rank + rt * 16 + r) * a.cols + 8 * c;
        const uint16_t* hi = lo + 8ll * a.cols;
        const uint16_t* x = a.x + (i64)max(token, 0) * a.x_stride + 8 * c;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // the next U chunks are on their way while these are multiplied
        uint4 wl[2][U], wh[2][U], wx[2][U];
        auto load = [&](int buf, int k) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k + 32 * u;
                const bool in = at + 8 * c < k1;
                wl[buf][u] = ldg(lo + at, in && lo_in);
                wh[buf][u] = ldg(hi + at, in && hi_in);
                wx[buf][u] = ldg(x + at, in && token >= 0);
            }
        };
        auto multiply = [&](int buf) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                mma32(d, wl[buf][u], wh[buf][u], wx[buf][u]);
        };
        constexpr int step = 32 * U * kWarps;
        load(0, k0);
        for (int k = k0; k < k1; k += 2 * step) {
            load(1, k + step);
            multiply(0);
            load(0, k + 2 * step);
            multiply(1);
        }
        // rows r, r + 8 of this tile by tokens 2c, 2c + 1
        __syncthreads();
        red[warp][r * kGroup + 2 * c] = d[0], red[warp][r * kGroup + 2 * c + 1] = d[1];
        red[warp][(r + 8) * kGroup + 2 * c] = d[2], red[warp][(r + 8) * kGroup + 2 * c + 1] = d[3];
        __syncthreads();
        if (tid < 16 * kGroup) {
            const int row = tid % 16, n = tid / 16, m = member_of(group, n);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += red[w][row * kGroup + n];
            if (m >= 0 && rt * 16 + row < a.rank)
                a.h[((i64)part * kMaxM + m) * a.rank + rt * 16 + row] = sum;
        }
    }
}

template <class T>
__device__ __forceinline__ float value(const T* p)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)*p << 16);
    else
        return *p;
}
template <class T>
__device__ __forceinline__ T rounded(float x)
{
    if constexpr (sizeof(T) == 2)
        return (uint16_t)kv::bf16x2(x, 0.0f);
    else
        return x;
}

// out = y + s B h.  A CTA takes a part of one group's tiles of NT times 16 rows: the parts
// of the group's h are added up in shared memory, then every warp takes every eighth tile,
// with all CH chunks of 32 of the rank.
template <class T, int CH, int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_b_kernel(LoraArgs a)
{
    __shared__ __align__(16) float s_h[kGroup][32 * CH + 4];
    const Groups g = find_groups(a);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const T* y = static_cast<const T*>(a.y);
    T* out = static_cast<T*>(a.out);
    const int parts = parts_of(a, g.n), tiles = (a.rows + 16 * NT - 1) / (16 * NT);
    const int split = g.n ? max(1, min((int)gridDim.x / g.n, (tiles + kWarps - 1) / kWarps)) : 1;       // CTAs of a group
    for (int item = blockIdx.x; item < g.n * split; item += gridDim.x) {
        const Group group = group_at(g, item / split);
        const int part = item % split, tile0 = (int)((i64)tiles * part / split), tile1 = (int)((i64)tiles * (part + 1) / split);
        const int mine[2] = {member_of(group, 2 * c), member_of(group, 2 * c + 1)};
        uint4 lo[CH][NT], hi[CH][NT];
        T yv[NT][2][2];
        auto load = [&](int tile) {
            const int n0 = tile * 16 * NT;
            const uint16_t* b = a.b + ((i64)group.adapter * a.rows + n0 + r) * a.rank + 8 * c;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int row = n0 + 16 * t + r;
                    const bool in = 32 * ch + 8 * c < a.rank;
                    lo[ch][t] = ldg(b + 16ll * t * a.rank + 32 * ch, in && row < a.rows);
                    hi[ch][t] = ldg(b + (16ll * t + 8) * a.rank + 32 * ch, in && row + 8 < a.rows);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = n0 + 16 * t + r + 8 * k;
                        yv[t][e][k] = y && mine[e] >= 0 && row < a.rows ? y[mine[e] * a.y_stride + row] : T(0);
                    }
        };
        if (tile0 + warp < tile1)
            load(tile0 + warp);
        const float s = a.scale ? a.scale[group.adapter] : 1.0f;
        if (item == blockIdx.x)
            asm volatile("griddepcontrol.wait;" ::: "memory");
        else
            __syncthreads();                                   // the last group's h is read no more
        for (int i = tid; i < kGroup * 8 * CH; i += kThreads) {
            const int n = i / (8 * CH), x = i % (8 * CH) * 4, m = member_of(group, n);
            float4 sum = make_float4(0, 0, 0, 0);
            if (m >= 0 && x < a.rank) {
                const float* h = a.h + (i64)m * a.rank + x;
                constexpr int U = 8;                           // parts whose loads go out together
                for (int p = 0; p < parts; p += U) {
                    float4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        v[u] = p + u < parts ? __ldcg(reinterpret_cast<const float4*>(h + (i64)(p + u) * kMaxM * a.rank)) : make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        sum.x += v[u].x, sum.y += v[u].y, sum.z += v[u].z, sum.w += v[u].w;
                }
            }
            *reinterpret_cast<float4*>(&s_h[n][x]) = sum;
        }
        __syncthreads();
        uint32_t h3[CH][3][4];            // this lane's eight of a chunk of its token's h, in three bf16 terms
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 h = *reinterpret_cast<const float2*>(&s_h[r][32 * ch + 8 * c + 2 * e]);
                float u = h.x, v = h.y;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    h3[ch][i][e] = kv::bf16x2(u, v);
                    u -= __uint_as_float(h3[ch][i][e] << 16);
                    v -= __uint_as_float(h3[ch][i][e] & 0xffff0000u);
                }
            }
        for (int tile = tile0 + warp; tile < tile1; tile += kWarps) {
            float d[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.0f;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma32(d[t], lo[ch][t], hi[ch][t], make_uint4(h3[ch][i][0], h3[ch][i][1], h3[ch][i][2], h3[ch][i][3]));
            T base[NT][2][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    base[t][e / 2][e % 2] = yv[t][e / 2][e % 2];
            if (tile + kWarps < tile1)
                load(tile + kWarps);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (mine[e] < 0)
                    continue;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = tile * 16 * NT + 16 * t + r + 8 * k;
                        if (row < a.rows)
                            out[mine[e] * a.out_stride + row] = rounded<T>(value(&base[t][e][k]) + s * d[t][2 * k + e]);
                    }
            }
        }
    }
    if ((int)blockIdx.x >= g.n * split)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    // tokens without an adapter
    if (a.y != a.out)
        for (int m = blockIdx.x; m < a.M; m += gridDim.x)
            if (adapter_of(g, m) < 0)
                for (int row = tid; row < a.rows; row += kThreads)
                    out[m * a.out_stride + row] = y ? y[m * a.y_stride + row] : T(0);
}

typedef void (*KernelB)(LoraArgs);
// NT: 4 KB of B a warp and step at the largest rank of each, 1 KB at rank 8
template <class T>
KernelB pick(int rank, int& rows)
{
    rows = rank <= 32 ? 64 : rank <= 64 ? 32 : 16;
    return rank <= 32 ? lora_b_kernel<T, 1, 4> : rank <= 64 ? lora_b_kernel<T, 2, 2> : lora_b_kernel<T, 4, 1>;
}

}  // namespace

size_t lora_workspace_bytes() { return (size_t)kMaxParts * kMaxM * 128 * sizeof(float); }

cudaError_t launch_lora(LoraArgs a, int num_sms, cudaStream_t s)
{
    a.ctas = 2 * num_sms;
    const int most = a.M * ((a.rank + 15) / 16) * ((a.cols + 255) / 256 < kMaxParts ? (a.cols + 255) / 256 : kMaxParts);
    lora_a_kernel<<<most < a.ctas ? most : a.ctas, kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    int rows;
    const KernelB b = a.type == MOE_DT_BF16 ? pick<uint16_t>(a.rank, rows) : pick<float>(a.rank, rows);
    const i64 items = (i64)a.M * ((a.rows + rows - 1) / rows), ctas = (items + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas < 2 * num_sms ? ctas : 2 * num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, b, a);
}

}  // namespace moe
