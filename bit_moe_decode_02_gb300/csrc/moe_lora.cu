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
constexpr int kTiles = 4;                 // tiles of 16 rows of B that a warp takes at once

// Tokens by adapter: groups of at most eight, in the order of their first tokens.
struct Groups {
    int n;
    int adapter[kMaxM];
    int member[kMaxM][kGroup];            // tokens, -1: none
    int of[kMaxM];                        // a token's adapter, -1: none
    int heads[2];
};
__device__ __forceinline__ void find_groups(const LoraArgs& a, Groups& g)
{
    const int tid = threadIdx.x;
    int mine = -1;
    if (tid < kMaxM) {
        mine = tid < a.M ? a.index[tid] : -1;
        if (mine >= a.n_adapters) {
            atomicExch(a.status, MOE_ERR_DEVICE_FAULT);
            mine = -1;
        }
        mine = mine < 0 ? -1 : mine;
        g.of[tid] = mine;
    }
    for (int i = tid; i < kMaxM * kGroup; i += kThreads)
        g.member[i / kGroup][i % kGroup] = -1;
    __syncthreads();
    int before = 0, head = tid;           // tokens before this one with its adapter; the first of its group
    if (tid < kMaxM) {
        if (mine >= 0)
            for (int m = 0; m < tid; ++m)
                before += g.of[m] == mine;
        const unsigned first = __ballot_sync(~0u, mine >= 0 && before % kGroup == 0);
        if ((tid & 31) == 0)
            g.heads[tid >> 5] = (int)first;
    }
    __syncthreads();
    if (tid < kMaxM && mine >= 0) {
        int skip = before / kGroup * kGroup;
        for (int m = 0; m <= tid; ++m)
            if (g.of[m] == mine && skip-- == 0)
                head = m;
        const unsigned lo = g.heads[0], hi = g.heads[1];
        const int at = head < 32 ? __popc(lo & ((1u << head) - 1)) : __popc(lo) + __popc(hi & ((1u << (head - 32)) - 1));
        g.member[at][before % kGroup] = tid;
        g.adapter[at] = mine;
    }
    if (tid == 0)
        g.n = __popc((unsigned)g.heads[0]) + __popc((unsigned)g.heads[1]);
    __syncthreads();
}

// Parts of h: as many as fill the CTAs, of 256 columns at least.
__device__ __forceinline__ int parts_of(const LoraArgs& a, int groups)
{
    const int items = groups * ((a.rank + 15) / 16), most = min(kMaxParts, (a.cols + 255) / 256);
    return items ? max(1, min(most, a.ctas / items)) : 1;
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
    __shared__ Groups g;
    __shared__ float red[kWarps][16 * kGroup];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_groups(a, g);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int rts = (a.rank + 15) / 16, parts = parts_of(a, g.n), items = g.n * rts * parts;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int part = item % parts, rt = item / parts % rts, grp = item / parts / rts;
        const int adapter = g.adapter[grp], token = g.member[grp][r];
        // chunks of 32 columns, in equal runs for the parts and their warps
        const int chunks = (a.cols + 31) / 32, runs = parts * kWarps, run = part * kWarps + warp;
        const int k0 = (int)((i64)chunks * run / runs) * 32, k1 = min((int)((i64)chunks * (run + 1) / runs) * 32, a.cols);
        const bool lo_in = rt * 16 + r < a.rank, hi_in = rt * 16 + r + 8 < a.rank;
        const uint16_t* lo = a.a + ((i64)adapter * a.rank + rt * 16 + r) * a.cols + 8 * c;
        const uint16_t* hi = lo + 8ll * a.cols;
        const uint16_t* x = a.x + (i64)max(token, 0) * a.x_stride + 8 * c;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int U = 6;
        for (int k = k0; k < k1; k += 32 * U) {
            uint4 wl[U], wh[U], wx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k + 32 * u;
                const bool in = at + 8 * c < k1;
                wl[u] = ldg(lo + at, in && lo_in);
                wh[u] = ldg(hi + at, in && hi_in);
                wx[u] = ldg(x + at, in && token >= 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                mma32(d, wl[u], wh[u], wx[u]);
        }
        // rows r, r + 8 of this tile by tokens 2c, 2c + 1
        __syncthreads();
        red[warp][r * kGroup + 2 * c] = d[0], red[warp][r * kGroup + 2 * c + 1] = d[1];
        red[warp][(r + 8) * kGroup + 2 * c] = d[2], red[warp][(r + 8) * kGroup + 2 * c + 1] = d[3];
        __syncthreads();
        if (tid < 16 * kGroup) {
            const int row = tid % 16, n = tid / 16, m = g.member[grp][n];
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

// out = y + s B h
template <class T>
__global__ void __launch_bounds__(kThreads, 2) lora_b_kernel(LoraArgs a)
{
    __shared__ Groups g;
    find_groups(a, g);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const T* y = static_cast<const T*>(a.y);
    T* out = static_cast<T*>(a.out);
    const int parts = parts_of(a, g.n), chunks = (a.rank + 31) / 32;
    const int tiles = (a.rows + 16 * kTiles - 1) / (16 * kTiles);
    const i64 items = (i64)g.n * tiles;
    bool waited = false;
    for (i64 item = (i64)blockIdx.x * kWarps + warp; item < items; item += (i64)gridDim.x * kWarps) {
        const int grp = (int)(item / tiles), n0 = (int)(item % tiles) * 16 * kTiles;
        const int adapter = g.adapter[grp], token = g.member[grp][r];
        float d[kTiles][4];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.0f;
        for (int ch = 0; ch < chunks; ++ch) {
            const int at = 32 * ch + 8 * c;
            uint4 wl[kTiles], wh[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const int row = n0 + 16 * t + r;
                const uint16_t* p = a.b + ((i64)adapter * a.rows + row) * a.rank + at;
                wl[t] = ldg(p, at < a.rank && row < a.rows);
                wh[t] = ldg(p + 8ll * a.rank, at < a.rank && row + 8 < a.rows);
            }
            if (!waited) {
                asm volatile("griddepcontrol.wait;" ::: "memory");
                waited = true;
            }
            // this lane's eight of the group's h, in three bf16 terms
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = 0.0f;
            if (token >= 0 && at < a.rank)
                for (int p = 0; p < parts; ++p) {
                    const float4* q = reinterpret_cast<const float4*>(a.h + ((i64)p * kMaxM + token) * a.rank + at);
                    const float4 u = __ldcg(q), v = __ldcg(q + 1);
                    h[0] += u.x, h[1] += u.y, h[2] += u.z, h[3] += u.w, h[4] += v.x, h[5] += v.y, h[6] += v.z, h[7] += v.w;
                }
            uint32_t t3[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float u = h[2 * e], v = h[2 * e + 1];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    t3[i][e] = kv::bf16x2(u, v);
                    u -= __uint_as_float(t3[i][e] << 16);
                    v -= __uint_as_float(t3[i][e] & 0xffff0000u);
                }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    mma32(d[t], wl[t], wh[t], make_uint4(t3[i][0], t3[i][1], t3[i][2], t3[i][3]));
        }
        const float s = a.scale ? a.scale[adapter] : 1.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = g.member[grp][2 * c + e];
            if (m < 0)
                continue;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = n0 + 16 * t + r + 8 * k;
                    if (row < a.rows) {
                        const float base = y ? value(y + m * a.y_stride + row) : 0.0f;
                        out[m * a.out_stride + row] = rounded<T>(base + s * d[t][2 * k + e]);
                    }
                }
        }
    }
    if (!waited)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    // tokens without an adapter
    if (a.y != a.out)
        for (int m = blockIdx.x; m < a.M; m += gridDim.x)
            if (g.of[m] < 0)
                for (int row = tid; row < a.rows; row += kThreads)
                    out[m * a.out_stride + row] = y ? y[m * a.y_stride + row] : T(0);
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
    const i64 tiles = (i64)a.M * ((a.rows + 16 * kTiles - 1) / (16 * kTiles)), ctas = (tiles + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas < a.ctas ? ctas : a.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return a.type == MOE_DT_BF16 ? cudaLaunchKernelEx(&cfg, lora_b_kernel<uint16_t>, a) : cudaLaunchKernelEx(&cfg, lora_b_kernel<float>, a);
}

}  // namespace moe
