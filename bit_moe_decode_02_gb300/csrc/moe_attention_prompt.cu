// moe_attention_prompt.cu -- attention of many tokens over the 8-bit paged cache
// (prompts and their chunks), on tcgen05.
//
// 4 D multiply-adds a (row, key) pair, both products as kind::f16 MMAs of 128 rows
// with fp32 accumulators in tensor memory.  What bounds it: a tile of 128 keys moves
// 320 KB through shared memory (192 KB of it MMA operands), 2,500 cycles at 128
// bytes a cycle, where the MMAs need 2,048; it takes 4,200, because a row tile's
// softmax (2,300) and its MMAs (1,300) wait for one another and only the other row
// tile's overlap.  Two prompts of 2,100 tokens over 3,000, 32 heads of 128 on 4 kv
// heads: 287 us, 953 TFLOP/s (0.51 of the measured bf16 rate).
//  - Work.  A CTA takes 256 rows (token, query head of one kv head) of one sequence,
//    as two tiles of 128, against tiles of 128 keys.  Heads that share K and V share
//    the tiles, whatever their number.
//  - Roles (24 warps).  Warp 0 streams the raw codes of a tile's blocks (bulk copies,
//    K and V apart) and their scales.  Warps 4-7 make them the f16 operands, in the
//    canonical K-major order, exactly: K as it lies, V as it lies too (transposed in
//    the cache).  Warp 1 issues the MMAs.  Warps 8-15 and 16-23 do the softmax of
//    one row tile each, two threads a row with 64 keys each: while one tile's is
//    under way, the other's MMAs run.
//  - Tensor memory: S0 S1 O0 O1, 128 columns each.  P replaces the scores it comes
//    from, as f16 (64 keys' in columns 0-31, the others' in 64-95), and is the second
//    product's A operand from there.
//  - Scales and maxima as in the decode kernel: K's scale multiplies a block's
//    scores, V's enters the exponent; O is rescaled in tensor memory only where a
//    row's maximum grows by more than 2^8, or the unit changes.  The unit is the
//    largest V scale of a tile, whether a row sees that block or not, which takes bits
//    of the other blocks' probabilities: a tile whose V scales are more than 2^6 apart
//    goes through as several, one block each.
#include <cstdint>

#include "attn_device.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kThreads = 768;
constexpr int kRows = 256;                // of a CTA
constexpr int kKeys = 128;                // of a tile
constexpr int kRing = 8;                  // tiles whose scales are kept: the loads are at most four ahead of the softmax

template <int D, int BLK>
struct Layout {
    static constexpr int NB = kKeys / BLK;                // cache blocks of a tile
    static constexpr int OP = kKeys * D * 2;              // bytes of an f16 operand: Q tile, K tile, V tile
    static constexpr int RAW = kKeys * D;                 // bytes of a tile's K or V codes
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * OP;
    static constexpr int OFF_V = OFF_K + 2 * OP;
    static constexpr int OFF_RAW = OFF_V + 2 * OP;
    static constexpr int OFF_SC = OFF_RAW + 2 * RAW;      // [kRing][4] (K scale, V scale), K scale < 0: no block
    static constexpr int OFF_BAR = OFF_SC + kRing * 4 * 8;
    static constexpr int OFF_INFO = OFF_BAR + 24 * 8;     // [kRing]: position of the first key, bit 0: the last tile
    static constexpr int OFF_MAX = OFF_INFO + kRing * 4;  // [2 row tiles][2 halves][128]
    static constexpr int SMEM = OFF_MAX + 2 * 2 * 128 * 4;   // 226.4 KB for D = 128, of 227
};

// The whole warp executes these, one elected lane (`one` != 0) issues: outside a
// branch the operands, the same in all lanes, stay in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint64_t* bar)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 ::"r"(tc::su32(bar)), "r"(one) : "memory");
}
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(one));
    return one;
}

#define MOE_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define MOE_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tm_ld32(uint32_t t, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : MOE_R8(r, 0), MOE_R8(r, 8), MOE_R8(r, 16), MOE_R8(r, 24) : "r"(t) : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t t, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
                 ::MOE_I8(r, 0), MOE_I8(r, 8), MOE_I8(r, 16), MOE_I8(r, 24), "r"(t) : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
                 ::MOE_I8(r, 0), MOE_I8(r, 8), "r"(t) : "memory");
}
#define MOE_IO8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
// Waits for this thread's loads; names the registers, so that no use of them is moved above it.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : MOE_IO8(r, 0), MOE_IO8(r, 8), MOE_IO8(r, 16), MOE_IO8(r, 24)::"memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
          "l"(reinterpret_cast<const unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A CTA's rows: the idx-th group of 256 rows, counted over the sequences and,
// within one, over its row tiles (the last, which see the most keys, first) and
// kv heads.  One warp computes it; false: there is no such group.
struct Work {
    int b, c0, n, len;
    int rt, h;
};
__device__ __forceinline__ bool find_work(const AttnArgs& a, int idx, Work& w)
{
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < a.c.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int c0 = 0, n = 0, len = 0;
        if (b < a.c.n_seqs && !kv::sequence(a.c, b, c0, n, len)) {
            atomicExch(a.c.status, MOE_ERR_DEVICE_FAULT);
            n = 0;
        }
        const int cnt = (n * a.group + kRows - 1) / kRows * a.c.H;
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, incl, o);
            if (lane >= o)
                incl += v;
        }
        const unsigned hit = __ballot_sync(~0u, idx < base + incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            w.b = b0 + src;
            w.c0 = __shfl_sync(~0u, c0, src);
            w.n = __shfl_sync(~0u, n, src);
            w.len = __shfl_sync(~0u, len, src);
            const int at = idx - base - __shfl_sync(~0u, incl - cnt, src), tiles = __shfl_sync(~0u, cnt, src) / a.c.H;
            w.rt = tiles - 1 - at / a.c.H;
            w.h = at % a.c.H;
            return true;
        }
        base += __shfl_sync(~0u, incl, 31);
    }
    return false;
}

template <int D, int FMT, int BLK>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(AttnArgs a)
{
    using L = Layout<D, BLK>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* status = a.c.status;
    Work w;
    if (!find_work(a, blockIdx.x, w))
        return;

    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
    uint64_t *raw_full = bar, *raw_empty = bar + 2, *k_full = bar + 4, *k_empty = bar + 6, *v_full = bar + 8, *v_empty = bar + 10;
    uint64_t *s_full = bar + 12, *p_full = bar + 14, *o_full = bar + 16, *q_full = bar + 18;
    float2* sc = reinterpret_cast<float2*>(sm + L::OFF_SC);
    int* info = reinterpret_cast<int*>(sm + L::OFF_INFO);

    const int rows = min(w.n * a.group - w.rt * kRows, kRows), na = rows > 128 ? 2 : 1;     // row tiles with rows
    const int i0 = w.rt * kRows / a.group, i1 = (w.rt * kRows + rows - 1) / a.group;        // first and last token
    const int pos0 = w.len - w.n + i0, pos1 = w.len - w.n + i1;
    const int tile0 = a.window > 0 && pos0 >= a.window ? (pos0 - a.window + 1) / kKeys : 0, nt = pos1 / kKeys - tile0 + 1;
    // `info` says which tile is the last one; this bounds the loops should a wait have given up
    const int most = nt * L::NB;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(raw_full + i, 1);
            tc::mbar_init(raw_empty + i, 4);
            tc::mbar_init(k_full + i, 4);
            tc::mbar_init(k_empty + i, na);
            tc::mbar_init(v_full + i, 4);
            tc::mbar_init(v_empty + i, na);
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, 8);
            tc::mbar_init(o_full + i, 1);
        }
        tc::mbar_init(q_full, 16);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::su32(&tmem_base)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;

    if (warp == 0) {
        // ---- raw codes and scales of each tile's blocks, of those that a row sees: a caller may
        // have given the ones before a window to other sequences
        const int jlo = a.window > 0 && pos0 >= a.window ? (pos0 - a.window + 1) / BLK : 0, jhi = pos1 / BLK;
        auto block_of = [&](int t) {
            const int j = (tile0 + t) * L::NB + lane;
            return lane < L::NB && t < nt && j >= jlo && j <= jhi ? kv::physical(a.c, w.b, j) : -1;
        };
        auto scales_of = [&](int id) {
            return id >= 0 ? *reinterpret_cast<const float2*>(a.c.scales + ((long long)id * a.c.H + w.h) * 2) : make_float2(-1.0f, 0.0f);
        };
        int id = block_of(0);
        float2 s = scales_of(id);
        int t = 0;
#pragma unroll 1
        for (int tile = 0; tile < nt; ++tile) {
            const int next = block_of(tile + 1);
            const uint8_t* src = a.c.codes + ((long long)id * a.c.H + w.h) * 2 * (BLK * D);
            // blocks with V scales far apart go one after another
            bool split = false;
            if constexpr (L::NB > 1) {
                float big = id >= 0 ? s.y : 0.0f, small = big > 0.0f ? big : INFINITY;
#pragma unroll
                for (int o = 1; o < L::NB; o <<= 1) {
                    big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
                    small = fminf(small, __shfl_xor_sync(~0u, small, o));
                }
                split = __shfl_sync(~0u, big > 64.0f * small, 0);
            }
            unsigned left = split ? __ballot_sync(~0u, id >= 0) : 0u;
            do {
                const unsigned now = split ? left & (~left + 1) : ~0u;
                left &= ~now;
                const bool have = id >= 0 && (now >> lane & 1);
                if (lane < L::NB)
                    sc[(t % kRing) * 4 + lane] = have ? s : make_float2(-1.0f, 0.0f);
                if (lane == 0)
                    info[t % kRing] = (tile0 + tile) * kKeys | (tile + 1 == nt && !left);
                const int n = __popc(__ballot_sync(~0u, have));
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (t >= 1)
                        tc::mbar_wait(raw_empty + v, (uint32_t)((t - 1) & 1), status);
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_expect_tx(raw_full + v, (uint32_t)n * (BLK * D));
                    __syncwarp();
                    if (have)
                        tc::bulk_copy(sm + L::OFF_RAW + v * L::RAW + lane * (BLK * D), src + v * (BLK * D), BLK * D, raw_full + v);
                }
                ++t;
            } while (left);
            id = next;
            s = scales_of(id);
        }
    } else if (warp == 1) {
        // ---- MMAs, the row tiles in turn: P V of a tile of keys and the scores of the
        // next go out as that row tile's P is ready, so that its softmax and the other's
        // MMAs come to overlap
        const uint32_t base_desc = (1u << 4) | ((uint32_t)(128 >> 4) << 24);     // fp32 sums, f16 operands, 128 rows
        const uint32_t id_s = base_desc | ((uint32_t)(kKeys >> 3) << 17), id_o = base_desc | ((uint32_t)(D >> 3) << 17);
        const uint64_t qd = tc::smem_desc(tc::su32(sm + L::OFF_Q), 128, D * 16), kd = tc::smem_desc(tc::su32(sm + L::OFF_K), 128, D * 16);
        const uint64_t vd = tc::smem_desc(tc::su32(sm + L::OFF_V), 128, 2048);
        const uint32_t one = elect_one();
        auto scores = [&](int x, int t) {
            const int st = t & 1;
            tc::mbar_wait(k_full + st, (uint32_t)(t >> 1 & 1), status);
            tc::tc_fence_after();
            {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(one, tmem + x * 128, qd + (x * L::OP + 256 * k >> 4), kd + (st * L::OP + 256 * k >> 4), id_s, k > 0);
                commit(one, s_full + x);
                commit(one, k_empty + st);
            }
            __syncwarp();
        };
        tc::mbar_wait(q_full, 0, status);
        for (int x = 0; x < na; ++x)
            scores(x, 0);
        for (int t = 0; t < most; ++t) {
            const int st = t & 1;
            const bool last = info[t % kRing] & 1;
            tc::mbar_wait(v_full + st, (uint32_t)(t >> 1 & 1), status);
            for (int x = 0; x < na; ++x) {
                tc::mbar_wait(p_full + x, (uint32_t)(t & 1), status);
                tc::tc_fence_after();
                {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_ts(one, tmem + 256 + x * 128, tmem + x * 128 + 8 * k + (k >= 4 ? 32 : 0), vd + (st * L::OP + 256 * k >> 4), id_o, t > 0 || k > 0);
                    commit(one, v_empty + st);
                    if (last)
                        commit(one, o_full + x);
                }
                __syncwarp();
                if (!last)
                    scores(x, t + 1);
            }
            if (last)
                break;
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- codes -> f16 operands (zero where there is no block)
        const int ct = tid - 128;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        // a warp's writes (and reads of the raw codes) are done
        auto arrive = [&](uint64_t* full, uint64_t* empty) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(full);
                tc::mbar_arrive(empty);
            }
        };
        for (int t = 0; t < most; ++t) {
            const int st = t & 1;
            const float2* tsc = sc + (t % kRing) * 4;
            tc::mbar_wait(raw_full, (uint32_t)(t & 1), status);
            const bool last = info[t % kRing] & 1;
            if (t >= 2)
                tc::mbar_wait(k_empty + st, (uint32_t)((t >> 1) - 1 & 1), status);
            {
                // K: this thread's token; its 16-code pieces in an order that spreads the banks
                const uint8_t* raw = sm + L::OFF_RAW + ct * D;
                uint8_t* out = sm + L::OFF_K + st * L::OP + (ct >> 3) * (D * 16) + (ct & 7) * 16;
                const bool have = tsc[ct / BLK].x >= 0.0f;
                uint4 w[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    w[i] = *reinterpret_cast<const uint4*>(raw + 16 * ((i + ct / (128 / D)) & (D / 16 - 1)));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int q = (i + ct / (128 / D)) & (D / 16 - 1);
                    const uint4 c = have ? w[i] : zero;
                    uint32_t h[8];
                    to_f16<FMT>(c.x, h[0], h[1]);
                    to_f16<FMT>(c.y, h[2], h[3]);
                    to_f16<FMT>(c.z, h[4], h[5]);
                    to_f16<FMT>(c.w, h[6], h[7]);
                    *reinterpret_cast<uint4*>(out + 256 * q) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(out + 256 * q + 128) = make_uint4(h[4], h[5], h[6], h[7]);
                }
            }
            arrive(k_full + st, raw_empty);

            tc::mbar_wait(raw_full + 1, (uint32_t)(t & 1), status);
            if (t >= 2)
                tc::mbar_wait(v_empty + st, (uint32_t)((t >> 1) - 1 & 1), status);
            {
                // V: this thread's d, 16 tokens at a time
                const int d = ct & (D - 1), part = ct / D;
                const uint8_t* raw = sm + L::OFF_RAW + L::RAW + d * BLK;
                uint8_t* out = sm + L::OFF_V + st * L::OP + (d >> 3) * 2048 + (d & 7) * 16;
                uint4 w[D / 16];
                bool have[L::NB];
#pragma unroll
                for (int b = 0; b < L::NB; ++b)
                    have[b] = tsc[b].x >= 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int q = ((i + d / (128 / BLK)) & (D / 16 - 1)) + part * (D / 16);
                    w[i] = *reinterpret_cast<const uint4*>(raw + q * 16 / BLK * (BLK * D) + q * 16 % BLK);
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int q = ((i + d / (128 / BLK)) & (D / 16 - 1)) + part * (D / 16);
                    bool ok = have[0];
#pragma unroll
                    for (int b = 1; b < L::NB; ++b)
                        ok = q * 16 / BLK == b ? have[b] : ok;
                    const uint4 c = ok ? w[i] : zero;
                    uint32_t h[8];
                    to_f16<FMT>(c.x, h[0], h[1]);
                    to_f16<FMT>(c.y, h[2], h[3]);
                    to_f16<FMT>(c.z, h[4], h[5]);
                    to_f16<FMT>(c.w, h[6], h[7]);
                    *reinterpret_cast<uint4*>(out + 256 * q) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(out + 256 * q + 128) = make_uint4(h[4], h[5], h[6], h[7]);
                }
            }
            arrive(v_full + st, raw_empty + 1);
            if (last)
                break;
        }
    } else if (warp >= 8) {
        // ---- softmax: two threads a row, one for each 64 keys of a tile
        const int x = (warp - 8) >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, row = w.rt * kRows + x * 128 + r;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;      // this warp's quarter of the tensor memory's lanes
        const uint32_t ts = tmem + x * 128 + half * 64 + lanes, to = tmem + 256 + x * 128 + half * (D / 2) + lanes;
        const bool in = x * 128 + r < rows;
        const int i = row / a.group, hq = w.h * a.group + row % a.group;
        float* mine = reinterpret_cast<float*>(sm + L::OFF_MAX) + (x * 2 + half) * 128 + r;
        const float* other = mine + (half ? -128 : 128);
        // the two warps that share 32 rows
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + x * 4 + (warp & 3)) : "memory"); };
        float f;
        {
            // the query row: f16, scaled, in the canonical order; half of it each
            uint32_t big = 0;
            const uint4* q = reinterpret_cast<const uint4*>(a.q + (long long)(w.c0 + i) * a.q_stride + (long long)hq * D);
            if (in)
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 v = q[k];
                    big = max(max(max(big, big_of(v.x)), max(big_of(v.y), big_of(v.z))), big_of(v.w));
                }
            const RowScale rs = row_scale(big, a.scale);
            f = rs.f;
            uint8_t* out = sm + L::OFF_Q + x * L::OP + (r >> 3) * (D * 16) + (r & 7) * 16;
#pragma unroll 4
            for (int k = half * (D / 16); k < (half + 1) * (D / 16); ++k) {
                const uint4 v = in ? q[k] : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(out + 128 * k) =
                    make_uint4(scale_pair(v.x, rs), scale_pair(v.y, rs), scale_pair(v.z, rs), scale_pair(v.w, rs));
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(q_full);
        }
        if (x < na) {
            const int phi = in ? w.len - w.n + i : -1, plo = in && a.window > 0 ? phi - a.window + 1 : 0;
            // positions that all rows of this tile see
            const int all_hi = w.len - w.n + (w.rt * kRows + x * 128) / a.group;
            const int all_lo = a.window > 0 ? w.len - w.n + (w.rt * kRows + min(rows, x * 128 + 128) - 1) / a.group - a.window + 1 : 0;
            float m = kNone, l = 0.0f, ref = 0.0f, vmax = 0.0f;
#pragma unroll 1
            for (int t = 0; t < most; ++t) {
                tc::mbar_wait(s_full + x, (uint32_t)(t & 1), status);
                tc::tc_fence_after();
                const int word = info[t % kRing], p0 = word & ~1;
                float top = 0.0f;
                bool whole = p0 >= all_lo && p0 + kKeys - 1 <= all_hi;
#pragma unroll
                for (int b = 0; b < L::NB; ++b) {
                    const float2 v = sc[(t % kRing) * 4 + b];
                    top = fmaxf(top, v.y);
                    whole = whole && v.x >= 0.0f;
                }
                // scores of 32 keys of this row, -inf where it does not see them
                auto take = [&](int g, uint32_t (&v)[32], float ks) {
                    tm_ld32(ts + 32 * g, v);
                    tm_wait_ld(v);
                    if (!whole) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int p = p0 + 64 * half + 32 * g + k;
                            if (ks < 0.0f || p < plo || p > phi)
                                v[k] = 0xff800000u;
                        }
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float ks = sc[(t % kRing) * 4 + (64 * half + 32 * g) / BLK].x;
                    uint32_t v[32];
                    take(g, v, ks);
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 4]));
#pragma unroll
                    for (int k = 8; k < 32; k += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = max3(y[e], __uint_as_float(v[k + e]), __uint_as_float(v[k + e + 4]));
                    mx = fmaxf(mx, max3(fmaxf(y[0], y[1]), y[2], y[3]) * fmaxf(ks * f, 1e-37f));
                }
                *mine = mx;
                pair_sync();
                mx = fmaxf(mx, *other);
                const bool unit = !(top <= 2.0f * ref && top >= 0.5f * ref);            // the same for all warps
                if (__any_sync(~0u, unit || mx > m + kSlack)) {                         // the same for both of a pair
                    const float mn = fmaxf(m, mx);
                    float al = ex2(m - mn);
                    m = mn;
                    l *= al;
                    if (unit) {
                        vmax = fmaxf(vmax, top);
                        const float now = new_unit(top, vmax);
                        al *= ref / now;
                        ref = now;
                    }
                    if (t > 0)
#pragma unroll 1
                        for (int ch = 0; ch < D / 64; ++ch) {
                            uint32_t v[32];
                            tm_ld32(to + 32 * ch, v);
                            tm_wait_ld(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(__uint_as_float(v[k]) * al);
                            tm_st32(to + 32 * ch, v);
                        }
                }
                const float iref = rcp(ref);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float2 kv = sc[(t % kRing) * 4 + (64 * half + 32 * g) / BLK];
                    const float c = fmaxf(kv.x * f, 1e-37f), ratio = fmaxf(kv.y * iref, 8.673617379884035e-19f);   // 2^-60
                    const float off = lg2(ratio) - m + kRoom;
                    uint32_t v[32], p[16];
                    take(g, v, kv.x);
                    const float2 cc = make_float2(c, c), oo = make_float2(off, off);
                    float2 part[2];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float2 z = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), cc, oo);
                        z.x = ex2(z.x);
                        z.y = ex2(z.y);
                        part[k / 2 & 1] = k > 2 ? add2(part[k / 2 & 1], z) : z;
                        p[k / 2] = pack_f16(z.x, z.y);
                    }
                    const float2 both = add2(part[0], part[1]);
                    l += (both.x + both.y) * rcp(ratio);
                    tm_st16(ts + 16 * g, p);
                }
                tm_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(p_full + x);
                if (word & 1)
                    break;
            }
            // ---- the row's result, half of its columns each
            pair_sync();                     // both have read the last maxima
            *mine = l;
            pair_sync();
            l = (l + *other) * kUnroom;
            tc::mbar_wait(o_full + x, 0, status);
            tc::tc_fence_after();
            const Final fin = finish(m, l, a.sinks, hq);
            const float mul = fin.mul * ref * kUnroom;
            uint16_t* out = a.out + ((long long)(w.c0 + i) * a.q_heads + hq) * D + half * (D / 2);
#pragma unroll
            for (int ch = 0; ch < D / 64; ++ch) {
                uint32_t v[32];
                tm_ld32(to + 32 * ch, v);
                tm_wait_ld(v);
                if (in)
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = kv::bf16x2(__uint_as_float(v[k + 2 * e]) * mul, __uint_as_float(v[k + 2 * e + 1]) * mul);
                        *reinterpret_cast<uint4*>(out + 32 * ch + k) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
            if (a.lse && in && half == 0)
                a.lse[(long long)(w.c0 + i) * a.q_heads + hq] = fin.lse;
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 3)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

typedef void (*Kernel)(AttnArgs);

template <int D, int FMT>
Kernel pick(int blk)
{
    return blk == 32 ? prompt_attn_kernel<D, FMT, 32> : blk == 64 ? prompt_attn_kernel<D, FMT, 64> : prompt_attn_kernel<D, FMT, 128>;
}
Kernel kernel_for(int d, int fmt, int blk)
{
    if (d == 64)
        return fmt == MOE_KV_E4M3 ? pick<64, MOE_KV_E4M3>(blk) : pick<64, MOE_KV_INT8>(blk);
    return fmt == MOE_KV_E4M3 ? pick<128, MOE_KV_E4M3>(blk) : pick<128, MOE_KV_INT8>(blk);
}
int smem_of(int d) { return d == 64 ? Layout<64, 64>::SMEM : Layout<128, 64>::SMEM; }   // whatever the block

}  // namespace

cudaError_t prepare_prompt_kernels()
{
    for (int d = 64; d <= 128; d *= 2)
        for (int fmt : {MOE_KV_E4M3, MOE_KV_INT8})
            for (int blk = 32; blk <= 128; blk *= 2) {
                const cudaError_t e = cudaFuncSetAttribute(kernel_for(d, fmt, blk), cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(d));
                if (e != cudaSuccess)
                    return e;
            }
    return cudaSuccess;
}

cudaError_t launch_attention_prompt(const AttnArgs& a, int, cudaStream_t s)
{
    // an upper bound on the groups of 256 rows: CTAs beyond the last one end at once
    const long long groups = ((long long)a.c.n_tokens * a.group / kRows + a.c.n_seqs) * a.c.H;
    kernel_for(a.c.D, a.c.fmt, a.c.blk)<<<(unsigned)groups, kThreads, smem_of(a.c.D), s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
