// moe_attention_prompt.cu -- attention of many tokens over the paged cache
// (prompts and their chunks), on tcgen05.
//
// 4 D multiply-adds a (row, key) pair, both products as kind::f16 MMAs of 128 rows
// with fp32 accumulators in tensor memory.  What bounds it: a tile of 128 keys moves
// 320 KB through shared memory (192 KB of it MMA operands), 2,500 cycles at 128
// bytes a cycle, where the MMAs need 2,048; it takes 3,900, because a row tile's
// softmax and its MMAs (1,300) wait for one another, but for the first half of P V, and
// otherwise only the other row tile's overlap.  Two prompts of 2,100 tokens over 3,000, 32 heads of 128 on 4 kv
// heads: 259 us, 1,058 TFLOP/s (0.56 of the measured bf16 rate); 275 with P handed over
// whole instead of 266 in halves and 264.6 in quarters.
//  - Work.  A CTA takes 256 rows (token, query head of one kv head) of one sequence,
//    as two tiles of 128, against tiles of 128 keys.  Heads that share K and V share
//    the tiles, whatever their number.
//  - Roles (24 warps).  Warp 0 streams the raw codes of a tile's blocks (bulk copies,
//    K and V apart) and their scales.  Warps 4-7 (2-7 in 4 bits) make them the f16 operands, in the
//    canonical K-major order, exactly: K as it lies, V as it lies too (transposed in
//    the cache).  Warp 1 issues the MMAs.  Warps 8-15 and 16-23 do the softmax of
//    one row tile each, two threads a row with 64 keys each: while one tile's is
//    under way, the other's MMAs run.
//  - Tensor memory: S0 S1 O0 O1, 128 columns each.  P replaces the scores it comes
//    from, as f16 (64 keys' in columns 0-31, the others' in 64-95), and is the second
//    product's A operand from there.
//  - Few groups of rows leave SMs idle, or the last ones of many do: then the keys of each of those are cut into
//    parts (prompt_cut; four tiles at least), a CTA each, whose results a second kernel joins in their order.
//    One sequence of 4,000 keys, 64 heads of 64 on 8, 80 tokens: 27 us, 60 by a CTA a group; 8 of them, 32 heads
//    of 128 on 4, 8 tokens: 25 and 53; 160 groups 65 and 85; the two prompts above 259 and 266.
//  - Scales and maxima as in the decode kernel: K's scale multiplies a block's
//    scores, V's enters the exponent; O is rescaled in tensor memory only where a
//    row's maximum grows by more than 2^8, or the unit changes.  The unit is the
//    largest V scale of a tile, whether a row sees that block or not, which takes bits
//    of the other blocks' probabilities: a tile whose V scales are more than 2^6 apart
//    goes through as several, one block each.
//  - In 4 bits a token's groups have scales of their own, which go into the f16 operands:
//    K's relative to the largest of a tile (Pass), V's to units of 32 columns of O each, so
//    that the softmax knows one scale a tile.  The same prompts, sinks besides: 271 us (350
//    before V's operands were stored without bank conflicts, 324 with a call at every wait, 305 with both
//    forms of a score's rounding in one loop).
#include <cstdint>

#include "attn_device.cuh"
#include "kv4_device.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kThreads = 768;
constexpr int kRows = kGroupRows;         // of a CTA
constexpr int kKeys = kTileKeys;          // of a tile
constexpr int kRing = 8;                  // tiles whose scales are kept: the loads are at most four ahead of the softmax

// A pass of a tile over a 4-bit cache: which of its keys take part, what their K's are scaled
// by, and the units of O's columns.
struct Pass {
    uint32_t keys[4];                     // a bit a key
    int kref;                             // K's f16 operand is its value times 2^(13 + 127 - kref)
    int unit[4];                          // of each group's V: its f16 operand is the value times 2^(13 + 127 - unit)
    int most[4];                          // largest exponent field of those operands' scales: 28, less in a later pass (0: none)
    uint32_t flags;                       // kCount: the probabilities join the sums; kAll: all keys
};
enum : uint32_t { kCount = 1, kAll = 2 };

template <int D, int FMT, int BLK>
struct Layout {
    static constexpr bool MX = FMT == MOE_KV_MXFP4;
    static constexpr int NB = kKeys / BLK;                // cache blocks of a tile
    static constexpr int CONVERT = MX ? 6 : 4;            // warps that make codes f16: the last of warps 0 to 7
    static constexpr int OP = kKeys * D * 2;              // bytes of an f16 operand: Q tile, K tile, V tile
    static constexpr int REC = MX ? kv4::record(BLK, D) : BLK * D;     // bytes of a block's K or V
    static constexpr int RAW = NB * REC;                  // bytes of a tile's K or V codes
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * OP;
    static constexpr int OFF_V = OFF_K + 2 * OP;
    static constexpr int OFF_RAW = OFF_V + 2 * OP;
    static constexpr int OFF_SC = OFF_RAW + 2 * RAW;      // [kRing][4] (K scale, V scale), K scale < 0: no block
    static constexpr int OFF_BAR = OFF_SC + kRing * 4 * 8;
    static constexpr int OFF_INFO = OFF_BAR + 24 * 8;     // [kRing]: position of the first key, bit 0: the last tile
    static constexpr int OFF_MAX = OFF_INFO + kRing * 4;  // [2 row tiles][2 halves][128]
    static constexpr int OFF_PASS = OFF_MAX + 2 * 2 * 128 * 4;         // MXFP4: [kRing]
    [[maybe_unused]] static constexpr int SMEM = OFF_PASS + (MX ? kRing * (int)sizeof(Pass) : 0);   // 226.4 KB for D = 128 in 8 bits, of 227
};

// A bounded wait, short where another one has given up already: a tile may go through in
// many passes, and the kernel has to end soon with its status set.
static __device__ __noinline__ void wait_on(uint64_t* bar, uint32_t parity, int* status)
{
#pragma unroll 1
    for (int i = 1; i < 1 << 22; ++i) {
        if (tc::mbar_try_wait(bar, parity))
            return;
        if (i % 4096 == 0 && *(volatile int*)status == MOE_ERR_DEVICE_TIMEOUT)
            return;
    }
    atomicExch(status, MOE_ERR_DEVICE_TIMEOUT);
}
// A wait that is over costs no call.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int* status)
{
    if (!tc::mbar_try_wait(bar, parity))
        wait_on(bar, parity, status);
}

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

// The rows of a group, and the tiles of keys that they see.
struct Extent {
    int rows;                             // of 256
    int pos0, pos1;                       // of the first and the last token
    int tile0, tiles;
    __device__ __forceinline__ Extent(const AttnArgs& a, const Work& w)
    {
        rows = min(w.n * a.group - w.rt * kRows, kRows);
        pos0 = w.len - w.n + w.rt * kRows / a.group;
        pos1 = w.len - w.n + (w.rt * kRows + rows - 1) / a.group;
        tile0 = a.window > 0 && pos0 >= a.window ? (pos0 - a.window + 1) / kKeys : 0;
        tiles = pos1 / kKeys - tile0 + 1;
    }
    // how many CTAs share them, of `most`
    __device__ __forceinline__ int parts(int most) const { return max(min(most, tiles / kPartTiles), 1); }
};

// A part's results: its 256 rows as attn_device.cuh keeps them, four columns of all rows after
// another, then the rows' maxima and sums.
__host__ __device__ constexpr int part_floats(int d) { return kRows * d + 2 * kRows; }

// The producer of a 4-bit cache: a tile's raw records, and how it goes through.  Keys whose
// largest scales are within 2^9 go together (K's f16 operand holds 2^36), the others in passes
// of their own; V's groups each have a unit that O's 32 columns are kept in, which moves where
// a tile's largest scale leaves [unit - 16, unit], and scales 2^28 and more below it go in
// passes of their own with the same probabilities.  One warp; nearly every tile is one pass.
template <int D, int BLK>
__device__ __forceinline__ void mx_produce(const AttnArgs& a, const Work& w, Pass* passes, int* info, uint8_t* raw, uint64_t* raw_full,
                                           uint64_t* raw_empty, int tile0, int nt, int jlo, int jhi, int see_lo, int see_hi)
{
    using L = Layout<D, MOE_KV_MXFP4, BLK>;
    constexpr int G = D / 32, N = D / 32;                 // N: words of a lane's scales, K's and V's
    const int lane = threadIdx.x & 31, sub = lane >> 3, r = lane & 7;
    int* status = a.c.status;
    auto block_of = [&](int t) {
        const int j = (tile0 + t) * L::NB + lane;
        return lane < L::NB && t < nt && j >= jlo && j <= jhi ? kv::physical(a.c, w.b, j) : -1;
    };
    // K: four keys (8 (r / 2) + 2 i + r % 2 of the 32, a byte each) in every group; V: 4 N keys of one group
    struct Scales {
        uint32_t k[N], v[N];
    };
    auto scales_of = [&](int id) {
        Scales z;
        const int mine = __shfl_sync(~0u, id, sub * 32 / BLK);
        const uint8_t* p = a.c.codes + ((long long)mine * a.c.H + w.h) * 2 * L::REC + BLK * D / 2 + sub * 32 % BLK / 32 * D + r * (4 * N);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 x = mine >= 0 ? *reinterpret_cast<const uint2*>(p + 4 * i) : make_uint2(0, 0);
            const uint2 y = mine >= 0 ? *reinterpret_cast<const uint2*>(p + L::REC + 4 * i) : make_uint2(0, 0);
            z.k[i] = x.x, z.k[i + 1] = x.y, z.v[i] = y.x, z.v[i + 1] = y.y;
        }
        return z;
    };
    const int g = r * 4 * N / 32, t4 = r * 4 * N % 32;    // V: this lane's group, its first key of the 32
    int unit = 28, vmax = 28;                             // of group g
    // block numbers two tiles ahead, scales one
    int id = block_of(0), next = block_of(1);
    Scales z = scales_of(id);
    int t = 0;
#pragma unroll 1
    for (int tile = 0; tile < nt; ++tile) {
        const int after = block_of(tile + 2);
        const Scales zn = scales_of(next);
        const int base = (tile0 + tile) * kKeys, here = base + 32 * sub;
        const bool block = __shfl_sync(~0u, id, sub * 32 / BLK) >= 0;
        const bool seen = __all_sync(~0u, block) && base >= see_lo && base + kKeys - 1 <= see_hi;       // every key, by some row
        uint32_t vb[N];
        int ke[4];                                        // a key's largest scale byte, -1: no row sees it
        {
            uint32_t even = 0, odd = 0;
#pragma unroll
            for (int x = 0; x < N; ++x) {
                even = max2(even, z.k[x] & 0x00ff00ffu);
                odd = max2(odd, z.k[x] >> 8 & 0x00ff00ffu);
                vb[x] = z.v[x];
            }
            ke[0] = even & 0xffffu, ke[1] = odd & 0xffffu, ke[2] = even >> 16, ke[3] = odd >> 16;
        }
        if (!seen) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = here + 8 * (r >> 1) + 2 * i + (r & 1);
                ke[i] = block && p >= see_lo && p <= see_hi ? ke[i] : -1;
            }
#pragma unroll
            for (int x = 0; x < N; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int p = here + t4 + 4 * x + k;
                    if (p < see_lo || p > see_hi)
                        vb[x] &= ~(0xffu << 8 * k);
                }
        }
        const uint8_t* src = a.c.codes + ((long long)id * a.c.H + w.h) * 2 * L::REC;
        const int n = __popc(__ballot_sync(~0u, id >= 0));
        unsigned rest = (ke[0] >= 0) | (ke[1] >= 0) << 1 | (ke[2] >= 0) << 2 | (ke[3] >= 0) << 3;
        bool again_k = false, again_v = false;
        uint32_t left[N];
        unsigned in = 0;
        int kref = 0;
#pragma unroll 1
        do {
            if (!again_v) {
                // the keys of this pass: the largest, and those within 2^9 of it (keys of zeros with the first)
                int big = -1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rest >> i & 1)
                        big = max(big, ke[i]);
                kref = max(__reduce_max_sync(~0u, big), 40);
                in = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((rest >> i & 1) && (ke[i] >= kref - 9 || ke[i] == 0))
                        in |= 1u << i;
                rest &= ~in;
                again_k = __any_sync(~0u, rest != 0);
#pragma unroll
                for (int x = 0; x < N; ++x)
                    left[x] = vb[x];
            }
            int big, small;                               // of the scales left, but 0
            {
                uint32_t top = 0, low = ~0u;
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const uint32_t e = left[x] & 0x00ff00ffu, o = left[x] >> 8 & 0x00ff00ffu;
                    uint32_t e1, o1;                      // 0 becomes the largest
                    asm("add.u16x2 %0, %1, %2;" : "=r"(e1) : "r"(e), "r"(0xffffffffu));
                    asm("add.u16x2 %0, %1, %2;" : "=r"(o1) : "r"(o), "r"(0xffffffffu));
                    top = max2(top, max2(e, o));
                    low = min2(low, min2(e1, o1));
                }
                big = max(top & 0xffffu, top >> 16);
                small = min(low & 0xffffu, low >> 16) + 1;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                if (o < 8 / G || o >= 8)
                    big = max(big, __shfl_xor_sync(~0u, big, o));
            vmax = max(vmax, big);
            const int done = again_v ? unit - 28 : 254;       // larger scales have been in an earlier pass
            if (big > 0 && (big > unit || big < unit - 16))
                unit = min(max(max(big + 1, vmax - 64), 28), 254);
            const int field = big > 0 ? min(done - unit, 0) + 28 : 0;
            bool more = false;
            if (__any_sync(~0u, small <= unit - 28)) {
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    uint32_t keep = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int b = left[x] >> 8 * k & 0xff;
                        if (b > 0 && b <= unit - 28 && b > vmax - 92)
                            keep |= 0xffu << 8 * k;
                    }
                    left[x] &= keep;
                    more |= keep != 0;
                }
            }
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bits |= (in >> i & 1) << (8 * (r >> 1) + 2 * i + (r & 1));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                bits |= __shfl_xor_sync(~0u, bits, o);
            Pass& p = passes[t % kRing];
            const bool first = !again_v;
            again_v = __any_sync(~0u, more);
            const bool last = tile + 1 == nt && !again_k && !again_v, whole = __all_sync(~0u, in == 15);
            if (r == 0)
                p.keys[sub] = bits;
            if (sub == 0 && r % (8 / G) == 0) {
                p.unit[g] = unit;
                p.most[g] = field;
            }
            if (lane == 0) {
                p.flags = (first ? kCount : 0u) | (whole ? kAll : 0u);
                p.kref = kref;
                info[t % kRing] = base | (int)last;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (t >= 1)
                    wait(raw_empty + v, (uint32_t)((t - 1) & 1), status);
                __syncwarp();
                if (lane == 0)
                    tc::mbar_expect_tx(raw_full + v, (uint32_t)n * L::REC);
                __syncwarp();
                if (id >= 0)
                    tc::bulk_copy(raw + v * L::RAW + lane * L::REC, src + v * L::REC, L::REC, raw_full + v);
            }
            ++t;
        } while (again_k || again_v);
        id = next;
        next = after;
        z = zn;
    }
    // nothing is on its way when the kernel ends, whoever gave up
    for (int v = 0; v < 2 && t > 0; ++v)
        wait(raw_full + v, (uint32_t)((t - 1) & 1), status);
}

template <int D, int FMT, int BLK>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(AttnArgs a, PromptCut cut)
{
    using L = Layout<D, FMT, BLK>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* status = a.c.status;
    Work w;
    const int after = (int)blockIdx.x - cut.whole;
    const int item = after < 0 ? blockIdx.x : cut.whole + after / cut.parts, part = after < 0 ? 0 : after % cut.parts;
    if (!find_work(a, item, w))
        return;
    const Extent e(a, w);
    const int parts = after < 0 ? 1 : e.parts(cut.parts);
    if (part >= parts)
        return;
    if (cut.parts > 1)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
    uint64_t *raw_full = bar, *raw_empty = bar + 2, *k_full = bar + 4, *k_empty = bar + 6, *v_full = bar + 8, *v_empty = bar + 10;
    uint64_t *s_full = bar + 12, *p_full = bar + 14, *o_full = bar + 16, *q_full = bar + 18, *p_half = bar + 20;
    float2* sc = reinterpret_cast<float2*>(sm + L::OFF_SC);
    int* info = reinterpret_cast<int*>(sm + L::OFF_INFO);

    const int rows = e.rows, na = rows > 128 ? 2 : 1;                                       // row tiles with rows
    const int pos0 = e.pos0, pos1 = e.pos1;
    const int skip = (int)((long long)e.tiles * part / parts);
    const int tile0 = e.tile0 + skip, nt = (int)((long long)e.tiles * (part + 1) / parts) - skip;
    // `info` says which tile is the last one; this bounds the loops should a wait have given up
    const int most = nt * (L::MX ? 256 : L::NB);
    Pass* passes = reinterpret_cast<Pass*>(sm + L::OFF_PASS);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(raw_full + i, 1);
            tc::mbar_init(raw_empty + i, L::CONVERT);
            tc::mbar_init(k_full + i, L::CONVERT);
            tc::mbar_init(k_empty + i, na);
            tc::mbar_init(v_full + i, L::CONVERT);
            tc::mbar_init(v_empty + i, na);
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_half + i, 8);
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
        if constexpr (L::MX)
            mx_produce<D, BLK>(a, w, passes, info, sm + L::OFF_RAW, raw_full, raw_empty, tile0, nt, jlo, jhi,
                               a.window > 0 && pos0 >= a.window ? pos0 - a.window + 1 : 0, pos1);
        else {
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
                            wait(raw_empty + v, (uint32_t)((t - 1) & 1), status);
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
            // nothing is on its way when the kernel ends, whoever gave up
            for (int v = 0; v < 2 && t > 0; ++v)
                wait(raw_full + v, (uint32_t)((t - 1) & 1), status);
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
            wait(k_full + st, (uint32_t)(t >> 1 & 1), status);
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
        wait(q_full, 0, status);
        for (int x = 0; x < na; ++x)
            scores(x, 0);
        for (int t = 0; t < most; ++t) {
            const int st = t & 1;
            const bool last = info[t % kRing] & 1;
            wait(v_full + st, (uint32_t)(t >> 1 & 1), status);
            for (int x = 0; x < na; ++x) {
                // the first 32 of every 64 keys, then the others
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    wait((g ? p_full : p_half) + x, (uint32_t)(t & 1), status);
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = i / 2 * 4 + 2 * g + i % 2;
                        mma_ts(one, tmem + 256 + x * 128, tmem + x * 128 + 8 * k + (k >= 4 ? 32 : 0), vd + (st * L::OP + 256 * k >> 4), id_o, t > 0 || k > 0);
                    }
                }
                commit(one, v_empty + st);
                if (last)
                    commit(one, o_full + x);
                __syncwarp();
                if (!last)
                    scores(x, t + 1);
            }
            if (last)
                break;
        }
    } else if (warp >= 8 - L::CONVERT && warp < 8) {
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
            wait(raw_full, (uint32_t)(t & 1), status);
            const bool last = info[t % kRing] & 1;
            if (t >= 2)
                wait(k_empty + st, (uint32_t)((t >> 1) - 1 & 1), status);
            if constexpr (L::MX) {
                // K: a key a lane, a group's 16 bytes of it at a time in an order that spreads the banks
                const Pass& p = passes[t % kRing];
                const int kref = p.kref;
#pragma unroll
                for (int i = 0; i < (D / 8 + L::CONVERT - 1) / L::CONVERT; ++i) {
                    const int u = i * L::CONVERT + warp - (8 - L::CONVERT);                // of 4 times 32 keys and D / 32 groups
                    if (u >= D / 8)
                        break;
                    const int key = u / (D / 32) * 32 + lane, g = (u + lane / (256 / D)) & (D / 32 - 1);
                    const uint8_t* rec = sm + L::OFF_RAW + key / BLK * L::REC;
                    const uint4 w = *reinterpret_cast<const uint4*>(rec + key % BLK * (D / 2) + 16 * g);
                    // 2^(13 + 127 + e - kref) in f16, with its subnormal numbers
                    const int e = rec[BLK * D / 2 + kv4::k_scale_at<D>(key % BLK, g)];
                    const bool have = p.keys[key >> 5] >> lane & 1;
                    const float f = have ? __uint_as_float((uint32_t)max(e - kref + 140, 0) << 23) : 0.0f;
                    const uint32_t z = pack_f16(f, f), words[4] = {w.x, w.y, w.z, w.w};
                    uint8_t* out = sm + L::OFF_K + st * L::OP + (key >> 3) * (D * 16) + (key & 7) * 16 + 512 * g;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t h[4];
                        kv4::to_f16(words[k], h);
                        *reinterpret_cast<uint4*>(out + 128 * k) = make_uint4(mul_f16(h[0], z), mul_f16(h[1], z), mul_f16(h[2], z), mul_f16(h[3], z));
                    }
                }
            } else {
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

            wait(raw_full + 1, (uint32_t)(t & 1), status);
            if (t >= 2)
                wait(v_empty + st, (uint32_t)((t >> 1) - 1 & 1), status);
            if constexpr (L::MX) {
                // V: eight tokens of four d's at a time, as the record's words lie
                const Pass& p = passes[t % kRing];
                // (r, c) so that eight lanes meet in no bank, neither loading nor storing
                const int r = lane & 7, c = ((r >> 1) + (lane >> 3)) & 3;
#pragma unroll
                for (int i = 0; i < (D / 8 + L::CONVERT - 1) / L::CONVERT; ++i) {
                    const int u = i * L::CONVERT + warp - (8 - L::CONVERT);
                    if (u >= D / 8)
                        break;
                    const int sub = u / (D / 32), g = u % (D / 32);
                    const uint8_t* rec = sm + L::OFF_RAW + L::RAW + sub * 32 / BLK * L::REC;
                    const int in = sub * 32 % BLK / 32 * (D / 32) + g;
                    const uint4 w = *reinterpret_cast<const uint4*>(rec + (in * 32 + r * 4 + c) * 16);
                    const uint2 b = *reinterpret_cast<const uint2*>(rec + BLK * D / 2 + in * 32 + 8 * c);
                    // 2^(13 + e - unit): exponent field e - unit + 28, where that is 1 to 28
                    const uint32_t base = (uint32_t)(p.unit[g] - 28) * 0x10001u, top = (uint32_t)p.most[g];
                    const uint32_t bytes[4] = {__byte_perm(b.x, 0, 0x4140), __byte_perm(b.x, 0, 0x4342), __byte_perm(b.y, 0, 0x4140),
                                               __byte_perm(b.y, 0, 0x4342)};
                    uint32_t z[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x = max2(bytes[k], base) - base;
                        // above: a token that no row sees, or one that an earlier pass has had
                        z[k] = ((x & 0xffffu) <= top ? x & 0xffffu : 0u) << 10 | ((x >> 16) <= top ? x >> 16 : 0u) << 26;
                    }
                    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t h[4];
                        kv4::to_f16(words[e], h);
                        *reinterpret_cast<uint4*>(sm + L::OFF_V + st * L::OP + (4 * g + e) * 2048 + r * 16 + (4 * sub + c) * 128) =
                            make_uint4(mul_f16(h[0], z[0]), mul_f16(h[1], z[1]), mul_f16(h[2], z[2]), mul_f16(h[3], z[3]));
                    }
                }
            } else {
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
            int was[D / 32];                  // MXFP4: O's units
#pragma unroll
            for (int g = 0; g < D / 32; ++g)
                was[g] = 28;
            auto was_of = [&](int ch) { return half ? was[D / 64 + ch] : was[ch]; };       // of this thread's columns
#pragma unroll 1
            for (int t = 0; t < most; ++t) {
                wait(s_full + x, (uint32_t)(t & 1), status);
                tc::tc_fence_after();
                const int word = info[t % kRing], p0 = word & ~1;
                float top = 0.0f;
                bool whole = p0 >= all_lo && p0 + kKeys - 1 <= all_hi;
                const Pass& pass = passes[t % kRing];
                if constexpr (L::MX) {
                    whole = whole && (pass.flags & kAll);
                } else {
#pragma unroll
                    for (int b = 0; b < L::NB; ++b) {
                        const float2 v = sc[(t % kRing) * 4 + b];
                        top = fmaxf(top, v.y);
                        whole = whole && v.x >= 0.0f;
                    }
                }
                // the scales of 32 keys: K's, V's
                const float kscale = L::MX ? __uint_as_float((uint32_t)pass.kref << 23) * 0x1p-13f : 0.0f;
                auto scales = [&](int g) { return L::MX ? make_float2(kscale, 1.0f) : sc[(t % kRing) * 4 + (64 * half + 32 * g) / BLK]; };
                // scores of 32 keys of this row, -inf where it does not see them
                auto take = [&](int g, uint32_t (&v)[32], float ks) {
                    tm_ld32(ts + 32 * g, v);
                    tm_wait_ld(v);
                    if (!whole) {
                        const uint32_t keys = L::MX ? pass.keys[2 * half + g] : ks < 0.0f ? 0u : ~0u;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int p = p0 + 64 * half + 32 * g + k;
                            if (!(keys >> k & 1) || p < plo || p > phi)
                                v[k] = 0xff800000u;
                        }
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float ks = scales(g).x;
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
                bool unit = !(top <= 2.0f * ref && top >= 0.5f * ref);                  // the same for all warps
                if constexpr (L::MX) {
                    unit = false;
#pragma unroll
                    for (int g = 0; g < D / 32; ++g)
                        unit |= pass.unit[g] != was[g];
                }
                if (__any_sync(~0u, unit || mx > m + kSlack)) {                         // the same for both of a pair
                    const float mn = fmaxf(m, mx);
                    float al = ex2(m - mn);
                    m = mn;
                    l *= al;
                    if (!L::MX && unit) {
                        vmax = fmaxf(vmax, top);
                        const float now = new_unit(top, vmax);
                        al *= ref / now;
                        ref = now;
                    }
                    if (t > 0)
#pragma unroll 1
                        for (int ch = 0; ch < D / 64; ++ch) {
                            uint32_t v[32];
                            const float by = L::MX ? al * ex2((float)max(was_of(ch) - pass.unit[half * (D / 64) + ch], -126)) : al;
                            tm_ld32(to + 32 * ch, v);
                            tm_wait_ld(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(__uint_as_float(v[k]) * by);
                            tm_st32(to + 32 * ch, v);
                        }
                    if constexpr (L::MX) {
#pragma unroll
                        for (int g = 0; g < D / 32; ++g)
                            was[g] = pass.unit[g];
                    }
                }
                const float iref = L::MX ? 1.0f : rcp(ref);
                // scores so large that their rounding is more than the room that a probability has: the
                // product is rounded as the maximum's was
                const bool far = __any_sync(~0u, fabsf(m) > 4194304.0f && m != kNone);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float2 kv = scales(g);
                    const float c = fmaxf(kv.x * f, 1e-37f), ratio = fmaxf(kv.y * iref, 8.673617379884035e-19f);   // 2^-60
                    const float off = lg2(ratio) - m + kRoom;
                    uint32_t v[32], p[16];
                    take(g, v, kv.x);
                    if (far)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            v[k] = __float_as_uint(__fmul_rn(__uint_as_float(v[k]), c));
                    const float by = far ? 1.0f : c;
                    const float2 cc = make_float2(by, by), oo = make_float2(off, off);
                    float2 part[2];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 x = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                        float2 z = fma2(x, cc, oo);
                        z.x = ex2(z.x);
                        z.y = ex2(z.y);
                        part[k / 2 & 1] = k > 2 ? add2(part[k / 2 & 1], z) : z;
                        p[k / 2] = pack_f16(z.x, z.y);
                    }
                    const float2 both = add2(part[0], part[1]);
                    if (!L::MX)
                        l += (both.x + both.y) * rcp(ratio);
                    else if (pass.flags & kCount)
                        l += both.x + both.y;
                    tm_st16(ts + 16 * g, p);
                    tm_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive((g ? p_full : p_half) + x);
                }
                if (word & 1)
                    break;
            }
            // ---- the row's result, half of its columns each
            pair_sync();                     // both have read the last maxima
            *mine = l;
            pair_sync();
            l = (l + *other) * kUnroom;
            wait(o_full + x, 0, status);
            tc::tc_fence_after();
            const Final fin = parts > 1 ? Final{pow2_under(l) * kDown, 0.0f} : finish(m, l, a.sinks, hq);
            float* share = reinterpret_cast<float*>(a.ws + kCounterBytes) + (long long)after * part_floats(D);
            uint16_t* out = a.out + ((long long)(w.c0 + i) * a.q_heads + hq) * D + half * (D / 2);
#pragma unroll
            for (int ch = 0; ch < D / 64; ++ch) {
                const float sums = fin.mul * kUnroom, unit = L::MX ? __uint_as_float((uint32_t)was_of(ch) << 23) * 0x1p-13f : ref, mul = sums * unit;
                uint32_t v[32];
                tm_ld32(to + 32 * ch, v);
                tm_wait_ld(v);
                if (parts > 1) {
                    if (in)
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(share + ((half * (D / 8) + 8 * ch + k / 4) * kRows + x * 128 + r) * 4) =
                                make_float4(__uint_as_float(v[k]) * sums * unit, __uint_as_float(v[k + 1]) * sums * unit,
                                            __uint_as_float(v[k + 2]) * sums * unit, __uint_as_float(v[k + 3]) * sums * unit);
                } else if (in)
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = kv::bf16x2(__uint_as_float(v[k + 2 * e]) * mul, __uint_as_float(v[k + 2 * e + 1]) * mul);
                        *reinterpret_cast<uint4*>(out + 32 * ch + k) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
            if (parts > 1 && in && half == 0)
                *reinterpret_cast<float2*>(share + kRows * D + 2 * (x * 128 + r)) = make_float2(m, l);
            if (parts == 1 && a.lse && in && half == 0)
                a.lse[(long long)(w.c0 + i) * a.q_heads + hq] = fin.lse;
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 3)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the parts of every group that has several, in their order: 32 rows a CTA, a warp for
// D / 8 columns of them.
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(AttnArgs a, PromptCut cut)
{
    constexpr int N = D / 32;             // float4 of a thread
    const int after = blockIdx.x / 8, row = blockIdx.x % 8 * 32 + (threadIdx.x & 31), at = threadIdx.x / 32 * N;
    Work w;
    const bool found = find_work(a, cut.whole + after, w);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!found)
        return;
    const Extent e(a, w);
    const int parts = e.parts(cut.parts);
    if (parts == 1 || row >= e.rows)
        return;
    const float* share = reinterpret_cast<const float*>(a.ws + kCounterBytes) + (long long)after * cut.parts * part_floats(D);
    auto ml_of = [&](int p) { return __ldcg(reinterpret_cast<const float2*>(share + (long long)p * part_floats(D) + kRows * D + 2 * row)); };
    float M = kNone, L = 0.0f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float2 ml = ml_of(p);
        const float m = fmaxf(M, ml.x);
        L = L * ex2(M - m) + ml.y * ex2(ml.x - m);
        M = m;
    }
    const float whole = pow2_under(L);
    float4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float2 ml = ml_of(p);
        const float f = pow2_in(ml.y) * ex2(ml.x - M) * whole;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(share + (long long)p * part_floats(D) + ((at + k) * kRows + row) * 4));
            v[k].x += y.x * f, v[k].y += y.y * f, v[k].z += y.z * f, v[k].w += y.w * f;
        }
    }
    const int i = (w.rt * kRows + row) / a.group, hq = w.h * a.group + (w.rt * kRows + row) % a.group;
    const Final fin = finish_mean(M, L, a.sinks, hq);
    uint16_t* out = a.out + ((long long)(w.c0 + i) * a.q_heads + hq) * D + 4 * at;
#pragma unroll
    for (int k = 0; k < N; k += 2)
        *reinterpret_cast<uint4*>(out + 4 * k) =
            make_uint4(kv::bf16x2(v[k].x * fin.mul, v[k].y * fin.mul), kv::bf16x2(v[k].z * fin.mul, v[k].w * fin.mul),
                       kv::bf16x2(v[k + 1].x * fin.mul, v[k + 1].y * fin.mul), kv::bf16x2(v[k + 1].z * fin.mul, v[k + 1].w * fin.mul));
    if (a.lse && at == 0)
        a.lse[(long long)(w.c0 + i) * a.q_heads + hq] = fin.lse;
}

typedef void (*Kernel)(AttnArgs, PromptCut);

template <int D, int FMT>
Kernel pick(int blk)
{
    return blk == 32 ? prompt_attn_kernel<D, FMT, 32> : blk == 64 ? prompt_attn_kernel<D, FMT, 64> : prompt_attn_kernel<D, FMT, 128>;
}
Kernel kernel_for(int d, int fmt, int blk)
{
    if (fmt == MOE_KV_MXFP4)
        return d == 64 ? pick<64, MOE_KV_MXFP4>(blk) : pick<128, MOE_KV_MXFP4>(blk);
    if (d == 64)
        return fmt == MOE_KV_E4M3 ? pick<64, MOE_KV_E4M3>(blk) : pick<64, MOE_KV_INT8>(blk);
    return fmt == MOE_KV_E4M3 ? pick<128, MOE_KV_E4M3>(blk) : pick<128, MOE_KV_INT8>(blk);
}
// whatever the block
int smem_of(int d, int fmt)
{
    if (fmt == MOE_KV_MXFP4)
        return d == 64 ? Layout<64, MOE_KV_MXFP4, 64>::SMEM : Layout<128, MOE_KV_MXFP4, 64>::SMEM;
    return d == 64 ? Layout<64, MOE_KV_INT8, 64>::SMEM : Layout<128, MOE_KV_INT8, 64>::SMEM;
}

}  // namespace

cudaError_t prepare_prompt_kernels()
{
    for (int d = 64; d <= 128; d *= 2)
        for (int fmt : {MOE_KV_E4M3, MOE_KV_INT8, MOE_KV_MXFP4})
            for (int blk = 32; blk <= 128; blk *= 2) {
                const cudaError_t e = cudaFuncSetAttribute(kernel_for(d, fmt, blk), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           smem_of(d, fmt));
                if (e != cudaSuccess)
                    return e;
            }
    return cudaSuccess;
}

size_t prompt_workspace_bytes(int num_sms) { return kCounterBytes + (size_t)num_sms * part_floats(128) * sizeof(float); }

cudaError_t launch_attention_prompt(const AttnArgs& a, int num_sms, cudaStream_t s)
{
    // CTAs beyond the last group or its last part end at once
    const PromptCut cut = attn::prompt_cut(a.call(), num_sms);
    kernel_for(a.c.D, a.c.fmt, a.c.blk)<<<(unsigned)(cut.whole + cut.rest * cut.parts), kThreads, smem_of(a.c.D, a.c.fmt), s>>>(a, cut);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || cut.rest == 0)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(cut.rest * (kRows / 32)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.c.D == 64 ? prompt_join_kernel<64> : prompt_join_kernel<128>, a, cut);
}

}  // namespace moe
