// moe_attention.cu -- attention over the 8-bit paged cache.
//
// out_i = sum_j e^{s_ij - m_i} v_j / (sum_j e^{s_ij - m_i} + e^{sink - m_i}),
// s_ij = scale q_i . k_j over the keys j that token i sees: its own position
// and before it, and with a window only the last `window` of them.
#include <cstdint>

#include "kv_device.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

// One warp per (token, query head), one key at a time.
__global__ void __launch_bounds__(128) attention_simple_kernel(AttnArgs a)
{
    const KvView& c = a.c;
    const int tok = blockIdx.x, lane = threadIdx.x & 31, hq = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (hq >= a.q_heads)
        return;
    const int h = hq / a.group, D = c.D, per = D / 32;
    int b = -1, c0 = 0, n = 0, len = 0;
    for (int i = 0; i < c.n_seqs; ++i) {
        int x0, xn, xl;
        if (!kv::sequence(c, i, x0, xn, xl)) {
            if (lane == 0)
                atomicExch(c.status, MOE_ERR_DEVICE_FAULT);
            continue;
        }
        if (tok >= x0 && tok < x0 + xn) {
            b = i;
            c0 = x0;
            n = xn;
            len = xl;
        }
    }
    if (b < 0)
        return;
    const int pos = len - n + (tok - c0);
    const int j0 = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
    float q[4], o[4] = {0, 0, 0, 0};
    for (int e = 0; e < per; ++e)
        q[e] = tc::bf16f(a.q[(long long)tok * a.q_stride + (long long)hq * D + lane * per + e]);
    float m = a.sinks ? a.sinks[hq] : -INFINITY, l = a.sinks ? 1.0f : 0.0f;
    for (int j = j0; j <= pos; ++j) {
        const int id = kv::physical(c, b, j / c.blk);
        if (id < 0)
            continue;
        const long long at = ((long long)id * c.H + h) * 2;
        const uint8_t* kc = c.codes + at * c.blk * D;
        const uint8_t* vc = kc + (long long)c.blk * D;
        const int r = j % c.blk;
        float s = 0.0f, d4[4];
        for (int e = 0; e < per; ++e) {
            kv::decode4(kc[r * D + lane * per + e], c.fmt, d4);
            s += q[e] * d4[0];
        }
        for (int x = 16; x; x >>= 1)
            s += __shfl_xor_sync(~0u, s, x);
        s *= c.scales[at] * a.scale;
        const float mn = fmaxf(m, s), al = m == mn ? 1.0f : expf(m - mn), p = expf(s - mn);
        l = l * al + p;
        m = mn;
        const float vs = c.scales[at + 1] * p;
        for (int e = 0; e < per; ++e) {
            kv::decode4(vc[(lane * per + e) * c.blk + r], c.fmt, d4);
            o[e] = o[e] * al + vs * d4[0];
        }
    }
    for (int e = 0; e < per; ++e)
        a.out[((long long)tok * a.q_heads + hq) * D + lane * per + e] = tc::f2bf16_rne(l > 0.0f ? o[e] / l : 0.0f);
    if (a.lse && lane == 0)
        a.lse[(long long)tok * a.q_heads + hq] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attention_workspace_bytes(int) { return 256; }
cudaError_t prepare_attention_kernels() { return cudaSuccess; }

cudaError_t launch_attention(const AttnArgs& a, int, cudaStream_t s)
{
    attention_simple_kernel<<<dim3(a.c.n_tokens, (a.q_heads + 3) / 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
