// moe_linear.cu -- y = x W^T + b for a few tokens, W in 4 bits (MXFP4, or int4
// with group scales), in the caller's layout.
#include <cstdint>

#include <cuda_fp16.h>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

// One warp per (row, token).
__global__ void __launch_bounds__(128) linear_simple_kernel(LinearArgs a)
{
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), m = blockIdx.y, lane = threadIdx.x & 31;
    if (row >= a.N)
        return;
    const uint8_t* codes = a.codes + (long long)row * (a.K / 2);
    const uint16_t* x = a.x + (long long)m * a.x_stride;
    float sum = 0.0f;
    for (int i = lane; i < a.K / 2; i += 32) {
        const uint32_t byte = codes[i];
        float2 w;
        float s;
        if (a.fmt == MOE_FMT_MXFP4) {
            w = tc::e2m1x2_to_f32(byte);
            const uint32_t e = static_cast<const uint8_t*>(a.scales)[(long long)row * (a.K / 32) + i / 16];
            s = e == 255 ? __uint_as_float(0x7fc00000u) : e == 0 ? __uint_as_float(0x400000u) : __uint_as_float(e << 23);
        } else {
            w = make_float2((float)(int)(byte & 15) - 8.0f, (float)(int)(byte >> 4) - 8.0f);
            s = __half2float(static_cast<const __half*>(a.scales)[(long long)row * (a.K / a.group) + 2 * i / a.group]);
        }
        sum += s * (w.x * tc::bf16f(x[2 * i]) + w.y * tc::bf16f(x[2 * i + 1]));
    }
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    if (lane)
        return;
    if (a.bias)
        sum += tc::bf16f(a.bias[row]);
    const long long at = (long long)m * a.out_stride + row;
    if (a.out_type == MOE_DT_BF16)
        static_cast<uint16_t*>(a.out)[at] = tc::f2bf16_rne(sum);
    else
        static_cast<float*>(a.out)[at] = sum;
}

}  // namespace

cudaError_t prepare_linear_kernels() { return cudaSuccess; }

cudaError_t launch_linear(const LinearArgs& a, int, cudaStream_t s)
{
    linear_simple_kernel<<<dim3((a.N + 3) / 4, a.M), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
