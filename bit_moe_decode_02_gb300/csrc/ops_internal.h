// ops_internal.h -- what the operators around the expert block share: the
// handle, the kernels' view of an 8-bit paged cache, and the launches that
// moe_ops.cu makes after its argument checks.  Not part of the public interface.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/moe.h"

struct moe_ops {
    int device = 0;
    int num_sms = 0;
    int clusters = 0;            // of moe_linear's CTAs that run at once
    int* status = nullptr;       // device word, as a moe_handle's
    uint8_t* ws = nullptr;       // workspace of the calls, ws_bytes: join counters (zero between calls), partial results
    size_t ws_bytes = 0;
};

namespace moe {

constexpr int kCounterBytes = 4096;      // of a workspace: one join counter per CTA
constexpr int kMaxSeqs = 1024;          // sequences of one batch
constexpr int kMaxBatchQ = 1 << 20;     // tokens of one batch

// One batch over one cache, as the kernels see it.
struct KvView {
    uint8_t* codes;          // [num_blocks][H][2][blk * D]
    float* scales;           // [num_blocks][H][2]
    const int* cu;           // [n_seqs + 1]
    const int* len;          // [n_seqs]
    const int* table;        // [n_seqs][table_stride]
    int n_seqs, n_tokens, table_stride;
    int num_blocks, H, D, blk, fmt;
    int* status;
};

cudaError_t launch_kv_write(const KvView& c, const uint16_t* k, const uint16_t* v, long long k_stride,
                            long long v_stride, cudaStream_t s);
cudaError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, long long k_stride, long long v_stride,
                           cudaStream_t s);

struct AttnArgs {
    KvView c;
    const uint16_t* q;       // [T] rows of q_heads * D, q_stride apart
    long long q_stride;
    int q_heads, group;      // group = q_heads / kv heads
    float scale;
    int window;              // 0: none
    const float* sinks;      // [q_heads] or nullptr
    uint16_t* out;           // [T][q_heads][D]
    float* lse;              // [T][q_heads] or nullptr
    uint8_t* ws;
};
cudaError_t prepare_attention_kernels();
cudaError_t prepare_prompt_kernels();
cudaError_t launch_attention_prompt(const AttnArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_attention(const AttnArgs& a, int num_sms, cudaStream_t s);

struct LinearArgs {
    const uint8_t* codes;    // [N][K/2]
    const void* scales;      // u8 [N][K/32] or fp16 [N][K/group]
    const uint16_t* bias;    // [N] or nullptr
    int N, K, fmt, group;
    const uint16_t* x;
    long long x_stride;
    int M;
    void* out;
    long long out_stride;
    int out_type;
    int* status;
};
cudaError_t prepare_linear_kernels(int* clusters);
cudaError_t launch_linear(const LinearArgs& a, int num_sms, int clusters, cudaStream_t s);

struct SampleArgs {
    const void* logits;
    int logits_type;
    long long stride;
    int M, V;
    moe_sample_params p;
    int* token;
    float* logprob;
};
cudaError_t prepare_sample_kernels();
cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s);

size_t attention_workspace_bytes(int num_sms);

}  // namespace moe
