// moe_ops.cu -- the C entry points of the operators around the expert block
// (declared in include/moe.h): the handle with their workspace, and the checks
// of every argument before anything is enqueued.
#include <cmath>
#include <new>

#include "moe_internal.h"
#include "ops_internal.h"

namespace {

using moe::set_error;

int cuda_fail(cudaError_t e, const char* what)
{
    return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void* a, long long an, const void* b, long long bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

int check_cache(const char* who, const moe_ops* o, const moe_kv_cache* c, const moe_kv_batch* b, moe::KvView* v)
{
    if (!o || !c || !b)
        return set_error(MOE_ERR_INVALID_ARG, "%s: the handle, the cache and the batch must not be NULL", who);
    if (!c->codes || !c->scales || !b->cu || !b->kv_len || !b->table)
        return set_error(MOE_ERR_INVALID_ARG, "%s: a pointer of the cache or the batch is NULL", who);
    if (c->format != MOE_KV_E4M3 && c->format != MOE_KV_INT8)
        return set_error(MOE_ERR_INVALID_ARG, "%s: unknown cache format %d", who, c->format);
    if (c->block != 32 && c->block != 64 && c->block != 128)
        return set_error(MOE_ERR_UNSUPPORTED, "%s: block=%d (32, 64 or 128)", who, c->block);
    if (c->head_dim != 64 && c->head_dim != 128)
        return set_error(MOE_ERR_UNSUPPORTED, "%s: head_dim=%d (64 or 128)", who, c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > 256)
        return set_error(MOE_ERR_INVALID_ARG, "%s: kv_heads=%d out of range 1..256", who, c->kv_heads);
    if (c->num_blocks < 1)
        return set_error(MOE_ERR_INVALID_ARG, "%s: num_blocks=%d must be positive", who, c->num_blocks);
    if (!aligned(c->codes, 16) || !aligned(c->scales, 8))
        return set_error(MOE_ERR_INVALID_ARG, "%s: codes must be 16-byte and scales 8-byte aligned", who);
    if (!aligned(b->cu, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4))
        return set_error(MOE_ERR_INVALID_ARG, "%s: cu, kv_len and table must be 4-byte aligned", who);
    if (b->n_seqs < 1 || b->n_seqs > moe::kMaxSeqs)
        return set_error(MOE_ERR_INVALID_ARG, "%s: n_seqs=%d out of range 1..%d", who, b->n_seqs, moe::kMaxSeqs);
    if (b->n_tokens < 1 || b->n_tokens > moe::kMaxBatchQ)
        return set_error(MOE_ERR_INVALID_ARG, "%s: n_tokens=%d out of range 1..%d", who, b->n_tokens, moe::kMaxBatchQ);
    if (b->table_stride < 1)
        return set_error(MOE_ERR_INVALID_ARG, "%s: table_stride=%d must be positive", who, b->table_stride);
    *v = moe::KvView{static_cast<uint8_t*>(c->codes), c->scales, b->cu, b->kv_len, b->table, b->n_seqs, b->n_tokens,
                     b->table_stride, c->num_blocks, c->kv_heads, c->head_dim, c->block, c->format, o->status};
    return MOE_OK;
}

// Rows of `width` bf16 each, `stride` elements apart, read or written 16 bytes at a time.
int check_rows(const char* who, const char* name, const void* p, long long stride, long long width)
{
    if (!p)
        return set_error(MOE_ERR_INVALID_ARG, "%s: %s must not be NULL", who, name);
    if (!aligned(p, 16) || stride % 8)
        return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with a stride that is a multiple of 8", who, name);
    if (stride < width)
        return set_error(MOE_ERR_INVALID_ARG, "%s: the stride of %s (%lld) is less than a row (%lld)", who, name, stride, width);
    return MOE_OK;
}

}  // namespace

int moe_ops_create(moe_ops** out)
{
    if (!out)
        return set_error(MOE_ERR_INVALID_ARG, "moe_ops_create: out is NULL");
    *out = nullptr;
    moe_ops* o = new (std::nothrow) moe_ops();
    if (!o)
        return set_error(MOE_ERR_OOM, "host allocation failed");
    cudaError_t e;
    if ((e = cudaGetDevice(&o->device)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&o->num_sms, cudaDevAttrMultiProcessorCount, o->device)) != cudaSuccess) {
        delete o;
        return cuda_fail(e, "moe_ops_create");
    }
    o->ws_bytes = moe::attention_workspace_bytes(o->num_sms);
    if ((e = cudaMalloc(&o->status, sizeof(int))) != cudaSuccess || (e = cudaMalloc(&o->ws, o->ws_bytes)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(o->status);
        const int sms = o->num_sms;
        delete o;
        return set_error(MOE_ERR_OOM, "moe_ops_create: workspace (%zu bytes) failed: %s", moe::attention_workspace_bytes(sms),
                         cudaGetErrorString(e));
    }
    if ((e = cudaMemset(o->status, 0, sizeof(int))) != cudaSuccess || (e = cudaMemset(o->ws, 0, o->ws_bytes)) != cudaSuccess ||
        (e = moe::prepare_attention_kernels()) != cudaSuccess || (e = moe::prepare_linear_kernels(&o->clusters)) != cudaSuccess ||
        (e = moe::prepare_sample_kernels()) != cudaSuccess || (e = cudaDeviceSynchronize()) != cudaSuccess) {
        moe_ops_destroy(o);
        return cuda_fail(e, "moe_ops_create");
    }
    *out = o;
    return MOE_OK;
}

void moe_ops_destroy(moe_ops* o)
{
    if (!o)
        return;
    cudaDeviceSynchronize();
    cudaFree(o->ws);
    cudaFree(o->status);
    delete o;
}

int moe_ops_get_status(moe_ops* o, void* stream)
{
    if (!o)
        return set_error(MOE_ERR_INVALID_ARG, "moe_ops_get_status: handle is NULL");
    cudaStream_t s = (cudaStream_t)stream;
    int st = 0;
    cudaError_t e;
    if ((e = cudaMemcpyAsync(&st, o->status, sizeof st, cudaMemcpyDeviceToHost, s)) != cudaSuccess ||
        (e = cudaStreamSynchronize(s)) != cudaSuccess)
        return cuda_fail(e, "moe_ops_get_status");
    if (st == 0)
        return MOE_OK;
    // a call that gave up may have left joins half done
    if ((e = cudaMemsetAsync(o->status, 0, sizeof(int), s)) != cudaSuccess ||
        (e = cudaMemsetAsync(o->ws, 0, moe::kCounterBytes, s)) != cudaSuccess ||
        (e = cudaStreamSynchronize(s)) != cudaSuccess)
        return cuda_fail(e, "moe_ops_get_status");
    return set_error(st, st == MOE_ERR_DEVICE_FAULT ? "a batch's lengths or a block number were out of range"
                                                    : "a device-side wait gave up");
}

int moe_kv_write(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* k_bf16,
                 long long k_stride, const void* v_bf16, long long v_stride, void* stream)
{
    moe::KvView v;
    int rc = check_cache("moe_kv_write", o, cache, batch, &v);
    if (rc == MOE_OK)
        rc = check_rows("moe_kv_write", "k", k_bf16, k_stride, (long long)v.H * v.D);
    if (rc == MOE_OK)
        rc = check_rows("moe_kv_write", "v", v_bf16, v_stride, (long long)v.H * v.D);
    if (rc != MOE_OK)
        return rc;
    const cudaError_t e = moe::launch_kv_write(v, static_cast<const uint16_t*>(k_bf16), static_cast<const uint16_t*>(v_bf16),
                                               k_stride, v_stride, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_kv_write");
}

int moe_kv_read(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, void* k_bf16, long long k_stride,
                void* v_bf16, long long v_stride, void* stream)
{
    moe::KvView v;
    int rc = check_cache("moe_kv_read", o, cache, batch, &v);
    if (rc == MOE_OK)
        rc = check_rows("moe_kv_read", "k", k_bf16, k_stride, (long long)v.H * v.D);
    if (rc == MOE_OK)
        rc = check_rows("moe_kv_read", "v", v_bf16, v_stride, (long long)v.H * v.D);
    if (rc != MOE_OK)
        return rc;
    const cudaError_t e = moe::launch_kv_read(v, static_cast<uint16_t*>(k_bf16), static_cast<uint16_t*>(v_bf16), k_stride,
                                              v_stride, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_kv_read");
}

int moe_attention(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* q_bf16, long long q_stride,
                  int q_heads, float scale, int window, const float* sinks, void* out_bf16, float* lse, void* stream)
{
    moe::AttnArgs a{};
    int rc = check_cache("moe_attention", o, cache, batch, &a.c);
    if (rc != MOE_OK)
        return rc;
    if (q_heads < 1 || q_heads > 1024 || q_heads % a.c.H)
        return set_error(MOE_ERR_INVALID_ARG, "moe_attention: q_heads=%d must be a multiple of kv_heads=%d, at most 1024",
                         q_heads, a.c.H);
    const long long width = (long long)q_heads * a.c.D;
    if ((rc = check_rows("moe_attention", "q", q_bf16, q_stride, width)) != MOE_OK)
        return rc;
    if (!out_bf16 || !aligned(out_bf16, 16) || !aligned(lse, 4) || !aligned(sinks, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_attention: out must be 16-byte aligned (and not NULL), lse and sinks 4-byte");
    if (!std::isfinite(scale))
        return set_error(MOE_ERR_INVALID_ARG, "moe_attention: scale must be finite");
    if (window < 0)
        return set_error(MOE_ERR_INVALID_ARG, "moe_attention: window=%d must not be negative", window);
    if (overlap(q_bf16, ((batch->n_tokens - 1ll) * q_stride + width) * 2, out_bf16, batch->n_tokens * width * 2))
        return set_error(MOE_ERR_INVALID_ARG, "moe_attention: q overlaps out");
    a.q = static_cast<const uint16_t*>(q_bf16);
    a.q_stride = q_stride;
    a.q_heads = q_heads;
    a.group = q_heads / a.c.H;
    a.scale = scale;
    a.window = window;
    a.sinks = sinks;
    a.out = static_cast<uint16_t*>(out_bf16);
    a.lse = lse;
    a.ws = o->ws;
    const cudaError_t e = moe::launch_attention(a, o->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_attention");
}

int moe_linear(moe_ops* o, const moe_linear_weights* w, const void* x_bf16, long long x_stride, int M, void* out,
               long long out_stride, int out_type, void* stream)
{
    if (!o || !w)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: the handle and the weights must not be NULL");
    if (w->format == MOE_FMT_MXFP4) {
        if (w->group != 32)
            return set_error(MOE_ERR_INVALID_ARG, "moe_linear: MXFP4 needs group == 32");
    } else if (w->format == MOE_FMT_INT4) {
        if (w->group != 32 && w->group != 64 && w->group != 128 && w->group != 256)
            return set_error(MOE_ERR_INVALID_ARG, "moe_linear: int4 needs group 32, 64, 128 or 256 (got %d)", w->group);
    } else {
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: unknown format %d", w->format);
    }
    if (w->rows < 1 || w->rows > 1 << 24)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: rows=%d out of range 1..2^24", w->rows);
    if (w->cols < 32 || w->cols > 32768 || w->cols % w->group)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: cols=%d must be a multiple of group, at most 32768", w->cols);
    if (!w->codes || !w->scales || !aligned(w->codes, 16) || !aligned(w->scales, 16) || !aligned(w->bias, 2))
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: codes and scales must be 16-byte aligned (and not NULL), bias 2-byte");
    if (M < 1 || M > 64)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: M=%d out of range 1..64", M);
    const int rc = check_rows("moe_linear", "x", x_bf16, x_stride, w->cols);
    if (rc != MOE_OK)
        return rc;
    if (out_type != MOE_DT_F32 && out_type != MOE_DT_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: unknown output type %d", out_type);
    const int size = out_type == MOE_DT_BF16 ? 2 : 4;
    if (!out || !aligned(out, size))
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: out must be aligned to its type (and not NULL)");
    if (out_stride < w->rows)
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: the stride of out (%lld) is less than a row (%d)", out_stride, w->rows);
    if (overlap(x_bf16, ((M - 1) * x_stride + w->cols) * 2, out, ((M - 1) * out_stride + w->rows) * size))
        return set_error(MOE_ERR_INVALID_ARG, "moe_linear: x overlaps out");
    moe::LinearArgs a{static_cast<const uint8_t*>(w->codes), w->scales, static_cast<const uint16_t*>(w->bias), w->rows, w->cols,
                      w->format, w->group, static_cast<const uint16_t*>(x_bf16), x_stride, M, out, out_stride, out_type,
                      o->status};
    const cudaError_t e = moe::launch_linear(a, o->num_sms, o->clusters, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_linear");
}

int moe_sample(moe_ops* o, const void* logits, int logits_type, long long stride, int M, int V, const moe_sample_params* p,
               int* token, float* logprob, void* stream)
{
    if (!o || !logits || !p || !token)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: the handle, logits, params and token must not be NULL");
    if (logits_type != MOE_DT_F32 && logits_type != MOE_DT_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: unknown logits type %d", logits_type);
    if (M < 1 || M > 65535)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: M=%d out of range 1..65535", M);
    if (V < 1 || V > 1 << 19)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: V=%d out of range 1..2^19", V);
    if (stride < V)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: stride=%lld is less than V=%d", stride, V);
    if (!p->u)
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: u must not be NULL");
    if (!aligned(logits, logits_type == MOE_DT_BF16 ? 2 : 4) || !aligned(token, 4) || !aligned(logprob, 4) ||
        !aligned(p->temperature, 4) || !aligned(p->top_k, 4) || !aligned(p->top_p, 4) || !aligned(p->min_p, 4) ||
        !aligned(p->u, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_sample: every array must be aligned to its type");
    moe::SampleArgs a{logits, logits_type, stride, M, V, *p, token, logprob};
    const cudaError_t e = moe::launch_sample(a, o->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_sample");
}
