// moe_ops.cu -- the C entry points of the operators around the expert block
// (declared in include/moe.h): the handle with their workspace, and the checks
// of every argument before anything is enqueued.
#include <cmath>
#include <new>
#include <type_traits>
#include <utility>

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
    const bool mx = c->format == MOE_KV_MXFP4;
    if (!c->codes || (!c->scales && !mx) || !b->cu || !b->kv_len || !b->table)
        return set_error(MOE_ERR_INVALID_ARG, "%s: a pointer of the cache or the batch is NULL", who);
    if (c->format != MOE_KV_E4M3 && c->format != MOE_KV_INT8 && !mx)
        return set_error(MOE_ERR_INVALID_ARG, "%s: unknown cache format %d", who, c->format);
    if (mx && c->scales)
        return set_error(MOE_ERR_INVALID_ARG, "%s: scales must be NULL (an MXFP4 cache holds them with its codes)", who);
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

size_t workspace_bytes(int num_sms)
{
    const size_t a = moe::attention_workspace_bytes(num_sms), l = moe::kCounterBytes + moe::lora_workspace_bytes();
    return a > l ? a : l;
}

// As check_rows, for rows of `size`-byte elements.
int check_rows_of(const char* who, const char* name, const void* p, long long stride, long long width, int size)
{
    if (!p)
        return set_error(MOE_ERR_INVALID_ARG, "%s: %s must not be NULL", who, name);
    if (!aligned(p, 16) || stride % (16 / size))
        return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with a stride of a multiple of 16 bytes", who, name);
    if (stride < width)
        return set_error(MOE_ERR_INVALID_ARG, "%s: the stride of %s (%lld) is less than a row (%lld)", who, name, stride, width);
    return MOE_OK;
}

// Rows of a tensor: `width` elements each, `stride` elements apart.
struct Rows {
    const void* p;
    long long stride, width;
};
// Whether two tensors' n rows, of as and bs bytes an element, share a byte.  Rows that lie within
// one another's strides (parts of a fused projection) do not where their columns do not.
bool rows_overlap(const Rows& a, int as, const Rows& b, int bs, int n)
{
    if (!overlap(a.p, ((n - 1) * a.stride + a.width) * as, b.p, ((n - 1) * b.stride + b.width) * bs))
        return false;
    const long long pitch = a.stride * as;
    if (n == 1 || pitch != b.stride * bs)
        return true;
    long long d = (long long)((intptr_t)b.p - (intptr_t)a.p) % pitch;
    d += d < 0 ? pitch : 0;
    return !(d >= a.width * as && pitch - d >= b.width * bs);
}
bool rows_overlap(const Rows& a, const Rows& b, int n, int size) { return rows_overlap(a, size, b, size, n); }
// The same for rows and one contiguous array.
bool rows_overlap(const Rows& a, int n, int size, const void* p, long long bytes)
{
    if (!overlap(a.p, ((n - 1) * a.stride + a.width) * size, p, bytes))
        return false;
    const long long pitch = a.stride * size, d = (long long)((intptr_t)p - (intptr_t)a.p), at = d % pitch;
    return d < 0 || at < a.width * size || at + bytes > pitch;
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
    o->ws_bytes = workspace_bytes(o->num_sms);
    if ((e = cudaMalloc(&o->status, sizeof(int))) != cudaSuccess || (e = cudaMalloc(&o->ws, o->ws_bytes)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(o->status);
        const int sms = o->num_sms;
        delete o;
        return set_error(MOE_ERR_OOM, "moe_ops_create: workspace (%zu bytes) failed: %s", workspace_bytes(sms),
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
    return set_error(st, st == MOE_ERR_DEVICE_FAULT ? "a batch's lengths, a block or an adapter number were out of range"
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
    const uint16_t *k = static_cast<const uint16_t*>(k_bf16), *x = static_cast<const uint16_t*>(v_bf16);
    const cudaError_t e = v.fmt == MOE_KV_MXFP4 ? moe::launch_kv4_write(v, k, x, k_stride, v_stride, (cudaStream_t)stream)
                                                : moe::launch_kv_write(v, k, x, k_stride, v_stride, (cudaStream_t)stream);
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
    uint16_t *k = static_cast<uint16_t*>(k_bf16), *x = static_cast<uint16_t*>(v_bf16);
    const cudaError_t e = v.fmt == MOE_KV_MXFP4 ? moe::launch_kv4_read(v, k, x, k_stride, v_stride, o->num_sms, (cudaStream_t)stream)
                                                : moe::launch_kv_read(v, k, x, k_stride, v_stride, (cudaStream_t)stream);
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
    if (rows_overlap(Rows{x_bf16, x_stride, w->cols}, 2, Rows{out, out_stride, w->rows}, size, M))
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

int moe_rope_turns(const moe_rope_config* c, unsigned long long* turns)
{
    if (!c || !turns)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: the configuration and turns must not be NULL");
    if (c->rot_dim < 2 || c->rot_dim > 512 || c->rot_dim % 2)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: rot_dim=%d must be even, 2..512", c->rot_dim);
    if (c->scaling < MOE_ROPE_PLAIN || c->scaling > MOE_ROPE_WAVELENGTH)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: unknown scaling %d", c->scaling);
    if (!(c->base > 1.0) || !std::isfinite(c->base))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: base must be finite and above 1");
    // (a speed above 2^53 would have no fraction of a turn left, and its rest no place in 64 bits)
    if (c->scaling != MOE_ROPE_PLAIN && (!(c->factor >= 0x1p-32) || !std::isfinite(c->factor)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: factor must be finite and at least 2^-32");
    if (c->scaling > MOE_ROPE_LINEAR && (!(c->length > 0.0) || !(c->low > 0.0) || !(c->high > c->low) || !std::isfinite(c->length) ||
                                         !std::isfinite(c->high)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope_turns: length and low must be positive and high above low, all finite");
    const double pi = 3.14159265358979323846;
    for (int i = 0; i < c->rot_dim / 2; ++i) {
        double f = std::pow(c->base, -2.0 * i / c->rot_dim);
        const double slow = f / c->factor;
        if (c->scaling == MOE_ROPE_LINEAR) {
            f = slow;
        } else if (c->scaling == MOE_ROPE_PARTS) {
            auto at = [&](double n) { return c->rot_dim * std::log(c->length / (2.0 * pi * n)) / (2.0 * std::log(c->base)); };
            const double lo = std::fmax(at(c->high), 0.0), hi = std::fmin(at(c->low), c->rot_dim / 2 - 1.0);
            const double x = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1.0 - x) + slow * x;
        } else if (c->scaling == MOE_ROPE_WAVELENGTH) {
            const double x = std::fmin(std::fmax((c->length * f / (2.0 * pi) - c->low) / (c->high - c->low), 0.0), 1.0);
            f = f * x + slow * (1.0 - x);
        }
        // f / 2 pi in two doubles, its fraction times 2^64
        const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;      // 1 / 2 pi
        const double p = f * hi, rest = std::fma(f, hi, -p) + f * lo, frac = p - std::floor(p);
        const unsigned long long whole = (unsigned long long)std::ldexp(frac, 64);
        turns[i] = whole + (unsigned long long)std::llrint(std::ldexp(rest, 64));
    }
    return MOE_OK;
}

int moe_rope(moe_ops* o, const moe_rope_table* r, const int* position, int n_tokens, int head_dim, int type, const void* q,
             long long q_stride, int q_heads, void* q_out, long long q_out_stride, const void* k, long long k_stride, int k_heads,
             void* k_out, long long k_out_stride, void* stream)
{
    if (!o || !r || !r->turns || !position)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: the handle, the table and position must not be NULL");
    if (type != MOE_DT_F32 && type != MOE_DT_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: unknown type %d", type);
    if (r->layout != MOE_ROPE_HALF && r->layout != MOE_ROPE_INTERLEAVED)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: unknown layout %d", r->layout);
    if (head_dim < 8 || head_dim > 512 || head_dim % 8)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: head_dim=%d must be a multiple of 8, at most 512", head_dim);
    if (r->rot_dim < 2 || r->rot_dim > head_dim || r->rot_dim % 2)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: rot_dim=%d must be even, 2..head_dim", r->rot_dim);
    if (!std::isfinite(r->mscale))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: mscale must be finite");
    if (n_tokens < 1 || n_tokens > moe::kMaxBatchQ)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: n_tokens=%d out of range 1..%d", n_tokens, moe::kMaxBatchQ);
    if (q_heads < 1 || q_heads > 1024 || k_heads < 0 || k_heads > 1024)
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: q_heads=%d out of range 1..1024 or k_heads=%d out of range 0..1024", q_heads, k_heads);
    if (!aligned(r->turns, 8) || !aligned(position, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: turns must be 8-byte and position 4-byte aligned");
    const int size = type == MOE_DT_BF16 ? 2 : 4;
    const Rows in[2] = {{q, q_stride, (long long)q_heads * head_dim}, {k, k_stride, (long long)k_heads * head_dim}};
    const Rows out[2] = {{q_out, q_out_stride, in[0].width}, {k_out, k_out_stride, in[1].width}};
    const char* const names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    const int n = k_heads ? 2 : 1;
    for (int i = 0; i < n; ++i) {
        int rc = check_rows_of("moe_rope", names[i][0], in[i].p, in[i].stride, in[i].width, size);
        if (rc == MOE_OK)
            rc = check_rows_of("moe_rope", names[i][1], out[i].p, out[i].stride, out[i].width, size);
        if (rc != MOE_OK)
            return rc;
    }
    bool same[2] = {false, false};
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            const bool here = i == j && out[i].p == in[i].p && (n_tokens == 1 || out[i].stride == in[i].stride);
            same[i] |= here;
            if (!here && rows_overlap(out[i], in[j], n_tokens, size))
                return set_error(MOE_ERR_INVALID_ARG, "moe_rope: %s overlaps %s (in place: the same rows)", names[i][1], names[j][0]);
        }
    for (int i = 0; i < n; ++i) {
        const bool at = rows_overlap(out[i], n_tokens, size, position, n_tokens * 4ll);
        if (at || rows_overlap(out[i], n_tokens, size, r->turns, r->rot_dim / 2 * 8ll))
            return set_error(MOE_ERR_INVALID_ARG, "moe_rope: %s overlaps %s", names[i][1], at ? "position" : "turns");
    }
    if (n == 2 && rows_overlap(out[0], out[1], n_tokens, size))
        return set_error(MOE_ERR_INVALID_ARG, "moe_rope: q_out overlaps k_out");
    moe::RopeArgs a{r->turns, position, q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, n_tokens, q_heads,
                    k_heads, head_dim, r->rot_dim, r->layout, type, r->mscale, !(same[0] && (n == 1 || same[1])), 0};
    const cudaError_t e = moe::launch_rope(a, o->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_rope");
}

int moe_kv_plan(moe_ops* o, const moe_kv_pool* p, const int* n_new, const int* kv_len, const int* state, int n_tokens, int* cu,
                int* kv_len_out, int* state_out, int* admitted, int* seq, int* position, long long* slot, void* stream)
{
    if (!o || !p || !p->ring || !p->table || !n_new || !kv_len || !state || !cu || !kv_len_out || !state_out)
        return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: only admitted, seq, position and slot may be NULL");
    if (p->n_seqs < 1 || p->n_seqs > moe::kMaxSeqs)
        return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: n_seqs=%d out of range 1..%d", p->n_seqs, moe::kMaxSeqs);
    if (p->ring_size < 1)
        return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: ring_size=%d must be positive", p->ring_size);
    if (p->table_stride < 1)
        return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: table_stride=%d must be positive", p->table_stride);
    if (p->block != 32 && p->block != 64 && p->block != 128)
        return set_error(MOE_ERR_UNSUPPORTED, "moe_kv_plan: block=%d (32, 64 or 128)", p->block);
    if (n_tokens < 1 || n_tokens > moe::kMaxBatchQ)
        return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: n_tokens=%d out of range 1..%d", n_tokens, moe::kMaxBatchQ);
    const long long n = p->n_seqs;
    // what is read, then what is written; kv_len and state may be updated in place
    const struct { const void* p; long long bytes; const char* name; } t[] = {
        {n_new, n * 4, "n_new"}, {kv_len, n * 4, "kv_len"}, {state, 8, "state"}, {p->ring, p->ring_size * 4ll, "ring"},
        {p->table, n * p->table_stride * 4, "table"}, {cu, (n + 1) * 4, "cu"}, {kv_len_out, n * 4, "kv_len_out"},
        {state_out, 8, "state_out"}, {admitted, 4, "admitted"}, {seq, n_tokens * 4ll, "seq"}, {position, n_tokens * 4ll, "position"},
        {slot, n_tokens * 8ll, "slot"}};
    constexpr int N = sizeof t / sizeof *t;
    for (int i = 0; i < N; ++i) {
        if (!aligned(t[i].p, t[i].p == slot ? 8 : 4))
            return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: every array must be aligned to its type (%s is not)", t[i].name);
        for (int j = i > 3 ? i : 3; j < N; ++j)
            if (i != j && t[i].p && t[j].p && !(i == 1 && j == 6 && t[i].p == t[j].p) && !(i == 2 && j == 7 && t[i].p == t[j].p) &&
                overlap(t[i].p, t[i].bytes, t[j].p, t[j].bytes))
                return set_error(MOE_ERR_INVALID_ARG, "moe_kv_plan: %s overlaps %s", t[j].name, t[i].name);
    }
    moe::PlanArgs a{p->ring, p->table, p->ring_size, p->n_seqs, p->table_stride, p->block == 32 ? 5 : p->block == 64 ? 6 : 7, n_new, kv_len, state, cu, kv_len_out,
                    state_out, admitted, seq, position, slot, n_tokens, o->status};
    const cudaError_t e = moe::launch_plan(a, o->num_sms, reinterpret_cast<unsigned*>(o->ws), (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_kv_plan");
}

int moe_lora(moe_ops* o, const moe_lora_weights* w, const int* index, const void* x_bf16, long long x_stride, int M, const void* y,
             long long y_stride, void* out, long long out_stride, int type, void* stream)
{
    if (!o || !w || !index)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: the handle, the weights and index must not be NULL");
    if (w->n_adapters < 1 || w->n_adapters > 65536)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: n_adapters=%d out of range 1..65536", w->n_adapters);
    if (w->rank < 8 || w->rank > 128 || w->rank % 8)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: rank=%d must be a multiple of 8, at most 128", w->rank);
    if (w->rows < 1 || w->rows > 1 << 24)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: rows=%d out of range 1..2^24", w->rows);
    if (w->cols < 8 || w->cols > 32768 || w->cols % 8)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: cols=%d must be a multiple of 8, at most 32768", w->cols);
    if (!w->a || !w->b || !aligned(w->a, 16) || !aligned(w->b, 16) || !aligned(w->scale, 4) || !aligned(index, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: a and b must be 16-byte aligned (and not NULL), scale and index 4-byte");
    if (M < 1 || M > 64)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: M=%d out of range 1..64", M);
    const int rc = check_rows("moe_lora", "x", x_bf16, x_stride, w->cols);
    if (rc != MOE_OK)
        return rc;
    if (type != MOE_DT_F32 && type != MOE_DT_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: unknown type %d", type);
    const int size = type == MOE_DT_BF16 ? 2 : 4;
    if (!out || !aligned(out, size) || !aligned(y, size))
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: out (not NULL) and y must be aligned to their type");
    if (out_stride < w->rows || (y && y_stride < w->rows))
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: the stride of out (%lld) or y (%lld) is less than a row (%d)", out_stride,
                         y_stride, w->rows);
    if (rows_overlap(Rows{x_bf16, x_stride, w->cols}, 2, Rows{out, out_stride, w->rows}, size, M))
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: x overlaps out");
    const bool same = y == out && (M == 1 || y_stride == out_stride);
    if (y && !same && rows_overlap(Rows{y, y_stride, w->rows}, Rows{out, out_stride, w->rows}, M, size))
        return set_error(MOE_ERR_INVALID_ARG, "moe_lora: y overlaps out (in place: the same rows)");
    moe::LoraArgs a{static_cast<const uint16_t*>(w->a), static_cast<const uint16_t*>(w->b), w->scale, index, w->n_adapters, w->rank,
                    w->rows, w->cols, M, type, static_cast<const uint16_t*>(x_bf16), y, out, x_stride, y_stride, out_stride,
                    reinterpret_cast<float*>(o->ws + moe::kCounterBytes), o->status, 0};
    const cudaError_t e = moe::launch_lora(a, o->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_lora");
}

// The calls with many arguments, for the Python binding: the same arguments as 64-bit
// words, in their order.  ctypes takes 0.11 us for each argument that it converts, 1.9 of
// the 9.5 us that a call of moe_rope took the host.
namespace {
template <class T>
T word(long long v)
{
    if constexpr (std::is_pointer_v<T>)
        return reinterpret_cast<T>(static_cast<intptr_t>(v));
    else
        return static_cast<T>(v);
}
template <class... A, size_t... I>
int call(int (*f)(A...), const long long* w, std::index_sequence<I...>)
{
    return f(word<A>(w[I])...);
}
template <class... A>
int call(int (*f)(A...), const long long* w)
{
    return call(f, w, std::index_sequence_for<A...>());
}
}  // namespace

extern "C" int moe_words_kv_write(const long long* w) { return call(moe_kv_write, w); }
extern "C" int moe_words_kv_read(const long long* w) { return call(moe_kv_read, w); }
extern "C" int moe_words_rope(const long long* w) { return call(moe_rope, w); }
extern "C" int moe_words_kv_plan(const long long* w) { return call(moe_kv_plan, w); }
extern "C" int moe_words_lora(const long long* w) { return call(moe_lora, w); }
