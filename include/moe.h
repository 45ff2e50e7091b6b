/*
 * moe.h -- C ABI of libmoe: the routed-expert block of a fine-grained
 * sparse-MoE decode step with 4-bit packed expert weights, on one GB300
 * (sm_103a).
 *
 * What one forward computes, per token m of a batch of M:
 *   1. router: the top_k experts with the largest logits (ties: lower expert
 *      index first; NaN orders as -inf) and a softmax over those top_k logits
 *      only ("Sovereign gpt-oss-20B (MXFP4) on Apple Silicon", section 3:
 *      top-4 routing of 32 experts; GPU top-k on the serving path in
 *      "Amortizing the per-token host-sync setup tax ...", section 3);
 *   2. per selected expert e: a = W_gu[e] x + b_gu[e] with W_gu dequantised
 *      on chip (gate rows [0, I), up rows [I, 2I)); h = silu(gate) * up with
 *      silu(g) = g / (1 + exp(-g)); y = W_d[e] h + b_d[e] (the "4 sequential
 *      experts x 2 small-block GEMVs" of the gpt-oss page, section 3);
 *   3. out[m] = r[m] + sum_s w[m][s] * y_{m,s}   (routing-weighted sum into
 *      the residual), rounded to bfloat16 (nearest even).
 *
 * Weight formats ("MXFP4 reader", gpt-oss page section 3; packed int4 with
 * on-chip dequantisation, "Single-stream int4 decode of a 30B MoE", sections
 * 1 and 6).  All matrices are row-major [N_out][K]; two 4-bit codes per byte,
 * the low nibble holding the even element:
 *   MOE_FMT_MXFP4: OCP MX v1.0 MXFP4 -- FP4 E2M1 codes, one E8M0 scale byte
 *                  (value 2^(s-127), 0xFF = NaN) per 32 consecutive elements
 *                  along K.  Scales u8 [N][K/32].
 *   MOE_FMT_INT4 : symmetric int4, W = (code - 8) * s, one fp16 scale per
 *                  `group` consecutive elements along K.  Scales fp16
 *                  [N][K/group].
 *
 * Precision: x, r and out are bfloat16; routing weights are fp32; dot
 * products are accumulated in fp32.  Denormal scales are kept (no flush to
 * zero).  How the activations reach the multiplier depends on the path:
 *   - MXFP4, M <= 4 (tensor cores, kind::mxf4): x and h' = w h enter as sums
 *     of 8 MXFP4 vectors (term j of a 32-element block has the shared
 *     exponent X0 - 2j, X0 the OCP MX exponent of the block; each term takes
 *     the nearest-even E2M1 codes of what the earlier ones left), within
 *     2^-15 of each block's largest magnitude;
 *   - MXFP4, M > 4 (batched grouped GEMMs): x and h are quantised to one
 *     MXFP4 vector each (OCP MX v1.0, nearest even);
 *   - int4: x enters as f16 after an exact power-of-two rescale, h as f16
 *     hi + lo (about 22 bits).
 *
 * Conventions:
 *   - Every call returns a moe_status (0 = MOE_OK).  Arguments are checked
 *     before anything is enqueued: a call that fails validation enqueues no
 *     work and leaves all buffers untouched.  moe_last_error() gives a
 *     message for the calling thread's last failure.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default).
 *     Forward calls are asynchronous on it.
 *   - Device pointers are plain CUDA device addresses (e.g. from a PyTorch
 *     tensor's data_ptr()); they are borrowed for the duration of the work
 *     enqueued by the call and never freed by the library.
 *   - A handle owns all the device memory it uses: the resident weights of
 *     every layer, a fixed workspace sized at moe_create, and a status word.
 *     No forward call allocates.
 *   - A handle is not thread-safe: use it from one host thread and one stream
 *     at a time.  Distinct handles are independent.
 *   - Failures detected on the device (a bounded wait that gave up, an index
 *     out of range) set the handle's status word; read it with
 *     moe_get_status().  Device code never traps.
 *   - A decode layer runs as one persistent launch with one CTA per SM whose
 *     CTAs wait for one another (a grid barrier before the output is summed;
 *     the pieces of a split unit exchange partial sums).  Work that other
 *     streams run at the same time can delay it; each wait gives up after
 *     about a second and reports MOE_ERR_DEVICE_TIMEOUT instead of hanging.
 */
#ifndef MOE_H
#define MOE_H

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_handle moe_handle;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,    /* bad pointer, size, layer, M or top_k   */
    MOE_ERR_UNSUPPORTED = -2,    /* a shape or format this build does not run */
    MOE_ERR_OOM = -3,            /* device allocation failed in moe_create */
    MOE_ERR_CUDA = -4,           /* a CUDA runtime call failed             */
    MOE_ERR_NOT_LOADED = -5,     /* forward on a layer whose experts were never loaded */
    MOE_ERR_DEVICE_TIMEOUT = -6, /* a device-side bounded wait gave up     */
    MOE_ERR_DEVICE_FAULT = -7    /* a device-side bounds check fired       */
} moe_status;

typedef enum { MOE_FMT_MXFP4 = 1, MOE_FMT_INT4 = 2 } moe_format;

typedef struct {
    int hidden;        /* H: model width, the K of gate_up and the N of down   */
    int intermediate;  /* I: expert width; gate_up has 2I rows                 */
    int num_experts;   /* E experts per layer                                  */
    int num_layers;    /* L layers held resident                               */
    int max_tokens;    /* largest M any forward will be given: 1..4 decode
                          only; 5..8192 also enables the batched path (MXFP4) */
    int max_top_k;     /* largest top_k any forward will be given (<= E)       */
    int format;        /* moe_format                                           */
    int group;         /* elements per scale along K: 32 (MXFP4) or e.g. 64 (int4) */
    int has_bias;      /* 1: bf16 biases b_gu [E][2I] and b_d [E][H] are loaded */
} moe_config;

/* Validate cfg and create a handle on the current CUDA device.  Allocates
 * the resident weight arena for all L layers plus a fixed workspace, and a
 * small pinned host staging buffer for moe_forward_host.
 * Requirements: H and I multiples of 64 and at most 3072; E in 1..256;
 * max_top_k in 1..min(E, 16); max_tokens in 1..8192, above 4 only with
 * MOE_FMT_MXFP4 (else MOE_ERR_UNSUPPORTED); MXFP4 needs group == 32; int4
 * needs group a multiple of 32 dividing both H and I.  Weights are repacked
 * at load into the layout their kernels stream, once: MXFP4 into 128-row
 * tiles whose bytes are the operands of the tensor-core MMA (gate and up rows
 * interleaved per 64), int4 into 16-row slabs of MMA fragments.  The codes,
 * scales and biases take the same bytes as in the caller layout (MXFP4 pads
 * the scales of a partial 128-row tile).  The formats are those of the
 * "MXFP4 reader" ("Sovereign gpt-oss-20B (MXFP4) on Apple Silicon", section 3)
 * and of packed int4 ("Single-stream int4 decode of a 30B MoE", section 1).
 * On success *out receives the handle; on failure *out is set to NULL and
 * nothing stays allocated. */
int moe_create(const moe_config* cfg, moe_handle** out);

/* Copy one layer's experts into the handle (the load-once tables the pages
 * build at start-up instead of per token: "Amortizing the per-token host-sync
 * setup tax ...", section 3).  Each pointer may be host or
 * device memory (any address the CUDA runtime can copy from); the caller keeps
 * ownership and may free or reuse its buffers once the call returns (the call
 * synchronises `stream`).  Layouts (E experts, caller order):
 *   gu_codes  u8 [E][2I][H/2]   gu_scales u8 [E][2I][H/32] | fp16 [E][2I][H/group]
 *   gu_bias bf16 [E][2I]        (NULL allowed only when has_bias == 0)
 *   dn_codes  u8 [E][H][I/2]    dn_scales u8 [E][H][I/32]  | fp16 [E][H][I/group]
 *   dn_bias bf16 [E][H]         (NULL allowed only when has_bias == 0)
 * A layer may be reloaded; the new weights replace the old ones. */
int moe_load_experts(moe_handle* h, int layer,
                     const void* gu_codes, const void* gu_scales, const void* gu_bias,
                     const void* dn_codes, const void* dn_scales, const void* dn_bias,
                     void* stream);

/* Checkpoint-layout flags of moe_load_experts_ex.  The pages verify the
 * MXFP4 reader's orientation against the reference checkpoint ("Sovereign
 * gpt-oss-20B (MXFP4) on Apple Silicon", section 3, "transpose orientation
 * verified"); these accept the layouts a checkpoint may use instead of the
 * caller layout above:
 *   MOE_LOAD_GATE_UP_INTERLEAVED: gate_up rows alternate, row 2j gate row j and
 *     row 2j+1 up row j (codes, scales and gu_bias alike);
 *   MOE_LOAD_TRANSPOSED: both projections stored [K][N] rather than [N][K]:
 *     codes u8 [E][K][N/2] (the element with the even index along N in the low
 *     nibble), scales [E][K/blk][N] (blk = 32 for MXFP4, group for int4); the
 *     biases are vectors and unchanged.  With both flags the transposed
 *     gate_up's N index is the alternating row order.
 * The conversion runs on the device at load time (one extra staging copy of
 * the layer); the resident layout and every forward are those of
 * moe_load_experts. */
typedef enum { MOE_LOAD_GATE_UP_INTERLEAVED = 1, MOE_LOAD_TRANSPOSED = 2 } moe_load_flags;
int moe_load_experts_ex(moe_handle* h, int layer,
                        const void* gu_codes, const void* gu_scales, const void* gu_bias,
                        const void* dn_codes, const void* dn_scales, const void* dn_bias,
                        int flags, void* stream);

/* Router weights of one layer, for calls that leave the logits to the
 * library (router_logits == NULL): logits[m][e] = b[e] + sum_h x[m][h] W[e][h]
 * over the layer's input x (the same bf16 values the experts see; in the
 * stack, the normalised residual), accumulated in fp32 -- the MoE block's
 * gate, whose top-k the pages keep on the GPU ("Amortizing the per-token
 * host-sync setup tax in fused all-layer q4 decode on Apple M1 Ultra",
 * section 3; "Sovereign gpt-oss-20B (MXFP4) on Apple Silicon", section 1,
 * top-4 of 32 experts).  w_bf16 [E][H], bias_bf16 [E] or NULL (zero); host or
 * device memory, copied before the call returns.  Summation order, the same
 * in every kernel (so the decode, int4 and batched paths give the same bits):
 * for each 8-element vector i = lane, lane + 32, ... of the row (lane =
 * 0..31), its elements in order, fused multiply-adds into the lane's sum;
 * then a butterfly over the 32 lanes; then + b[e].  The decode kernels
 * compute the logits inside the layer launch (each CTA a few experts, shared
 * through the grid-wide exchange that publishes the layer's input), so a
 * whole decode step with data-dependent routing stays one launch; the batched
 * path runs one more small kernel first.  A layer may be reloaded. */
int moe_load_router(moe_handle* h, int layer, const void* w_bf16, const void* bias_bf16);

/* One layer.  x bf16 [M][H] (the layer input, already normalised),
 * router_logits fp32 [M][E] -- or NULL: computed from x by the layer's
 * router weights (moe_load_router; MOE_ERR_NOT_LOADED without them) --,
 * out bf16 [M][H]: the residual r on entry and r + MoE(x) on return.
 * 1 <= M <= max_tokens, 1 <= top_k <= max_top_k.  x must not overlap out
 * (checked).  All three are device pointers.
 * M <= 4 runs the decode kernel (one persistent launch).  M > 4 runs the
 * batched path: per-expert grouped GEMMs on the tensor cores
 * (tcgen05.mma kind::mxf4) with x and h quantised to MXFP4 per 32 along K by
 * the OCP MX v1.0 rule (shared exponent floor(log2 amax) - 2, E2M1 nearest-
 * even with saturation); six launches (route, plan, quantise x, the gate_up
 * and down GEMMs, combine), seven when the router weights compute the
 * logits.  moe_set_batched_numerics(MOE_BATCHED_BF16) swaps the quantised
 * GEMMs for kind::f16 ones on weights dequantised to bf16.  Grouped-expert
 * GEMM batching is the lever "Sovereign gpt-oss-20B (MXFP4) on Apple
 * Silicon", section 5, names as untried; the activation quantisation is this
 * library's reading (the tensor-core instruction needs FP4 on both sides). */
int moe_forward(moe_handle* h, int layer, const void* x_bf16, const float* router_logits,
                int M, int top_k, void* out_bf16, void* stream);

/* The SwiGLU form of every forward on this handle (decode, int4, batched, the
 * stack), from the next call on:
 *   h = gc * sigmoid(alpha * gc) * (uc + beta),
 *   gc = min(g, limit), uc = clamp(u, -limit, limit),
 * with g, u the gate and up sums (bias included).  The default (1, +inf, 0)
 * is the plain silu(g) * u of the pages' layer; the expert activation of the
 * gpt-oss model in its public reference implementation is (1.702, 7, 1) --
 * the pages name the model, not these constants.  alpha and beta finite,
 * limit > 0 (+inf for no clamp); else MOE_ERR_INVALID_ARG.
 * moe_forward_noalloc always takes the plain form. */
int moe_set_swiglu(moe_handle* h, float alpha, float limit, float beta);

/* Numerics of the batched path (M > 4) on this handle:
 *   MOE_BATCHED_MXFP4 (default): tcgen05.mma kind::mxf4 -- x and h quantised
 *     to MXFP4 per 32 along K (the OCP MX rule), as that instruction needs;
 *   MOE_BATCHED_BF16: tcgen05.mma kind::f16 -- every weight dequantised to
 *     bf16 in shared memory (exactly: e2m1 * 2^(s-127) is a bf16 value), x as
 *     given and h as bf16 hi + lo (hi = bf16(h), lo = bf16(h - hi)), fp32
 *     accumulation: no activation quantisation, at the cost of the
 *     dequantisation on the CUDA cores.
 * The grouped-expert GEMM is the lever "Sovereign gpt-oss-20B (MXFP4) on
 * Apple Silicon", section 5, names as untried; the two numerics are this
 * library's.  The first switch to bf16 allocates its activation tiles.
 * MOE_ERR_UNSUPPORTED on a handle with max_tokens <= 4. */
typedef enum { MOE_BATCHED_MXFP4 = 0, MOE_BATCHED_BF16 = 1 } moe_batched_numerics;
int moe_set_batched_numerics(moe_handle* h, int numerics);

/* Debug: the router logits of the last call that computed them (the last
 * layer call of a decode launch, or the batched call), fp32 [M][E], copied to
 * the device buffer out_dev on `stream`. */
int moe_debug_router_logits(moe_handle* h, float* out_dev, int M, void* stream);

/* The same layer with host buffers (any host memory, pinned or not): packs x,
 * the residual and the logits into the handle's pinned staging buffer, which
 * is mapped into the device's address space; the layer kernel reads its
 * inputs from it and writes its result into it directly over the host-device
 * link (no separate copies).  Synchronises `stream`, then copies the result
 * into out_bf16.  Argument checks as for moe_forward; router_logits may be
 * NULL (the in-kernel router). */
int moe_forward_host(moe_handle* h, int layer, const void* x_bf16, const float* router_logits,
                     int M, int top_k, void* out_bf16, void* stream);

/* The whole L-layer expert stack for one decode step ("one command buffer per
 * decode", "Single-stream int4 decode of a 30B MoE", sections 1 and 6).  For
 * l = 0..L-1:
 *   x_l = bf16(r_l / sqrt(mean(r_l^2) + 1e-6))   (weightless RMSNorm, per token)
 *   r_{l+1} = bf16(r_l + MoE_l(x_l))
 * The pages name a residual add between layers but no coupling; the
 * normalised input is this library's reading (a literal x + MoE(x) chain
 * overflows within a few layers on these value distributions).
 * resid bf16 [M][H] holds r_0 on entry and r_L on return; logits fp32
 * [L][M][E], or NULL: each layer's logits from its router weights applied to
 * x_l (moe_load_router, every layer), so that the routing of layer l+1
 * depends on the output of layer l inside the one launch.  Layer l+1 reads
 * its logits only after layer l's output is complete.  Device pointers.  One persistent launch for all L layers (grid
 * barriers between them), both formats.  Decode sizes only: M <= 4 (else
 * MOE_ERR_UNSUPPORTED). */
int moe_forward_stack(moe_handle* h, void* resid_bf16, const float* router_logits,
                      int M, int top_k, void* stream);

/* n decode steps of the whole stack in one persistent launch (n tokens, each
 * through all L layers; P2's "all decode tokens into a single command
 * buffer"): step t runs the L layers of moe_forward_stack on its own residual
 * resid[t] (bf16 [n][M][H]: r_0 of step t on entry, its r_L on return) with
 * logits[t] (fp32 [n][L][M][E], or NULL: the in-kernel router, as for
 * moe_forward_stack), steps one after another, exactly as n
 * moe_forward_stack calls in that order would (bit-identical results).  Each
 * layer call reads its logits only after the previous call's output is
 * complete.  Device pointers, 16-byte aligned; decode sizes only (M <= 4);
 * n * L <= 2^30. */
int moe_forward_stack_steps(moe_handle* h, int n, void* resid_bf16, const float* router_logits,
                            int M, int top_k, void* stream);

/* n single-layer decode steps in sequence: step s runs resident layer
 * (layer0 + s) mod L on x[s], logits[s] and out[s] (x bf16 [n][M][H],
 * router_logits fp32 [n][M][E] or NULL for the in-kernel router, out bf16
 * [n][M][H]: the residual of each step
 * on entry, r + MoE(x) on return), exactly as n moe_forward calls in that order
 * would (bit-identical results).  Step s + 1 reads its routing and inputs only
 * after step s's output is complete.  One persistent launch for all n steps,
 * both formats ("all decode tokens in a single command buffer", "Single-stream
 * int4 decode of a 30B MoE", section 1).  Decode sizes only (M <= 4); x must
 * not overlap out; 16-byte aligned.  x, logits and out may be device memory
 * or page-locked host memory mapped into the device's address space at the
 * same address (cudaHostAlloc / cudaMallocHost, or cudaHostRegister with
 * cudaHostRegisterMapped, on a system with unified addressing): the kernel
 * then reads each step's inputs and writes each step's result over the
 * host-device link itself, and the host sees every step's result once
 * `stream` has been synchronised.  Host memory that is not mapped so is
 * rejected (MOE_ERR_INVALID_ARG).  moe_last_bytes then counts each step's
 * distinct experts (a layer run by several steps counts its last step's, n
 * times over). */
int moe_forward_steps(moe_handle* h, int n, int layer0, const void* x_bf16, const float* router_logits,
                      int M, int top_k, void* out_bf16, void* stream);

/* Measurement: the streaming floor of this GPU for decode-sized weight reads.
 * Reads the first `bytes` bytes of resident layers layer0 .. layer0 + n - 1,
 * one layer after another with a grid barrier between them (as dependent
 * decode layers are), with the copy engine and stage sizes of the decode
 * kernels (one CTA per SM, bulk copies of 32 KB, 128 KB in flight per SM) and
 * no compute.  bytes: a multiple of 16, at most one layer's arena.  Device
 * work on `stream`; errors as MOE_ERR_INVALID_ARG. */
int moe_debug_stream_weights(moe_handle* h, int layer0, int n, long long bytes, void* stream);

/* Synchronise `stream` and return (and clear) the handle's device status:
 * MOE_OK, MOE_ERR_DEVICE_TIMEOUT or MOE_ERR_DEVICE_FAULT.  After a non-OK
 * status the handle's cross-CTA counters are reset, so it can be used again.
 * (Failure detection: the pages describe none for the GPU path; every wait in
 * this library is bounded and reports here instead of hanging.) */
int moe_get_status(moe_handle* h, void* stream);

/* Debug: decode one stored expert projection to fp32, exactly (each element
 * is e2m1 * 2^(s-127) or (q - 8) * fp16 scale, rounded to fp32 once), from
 * the very bytes the forward kernels stream: MXFP4 from the tile layout, int4
 * from the slabs.  proj 0 = gate_up ([2I][H], caller row order), 1 = down
 * ([H][I]).  out_dev fp32 device buffer of N*K elements.  The bit-exact check
 * of the "MXFP4 reader" against its golden, gpt-oss page section 1. */
int moe_debug_dequant(moe_handle* h, int layer, int expert, int proj, float* out_dev,
                      void* stream);

/* Debug: the router alone.  logits fp32 [M][E] device; idx int32 [M][top_k]
 * and w fp32 [M][top_k] device outputs, selection order (largest first).
 * M up to 65536 here. */
int moe_debug_route(moe_handle* h, const float* logits, int M, int top_k, int* idx, float* w,
                    void* stream);

/* Debug: the batched path's MX quantiser on a flat fp32 vector.  in fp32 [n]
 * device, n a multiple of 32; codes u8 [n/2] (low nibble = even element) and
 * scales u8 [n/32] (E8M0) device outputs, natural order.  No handle needed.
 * in and codes 16-byte aligned. */
int moe_debug_mx_quantize(const float* in, long long n, unsigned char* codes,
                          unsigned char* scales, void* stream);

/* Debug: the quantised h of the last batched forward (M > 4) on this handle,
 * in (token, choice) order: codes u8 [M*top_k][I/2] and E8M0 scales u8
 * [M*top_k][I/32], device outputs (codes 16-byte aligned).  Choice s of token
 * m is the s-th selected expert (largest logit first). */
int moe_debug_batched_h(moe_handle* h, unsigned char* codes, unsigned char* scales, void* stream);

/* Debug: the expert stack run layer by layer with the same kernels as
 * moe_forward_stack (one launch per layer), recording the residual after
 * every layer.  resid bf16 [M][H] is updated in place as in
 * moe_forward_stack; trace bf16 [L+1][M][H] device buffer receives r_0 ..
 * r_L.  router_logits NULL: the in-kernel router, as in moe_forward_stack. */
int moe_debug_stack_trace(moe_handle* h, void* resid_bf16, const float* router_logits, int M,
                          int top_k, void* trace_bf16, void* stream);

/* Debug: moe_forward that also writes the fp32 result before its bf16
 * rounding, out_f32 fp32 [M][H] device (16-byte aligned), for checking the
 * fp32-accumulated output itself.  Everything else as moe_forward. */
int moe_debug_forward_f32(moe_handle* h, int layer, const void* x_bf16, const float* router_logits,
                          int M, int top_k, void* out_bf16, float* out_f32, void* stream);

/* Debug (failure detection): the cross-CTA waits of the MXFP4 decode layer
 * give up after `spin_limit` polls (0 restores the default, about a second),
 * and CTA `skip_cta` (-1: none) skips its arrival at the layer's grid barrier,
 * so that the other CTAs' waits run out.  Applies to moe_forward and
 * moe_debug_forward_f32 calls made after it (stack graphs already captured keep
 * the settings they were captured with).  A call whose wait ran out reports
 * MOE_ERR_DEVICE_TIMEOUT through moe_get_status, which also resets the
 * counters so the handle works again.  Every access stays inside the handle's
 * buffers; nothing traps. */
int moe_debug_set_wait(moe_handle* h, int spin_limit, int skip_cta);

/* Algorithmic expert bytes moved by the last forward call on this handle:
 * codes + scales + biases of the distinct experts selected in each layer,
 * counted once per layer (the byte counters of the pages' tracing, TinyTitan
 * tracker).  Synchronises `stream` (so the signature takes the stream and
 * returns a status, writing *bytes).  Returns MOE_OK and writes *bytes, or an
 * error. */
int moe_last_bytes(moe_handle* h, void* stream, long long* bytes);

/* Bytes of one expert (codes + scales + biases) for this handle's config. */
long long moe_expert_bytes(const moe_handle* h);

/* Number of kernel launches the last forward call enqueued (for the caller's
 * launch accounting; a graph replay counts the kernels inside it). */
int moe_last_launches(const moe_handle* h);

/* Message for the calling thread's most recent failure ("" if none). */
const char* moe_last_error(void);

/* One decode layer for callers that cannot allocate device memory.
 *
 * The pages describe no such call; it exists for users of this library whose
 * runtime forbids cudaMalloc: an inference engine that serves every buffer
 * from its own pre-sized pool, code running while a CUDA graph is captured, or
 * a plug-in that may not touch the CUDA allocator.  Such a caller cannot create
 * a moe_handle (moe_create allocates), so here every input and output is the
 * caller's memory and the call allocates nothing: no cudaMalloc, cudaFree or
 * allocating library routine.
 *
 * Computes the same layer as moe_forward: out = r + sum_s w_s * y_s for the
 * top_k experts of each token.  The weights are the caller-layout tensors of
 * moe_load_experts for one layer (E experts), on the device; x bf16 [M][H],
 * router_logits fp32 [M][E] and out bf16 [M][H] (the residual on entry) are
 * device pointers; x must not overlap out.  Alignment: x, out and the code
 * and scale arrays 16-byte aligned, router_logits 4-byte, biases 2-byte
 * (else MOE_ERR_INVALID_ARG).  cfg gives H, I, E, format, group and has_bias
 * (its num_layers, max_tokens and max_top_k are ignored).
 *
 * Scratch (h, the per-slot down outputs and the output-tile counters) is one
 * file-scope __device__ array of 1,574,400 bytes that every GPU which loads the
 * library holds until the process exits.  It fixes the limits: M <= 4,
 * top_k <= 16, H and I multiples of 32 and at most 3072; larger sizes return
 * MOE_ERR_INVALID_ARG with a message.  The first call on a device looks up the
 * array's device address (cudaGetSymbolAddress) for that device; make that
 * first call before any stream capture.  Every call uses the same array, and
 * it keeps the contents of the last call (the tile counters are cleared at the
 * start of each call), so calls that overlap on the GPU -- on two streams, or
 * from two threads -- race and must be serialised by the caller.  Runs
 * asynchronously on `stream`. */
int moe_forward_noalloc(const moe_config* cfg, const void* gu_codes, const void* gu_scales,
                        const void* gu_bias, const void* dn_codes, const void* dn_scales,
                        const void* dn_bias, const void* x_bf16, const float* router_logits,
                        int M, int top_k, void* out_bf16, void* stream);

/* Release a handle and all device memory it owns.  NULL is a no-op. */
void moe_destroy(moe_handle* h);

/* ======================================================================
 * The operators around the expert block in a decode step, and in the prompt
 * before it: a paged key/value cache in 8 or 4 bits, attention over it, projections
 * with 4-bit weights, and sampling.  The pages name them as the rest of the
 * decode ("Sovereign gpt-oss-20B (MXFP4) on Apple Silicon", sections 1 and 3:
 * attention with sinks and a sliding window, the LM head; the "greedy, KV"
 * decode loop of "Single-stream int4 decode of a 30B MoE").
 *
 * All tensors, the cache and the weights among them, are the caller's device
 * memory, borrowed for the work that a call enqueues.  A moe_ops handle holds
 * the workspace and a status word; the conventions at the top of this file
 * (status codes, checks before anything is enqueued, streams, one thread and
 * one stream at a time per handle, nothing allocated by a call, no host work
 * that depends on device values) hold for it too.  Each call is one launch
 * (moe_linear: one for each pass of up to 16 tokens; moe_lora: two; moe_attention: two where few rows
 * share out many keys) and can be captured in a CUDA graph.  What a device-side check finds (metadata that does not describe the
 * batch, a block number outside the cache) sets MOE_ERR_DEVICE_FAULT in the
 * handle's status word and skips that sequence or block.
 * ====================================================================== */

typedef struct moe_ops moe_ops;

/* A handle on the current device: allocates the workspace (22.7 MB on 152 SMs,
 * whatever the sizes of later calls). */
int moe_ops_create(moe_ops** out);

/* Synchronise `stream`; return (and clear) the handle's device status: MOE_OK,
 * MOE_ERR_DEVICE_FAULT or MOE_ERR_DEVICE_TIMEOUT, or MOE_ERR_CUDA.  After a
 * non-OK status the handle can be used again. */
int moe_ops_get_status(moe_ops* o, void* stream);

/* Release the workspace.  NULL is a no-op. */
void moe_ops_destroy(moe_ops* o);

/* An 8-bit paged cache of one layer: num_blocks blocks of `block` tokens each,
 * with one fp32 scale for each (block, head, K or V).
 *   codes  u8 [num_blocks][kv_heads][2][block * head_dim], 16-byte aligned:
 *          K codes as [block][head_dim], then V codes as [head_dim][block]
 *          (transposed: attention multiplies V along the tokens);
 *   scales fp32 [num_blocks][kv_heads][2] (K, V), 8-byte aligned.
 * A value is its code times the scale.  MOE_KV_INT8: codes -127..127.
 * MOE_KV_E4M3: OCP FP8 E4M3 codes and scales that are powers of two.  A cache
 * holds no NaN code (0x7f, 0xff: none is ever written) and no scale that is negative,
 * infinite or NaN; what attention makes of one is not defined, but stays in the
 * sequences whose tables name the block.  block 32, 64 or 128; head_dim 64 or 128; kv_heads
 * 1..256.
 *
 * In 4 bits, MOE_KV_MXFP4: FP4 E2M1 codes with an E8M0 scale byte s (the value is the
 * code times 2^(s - 127); 0: a group of zeros) for each group of 32 values of one token
 * and head, d = 32 g .. 32 g + 31.  `scales` is NULL:
 *   codes  u8 [num_blocks][kv_heads][2][block * head_dim * 17 / 32], 16-byte aligned: for
 *          K, then for V, the block's codes and after them its scale bytes, 32 tokens at
 *          a time.  With t of the block, u = t % 32, d = 32 g + 8 e + r (e 0..3, r 0..7):
 *   K code  byte t * head_dim / 2 + d / 2, the even d in the low nibble;
 *   K scale byte (t / 32) * head_dim + ((2 (u / 8) + u % 2) * head_dim / 32 + g) * 4 +
 *           (u / 2) % 4;
 *   V code  byte (((t / 32) * head_dim / 32 + g) * 8 + r) * 64 + (u / 8) * 16 + 4 e +
 *           (u % 8) / 2, the even t in the low nibble;
 *   V scale byte ((t / 32) * head_dim / 32 + g) * 32 + u.
 * An MXFP4 cache holds no scale byte 255 where a token is. */
typedef enum { MOE_KV_E4M3 = 1, MOE_KV_INT8 = 2, MOE_KV_MXFP4 = 4 } moe_kv_format;
typedef struct {
    void* codes;
    float* scales;
    int num_blocks, kv_heads, head_dim, block, format;
} moe_kv_cache;

/* A batch of tokens of several sequences, all device arrays of int32:
 *   cu     [n_seqs + 1]: tokens cu[b] .. cu[b+1] - 1 of the batch belong to
 *          sequence b (0 <= cu[b] <= cu[b+1] <= n_tokens);
 *   kv_len [n_seqs]: the sequence's cached tokens, the batch's own included:
 *          they are its last ones, at positions kv_len - n .. kv_len - 1;
 *   table  [n_seqs][table_stride]: the cache block of each `block` positions
 *          (only entries below ceil(kv_len / block) are read).
 * n_seqs 1..1024, n_tokens 1..2^20; a sequence may have no tokens. */
typedef struct {
    const int* cu;
    const int* kv_len;
    const int* table;
    int n_seqs, n_tokens, table_stride;
} moe_kv_batch;

/* Quantise the batch's keys and values (bf16 [n_tokens][kv_heads][head_dim],
 * rows k_stride / v_stride elements apart) into the cache.  For each (block,
 * head) and K and V apart, with a the largest finite magnitude among the new
 * values (at least 2^-100):
 *   INT8 scale a / 127 (rounded to fp32); E4M3: the smallest 2^e with
 *   a <= 448 * 2^e;
 *   a block whose first token is written takes that scale, and its unwritten
 *   tokens get code 0; a block that already holds earlier tokens of the
 *   sequence keeps its scale, or takes the new one if that is larger: then the
 *   earlier tokens' codes c become round(c * (old * (1 / new)));
 *   code = round(x * (1 / scale)), to nearest even, saturating; a NaN becomes
 *   0 and an infinity the largest code.
 * (1 / scale and the products are single fp32 operations.)  MXFP4, for each group
 * apart, with a its largest finite magnitude: below 2^-100 its codes and its scale
 * byte are 0; else the scale is the smallest 2^e with a <= 6 * 2^e, the byte e + 127,
 * and a code the nearest E2M1 value to x / 2^e, ties to the even code, saturating; a NaN
 * becomes 0 and an infinity +-6.  What a token becomes depends on nothing else, and
 * other tokens' codes stay; a block whose first token is written has its unwritten
 * tokens' codes and scale bytes set to 0.  Sequences must not share a block that is
 * written.  The rows are 16-byte aligned and the strides multiples of 8. */
int moe_kv_write(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* k_bf16,
                 long long k_stride, const void* v_bf16, long long v_stride, void* stream);

/* Read the batch's tokens back: code * scale, rounded to bf16 (MXFP4: exact, but for
 * magnitudes that round up to 2^128, which are infinite), into rows
 * k_stride / v_stride elements apart.  Conditions as for moe_kv_write; the
 * same batch names the tokens (so cu and kv_len of another batch, say all of
 * a prefix, read those). */
int moe_kv_read(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, void* k_bf16,
                long long k_stride, void* v_bf16, long long v_stride, void* stream);

/* Attention of the batch's tokens over the cache (which holds their own keys
 * and values already).  q bf16 [n_tokens][q_heads][head_dim], rows q_stride
 * elements apart (16-byte aligned, a multiple of 8); query head h reads kv
 * head h / (q_heads / kv_heads); q_heads a multiple of kv_heads, at most 1024.
 * The token at position i sees positions j <= i, and with window > 0 only
 * j > i - window; blocks wholly before the window of a sequence's first token of
 * the batch are not read, and neither are their entries of the table.
 * s_j = scale q . k_j;
 *   out = sum_j e^(s_j - m) v_j / (sum_j e^(s_j - m) + e^(sink - m)),
 * m the largest of them, sinks fp32 [q_heads] or NULL (no such term).
 * out bf16 [n_tokens][q_heads][head_dim], contiguous, 16-byte aligned; must not
 * overlap q (checked).  lse fp32 [n_tokens][q_heads] or NULL: m + log of the
 * denominator.  A row of which nothing is visible (its blocks are missing)
 * is 0, with the sink (or -inf) as its lse.  A row whose q or sink has a NaN is NaN,
 * and so is its lse; other rows are not touched by it.
 * Scores and sums are fp32, and parts of a row that are summed apart are joined so that out
 * is finite wherever its value is (and off by no more than 2^-137 beside the rest, which
 * shows below 2^-126 only); q enters as f16 after an exact power-of-two rescale
 * of each row, codes are exact in f16, and e^(s_j - m) enters the second
 * product as 11 bits down to 2^-20, below that within 2^-31.  MXFP4: of a key, groups whose
 * scale is below 2^-27 of its largest group's count as 0; V's groups whose scale is below
 * 2^-64 of the largest that the call's earlier keys of that sequence have in that group, or
 * below 2^-118, may count as 0; and a probability loses at most 2^-31 in units of that largest
 * scale.  The (sequence,
 * 16 rows, kv head, block) combinations of one call number less than 2^31, of MXFP4 with
 * 8 rows or fewer a sequence and kv head on average those of 8 rows (else nothing is
 * written, MOE_ERR_DEVICE_FAULT). */
int moe_attention(moe_ops* o, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* q_bf16,
                  long long q_stride, int q_heads, float scale, int window, const float* sinks, void* out_bf16,
                  float* lse, void* stream);

/* A step's batch, made on the GPU from the requests' lengths: block tables, and for
 * each token its sequence, position and slot.
 *
 * Free blocks lie in a ring: entries state[0], state[0] + 1, ... (modulo ring_size) of
 * `ring`, state[1] of them.  ring_size is the number of the cache's blocks, so that
 * the ring holds them all. */
typedef struct {
    int* ring;                    /* [ring_size] */
    int* table;                   /* [n_seqs][table_stride]: the sequences' blocks, as in moe_kv_batch */
    int ring_size, n_seqs, table_stride, block;
} moe_kv_pool;

/* For each sequence b, n_new[b] tokens are to be added to the kv_len[b] that it has
 * (-1: it has ended, and its blocks go back to the ring).  All arrays are the caller's
 * device memory.
 *   - Sequences are served in order.  The first whose tokens pass n_tokens, or whose new
 *     blocks pass the free ones, and every one after it, get no tokens in this step;
 *     admitted[0] is the number of those before it (n_seqs: all).
 *   - The blocks that sequence b comes to need, ceil((kv_len + n) / block) less those
 *     that it has, are taken from the ring's front, in order, and entered in its row of
 *     the table; its other entries stay as they are.
 *   - Blocks of ended sequences, admitted or not, go to the ring's end, in order (and
 *     are free from the next call on); their rows of the table stay as they are.
 *   - cu [n_seqs + 1] and kv_len_out [n_seqs] are what a moe_kv_batch takes: the served
 *     tokens' prefix sums, and the lengths with them (0 for an ended sequence).
 *   - state_out [2]: the ring's state after it.
 *   - For token t < cu[n_seqs]: seq[t], position[t] (of its sequence) and slot[t] = its
 *     block * `block` + its place in it; all three are -1 from cu[n_seqs] to n_tokens - 1.
 * admitted, seq, position and slot may be NULL.  kv_len_out may be kv_len and state_out
 * may be state (updated in place); else a call with the same inputs gives the same
 * outputs, whatever an earlier one did.  No other arrays may overlap (checked).
 * A sequence whose length is negative or whose n_new is below -1, or whose tokens do not
 * fit its row of the table, gets none and keeps its length; a state outside the ring serves no one; where more
 * blocks come back than the ring has room for none does, and ended sequences keep their
 * lengths: each sets MOE_ERR_DEVICE_FAULT.  So does a block number outside 0 ..
 * ring_size - 1; it is passed on as it is, and its tokens' slots are -1.
 * n_seqs 1..1024, n_tokens 1..2^20, block as in moe_kv_cache. */
int moe_kv_plan(moe_ops* o, const moe_kv_pool* pool, const int* n_new, const int* kv_len, const int* state,
                int n_tokens, int* cu, int* kv_len_out, int* state_out, int* admitted, int* seq, int* position,
                long long* slot, void* stream);

typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1 } moe_dtype;

/* Rotary positions.  Of each head's head_dim values the first rot_dim turn, in pairs:
 * (u, v) becomes mscale (u cos t - v sin t, v cos t + u sin t), t = position * f_i for
 * pair i; the others stay.  Pair i is (i, i + rot_dim / 2) or (2 i, 2 i + 1). */
typedef enum { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 } moe_rope_layout;

/* f_i = base^(-2 i / rot_dim), and for longer contexts than a model was trained on (factor at
 * least 2^-32):
 *   LINEAR      f_i / factor;
 *   PARTS       f_i (1 - x) + f_i / factor * x, x = (i - a) / max(b - a, 0.001) held to
 *               0..1, a = max(at(high), 0), b = min(at(low), rot_dim / 2 - 1),
 *               at(n) = rot_dim log(length / (2 pi n)) / (2 log base): pairs that turn
 *               more than `high` times within `length` positions keep their speed, those
 *               that turn less than `low` times are slowed down.  Some models round a and b
 *               to whole pairs, or hold b to rot_dim - 1: their tables are the caller's to
 *               make (moe_rope_table takes any);
 *   WAVELENGTH  f_i x + f_i / factor (1 - x), x = (length f_i / (2 pi) - low) /
 *               (high - low) held to 0..1. */
typedef enum { MOE_ROPE_PLAIN = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_PARTS = 2, MOE_ROPE_WAVELENGTH = 3 } moe_rope_scaling;
typedef struct {
    int rot_dim, scaling;
    double base, factor, length, low, high;
} moe_rope_config;

/* The table of a configuration: turns[i] = f_i / (2 pi), modulo 1, times 2^64, for
 * rot_dim / 2 pairs, in host memory (no GPU is needed); copy it to the device once. */
int moe_rope_turns(const moe_rope_config* c, unsigned long long* turns);

typedef struct {
    const unsigned long long* turns;    /* [rot_dim / 2], device */
    int rot_dim, layout;
    float mscale;
} moe_rope_table;

/* Turn queries [n_tokens][q_heads][head_dim] and keys [n_tokens][k_heads][head_dim] (k_heads
 * 0: none) by their positions, int32 [n_tokens]; a negative one leaves the row's output as
 * it is.  All of one type (moe_dtype), rows strides elements apart, 16-byte aligned, the
 * strides multiples of 16 bytes; the rows may be parts of a fused projection.  q_out may be
 * q and k_out k (the same rows, in place); else outputs must not overlap any array of the
 * call (checked).  position * f_i / (2 pi) is kept modulo 1 in 64 bits, so an angle is off by no
 * more than position * 2^-55 turns (times f_i where that is above 1) beside fp32 rounding of
 * what is left; cosine, sine and products are fp32, the result is rounded once.  head_dim a
 * multiple of 8, 8..512; rot_dim even, 2..head_dim; n_tokens 1..2^20. */
int moe_rope(moe_ops* o, const moe_rope_table* r, const int* position, int n_tokens, int head_dim, int type,
             const void* q, long long q_stride, int q_heads, void* q_out, long long q_out_stride, const void* k,
             long long k_stride, int k_heads, void* k_out, long long k_out_stride, void* stream);

/* A matrix of 4-bit weights W [rows][cols], format and group as in moe_config:
 *   codes  u8 [rows][cols/2]; scales u8 [rows][cols/32] (MXFP4) or fp16
 *          [rows][cols/group] (int4); both 16-byte aligned;
 *   bias   bf16 [rows] or NULL.
 * cols a multiple of 32 (MXFP4) or of group (int4: 32, 64, 128 or 256), at most
 * 32768; rows 1..2^24. */
typedef struct {
    const void* codes;
    const void* scales;
    const void* bias;
    int rows, cols, format, group;
} moe_linear_weights;

/* out[m] = W x[m] + bias for M = 1..64 tokens (the decode projections and the
 * LM head; "Single-stream int4 decode of a 30B MoE", sections 1 and 6: packed
 * int4 dequantised on chip).  x bf16 [M][cols], rows x_stride elements apart
 * (16-byte aligned, a multiple of 8); out fp32 or bf16 [M][rows], rows
 * out_stride elements apart.  x enters as f16 after an exact power-of-two
 * rescale of a token (or of a quarter of its columns), which keeps what is above
 * 2^-37 of its largest element (int4: every other element above 2^-33); weights are
 * exact in f16, sums are fp32.  A token's result does not depend on the other
 * tokens; a token with an infinity or NaN has no finite result (int4: NaN).  x and
 * out must not overlap. */
int moe_linear(moe_ops* o, const moe_linear_weights* w, const void* x_bf16, long long x_stride, int M, void* out,
               long long out_stride, int out_type, void* stream);

/* Low-rank adapters beside a shared projection, one for each token:
 *   a bf16 [n_adapters][rank][cols], b bf16 [n_adapters][rows][rank], 16-byte aligned;
 *   scale fp32 [n_adapters] or NULL (1).
 * rank a multiple of 8, 8..128 (pad with zeros); cols a multiple of 8, at most 32768;
 * rows 1..2^24; n_adapters 1..65536. */
typedef struct {
    const void* a;
    const void* b;
    const float* scale;
    int n_adapters, rank, rows, cols;
} moe_lora_weights;

/* out[m] = y[m] + scale[i] * b[i] (a[i] x[m]), i = index[m], for M = 1..64 tokens: index
 * int32 [M], -1 (or less): no adapter, out[m] = y[m]; one that is not below n_adapters sets
 * MOE_ERR_DEVICE_FAULT and counts as -1.  x bf16 [M][cols], rows x_stride elements apart
 * (16-byte aligned, a multiple of 8); y and out fp32 or bf16 [M][rows], rows y_stride and
 * out_stride elements apart; y may be NULL (0), or out (what moe_linear left there); else
 * they must not overlap, nor x and out (checked).  An adapter's weights are read once for
 * every eight tokens that share it.  a x is kept in fp32, sums are fp32, the result is rounded
 * once; a token's result does not depend on the others, but for the order of its sums.  A
 * token with an infinity or NaN in x, or whose a x overflows, has no finite result.  Two
 * launches. */
int moe_lora(moe_ops* o, const moe_lora_weights* w, const int* index, const void* x_bf16, long long x_stride, int M,
             const void* y, long long y_stride, void* out, long long out_stride, int type, void* stream);

/* Per-row device arrays [M]; every one but u may be NULL. */
typedef struct {
    const float* temperature;   /* NULL: 1.  <= 0 (or NaN): the largest logit, lowest index first */
    const int* top_k;           /* <= 0 or >= V: off */
    const float* top_p;         /* >= 1: off; <= 0: the first token alone */
    const float* min_p;         /* <= 0: off; > 1 counts as 1 */
    const float* u;             /* in [0, 1); clamped to [0, 1 - 2^-24] */
} moe_sample_params;

/* One token for each of M rows of logits [M][V] (fp32 or bf16, rows `stride`
 * elements apart), V 1..2^19.  Order: larger logit first, ties to the lower
 * index; NaN counts as -inf.  With l* the largest logit and z = (l - l*) *
 * (1 / T), a token's weight is round(e^z * 2^31), an integer, so that sums are
 * exact in any order.  Kept are, one filter after another:
 *   top-k: the first k;
 *   top-p: the shortest prefix of those whose weights reach top_p times the sum
 *          of all of those (product in fp64, at least one token);
 *   min-p: those whose weight is at least min_p * 2^31.
 * token[m]: the first kept one, by index, at which the running sum of weights
 * exceeds u times their sum.  logprob[m] (or NULL): z - log(sum / 2^31) of that
 * token; 0 where T <= 0.  A row of -inf only gives its lowest index and
 * logprob -inf; with +inf among the logits only those have weight. */
int moe_sample(moe_ops* o, const void* logits, int logits_type, long long stride, int M, int V,
               const moe_sample_params* p, int* token, float* logprob, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
