/*
 * wl.h -- C ABI of libwl.so, weightless linear projections on GB300 (sm_103a).
 *
 * A weightless projection never holds its dense weight.  Each weight is the
 * theta bundle of the "Serve and generate with weightless" page (overview):
 * a W0 block shared per band of layers, a per-output-row scale s and a rank-r
 * delta U, V.  Every call rebuilds the projection inside the kernel
 * ("In-kernel reconstruction" page, formula section):
 *
 *     y[t,o] = s[o] * sum_i W0[o,i] x[t,i] + sum_k U[o,k] * sum_i V[i,k] x[t,i]
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Layouts (row-major, contiguous, PyTorch Linear convention):
 *    x  [T, in]   bf16          W0 [out, in] bf16        s [out] fp32
 *    U  [out, r]  bf16          V  [in, r]   bf16        y [T, out] bf16 or fp32
 *  Precision: bf16 inputs, fp32 accumulation, fp32 combine, one final
 *    round-to-nearest-even cast to the output type ("In-kernel
 *    reconstruction": the custom-op path accumulates in float32; the GEMM
 *    path does its final combine in float32 before the cast).
 *  Memory: every pointer is device memory owned by the caller.  The library
 *    allocates nothing in these calls.  Outputs must not alias inputs.
 *  Streams: `stream` is a cudaStream_t (NULL = legacy default stream).  Calls
 *    are asynchronous on that stream; results are ready when it is.  The
 *    decode-size launches (wl_linear, wl_qkv_fused, wl_mlp_geglu_fused at
 *    T <= 8) use programmatic dependent launch: they start streaming W0, s,
 *    U and V while the previous kernel on the stream finishes, and read x
 *    (and write y) only after it has completed.  So the weights must not be
 *    written by the kernel launched immediately before the call on the same
 *    stream; weights written by a copy (cudaMemcpy*), on another stream
 *    joined by an event, or by any earlier kernel are fine.
 *    The decoder-layer operators below launch the same way but touch no
 *    caller memory before everything ahead of them on the stream is complete.
 *  Errors: return codes only; nothing is thrown or aborted across the ABI.
 *    Arguments are checked before anything is launched; on error nothing is
 *    launched and wl_last_error() describes the failure.  A failed launch
 *    returns WL_ERR_CUDA.  Kernel-side bounded waits that give up record
 *    WL_ERR_TIMEOUT in a device status word, read by wl_device_status().
 *  Limits: T >= 1, in >= 8, out >= 1, in % 8 == 0, 0 <= r <= WL_MAX_RANK;
 *    x, W0 and y must be 16-byte aligned (in % 8 == 0 keeps every row of x
 *    and W0 aligned when the base is); U and V may be NULL only if r == 0.
 */
#ifndef WL_H_
#define WL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    WL_OK = 0,
    WL_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or rank        */
    WL_ERR_UNSUPPORTED = 2, /* valid arguments this build cannot run       */
    WL_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed        */
    WL_ERR_TIMEOUT = 4,     /* a bounded device-side wait gave up          */
    WL_ERR_WORKSPACE = 5,   /* workspace missing, misaligned or too small  */
    WL_ERR_INTERNAL = 6     /* a plan broke an invariant of the library;
                               nothing was launched (a library bug)        */
} wl_status;

typedef enum { WL_OUT_BF16 = 0, WL_OUT_F32 = 1 } wl_out_dtype;

/* One projection's theta bundle: W0 [out, in], s [out], U [out, r], V [in, r]. */
typedef struct {
    const void *W0;
    const float *s;
    const void *U;
    const void *V;
    int64_t out;
} wl_proj;

#define WL_MAX_RANK 128

/*
 * wl_linear -- one weightless projection, y = s*(x W0^T) + (x V) U^T.
 * Source: "In-kernel reconstruction", formula section (per-element form) and
 * "The GEMM path" (the same map as s[None,:]*(x@W0.T) + (x@V)@U.T).
 * x [T,in] bf16, W0 [out,in] bf16, s [out] fp32, U [out,r] bf16, V [in,r] bf16,
 * y [T,out] of type ydt.  Small T (decode) streams W0 once from HBM with the
 * rank-r term and the scale folded into the same launch; large T (prefill)
 * runs the dense contraction on the tensor cores with the low-rank term in
 * the epilogue.  Both give the same result within fp32 accumulation order.
 */
wl_status wl_linear(const void *x, const void *W0, const float *s, const void *U,
                    const void *V, void *y, int64_t T, int64_t in, int64_t out,
                    int64_t r, wl_out_dtype ydt, void *stream);

/*
 * wl_qkv_fused -- the three attention projections that share one input x, in
 * one launch that reads x once ("In-kernel reconstruction", "Q/K/V fusion").
 * Each of q, k, v is a full theta bundle with its own out (in and r shared);
 * yq [T,q.out], yk [T,k.out], yv [T,v.out].  Equal, within accumulation
 * order, to three wl_linear calls.
 */
wl_status wl_qkv_fused(const void *x, wl_proj q, wl_proj k, wl_proj v, void *yq,
                       void *yk, void *yv, int64_t T, int64_t in, int64_t r,
                       wl_out_dtype ydt, void *stream);

/*
 * wl_mlp_workspace_bytes -- bytes of device workspace wl_mlp_geglu_fused
 * needs for these sizes (the intermediate h = gelu(g)*u and the partial sums
 * of the down projection's low-rank input h V_down).  Calls of up to 8 tokens
 * run the HBM-streaming kernels unless no launch plan of theirs fits shared
 * memory for these sizes (then the tensor-core kernels run); the size covers
 * both.  Returns 0 for invalid sizes.
 */
size_t wl_mlp_workspace_bytes(int64_t T, int64_t hidden, int64_t inter, int64_t r,
                              wl_out_dtype ydt);

/*
 * wl_mlp_geglu_fused -- the gated MLP of a weightless layer in one call
 * ("In-kernel reconstruction", custom-op path: gate, up, activation and down
 * fused into one dispatch):
 *     g = wl(x; gate), u = wl(x; up)          [T, inter]
 *     h = gelu_tanh(g) * u                    [T, inter]
 *     y = wl(h; down)                         [T, hidden]   (down.out == hidden)
 * gelu_tanh(v) = 0.5 v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))).
 * workspace: caller-owned device memory of at least
 * wl_mlp_workspace_bytes(T, hidden, inter, r, ydt) bytes, 256-byte aligned;
 * its contents need no initialisation.  Calls sharing one workspace must not
 * overlap in time (calls on one stream never do).
 */
wl_status wl_mlp_geglu_fused(const void *x, wl_proj gate, wl_proj up, wl_proj down,
                             void *y, int64_t T, int64_t hidden, int64_t inter,
                             int64_t r, void *workspace, size_t ws_bytes,
                             wl_out_dtype ydt, void *stream);

/*
 * wl_mlp_geglu_fused_noalloc -- the same fused GeGLU MLP as
 * wl_mlp_geglu_fused, for callers that cannot allocate device memory (code
 * that may not call cudaMalloc, such as a host callback, an allocator hook or
 * a process whose device-memory budget is fixed at start-up).  It takes no
 * workspace: it uses a 4 MiB scratch array built into libwl.so, which every
 * GPU that loads the library holds until the process exits.  The documentation
 * pages have no counterpart to this call; it exists for such callers.
 *   - Sizes whose workspace (wl_mlp_workspace_bytes) exceeds 4 MiB are
 *     rejected with WL_ERR_UNSUPPORTED and a message; nothing is launched.
 *   - The first call on a device looks up the scratch address for that device
 *     (make it before any stream capture on that device).
 *   - The scratch keeps whatever the previous call left; nothing in it has to
 *     start at zero.  No call allocates or frees memory.
 *   - All calls share the one scratch array: calls that overlap on the GPU
 *     (different streams, or different host threads) race and give wrong
 *     results.  Serialise them.
 */
wl_status wl_mlp_geglu_fused_noalloc(const void *x, wl_proj gate, wl_proj up, wl_proj down,
                                     void *y, int64_t T, int64_t hidden, int64_t inter,
                                     int64_t r, wl_out_dtype ydt, void *stream);

/*
 * fp32 encoding ("Serve and generate with weightless", "Supported encodings
 * and devices": the architectures default to bfloat16 and also support
 * float32).  The same projection with x, W0, s, U and V all fp32:
 *     y = s*(x W0^T) + (x V) U^T
 * computed with fp32 multiply-adds throughout (no bf16 or tf32 rounding of
 * any operand); y is fp32 or bf16 (ydt).  Layouts as above with 4-byte
 * elements: x [T,in], W0 [out,in], s [out], U [out,r], V [in,r], y [T,out].
 * Limits and errors as wl_linear; pointers 16-byte aligned except s, U, V
 * (4-byte).  Equal, within fp32 accumulation order, to the fp64 product of
 * the fp32 values.
 */
typedef struct {
    const float *W0;
    const float *s;
    const float *U;
    const float *V;
    int64_t out;
} wl_proj_f32;

wl_status wl_linear_f32(const float *x, const float *W0, const float *s, const float *U,
                        const float *V, void *y, int64_t T, int64_t in, int64_t out,
                        int64_t r, wl_out_dtype ydt, void *stream);

/* Q, K, V of one fp32 x in one launch (x read once per token tile). */
wl_status wl_qkv_fused_f32(const float *x, wl_proj_f32 q, wl_proj_f32 k, wl_proj_f32 v,
                           void *yq, void *yk, void *yv, int64_t T, int64_t in, int64_t r,
                           wl_out_dtype ydt, void *stream);

/*
 * wl_materialize -- W_eff = s*W0 + U V^T, formed once (the load-time
 * precompute of "Serve and generate with weightless", "Set the fast path on
 * NVIDIA").  W_eff [out, in] of type dt (fp32 or bf16).  Bit-exact with one
 * fixed fp32 order per element:
 *     d = +0; for k = 0..r-1: d = fma(U[o,k], V[i,k], d)
 *     w = fl(s[o] * W0[o,i]); if r > 0: w = fl(w + d)
 * then, for bf16, one round-to-nearest-even.
 */
wl_status wl_materialize(const void *W0, const float *s, const void *U, const void *V,
                         void *W_eff, int64_t out, int64_t in, int64_t r,
                         wl_out_dtype dt, void *stream);

/*
 * Decomposition of dense projection weights into theta bundles (the pages'
 * weight adapter "auto-decomposes" a checkpoint into the bundle: "Serve and
 * generate with weightless", "How the custom architecture loads").  One call
 * handles one band: the n layers of one projection family that share a W0.
 * Steps (the pages fix only the passthrough point G = num_layers, where each
 * reconstructed weight equals the original; the rest is this library's
 * reading):
 *   W0 = mean of the n weights (fp32 sum, bf16 round-to-nearest-even);
 *   s_l[o] = <W_l[o], W0[o]> / <W0[o], W0[o]> (1 where the W0 row is zero);
 *   U_l, V_l: rank-r truncated SVD of R_l = W_l - diag(s_l) W0, split evenly
 *   (U = U_r S^1/2, V = V_r S^1/2), by randomized subspace iteration from the
 *   caller's Gaussian start omega [in, r + p] fp32 with `iters` power
 *   iterations (Halko, Martinsson and Tropp 2011), then bf16.
 * With n = 1 the bundle is the passthrough one: W0 = W, s = 1, U = V = 0.
 * W: host array of n device pointers to bf16 [out, in] (16-byte aligned).
 * Outputs (device, caller-owned): W0 bf16 [out, in]; s fp32 [n, out];
 * U bf16 [n, out, r]; V bf16 [n, in, r].  workspace: at least
 * wl_decompose_workspace_bytes(out, in, r, p) bytes, 256-byte aligned.
 * Limits: 1 <= n <= 64, in % 8 == 0, 0 <= r <= min(out, in, 128),
 * 0 <= p, r + p <= 160, 0 <= iters <= 64.  Asynchronous on `stream`.
 */
size_t wl_decompose_workspace_bytes(int64_t out, int64_t in, int64_t r, int64_t p);

wl_status wl_decompose_band(const void *const *W, int64_t n, int64_t out, int64_t in, int64_t r,
                            int64_t p, int64_t iters, const float *omega, void *W0, float *s,
                            void *U, void *V, void *workspace, size_t ws_bytes, void *stream);

/*
 * Decoder-layer stacks at decode size, in one launch per step.
 *
 * A weightless decoder layer applies its projections in a chain ("Serve and
 * generate with weightless": every linear layer of the model is a theta
 * bundle; "In-kernel reconstruction", formula section, per projection):
 *     q, k, v = wl(x_l; q), wl(x_l; k), wl(x_l; v)
 *     o       = wl(q; o)                  (q stands in for attention, which
 *                                          is not part of the method)
 *     g, u    = wl(o; gate), wl(o; up);   h = gelu_tanh(g) * u
 *     x_{l+1} = wl(h; down)
 * Every output is bf16 (round-to-nearest-even of the fp32 result, as for
 * wl_linear with WL_OUT_BF16); h keeps fp32 accuracy inside the launch (it
 * enters the down projection as a bf16 pair hi + lo).  Each output of each
 * layer equals, within fp32 accumulation order, the single-projection calls
 * on that layer's bf16 inputs.  At batch 1 a launch per projection costs more than its weight
 * traffic ("What weightless inference costs": at batch-1 decode extra
 * dispatches, not extra arithmetic, dominate), so one launch streams the
 * weights of all L layers and follows the data dependencies inside it.
 */
typedef struct {
    wl_proj q, k, v, o, gate, up, down; /* gate.out == up.out == inter, o.out == down.out == hidden */
} wl_layer;

/* Output buffers of one layer, bf16 [T, n], row-major, 16-byte aligned. */
typedef struct {
    void *yq; /* [T, q.out]  */
    void *yk; /* [T, k.out]  */
    void *yv; /* [T, v.out]  */
    void *yo; /* [T, hidden] */
    void *ym; /* [T, hidden]: the layer's output and the next layer's input */
} wl_layer_out;

typedef struct wl_stack_s *wl_stack;

/*
 * wl_stack_create -- bind L layers and their output buffers (all device
 * memory owned by the caller, which must outlive the stack) into a stack for
 * T tokens on the current device.  Allocates the stack's own device tables
 * and scratch (cudaMalloc; freed by wl_stack_destroy) and uploads them
 * synchronously: call it outside stream capture.
 * Limits: 1 <= T <= 32, 0 <= r <= 32; hidden, q.out and gate.out multiples
 * of 64; every layer with the shapes of layer 0; W0 and V 16-byte aligned.
 * 1..4 tokens and 5..32 tokens run different kernels (the second reduces each
 * output row tile once and hands it on as bf16).
 * Output buffers of different layers must be distinct and may not alias any
 * input.  Sizes outside these limits give WL_ERR_UNSUPPORTED (use the
 * per-projection calls).  On error *out is NULL.
 */
wl_status wl_stack_create(wl_stack *out, const wl_layer *layers, const wl_layer_out *outs,
                          int64_t L, int64_t T, int64_t hidden, int64_t r);

/*
 * wl_stack_decode -- one pass over all layers of the stack for input x
 * [T, hidden] bf16 (device, 16-byte aligned), asynchronous on `stream`.
 * Writes every output of every layer.  Launches must not overlap: calls on
 * one stream never do.  Each step first runs a small kernel that writes V^T
 * of every projection (and, above 4 tokens, clears the step's flags).  The launch is cooperative (one CTA per SM); it
 * cannot be captured into a CUDA graph on drivers that refuse cooperative
 * launches in capture.
 */
wl_status wl_stack_decode(wl_stack stack, const void *x, void *stream);

/* Free the stack's device memory (after its last launch has completed). */
void wl_stack_destroy(wl_stack stack);

/*
 * Decoder-layer operators around the projections
 * ----------------------------------------------
 * The pages' models are decoders: between the Q/K/V and the O projection sit
 * rotary positions, a key/value cache and attention, and between the blocks
 * norms and the residual stream.  The pages leave these to the serving
 * framework; the entry points below are this library's own.
 *
 * A paged cache holds, per page, kv head and slot, one row of `dim` codes of
 * k and one of v, and one fp32 scale for each row; a value is code * scale.
 *   WL_CACHE_E4M3: 8-bit floats (4 exponent, 3 mantissa bits, no infinity);
 *     the scale is the smallest power of two 2^e, e >= -126, with
 *     max|row| <= 448 * 2^e (1 for a row of zeros).  A power of two loses
 *     nothing against max/448: the codes keep their 4 significant bits.
 *   WL_CACHE_BF16: codes are the values rounded to bf16, the scale is 1.
 *   A row with a NaN or an infinity (bf16: also one with a value that rounds to
 *     an infinity) is stored as codes 0 and scale NaN: all of it reads back as
 *     NaN, and only queries that see it become NaN.
 */
typedef enum { WL_CACHE_E4M3 = 0, WL_CACHE_BF16 = 1 } wl_cache_format;

typedef struct {
    void *k, *v;              /* [pages, kv_heads, page_size, dim], 1 or 2 bytes per code, 16-byte aligned */
    float *k_scale, *v_scale; /* [pages, kv_heads, page_size] */
    int64_t pages, kv_heads, page_size, dim;
    wl_cache_format format;
} wl_cache;

/*
 * The sequences of a call, in device memory: sequence b holds len[b] positions
 * in the cache, and the call is about its next count[b] <= n ones (count NULL:
 * n each).  Cache position j of sequence b lies in page
 * pages[b * max_pages + j / page_size], slot j % page_size.  The kernels check
 * what they read: counts are clamped to [0, n], lengths to [0, max_pages *
 * page_size]; a position past the table or with a page outside [0, cache.pages)
 * is not written, reads as zero, is seen by no query, and is reported by
 * wl_device_status() as WL_ERR_INVALID_ARG.
 */
typedef struct {
    const int32_t *pages; /* [batch, max_pages] */
    const int32_t *len;   /* [batch] */
    const int32_t *count; /* [batch] or NULL */
    int64_t batch, max_pages, n;
} wl_seqs;

/*
 * Rotary positions.  Pair i of a head turns by position * phase[i] * 2^-64
 * turns; the product wraps at one turn, so no position loses accuracy in a range
 * reduction.  The angle is then held in fp32, right to 2^-26 turn (9.4e-8
 * radian); cos and sin are multiplied by amplitude.  Pairs are
 * (i, i + rot/2), or (2i, 2i + 1) if interleaved; dims >= rot are not changed.
 */
typedef struct {
    const uint64_t *phase; /* device, [rot/2] */
    int64_t rot;           /* even, 0 <= rot <= dim; 0: no rotation */
    int32_t interleaved;
    float amplitude;
} wl_rope;

typedef enum {
    WL_ROPE_PLAIN = 0,  /* f_i = base^(-2i/rot) radians per position */
    WL_ROPE_LINEAR = 1, /* f_i / factor: positions interpolated */
    WL_ROPE_BASE = 2,   /* base * factor^(rot/(rot-2)): the slowest pair is interpolated, the fastest kept */
    WL_ROPE_RAMP = 3    /* between both, by how often a pair turns in orig_len positions: >= fast turns kept, <= slow
                           turns interpolated; amplitude 0.1 ln(factor) + 1 (the YaRN method, Peng et al. 2023) */
} wl_rope_scaling;

/*
 * wl_rope_phases -- fills phase[rot/2] and *amplitude in HOST memory (copy the
 * table to the device for wl_rope).  factor >= 1; orig_len, fast and slow are
 * read by WL_ROPE_RAMP only (orig_len >= 1, fast > slow > 0).  Host-only.
 */
wl_status wl_rope_phases(int64_t rot, double base, wl_rope_scaling scaling, double factor, double orig_len,
                         double fast, double slow, uint64_t *phase, float *amplitude);

/*
 * wl_rope_append -- what follows wl_qkv_fused, in one launch: q_out = rotated
 * q (bf16), and k (rotated) and v written to the cache at positions len[b] ..
 * len[b] + count[b] - 1, quantised from the fp32 rotated values.
 * q [batch*n, q_heads*dim], k and v [batch*n, kv_heads*dim] of type xdt (bf16
 * or fp32), token (b, i) in row b*n + i, rows q_stride, k_stride, v_stride
 * elements apart; q_out bf16 contiguous; rows i >= count[b] of q_out are zero.
 * positions [batch*n] int32: the rotary position of each token (NULL: len[b] +
 * i; a drafted tree gives len[b] + depth).  q and q_out may both be NULL: only
 * the cache is written.
 * Limits: dim a multiple of 16, 16 <= dim <= 256; strides multiples of 8;
 * q, k, v, q_out 16-byte aligned.
 */
wl_status wl_rope_append(const void *q, const void *k, const void *v, void *q_out, int64_t q_heads, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, wl_out_dtype xdt, const int32_t *positions, wl_rope rope,
                         wl_cache cache, wl_seqs seqs, void *stream);

/*
 * wl_cache_read -- k_out and v_out [batch, n, kv_heads, dim] (type dt): the
 * values at positions len[b] + i for i < count[b], zero beyond.  e4m3 values
 * are exact in either type but for over- or underflow of the type's range.
 */
wl_status wl_cache_read(wl_cache cache, wl_seqs seqs, void *k_out, void *v_out, wl_out_dtype dt, void *stream);

/*
 * wl_tree_attention -- attention of the 1 <= n <= 64 newest tokens of each
 * sequence (their k and v already in the cache at len[b] + i) over its cache:
 * token i sees the len[b] positions before them and those new tokens j with
 * bit j of mask[b*n + i] set (its ancestors and itself in a drafted tree).
 * mask NULL: token i sees new tokens 0..i, so n = 1 is plain decoding and a
 * prompt goes through in chunks of 64.  Softmax of scale * q.k in fp32; query
 * head h reads kv head h / (q_heads / kv_heads).  A token that sees nothing,
 * and rows i >= count[b], give zeros.
 *
 * Number formats.  Scores, running references and sums are fp32.  bf16 caches
 * are multiplied by q as it is and by weights of 16 bits.  e4m3 caches are
 * multiplied by pairs of e4m3 parts, which hold 8 bits:
 *   q: an element keeps all its bits down to 2^-14 of the largest of its row
 *     (2^-10 where other rows of the call are up to 16 times larger), fewer
 *     below, and is dropped below 2^-22 (2^-18).
 *   weights p * v_scale: 8 bits down to 2^-11 of the row's largest, fewer below,
 *     dropped below 2^-20.  What is dropped still counts in the softmax's sum,
 *     so a result can lose 2^-20 of the largest weight for each position: 0.8 %
 *     at most in 8192 positions, after which fp32 sums take over, and only if
 *     nearly all of them lie just below that line.
 *   rows of v of scale below 2^-104 count as if they had that scale.
 * q and out bf16 [batch, n, q_heads, dim], contiguous, 16-byte aligned.
 * workspace: wl_tree_attention_workspace_bytes(...) bytes (0 for invalid
 * sizes), 256-byte aligned, contents need no initialisation; calls that share
 * it must not overlap in time.
 */
size_t wl_tree_attention_workspace_bytes(int64_t batch, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim);

wl_status wl_tree_attention(const void *q, int64_t q_heads, const uint64_t *mask, float scale, wl_cache cache,
                            wl_seqs seqs, void *out, void *workspace, size_t ws_bytes, void *stream);

/*
 * wl_norm_residual -- what lies between two blocks, in one launch:
 *     u  = y, or rms(y) * (w_offset + w_post)      (w_post NULL: y itself)
 *     x' = alpha * x + beta * gate * u             (gate NULL: 1; y NULL: x' = alpha * x)
 *     h  = rms(x') * (w_offset + w_pre)            (h NULL: not formed)
 * with rms(a) = a / sqrt(mean(a^2) + eps), all in fp32; h takes x' before its
 * rounding to x_out.  y and gate [T, H] of type ydt (gate rows gate_stride
 * elements apart, 0: one row for all tokens), x and x_out [T, H] of type xdt
 * (x_out may be x itself; it may be NULL if y is), h [T, H] of type hdt,
 * w_post and w_pre [H] fp32.
 * Limits: T >= 1, H a multiple of 8, 8 <= H <= 16384; everything 16-byte aligned.
 */
wl_status wl_norm_residual(const void *y, const void *gate, int64_t gate_stride, const void *x, const float *w_post,
                           const float *w_pre, void *x_out, void *h, int64_t T, int64_t H, float alpha, float beta,
                           float eps, float w_offset, wl_out_dtype ydt, wl_out_dtype xdt, wl_out_dtype hdt,
                           void *stream);

/*
 * Operators between a step's last states and the next step
 * --------------------------------------------------------
 * The dense projection that no bundle covers (the vocabulary), the choice of
 * the next tokens, and the cache pages of the sequences as they grow and
 * shrink.  They launch like the decoder-layer operators (dependent launches
 * that touch no caller memory before all ahead of them is complete).
 *
 * 8-bit floats with a scale for each block of 128: a matrix [rows, in] of e4m3
 * codes (4 exponent, 3 mantissa bits, largest 448, no infinity), row-major and
 * contiguous, and fp32 scales [ceil(in/128), ceil(rows/group)]: the value at
 * (row, i) is code * scale[i/128][row/group].  group is 1 for activations (a
 * scale for 128 elements of a row) and 128 for weights (128 x 128 blocks).
 */

/*
 * wl_quant_f8 -- codes and scales of x [rows, in] (bf16 or fp32, rows x_stride
 * elements apart).  A block's scale is the smallest power of two 2^e, e >=
 * -126, with max|block| <= 448 * 2^e (1 for a block of zeros), so the division
 * is exact and only the rounding to 4 significant bits is lost; codes are
 * rounded to nearest, ties to even.  A block with a NaN or an infinity gets
 * codes 0 and scale NaN: all of it reads as NaN.
 * Limits: 1 <= rows <= 2^30; in a multiple of 16, 16 <= in <= 2^20; group 1 or
 * 128; x_stride a multiple of 8, at least in; x and codes 16-byte aligned.
 */
wl_status wl_quant_f8(const void *x, int64_t x_stride, wl_out_dtype xdt, int64_t rows, int64_t in, int64_t group,
                      void *codes, float *scales, void *stream);

/*
 * wl_linear_f8 -- y[t,o] = sum_b x_scale[b][t] w_scale[b][o/128] sum_{i in
 * block b} W[o,i] x[t,i], x [T, in] and W [out, in] e4m3 codes, x_scale
 * [ceil(in/128), T] and w_scale [ceil(in/128), ceil(out/128)] any fp32, y [T,
 * out] of type ydt.  Products of a block are summed by the tensor cores (fp32),
 * blocks are scaled and summed in fp32, and a result is rounded once.  A block is
 * scaled by the product of its two scales rounded to fp32: one past fp32's range
 * is an infinity (a block's sum of 0 times it NaN), one below 2^-126 has fewer bits.
 * Limits: 1 <= T, out <= 2^30; in a multiple of 16, 16 <= in <= 2^20; x, W and
 * y 16-byte aligned.
 */
wl_status wl_linear_f8(const void *x, const float *x_scale, const void *W, const float *w_scale, void *y, int64_t T,
                       int64_t in, int64_t out, wl_out_dtype ydt, void *stream);

/*
 * wl_verify -- which drafted tokens of each sequence hold, and the token after
 * them, from given random numbers.  Node i < count[b] <= n of sequence b (count
 * NULL: n) is a token of the last step; node 0 is known, the others are drafted:
 * mask[b*n + i] has bit j set where node j is i or an ancestor of it (as for
 * wl_tree_attention; NULL: a chain), and node i's parent is the highest node
 * below i among them.  Row b*n + i of logits [batch*n, vocab] (rows
 * logits_stride elements apart, bf16 or fp32) is the model's for the token after
 * node i.  From u = node 0 on, with weights w_i = exp((logit_i - max) / t):
 *     R = w;  for u's children c in order, token k = tokens[b*n + c], r =
 *     uniforms[b*n + c], S = sum R:
 *         accept c if  r * q_k * S < R_k:  u = c, and from the beginning;
 *         else R = max(R - S q, 0)
 * q: row b*n + u of draft [batch*n, vocab] (bf16 or fp32), the distribution
 * that u's children were drawn from; draft NULL: each child is certain, q is 1
 * at its own token.  Where no child is left, next[b] is the lowest i with R_i >
 * 0 and R_0 + ... + R_i > uniforms[b*n] * S (the last with R_i > 0 where rounding
 * leaves none); if R has no mass left, drawn from w.  So a sequence of accepted
 * tokens is distributed as the model alone would draw it.  A temperature t below
 * 1e-6 takes the most likely token, the lowest of equal ones, and accepts a
 * child if it is that one; random numbers and draft are not used.
 *     path[b*n ...]: the accepted nodes, node 0 first, then -1;  accepted[b]:
 *     how many (0 where count[b] is 0, with next[b] = -1).
 * t is temperatures[b] (device) or, where that is NULL, temperature (64 bits: 0.8 is not rounded); above 1e30 it counts as
 * 1e30, so that an infinite one leaves masks of fp32's lowest value masks.  Logits of
 * -infinity are tokens of no weight.  A row with a NaN or +infinity or with no
 * finite logit, or a t that is NaN, ends the path there with next[b] = -1.  Tokens outside
 * [0, vocab) are rejected.  Decisions are those of exact arithmetic where no
 * border lies within 2^-29 of the sum of the row's w, after rejections too.
 * Limits: 1 <= batch <= 65536, 1 <= n <= 64, 1 <= vocab <= 2^24; strides at
 * least vocab.
 */
wl_status wl_verify(const void *logits, int64_t logits_stride, wl_out_dtype ldt, const void *draft, int64_t draft_stride,
                    wl_out_dtype ddt, const int32_t *tokens, const float *uniforms, const uint64_t *mask,
                    const int32_t *count, const float *temperatures, double temperature, int64_t batch, int64_t n,
                    int64_t vocab, int32_t *path, int32_t *accepted, int32_t *next, void *stream);

/*
 * wl_page_plan -- makes each sequence's row of the page table pages [batch,
 * max_pages] fit len[b] + count[b] positions (count NULL: n each; n = 0: len[b]
 * alone): need = ceil((len + count) / page_size), at most max_pages.  held[b]
 * is how many entries of the row are in use.  Pages past need go back to the pool and
 * their entries become -1; then missing pages are taken from it, sequences in order,
 * all that a sequence is missing or none: once one goes without, those after it that
 * miss pages do too.  The pool is a stack free_pages[0 .. top-1] of at most
 * pool_pages page numbers (entries at and above top mean nothing): of the
 * pages given back by a call the first of the first sequence ends on top, and pages
 * are taken from the top, so a call that undoes the one before restores everything.
 *     room[b]: how many of the count[b] new positions have pages;
 *     slots[b*n + i] (NULL: not wanted): the cache row page * page_size + offset
 *     of position len[b] + i, i < room[b], else -1.
 * All of it is device memory, read and written when the kernels run; calls on one
 * pool must not overlap.  Lengths and counts below 0 count as 0 and counts above n
 * as n; held and top are taken as within [0, max_pages] and [0, pool_pages].
 * Limits: 1 <= batch <= 65536, n >= 0, batch * n <= 2^30, batch * max_pages <=
 * 2^30; max_pages and page_size as for wl_seqs; 1 <= pool_pages < 2^30.
 */
wl_status wl_page_plan(int32_t *free_pages, int32_t *top, int64_t pool_pages, int64_t page_size, int32_t *pages,
                       int32_t *held, const int32_t *len, const int32_t *count, int64_t batch, int64_t max_pages,
                       int64_t n, int32_t *room, int64_t *slots, void *stream);

/*
 * wl_band_of_layer -- which of the G shared W0 blocks layer `layer` of an
 * L-layer stack uses: floor(layer * G / L) (contiguous bands).  G = L is the
 * passthrough point (one W0 per layer, "Set the fast path on NVIDIA"); G = 1
 * shares one block ("What weightless inference costs", Compression).
 * Returns -1 unless 0 <= layer < L and 1 <= G <= L.  Host-only, exact.
 */
int64_t wl_band_of_layer(int64_t layer, int64_t L, int64_t G);

/*
 * wl_device_status -- synchronise `stream`, then read and clear the device
 * status word of the current device.  Returns WL_ERR_TIMEOUT if a bounded
 * wait in a kernel of this library gave up since the last read,
 * WL_ERR_INVALID_ARG if a kernel met a cache position without a valid page,
 * WL_ERR_CUDA if the synchronisation failed, else WL_OK.
 */
wl_status wl_device_status(void *stream);

/*
 * wl_selftest_wait -- diagnostic for the failure detection above (the pages
 * have no counterpart): launches on `stream` one kernel that waits, through
 * the same bounded-wait code as the projection kernels' ring stages, on a
 * barrier that nothing arrives on.  The wait gives up after its limit (4e9 SM
 * cycles, about 2 s), so the next wl_device_status(stream) returns
 * WL_ERR_TIMEOUT; the GPU context stays usable.  Returns WL_OK once launched,
 * WL_ERR_CUDA if the launch failed.
 */
wl_status wl_selftest_wait(void *stream);

/* Message for the last error on the calling thread ("" if none). */
const char *wl_last_error(void);

/* Library version string. */
const char *wl_version(void);

#ifdef __cplusplus
}
#endif

#endif /* WL_H_ */
