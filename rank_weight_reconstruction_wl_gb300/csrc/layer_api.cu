// layer_api.cu -- the C ABI of the decoder-layer operators: argument checks
// and dispatch (rotary append to a paged cache, cache read, tree attention,
// norm and residual), and the host-side rotary table.
#include <math.h>

#include "wl_internal.cuh"

using namespace wl;

#define WL_TRY(expr)                    \
    do {                                \
        wl_status _s = (expr);          \
        if (_s != WL_OK) return _s;     \
    } while (0)

static bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static constexpr int64_t kMaxCount = (int64_t)1 << 30;
static constexpr int64_t kMaxBatch = (int64_t)1 << 16;

static wl_status check_dtype(int dt)
{
    if (dt != WL_OUT_BF16 && dt != WL_OUT_F32) return fail(WL_ERR_INVALID_ARG, "unknown dtype %d", dt);
    return WL_OK;
}

static wl_status check_cache(const wl_cache &c)
{
    if (c.format != WL_CACHE_E4M3 && c.format != WL_CACHE_BF16)
        return fail(WL_ERR_INVALID_ARG, "unknown cache format %d", (int)c.format);
    if (c.dim < 16 || c.dim > 256 || c.dim % 16)
        return fail(WL_ERR_INVALID_ARG, "dim must be a multiple of 16 in [16, 256], got %lld", (long long)c.dim);
    if (c.pages < 1 || c.pages >= kMaxCount || c.page_size < 1 || c.page_size > (1 << 20))
        return fail(WL_ERR_INVALID_ARG, "cache: need 1 <= pages < 2^30 and 1 <= page_size <= 2^20");
    if (c.kv_heads < 1 || c.kv_heads > 4096) return fail(WL_ERR_INVALID_ARG, "kv_heads must be in [1, 4096]");
    if (!c.k || !c.v || !c.k_scale || !c.v_scale) return fail(WL_ERR_INVALID_ARG, "cache: k, v and scales must not be NULL");
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
        return fail(WL_ERR_INVALID_ARG, "cache: k and v must be 16-byte aligned, scales 4-byte");
    return WL_OK;
}

static wl_status check_seqs(const wl_seqs &s, int64_t page_size)
{
    if (s.batch < 1 || s.batch > kMaxBatch) return fail(WL_ERR_INVALID_ARG, "batch must be in [1, 65536], got %lld", (long long)s.batch);
    if (s.n < 1 || s.n > kMaxCount || s.batch * s.n > kMaxCount)
        return fail(WL_ERR_INVALID_ARG, "n must be >= 1 and batch * n <= 2^30, got n = %lld", (long long)s.n);
    if (s.max_pages < 1 || s.max_pages * page_size > kMaxCount)
        return fail(WL_ERR_INVALID_ARG, "max_pages must be >= 1 and max_pages * page_size <= 2^30");
    if (!s.pages || !s.len) return fail(WL_ERR_INVALID_ARG, "pages and len must not be NULL");
    if (!aligned(s.pages, 4) || !aligned(s.len, 4) || !aligned(s.count, 4))
        return fail(WL_ERR_INVALID_ARG, "pages, len and count must be 4-byte aligned");
    return WL_OK;
}

static wl_status check_heads(int64_t q_heads, int64_t kv_heads)
{
    if (q_heads < 1 || q_heads > 4096 || q_heads % kv_heads)
        return fail(WL_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads in [1, 4096], got %lld", (long long)q_heads);
    return WL_OK;
}

extern "C" {

wl_status wl_rope_phases(int64_t rot, double base, wl_rope_scaling scaling, double factor, double orig_len, double fast,
                         double slow, uint64_t *phase, float *amplitude)
{
    clear_error();
    if (rot < 0 || rot > 256 || rot % 2) return fail(WL_ERR_INVALID_ARG, "rot must be even and in [0, 256], got %lld", (long long)rot);
    if (!(base > 1.0) || !isfinite(base)) return fail(WL_ERR_INVALID_ARG, "base must be finite and > 1");
    if (scaling < WL_ROPE_PLAIN || scaling > WL_ROPE_RAMP) return fail(WL_ERR_INVALID_ARG, "unknown rotary scaling %d", (int)scaling);
    if (scaling != WL_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return fail(WL_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (scaling == WL_ROPE_RAMP && (!(orig_len >= 1.0) || !isfinite(orig_len) || !(slow > 0.0) || !(fast > slow) || !isfinite(fast)))
        return fail(WL_ERR_INVALID_ARG, "the ramp needs orig_len >= 1 and fast > slow > 0");
    if ((rot > 0 && !phase) || !amplitude) return fail(WL_ERR_INVALID_ARG, "phase and amplitude must not be NULL");
    const double two_pi = 6.283185307179586476925;
    if (scaling == WL_ROPE_BASE && rot > 2) base *= pow(factor, (double)rot / (double)(rot - 2));
    double lo = 0.0, hi = 1.0;
    if (scaling == WL_ROPE_RAMP) {
        // the pair that turns t times in orig_len positions: i = rot ln(orig_len / (2 pi t)) / (2 ln base)
        lo = fmax(0.0, floor(rot * log(orig_len / (fast * two_pi)) / (2.0 * log(base))));
        hi = fmin(rot - 1.0, ceil(rot * log(orig_len / (slow * two_pi)) / (2.0 * log(base))));
        if (hi <= lo) hi = lo + 0.001;
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * (double)i / (double)rot);
        if (scaling == WL_ROPE_LINEAR) f /= factor;
        if (scaling == WL_ROPE_RAMP) {
            const double keep = 1.0 - fmin(1.0, fmax(0.0, ((double)i - lo) / (hi - lo)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        // f <= 1 radian per position: under 2^62 in units of 2^-64 turn
        phase[i] = (uint64_t)nearbyint(ldexp(f / two_pi, 64));
    }
    *amplitude = scaling == WL_ROPE_RAMP ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return WL_OK;
}

wl_status wl_rope_append(const void *q, const void *k, const void *v, void *q_out, int64_t q_heads, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, wl_out_dtype xdt, const int32_t *positions, wl_rope rope,
                         wl_cache cache, wl_seqs seqs, void *stream)
{
    clear_error();
    WL_TRY(check_cache(cache));
    WL_TRY(check_seqs(seqs, cache.page_size));
    WL_TRY(check_dtype(xdt));
    if ((q == nullptr) != (q_out == nullptr)) return fail(WL_ERR_INVALID_ARG, "q and q_out must both be given or both be NULL");
    if (!k || !v) return fail(WL_ERR_INVALID_ARG, "k and v must not be NULL");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
        return fail(WL_ERR_INVALID_ARG, "q, k, v and q_out must be 16-byte aligned");
    if (!aligned(positions, 4)) return fail(WL_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    const int64_t kvw = cache.kv_heads * cache.dim;
    if (q) {
        WL_TRY(check_heads(q_heads, cache.kv_heads));
        if (q_stride % 8 || q_stride < q_heads * cache.dim)
            return fail(WL_ERR_INVALID_ARG, "q_stride must be a multiple of 8 and at least q_heads * dim");
    }
    if (k_stride % 8 || v_stride % 8 || k_stride < kvw || v_stride < kvw)
        return fail(WL_ERR_INVALID_ARG, "k_stride and v_stride must be multiples of 8 and at least kv_heads * dim");
    if (rope.rot < 0 || rope.rot > cache.dim || rope.rot % 2)
        return fail(WL_ERR_INVALID_ARG, "rot must be even and in [0, dim], got %lld", (long long)rope.rot);
    if (rope.rot > 0 && (!rope.phase || !aligned(rope.phase, 8)))
        return fail(WL_ERR_INVALID_ARG, "phase must be non-NULL and 8-byte aligned when rot > 0");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    return launch_rope_append(q, k, v, static_cast<bf16 *>(q_out), q ? q_heads : 0, q_stride, k_stride, v_stride, xdt,
                              positions, rope, cache, seqs, di, static_cast<cudaStream_t>(stream));
}

wl_status wl_cache_read(wl_cache cache, wl_seqs seqs, void *k_out, void *v_out, wl_out_dtype dt, void *stream)
{
    clear_error();
    WL_TRY(check_cache(cache));
    WL_TRY(check_seqs(seqs, cache.page_size));
    WL_TRY(check_dtype(dt));
    if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(WL_ERR_INVALID_ARG, "k_out and v_out must be non-NULL and 16-byte aligned");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    return launch_cache_read(cache, seqs, k_out, v_out, dt, di, static_cast<cudaStream_t>(stream));
}

size_t wl_tree_attention_workspace_bytes(int64_t batch, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim)
{
    if (batch < 1 || batch > kMaxBatch || n < 1 || n > kMaxTree || kv_heads < 1 || kv_heads > 4096 || q_heads < 1 ||
        q_heads > 4096 || q_heads % kv_heads || dim < 16 || dim > 256 || dim % 16)
        return 0;
    return tree_attention_workspace_bytes(batch, n, q_heads, kv_heads, dim);
}

wl_status wl_tree_attention(const void *q, int64_t q_heads, const uint64_t *mask, float scale, wl_cache cache,
                            wl_seqs seqs, void *out, void *workspace, size_t ws_bytes, void *stream)
{
    clear_error();
    WL_TRY(check_cache(cache));
    WL_TRY(check_seqs(seqs, cache.page_size));
    WL_TRY(check_heads(q_heads, cache.kv_heads));
    if (seqs.n > kMaxTree) return fail(WL_ERR_INVALID_ARG, "n must be in [1, %d], got %lld", kMaxTree, (long long)seqs.n);
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
        return fail(WL_ERR_INVALID_ARG, "q and out must be non-NULL and 16-byte aligned");
    if (!aligned(mask, 8)) return fail(WL_ERR_INVALID_ARG, "mask must be 8-byte aligned");
    if (!isfinite(scale)) return fail(WL_ERR_INVALID_ARG, "scale must be finite");
    const size_t need = tree_attention_workspace_bytes(seqs.batch, seqs.n, q_heads, cache.kv_heads, cache.dim);
    if (!workspace || !aligned(workspace, 256))
        return fail(WL_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
    if (ws_bytes < need) return fail(WL_ERR_WORKSPACE, "workspace too small: %zu bytes, need %zu", ws_bytes, need);
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    return launch_tree_attention(static_cast<const bf16 *>(q), q_heads, mask, scale, cache, seqs, static_cast<bf16 *>(out),
                                 workspace, di, static_cast<cudaStream_t>(stream));
}

wl_status wl_norm_residual(const void *y, const void *gate, int64_t gate_stride, const void *x, const float *w_post,
                           const float *w_pre, void *x_out, void *h, int64_t T, int64_t H, float alpha, float beta,
                           float eps, float w_offset, wl_out_dtype ydt, wl_out_dtype xdt, wl_out_dtype hdt, void *stream)
{
    clear_error();
    if (T < 1 || T > kMaxCount) return fail(WL_ERR_INVALID_ARG, "T must be in [1, 2^30], got %lld", (long long)T);
    if (H < 8 || H > 16384 || H % 8) return fail(WL_ERR_INVALID_ARG, "H must be a multiple of 8 in [8, 16384], got %lld", (long long)H);
    WL_TRY(check_dtype(ydt));
    WL_TRY(check_dtype(xdt));
    WL_TRY(check_dtype(hdt));
    if (!x) return fail(WL_ERR_INVALID_ARG, "x must not be NULL");
    if (y && !x_out) return fail(WL_ERR_INVALID_ARG, "x_out must not be NULL when y is given");
    if (!y && (gate || w_post)) return fail(WL_ERR_INVALID_ARG, "gate and w_post need y");
    if (!x_out && !h) return fail(WL_ERR_INVALID_ARG, "x_out and h must not both be NULL");
    if (h && !w_pre) return fail(WL_ERR_INVALID_ARG, "h needs w_pre");
    if (gate && gate_stride != 0 && (gate_stride < H || gate_stride % 8))
        return fail(WL_ERR_INVALID_ARG, "gate_stride must be 0, or a multiple of 8 and at least H");
    if (!aligned(y, 16) || !aligned(gate, 16) || !aligned(x, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
        !aligned(x_out, 16) || !aligned(h, 16))
        return fail(WL_ERR_INVALID_ARG, "all pointers must be 16-byte aligned");
    if (!(eps >= 0.0f) || !isfinite(eps)) return fail(WL_ERR_INVALID_ARG, "eps must be finite and >= 0");
    wl_status st = WL_OK;
    if (!device_info(&st)) return st;
    return launch_norm_residual(y, gate, gate_stride, x, w_post, w_pre, x_out, h, T, H, alpha, beta, eps, w_offset, ydt, xdt,
                                hdt, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
