// step_api.cu -- the C ABI of the operators between a step's last states and
// the next step: argument checks and dispatch (8-bit quantiser and product,
// verification of drafted tokens, page plan).
#include <math.h>

#include "wl_internal.cuh"

using namespace wl;

static bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static constexpr int64_t kMaxCount = (int64_t)1 << 30;
static constexpr int64_t kMaxBatch = (int64_t)1 << 16;
static constexpr int64_t kMaxIn = (int64_t)1 << 20;
static constexpr int64_t kMaxVocab = (int64_t)1 << 24;

static bool known(int dt) { return dt == WL_OUT_BF16 || dt == WL_OUT_F32; }

extern "C" {

wl_status wl_quant_f8(const void *x, int64_t x_stride, wl_out_dtype xdt, int64_t rows, int64_t in, int64_t group,
                      void *codes, float *scales, void *stream)
{
    clear_error();
    if (!known(xdt)) return fail(WL_ERR_INVALID_ARG, "unknown dtype %d", (int)xdt);
    if (rows < 1 || rows > kMaxCount) return fail(WL_ERR_INVALID_ARG, "rows must be in [1, 2^30], got %lld", (long long)rows);
    if (in < 16 || in > kMaxIn || in % 16)
        return fail(WL_ERR_INVALID_ARG, "in must be a multiple of 16 in [16, 2^20], got %lld", (long long)in);
    if (group != 1 && group != 128) return fail(WL_ERR_INVALID_ARG, "group must be 1 or 128, got %lld", (long long)group);
    if (x_stride % 8 || x_stride < in) return fail(WL_ERR_INVALID_ARG, "x_stride must be a multiple of 8 and at least in");
    if (!x || !codes || !scales) return fail(WL_ERR_INVALID_ARG, "x, codes and scales must not be NULL");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(WL_ERR_INVALID_ARG, "x and codes must be 16-byte aligned, scales 4-byte");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    return launch_quant_f8(x, x_stride, xdt, rows, in, group, static_cast<uint8_t *>(codes), scales, di,
                           static_cast<cudaStream_t>(stream));
}

wl_status wl_linear_f8(const void *x, const float *x_scale, const void *W, const float *w_scale, void *y, int64_t T,
                       int64_t in, int64_t out, wl_out_dtype ydt, void *stream)
{
    clear_error();
    if (!known(ydt)) return fail(WL_ERR_INVALID_ARG, "unknown dtype %d", (int)ydt);
    if (T < 1 || T > kMaxCount) return fail(WL_ERR_INVALID_ARG, "T must be in [1, 2^30], got %lld", (long long)T);
    if (out < 1 || out > kMaxCount) return fail(WL_ERR_INVALID_ARG, "out must be in [1, 2^30], got %lld", (long long)out);
    if (in < 16 || in > kMaxIn || in % 16)
        return fail(WL_ERR_INVALID_ARG, "in must be a multiple of 16 in [16, 2^20], got %lld", (long long)in);
    if (!x || !x_scale || !W || !w_scale || !y) return fail(WL_ERR_INVALID_ARG, "x, W, their scales and y must not be NULL");
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
        return fail(WL_ERR_INVALID_ARG, "x, W and y must be 16-byte aligned, scales 4-byte");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    return launch_linear_f8(static_cast<const uint8_t *>(x), x_scale, static_cast<const uint8_t *>(W), w_scale, y, T, in, out,
                            ydt, di, static_cast<cudaStream_t>(stream));
}

wl_status wl_verify(const void *logits, int64_t logits_stride, wl_out_dtype ldt, const void *draft, int64_t draft_stride,
                    wl_out_dtype ddt, const int32_t *tokens, const float *uniforms, const uint64_t *mask,
                    const int32_t *count, const float *temperatures, double temperature, int64_t batch, int64_t n,
                    int64_t vocab, int32_t *path, int32_t *accepted, int32_t *next, void *stream)
{
    clear_error();
    if (!known(ldt) || !known(ddt)) return fail(WL_ERR_INVALID_ARG, "unknown dtype %d", known(ldt) ? (int)ddt : (int)ldt);
    if (batch < 1 || batch > kMaxBatch) return fail(WL_ERR_INVALID_ARG, "batch must be in [1, 65536], got %lld", (long long)batch);
    if (n < 1 || n > kMaxTree) return fail(WL_ERR_INVALID_ARG, "n must be in [1, %d], got %lld", kMaxTree, (long long)n);
    if (vocab < 1 || vocab > kMaxVocab) return fail(WL_ERR_INVALID_ARG, "vocab must be in [1, 2^24], got %lld", (long long)vocab);
    if (!logits || !tokens || !uniforms || !path || !accepted || !next)
        return fail(WL_ERR_INVALID_ARG, "logits, tokens, uniforms and the outputs must not be NULL");
    if (logits_stride < vocab || (draft && draft_stride < vocab))
        return fail(WL_ERR_INVALID_ARG, "logits_stride and draft_stride must be at least vocab");
    if (!aligned(logits, ldt == WL_OUT_F32 ? 4 : 2) || !aligned(draft, ddt == WL_OUT_F32 ? 4 : 2))
        return fail(WL_ERR_INVALID_ARG, "logits and draft must be aligned to their elements");
    if (!aligned(tokens, 4) || !aligned(uniforms, 4) || !aligned(mask, 8) || !aligned(count, 4) || !aligned(temperatures, 4) ||
        !aligned(path, 4) || !aligned(accepted, 4) || !aligned(next, 4))
        return fail(WL_ERR_INVALID_ARG, "mask must be 8-byte aligned, the other small tensors 4-byte");
    if (!temperatures && (!(temperature >= 0.0) || !isfinite(temperature)))
        return fail(WL_ERR_INVALID_ARG, "temperature must be finite and >= 0");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    const VerifyArgs a{logits, draft, logits_stride, draft_stride, tokens, uniforms, mask, count, temperatures, temperature,
                       (int)batch, (int)n, (int)vocab, path, accepted, next};
    return launch_verify(a, ldt, ddt, di, static_cast<cudaStream_t>(stream));
}

wl_status wl_page_plan(int32_t *free_pages, int32_t *top, int64_t pool_pages, int64_t page_size, int32_t *pages,
                       int32_t *held, const int32_t *len, const int32_t *count, int64_t batch, int64_t max_pages,
                       int64_t n, int32_t *room, int64_t *slots, void *stream)
{
    clear_error();
    if (pool_pages < 1 || pool_pages >= kMaxCount || page_size < 1 || page_size > (1 << 20))
        return fail(WL_ERR_INVALID_ARG, "need 1 <= pool_pages < 2^30 and 1 <= page_size <= 2^20");
    if (batch < 1 || batch > kMaxBatch) return fail(WL_ERR_INVALID_ARG, "batch must be in [1, 65536], got %lld", (long long)batch);
    if (n < 0 || n > kMaxCount || batch * n > kMaxCount)
        return fail(WL_ERR_INVALID_ARG, "n must be >= 0 and batch * n <= 2^30, got n = %lld", (long long)n);
    if (max_pages < 1 || max_pages > kMaxCount || max_pages * page_size > kMaxCount)
        return fail(WL_ERR_INVALID_ARG, "max_pages must be >= 1 and max_pages * page_size <= 2^30");
    if (batch * max_pages > kMaxCount) return fail(WL_ERR_INVALID_ARG, "batch * max_pages must be <= 2^30");
    if (!free_pages || !top || !pages || !held || !len || !room)
        return fail(WL_ERR_INVALID_ARG, "the pool, pages, held, len and room must not be NULL");
    if (!aligned(free_pages, 4) || !aligned(top, 4) || !aligned(pages, 4) || !aligned(held, 4) || !aligned(len, 4) ||
        !aligned(count, 4) || !aligned(room, 4) || !aligned(slots, 8))
        return fail(WL_ERR_INVALID_ARG, "slots must be 8-byte aligned, the other tensors 4-byte");
    wl_status st = WL_OK;
    const DeviceInfo *di = device_info(&st);
    if (!di) return st;
    const PlanArgs a{free_pages, top, pages, held, len, count, room, slots, (int)pool_pages, (int)page_size, (int)batch,
                     (int)max_pages, (int)n};
    return launch_page_plan(a, di, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
