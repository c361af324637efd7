// rope_cache.cu -- rotary positions with the quantising cache write, and the
// cache read.
#include "cache_row.cuh"

namespace wl {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const void *q, *k, *v;
    bf16 *q_out;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *positions;
    const uint64_t *phase;
    int q_heads, rot, interleaved, width;  // width: lanes of a row, a power of two >= dim / 8
    float amplitude;
    CacheArgs c;
};

// One CTA per token.  `width` lanes share a row (one head of q, k or v), 8
// elements each.
//   angle = frac(position * phase / 2^64) turns, from the wrapped 64-bit
//   product, so no position loses accuracy in a range reduction;
//   (a, b) -> A (a cos - b sin, a sin + b cos);
//   k, v: e = row exponent of max|x|, code = e4m3(x 2^-e), scale = 2^e.
template <typename X, bool kE4M3>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a)
{
    __shared__ float2 trig[128];
    __shared__ float row_buf[kRopeThreads * 8];
    const CacheArgs &c = a.c;
    const int tok = blockIdx.x, b = tok / c.n, i = tok - b * c.n;
    const int len = seq_len(c, b);
    const bool live = i < seq_count(c, b);
    if (live && threadIdx.x < a.rot / 2) {
        const int pos = a.positions ? a.positions[tok] : len + i;
        const uint64_t turn = (uint64_t)(int64_t)pos * a.phase[threadIdx.x];
        float s, co;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // 2^-31: half turns
        trig[threadIdx.x] = make_float2(co * a.amplitude, s * a.amplitude);
    }
    __syncthreads();
    const int w = a.width, g = threadIdx.x / w, ngroups = kRopeThreads / w;
    const int e0 = (threadIdx.x % w) * 8, half = a.rot / 2;
    const bool mine = e0 < c.dim;
    float *buf = row_buf + g * w * 8;
    const int rows = a.q_heads + 2 * c.kv_heads;
    for (int r0 = 0; r0 < rows; r0 += ngroups) {
        const int r = r0 + g;
        const bool isq = r < a.q_heads, isv = r >= a.q_heads + c.kv_heads, on = r < rows && mine;
        const int h = isq ? r : (r - a.q_heads) % c.kv_heads;
        float v[8] = {};
        if (on && live) {
            const X *src = isq ? static_cast<const X *>(a.q) + tok * a.q_stride
                               : isv ? static_cast<const X *>(a.v) + tok * a.v_stride : static_cast<const X *>(a.k) + tok * a.k_stride;
            load8(src + (int64_t)h * c.dim + e0, v);
        }
        if (on) store8(buf + e0, v);
        __syncwarp();
        if (on && live && !isv) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = e0 + j;
                if (e < a.rot) {
                    const int pair = a.interleaved ? e >> 1 : (e < half ? e : e - half);
                    const bool second = a.interleaved ? (e & 1) : e >= half;
                    const int other = a.interleaved ? e ^ 1 : (second ? e - half : e + half);
                    const float2 t = trig[pair];
                    v[j] = second ? buf[other] * t.y + v[j] * t.x : v[j] * t.x - buf[other] * t.y;
                }
            }
        }
        __syncwarp();
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
        for (int d = w / 2; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (!on) continue;
        if (isq) {
            store8(a.q_out + ((int64_t)tok * a.q_heads + h) * c.dim + e0, v);
            continue;
        }
        if (!live) continue;
        const int64_t at = cache_row(c, b, h, len + i);
        if (at < 0) {
            if (e0 == 0) atomicOr(c.status, kStatusPage);
            continue;
        }
        const bool bad = amax >= 0x7f800000u;  // a NaN or an infinity in the row
        float scale = 1.0f;
        if (kE4M3 && !bad) {
            const int e = row_exponent(amax);
            scale = exp2_int(e);
            const float inv = exp2_int(-e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv;
        }
        if (bad) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            scale = __uint_as_float(0x7fc00000u);
        }
        char *codes = isv ? c.v : c.k;
        if (kE4M3)
            *reinterpret_cast<uint2 *>(codes + at * c.dim + e0) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
        else
            store8(reinterpret_cast<bf16 *>(codes) + at * c.dim + e0, v);
        if (e0 == 0) (isv ? c.v_scale : c.k_scale)[at] = scale;
    }
}

template <bool kE4M3>
static void rope_launch(const RopeArgs &a, int xdt, int64_t tokens, cudaStream_t st)
{
    if (xdt == WL_OUT_F32)
        rope_append_kernel<float, kE4M3><<<(unsigned)tokens, kRopeThreads, 0, st>>>(a);
    else
        rope_append_kernel<bf16, kE4M3><<<(unsigned)tokens, kRopeThreads, 0, st>>>(a);
}

wl_status launch_rope_append(const void *q, const void *k, const void *v, bf16 *q_out, int64_t q_heads, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, int xdt, const int32_t *positions, const wl_rope &rope,
                             const wl_cache &cache, const wl_seqs &seqs, const DeviceInfo *di, cudaStream_t st)
{
    RopeArgs a;
    a.q = q, a.k = k, a.v = v, a.q_out = q_out;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.positions = positions, a.phase = rope.phase;
    a.q_heads = (int)q_heads, a.rot = (int)rope.rot, a.interleaved = rope.interleaved, a.amplitude = rope.amplitude;
    a.c = cache_args(cache, seqs, di->status);
    a.width = 2;
    while (a.width * 8 < a.c.dim) a.width *= 2;
    if (cache.format == WL_CACHE_E4M3)
        rope_launch<true>(a, xdt, seqs.batch * seqs.n, st);
    else
        rope_launch<false>(a, xdt, seqs.batch * seqs.n, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_rope_append launch");
}

// ------------------------------------------------------------------ read --
// A thread decodes 16 consecutive codes of one row of k or v (blockIdx.y).
template <typename Y, bool kE4M3>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheArgs c, Y *k_out, Y *v_out)
{
    const int chunks = c.dim / 16;
    const int64_t items = (int64_t)c.batch * c.n * c.kv_heads * chunks;
    const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (it >= items) return;
    const int ch = (int)(it % chunks);
    const int64_t row = it / chunks;
    const int h = (int)(row % c.kv_heads);
    const int64_t tok = row / c.kv_heads;
    const int b = (int)(tok / c.n), i = (int)(tok % c.n);
    Y *out = (blockIdx.y ? v_out : k_out) + row * c.dim + ch * 16;
    float v[16] = {};
    if (i < seq_count(c, b)) {
        const int64_t at = cache_row(c, b, h, seq_len(c, b) + i);
        if (at < 0) {
            if (ch == 0) atomicOr(c.status, kStatusPage);
        } else {
            const float scale = (blockIdx.y ? c.v_scale : c.k_scale)[at];
            const char *src = (blockIdx.y ? c.v : c.k) + (at * c.dim + ch * 16) * (kE4M3 ? 1 : 2);
            if (kE4M3) {
                const uint4 u = *reinterpret_cast<const uint4 *>(src);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = e4m3x2_f32((w[j / 2] >> (16 * (j & 1))) & 0xffffu);
                    v[2 * j] = f.x;
                    v[2 * j + 1] = f.y;
                }
            } else {
                load8(reinterpret_cast<const bf16 *>(src), v);
                load8(reinterpret_cast<const bf16 *>(src) + 8, v + 8);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= scale;
        }
    }
    store8(out, v);
    store8(out + 8, v + 8);
}

wl_status launch_cache_read(const wl_cache &cache, const wl_seqs &seqs, void *k_out, void *v_out, int dt,
                            const DeviceInfo *di, cudaStream_t st)
{
    const CacheArgs c = cache_args(cache, seqs, di->status);
    const int64_t items = seqs.batch * seqs.n * cache.kv_heads * (cache.dim / 16);
    if ((items + 255) / 256 > 0x7fffffff) return fail(WL_ERR_UNSUPPORTED, "wl_cache_read: too many elements for one call");
    const dim3 grid((unsigned)((items + 255) / 256), 2);
    const bool e4 = cache.format == WL_CACHE_E4M3;
    if (dt == WL_OUT_F32) {
        float *ko = static_cast<float *>(k_out), *vo = static_cast<float *>(v_out);
        e4 ? cache_read_kernel<float, true><<<grid, 256, 0, st>>>(c, ko, vo) : cache_read_kernel<float, false><<<grid, 256, 0, st>>>(c, ko, vo);
    } else {
        bf16 *ko = static_cast<bf16 *>(k_out), *vo = static_cast<bf16 *>(v_out);
        e4 ? cache_read_kernel<bf16, true><<<grid, 256, 0, st>>>(c, ko, vo) : cache_read_kernel<bf16, false><<<grid, 256, 0, st>>>(c, ko, vo);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_cache_read launch");
}

}  // namespace wl
