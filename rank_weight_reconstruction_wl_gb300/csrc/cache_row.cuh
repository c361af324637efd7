// cache_row.cuh -- device helpers shared by the kernels that write, read and
// attend over a paged cache: where a position lives, how a row is coded.
#pragma once

#include <cuda_fp8.h>

#include <utility>

#include "wl_internal.cuh"

namespace wl {

// x / d for 0 <= x < 2^31 by a multiplication: with 2^L >= d the smallest,
// umulhi(2 x, floor(2^(31 + L) / d) + 1) >> L is exact (Granlund and
// Montgomery 1994).
struct FastDiv {
    uint32_t d, mul, shr;
    __device__ __forceinline__ int div(int x) const { return (int)(__umulhi((uint32_t)x << 1, mul) >> shr); }
};

inline FastDiv fast_div(int64_t d)
{
    FastDiv f;
    f.d = (uint32_t)d;
    f.shr = 0;
    while (((int64_t)1 << f.shr) < d) ++f.shr;
    f.mul = (uint32_t)(((uint64_t)1 << (31 + f.shr)) / (uint64_t)d + 1);
    return f;
}

// wl_cache and wl_seqs as the kernels take them.
struct CacheArgs {
    char *k, *v;
    float *k_scale, *v_scale;
    const int32_t *pages, *len, *count;
    int64_t npages;
    int kv_heads, page_size, page_shift, dim, batch, n, max_pages;  // page_shift: log2(page_size), -1 where it is none
    unsigned *status;
};

inline CacheArgs cache_args(const wl_cache &c, const wl_seqs &s, unsigned *status)
{
    CacheArgs a;
    a.k = static_cast<char *>(c.k);
    a.v = static_cast<char *>(c.v);
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.pages = s.pages;
    a.len = s.len;
    a.count = s.count;
    a.npages = c.pages;
    a.kv_heads = (int)c.kv_heads;
    a.page_size = (int)c.page_size;
    a.page_shift = -1;
    for (int b = 0; b < 31; ++b)
        if (c.page_size == ((int64_t)1 << b)) a.page_shift = b;
    a.dim = (int)c.dim;
    a.batch = (int)s.batch;
    a.n = (int)s.n;
    a.max_pages = (int)s.max_pages;
    a.status = status;
    return a;
}

// Length and count of a sequence, clamped to what the table can hold.
__device__ __forceinline__ int seq_len(const CacheArgs &a, int b)
{
    return min(max(__ldg(a.len + b), 0), a.max_pages * a.page_size);
}
__device__ __forceinline__ int seq_count(const CacheArgs &a, int b)
{
    return a.count ? min(max(__ldg(a.count + b), 0), a.n) : a.n;
}

// Row index (of the codes' [dim] rows and of the scales) of position j of
// sequence b, head h; -1 where the table or its entry does not cover j.
__device__ __forceinline__ int64_t cache_row(const CacheArgs &a, int b, int h, int j)
{
    const int p = a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size;
    const int slot = a.page_shift >= 0 ? j & (a.page_size - 1) : j - p * a.page_size;
    if (p >= a.max_pages) return -1;
    const int page = __ldg(a.pages + (int64_t)b * a.max_pages + p);
    if (page < 0 || page >= a.npages) return -1;
    return ((int64_t)page * a.kv_heads + h) * a.page_size + slot;
}

// Exponent e of an e4m3 row's scale 2^e: the smallest e >= -126 with
// amax <= 448 * 2^e = 1.75 * 2^(e + 8).  amax_bits: bits of a positive finite
// fp32 number (0: e = 0, any scale holds a row of zeros).
__device__ __forceinline__ int row_exponent(uint32_t amax_bits)
{
    if (amax_bits == 0) return 0;
    const int k = (int)(amax_bits >> 23) - 127;  // subnormals: -127, clamped below
    return max((amax_bits & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7, -126);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Two e4m3 codes as fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 consecutive elements (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const bf16 *p, float v[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf_lo(w[i]);
        v[2 * i + 1] = bf_hi(w[i]);
    }
}
__device__ __forceinline__ void load8(const float *p, float v[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(bf16 *p, const float v[8])
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float v[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A launch that may begin while the kernel before it on the stream finishes:
// its blocks set themselves up and call pdl_wait() before they touch memory
// that others write.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A &&...args)
{
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace wl
