// tree_attention.cu -- attention of a tree of new tokens over a paged cache.
#include "cache_row.cuh"

namespace wl {

constexpr int kTaThreads = 128;

struct TaArgs {
    const bf16 *q;
    const uint64_t *mask;
    bf16 *out;
    int q_heads;
    float scale;
    CacheArgs c;
};

// One CTA per (query head, token): softmax with a running maximum over tiles
// of 128 positions, one position per thread for the scores, two dims per
// thread for the output.
template <bool kE4M3>
__global__ void __launch_bounds__(kTaThreads) tree_attention_kernel(const __grid_constant__ TaArgs a)
{
    __shared__ float sq[256], sp[kTaThreads], red[4];
    __shared__ int64_t srow[kTaThreads];
    const CacheArgs &c = a.c;
    const int h = blockIdx.x, tok = blockIdx.y, b = tok / c.n, i = tok - b * c.n, t = threadIdx.x;
    const int len = seq_len(c, b), cnt = seq_count(c, b);
    const int hk = h / (a.q_heads / c.kv_heads);
    const int64_t o = ((int64_t)tok * a.q_heads + h) * c.dim;
    const uint64_t m = a.mask ? a.mask[tok] : (i >= 63 ? ~0ull : (2ull << i) - 1);
    for (int d = t; d < c.dim; d += kTaThreads) sq[d] = bf2f(a.q[o + d]);
    __syncthreads();
    const int total = i < cnt ? len + cnt : 0;
    float top = -3.0e38f, sum = 0.0f, acc0 = 0.0f, acc1 = 0.0f;
    for (int j0 = 0; j0 < total; j0 += kTaThreads) {
        const int j = j0 + t;
        float s = -INFINITY;
        int64_t row = -1;
        if (j < total && (j < len || ((m >> (j - len)) & 1))) {
            row = cache_row(c, b, hk, j);
            if (row < 0) {
                atomicOr(c.status, kStatusPage);
            } else {
                float dot = 0.0f;
                if (kE4M3) {
                    const char *k = c.k + row * c.dim;
                    for (int d = 0; d < c.dim; d += 4) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(k + d);
                        const float2 f = e4m3x2_f32(w & 0xffffu), g = e4m3x2_f32(w >> 16);
                        dot += f.x * sq[d] + f.y * sq[d + 1] + g.x * sq[d + 2] + g.y * sq[d + 3];
                    }
                } else {
                    const bf16 *k = reinterpret_cast<const bf16 *>(c.k) + row * c.dim;
                    for (int d = 0; d < c.dim; ++d) dot += bf2f(k[d]) * sq[d];
                }
                s = dot * c.k_scale[row] * a.scale;
            }
        }
        float mx = s;
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (t % 32 == 0) red[t / 32] = mx;
        __syncthreads();
        const float now = fmaxf(top, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float f = expf(top - now);
        top = now;
        sp[t] = row < 0 ? 0.0f : expf(s - now);
        srow[t] = row;
        __syncthreads();
        sum *= f, acc0 *= f, acc1 *= f;
        for (int u = 0; u < kTaThreads; ++u) {
            if (srow[u] < 0) continue;
            sum += sp[u];
            const float p = sp[u] * c.v_scale[srow[u]];
            const int64_t r = srow[u] * c.dim;
            if (t < c.dim) acc0 += p * (kE4M3 ? e4m3x2_f32((uint8_t)c.v[r + t]).x : bf2f(reinterpret_cast<const bf16 *>(c.v)[r + t]));
            if (t + 128 < c.dim) acc1 += p * (kE4M3 ? e4m3x2_f32((uint8_t)c.v[r + t + 128]).x : bf2f(reinterpret_cast<const bf16 *>(c.v)[r + t + 128]));
        }
        __syncthreads();
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (t < c.dim) a.out[o + t] = __float2bfloat16_rn(acc0 * inv);
    if (t + 128 < c.dim) a.out[o + t + 128] = __float2bfloat16_rn(acc1 * inv);
}

size_t tree_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 256; }

wl_status launch_tree_attention(const bf16 *q, int64_t q_heads, const uint64_t *mask, float scale, const wl_cache &cache,
                                const wl_seqs &seqs, bf16 *out, void *, const DeviceInfo *di, cudaStream_t st)
{
    TaArgs a{q, mask, out, (int)q_heads, scale, cache_args(cache, seqs, di->status)};
    if (seqs.batch * seqs.n > 65535) return fail(WL_ERR_UNSUPPORTED, "wl_tree_attention: batch * n must be at most 65535");
    const dim3 grid((unsigned)q_heads, (unsigned)(seqs.batch * seqs.n));
    if (cache.format == WL_CACHE_E4M3)
        tree_attention_kernel<true><<<grid, kTaThreads, 0, st>>>(a);
    else
        tree_attention_kernel<false><<<grid, kTaThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_tree_attention launch");
}

}  // namespace wl
