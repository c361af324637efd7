// norm_residual.cu -- norm after a block, gate, residual update and norm
// before the next block, in one pass over the row.
//
//     u  = y  or  y / rms(y) * (w_offset + w_post)
//     x' = alpha x + beta gate u
//     h  = x' / rms(x') * (w_offset + w_pre),   rms(a) = sqrt(mean a^2 + eps)
//
// One CTA per token.  The row stays in registers between the two sums of
// squares, so y and x are read once and x' and h written once.  Sums of squares
// and the row are fp32; a row is rounded once, where it is stored.  Bound by
// DRAM bytes: 4096 tokens of 5376, y and h bf16, x fp32: 48 us, 5.5 TB/s.
#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace wl {

struct NormArgs {
    const void *y, *gate, *x;
    const float *w_post, *w_pre;
    void *x_out, *h;
    int64_t gate_stride;
    int H;
    float alpha, beta, eps, w_offset;
};

// Sum over the CTA; every thread gets the same value (fixed order).
__device__ __forceinline__ float block_sum(float v, float *red)
{
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
    return s;
}

// 8 elements as loaded.
template <typename T>
struct Chunk8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);  // coherent: x_out may be x
    }
    __device__ __forceinline__ float operator[](int j) const
    {
        const uint4 &q = w[sizeof(T) == 4 ? j / 4 : 0];
        const int k = sizeof(T) == 4 ? j % 4 : j / 2;
        const uint32_t u = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
        return sizeof(T) == 4 ? __uint_as_float(u) : (j & 1) ? bf_hi(u) : bf_lo(u);
    }
};

// V: chunks of 8 elements per thread, kept as loaded until they are used, so
// that several rows fit an SM's registers and their loads overlap.
template <typename Y, typename X, typename O, int V>
__global__ void __launch_bounds__(V == 1 ? 256 : V == 2 ? 384 : 256) norm_residual_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float red[2][32];
    pdl_wait();
    pdl_trigger();  // only now: a kernel after this one may rely on all before it
    const int nchunk = a.H / 8;
    const int64_t row = (int64_t)blockIdx.x * a.H;
    Chunk8<Y> y[V];
    Chunk8<X> xr[V];
    float x[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunk) {
            if (a.y) y[i].load(static_cast<const Y *>(a.y) + row + c * 8);
            xr[i].load(static_cast<const X *>(a.x) + row + c * 8);
        }
    }
    float f = a.beta;
    if (a.y && a.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (threadIdx.x + i * blockDim.x < nchunk)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
        f *= rsqrtf(block_sum(ss, red[0]) / (float)a.H + a.eps);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunk) {
            if (a.y) {
                float m[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) m[j] = f * y[i][j];
                if (a.w_post) {
                    float w[8];
                    load8(a.w_post + c * 8, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) m[j] *= a.w_offset + w[j];
                }
                if (a.gate) {
                    float g[8];
                    load8(static_cast<const Y *>(a.gate) + blockIdx.x * a.gate_stride + c * 8, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) m[j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(a.alpha, xr[i][j], m[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = a.alpha * xr[i][j];
            }
            if (a.x_out) store8(static_cast<X *>(a.x_out) + row + c * 8, x[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
        }
    }
    if (!a.h) return;
    f = rsqrtf(block_sum(ss, red[1]) / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunk) {
            float w[8];
            load8(a.w_pre + c * 8, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= f * (a.w_offset + w[j]);
            store8(static_cast<O *>(a.h) + row + c * 8, x[i]);
        }
    }
}

template <typename Y, typename X, typename O>
static cudaError_t norm_launch(const NormArgs &a, int64_t T, cudaStream_t st)
{
    const int nchunk = a.H / 8;
    // Chunks per thread: few, so that enough CTAs are resident for the loads of
    // one to run during the sums of another (rows of 5376: 49.6 us with two
    // chunks per thread, 54.9 with four), but one only up to 256 threads, whose
    // two sums are short.
    const int V = nchunk <= 256 ? 1 : nchunk <= 768 ? 2 : nchunk <= 1024 ? 4 : 8;
    const int threads = ((nchunk + V - 1) / V + 31) / 32 * 32;
    const unsigned grid = (unsigned)T;
    switch (V) {
    case 1: return launch_dependent(norm_residual_kernel<Y, X, O, 1>, dim3(grid), threads, 0, st, a);
    case 2: return launch_dependent(norm_residual_kernel<Y, X, O, 2>, dim3(grid), threads, 0, st, a);
    case 4: return launch_dependent(norm_residual_kernel<Y, X, O, 4>, dim3(grid), threads, 0, st, a);
    default: return launch_dependent(norm_residual_kernel<Y, X, O, 8>, dim3(grid), threads, 0, st, a);
    }
}

wl_status launch_norm_residual(const void *y, const void *gate, int64_t gate_stride, const void *x, const float *w_post,
                               const float *w_pre, void *x_out, void *h, int64_t T, int64_t H, float alpha, float beta,
                               float eps, float w_offset, int ydt, int xdt, int hdt, cudaStream_t st)
{
    const NormArgs a{y, gate, x, w_post, w_pre, x_out, h, gate_stride, (int)H, alpha, beta, eps, w_offset};
    const int kind = (ydt == WL_OUT_F32 ? 4 : 0) + (xdt == WL_OUT_F32 ? 2 : 0) + (hdt == WL_OUT_F32 ? 1 : 0);
    cudaError_t e;
    switch (kind) {
    case 0: e = norm_launch<bf16, bf16, bf16>(a, T, st); break;
    case 1: e = norm_launch<bf16, bf16, float>(a, T, st); break;
    case 2: e = norm_launch<bf16, float, bf16>(a, T, st); break;
    case 3: e = norm_launch<bf16, float, float>(a, T, st); break;
    case 4: e = norm_launch<float, bf16, bf16>(a, T, st); break;
    case 5: e = norm_launch<float, bf16, float>(a, T, st); break;
    case 6: e = norm_launch<float, float, bf16>(a, T, st); break;
    default: e = norm_launch<float, float, float>(a, T, st); break;
    }
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_norm_residual launch");
}

}  // namespace wl
