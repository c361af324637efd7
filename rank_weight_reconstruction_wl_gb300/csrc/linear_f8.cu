// linear_f8.cu -- product of two e4m3 matrices with a scale for each block of
// 128 along the sum.
//
//     y[t,o] = sum_b x_scale[b][t] w_scale[b][o / 128] sum_{i in block b} W[o,i] x[t,i]
#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace wl {

struct LinearF8Args {
    const uint8_t *x, *W;
    const float *xs, *ws;
    void *y;
    int64_t T, out;
    int in, ob, ydt;
};

// A 32 x 32 tile per CTA, two rows of outputs per thread.
__global__ void __launch_bounds__(512) linear_f8_kernel(const __grid_constant__ LinearF8Args a)
{
    __shared__ float xt[32][33], wt[32][33];
    pdl_wait();
    pdl_trigger();
    const int64_t o0 = (int64_t)blockIdx.x * 32, t0 = (int64_t)blockIdx.y * 32;
    const int i = threadIdx.x % 32, j = threadIdx.x / 32;
    float acc[2] = {0.0f, 0.0f}, part[2] = {0.0f, 0.0f};
    for (int k0 = 0; k0 < a.in; k0 += 32) {
        for (int r = j; r < 32; r += 16) {
            const bool in = k0 + i < a.in;
            xt[r][i] = in && t0 + r < a.T ? e4m3x2_f32(a.x[(t0 + r) * a.in + k0 + i]).x : 0.0f;
            wt[r][i] = in && o0 + r < a.out ? e4m3x2_f32(a.W[(o0 + r) * a.in + k0 + i]).x : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 32; ++k)
            for (int h = 0; h < 2; ++h) part[h] = fmaf(wt[i][k], xt[j + 16 * h][k], part[h]);
        __syncthreads();
        if ((k0 + 32) % 128 == 0 || k0 + 32 >= a.in) {
            const int64_t b = k0 / 128;
            for (int h = 0; h < 2; ++h) {
                const int64_t t = t0 + j + 16 * h, o = o0 + i;
                if (t < a.T && o < a.out) acc[h] = fmaf(part[h], a.xs[b * a.T + t] * a.ws[b * a.ob + o / 128], acc[h]);
                part[h] = 0.0f;
            }
        }
    }
    for (int h = 0; h < 2; ++h) {
        const int64_t t = t0 + j + 16 * h, o = o0 + i;
        if (t < a.T && o < a.out) store_out(a.y, a.ydt, t * a.out + o, acc[h]);
    }
}

wl_status launch_linear_f8(const uint8_t *x, const float *x_scale, const uint8_t *W, const float *w_scale, void *y, int64_t T,
                           int64_t in, int64_t out, int ydt, const DeviceInfo *di, cudaStream_t st)
{
    (void)di;
    if (T > 32 * 65535) return fail(WL_ERR_UNSUPPORTED, "T = %lld", (long long)T);
    const LinearF8Args a{x, W, x_scale, w_scale, y, T, out, (int)in, (int)((out + 127) / 128), ydt};
    const cudaError_t e = launch_dependent(linear_f8_kernel, dim3((unsigned)((out + 31) / 32), (unsigned)((T + 31) / 32)), 512, 0, st, a);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_linear_f8 launch");
}

}  // namespace wl
