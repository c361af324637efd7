// quant_f8.cu -- rows or weights as e4m3 codes with a power-of-two scale for
// each block of 128.
//
//     e = smallest integer >= -126 with max|block| <= 448 * 2^e,  code = e4m3(x / 2^e)
//
// x is read once, a code and 1/32 byte of scale written per element; a block is
// kept in registers between its maximum and its codes.  4096 rows of 5376: fp32
// 17.3 us, 0.94 of the copy rate; bf16 12.9 us, 0.76, as the instructions of an
// element are the same for half of the bytes.  Blocks of 128 x 128 of 262144 x
// 1152: fp32 231 us, 0.97; bf16 225 us, 0.59: a CTA's loads, reduction and stores
// follow one another, and two CTAs an SM (99 registers) hide too little of it.
#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace wl {

struct QuantArgs {
    const void *x;
    int64_t x_stride, rows;
    uint8_t *codes;
    float *scales;
    int in, nb, rows_per_cta;
    FastDiv by_nb;
};

__device__ __forceinline__ uint32_t amax8(const float v[8])
{
    // magnitudes as integers order like the numbers, with infinities and NaN above all
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// 8 codes of v and, where `first`, the block's scale.
__device__ __forceinline__ void put_codes(uint8_t *codes, float *scale, bool first, const float v[8], uint32_t amax)
{
    uint2 c = make_uint2(0, 0);
    float sc = __uint_as_float(0x7fc00000u);
    if (amax < 0x7f800000u) {
        const int e = row_exponent(amax);
        sc = exp2_int(e);
        // x / 2^e by two factors: 2^-e alone passes fp32's range for e = -126 .. 127
        const float f = exp2_int(min(max(-e, -126), 126)), g = exp2_int(-e - min(max(-e, -126), 126));
        c.x = e4m3x4(v[0] * f * g, v[1] * f * g, v[2] * f * g, v[3] * f * g);
        c.y = e4m3x4(v[4] * f * g, v[5] * f * g, v[6] * f * g, v[7] * f * g);
    }
    *reinterpret_cast<uint2 *>(codes) = c;
    if (first) *scale = sc;
}

// group 1: 16 lanes of 8 elements each per block.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int64_t row0 = (int64_t)blockIdx.x * a.rows_per_cta;
    const int units = (int)min((int64_t)a.rows_per_cta, a.rows - row0) * a.nb;
    const int lane = threadIdx.x % 16;
    constexpr int U = 4;
    for (int u0 = threadIdx.x / 16; u0 < units; u0 += 16 * U) {
        float v[U][8];
        int64_t row[U];
        int kb[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = min(u0 + 16 * j, units - 1);
            const int r = a.by_nb.div(u);
            row[j] = row0 + r;
            kb[j] = u - r * a.nb;
            const int i = kb[j] * 128 + lane * 8;
            if (i < a.in) {
                load8(static_cast<const T *>(a.x) + row[j] * a.x_stride + i, v[j]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            uint32_t m = amax8(v[j]);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            const int i = kb[j] * 128 + lane * 8;
            if (u0 + 16 * j < units && i < a.in)
                put_codes(a.codes + row[j] * a.in + i, a.scales + (int64_t)kb[j] * a.rows + row[j], lane == 0, v[j], m);
        }
    }
}

// group 128: a CTA per block, 16 lanes per row, 16 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const __grid_constant__ QuantArgs a, int64_t groups)
{
    __shared__ uint32_t red[8];
    pdl_wait();
    pdl_trigger();
    const int kb = blockIdx.y;
    const int64_t g = blockIdx.x;
    const int i = kb * 128 + threadIdx.x % 16 * 8, r = threadIdx.x / 16;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = g * 128 + r + 16 * j;
        if (i < a.in && row < a.rows) {
            load8(static_cast<const T *>(a.x) + row * a.x_stride + i, v[j]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, amax8(v[j]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, red[w]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = g * 128 + r + 16 * j;
        if (i < a.in && row < a.rows)
            put_codes(a.codes + row * a.in + i, a.scales + (int64_t)kb * groups + g, threadIdx.x == 0 && j == 0, v[j], m);
    }
}

wl_status launch_quant_f8(const void *x, int64_t x_stride, int xdt, int64_t rows, int64_t in, int64_t group, uint8_t *codes,
                          float *scales, const DeviceInfo *di, cudaStream_t st)
{
    QuantArgs a{x, x_stride, rows, codes, scales, (int)in, (int)((in + 127) / 128), 1, fast_div((in + 127) / 128)};
    cudaError_t e;
    if (group == 1) {
        // rows of a CTA: up to 8, so that their scales, neighbours in memory, are written together, while 8 CTAs an SM are left
        const int64_t most = rows / (8 * di->sm_count);
        a.rows_per_cta = (int)(most < 1 ? 1 : most > 8 ? 8 : most);
        const dim3 grid((unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta));
        e = xdt == WL_OUT_F32 ? launch_dependent(quant_rows_kernel<float>, grid, 256, 0, st, a)
                              : launch_dependent(quant_rows_kernel<bf16>, grid, 256, 0, st, a);
    } else {
        const int64_t groups = (rows + 127) / 128;
        const dim3 grid((unsigned)groups, (unsigned)a.nb);
        e = xdt == WL_OUT_F32 ? launch_dependent(quant_blocks_kernel<float>, grid, 256, 0, st, a, groups)
                              : launch_dependent(quant_blocks_kernel<bf16>, grid, 256, 0, st, a, groups);
    }
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_quant_f8 launch");
}

}  // namespace wl
