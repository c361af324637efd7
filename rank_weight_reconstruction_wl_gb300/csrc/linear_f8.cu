// linear_f8.cu -- product of two e4m3 matrices with a scale for each block of
// 128 along the sum, on the fifth-generation tensor cores.
//
//     y[t,o] = sum_b x_scale[b][t] w_scale[b][o / 128] sum_{i in block b} W[o,i] x[t,i]
//
// All three kernels walk over the blocks of 128: TMA boxes of both operands into
// a ring of stages, four MMAs (K = 32) into a tensor-memory accumulator of the
// block's own, and from there, scaled, into registers: acc += d * (x_scale
// w_scale).  So the block sums are scaled in fp32 whatever the scales are, and the
// MMAs of the next blocks run meanwhile in other accumulators.  They differ in
// what is M and what an SM holds:
//   few tokens (linear_f8_kernel): W is M, so that one token costs 16
//     columns, not 128 padded rows; tiles of a height that fills whole waves of
//     SMs, or the sum split over a cluster.  Bound by HBM: 1 x 1152 -> 262144
//     51 us, 0.88 of the copy rate; 1 x 5376 -> 21504 22 us.
//   up to 128 tokens (linear_f8_few_kernel): tokens are M; each byte of W is read
//     once.  96 x 1152 -> 262144 59 us, 0.87 of the copy rate.
//   more (linear_f8_pair_kernel): two SMs share 256 x 256 tiles.  Bound by the
//     way of a block through its accumulator: 4096 x 5376 -> 21504 369 us, 2.6
//     PFLOP/s (340 to 360 in replays of a graph, by the box).
// From 33 tokens on the one that is thought to be the fastest is taken (64 x 1152 -> 262144: the first 65 us, the second 59).
//
// linear_f8_kernel: a CTA takes a tile of up to 128 rows of W by N tokens.  Stages
// and hand-overs are of two blocks: a block alone took 0.36 us however small its
// tile, most of it barriers' round trips.  Warps 0-7 scale and store (4 warps per
// half of the tokens; a warp's lanes are 32 rows of W), warp 8 loads, warp 9
// multiplies.
#include <cooperative_groups.h>

#include "cache_row.cuh"
#include "dec_ptx.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace wl {

struct LinearF8Args {
    const float *xs, *ws;
    void *y;
    int64_t T, out;
    int nkb, ob, nt;  // blocks of 128 along the sum, along out; token tiles
    int rows;         // rows of W of a tile, a multiple of 8
    int stages;       // of the ring
    int64_t tiles;
    unsigned *status;
};

constexpr int kF8Threads = 320, kF8Ring = 192 * 1024;
constexpr int kF8Stages = 16;  // at most: tiles of 32 rows by 16 tokens

template <int N>
struct F8Shape {
    static constexpr int NB = 4;                 // pairs of accumulators
    static constexpr int COLS = 2 * N * NB;      // 128 .. 512: a power of two
    static constexpr int HALF = N / 2;           // tokens of a warp
    static constexpr int SCALES = 8 * 2 * 4 * HALF * 4;
    // the MMAs read 128 rows whatever the tile's height: past the last stage too
    static constexpr int SMEM = 1024 + kF8Ring + 16384 + SCALES;
};

// Instruction descriptor of kind::f8f6f4: e4m3 A and B, both K-major, fp32 D.
__host__ __device__ constexpr uint32_t f8_idesc(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void f8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ uint32_t f8_elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p;
}

template <int C>
__device__ __forceinline__ void f8_tmem_ld(uint32_t taddr, uint32_t *r)
{
    if constexpr (C == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    } else if constexpr (C == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
            "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
              "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
              "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(taddr));
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
    }
}
// Waits for this thread's loads; the registers are operands so that nothing reads them before.
template <int C>
__device__ __forceinline__ void f8_tmem_wait(uint32_t *r)
{
    if constexpr (C == 32) {
        f8_tmem_wait<16>(r);
        f8_tmem_wait<16>(r + 16);
    } else if constexpr (C == 8) {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
    } else {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                       "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
    }
}

// The bounded wait without a call: code that holds the sums in registers would have to save them around one, and
// register splits allow none.  CLUSTER: others of the cluster arrive.
template <bool CLUSTER = false>
__device__ __forceinline__ bool f8_wait(uint64_t *bar, unsigned parity, unsigned *status, unsigned site)
{
    if (CLUSTER ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity)) return true;
    const long long t0 = wait_clock();
    while (!(CLUSTER ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity))) {
        if (wait_clock() - t0 > kWaitLimitCycles) {
            atomicOr(status, kStatusTimeout | site);
            return false;
        }
    }
    return true;
}

// Waits until every stage that was filled has been handed back; st and phase as for the next item (of a stage that was
// never filled the first wait's parity passes).  A commit arrives on its barrier by itself some time after the MMAs, in a
// pair on the peer's too, and this memory is another CTA's once the kernel has ended.
template <bool CLUSTER = false>
__device__ __forceinline__ bool f8_ring_tail(uint64_t *empty, int stages, uint32_t st, uint32_t phase, unsigned *status)
{
    for (int i = 0; i < stages; ++i) {
        if (!f8_wait<CLUSTER>(&empty[st], phase, status, kWaitRingEmpty)) return false;
        if (++st == stages) st = 0, phase ^= 1;
    }
    return true;
}

// acc += d * s for two columns.
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t d0, uint32_t d1, uint64_t s)
{
    asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}" : "+l"(acc) : "r"(d0), "r"(d1), "l"(s));
}

__device__ __forceinline__ float f8_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f8_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// A warp's 32 rows of W (row o its lane's, in the tile where `in`) by COLS tokens from t0 on; pairs of tokens in acc.
// Tiles are multiples of 8 rows high, so that of two neighbouring rows both or none are in it.
template <int COLS>
__device__ __forceinline__ void f8_store(const LinearF8Args &a, int ydt, int64_t t0, int64_t o, bool in, const uint64_t acc[COLS / 2])
{
    const int n = (int)min((int64_t)COLS, a.T - t0);
    if (ydt == WL_OUT_F32) {
        float *y = static_cast<float *>(a.y) + t0 * a.out + o;
        if (in && o < a.out)
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                if (c < n) *y = c & 1 ? f8_hi(acc[c / 2]) : f8_lo(acc[c / 2]);
                y += a.out;
            }
    } else if (a.out % 2 == 0) {
        // neighbouring lanes trade halves: 4 bytes of one token each
        const int odd = threadIdx.x & 1;
        bf16 *y = static_cast<bf16 *>(a.y) + (t0 + odd) * a.out + o - odd;
        in = in && o - odd < a.out;
#pragma unroll
        for (int c = 0; c < COLS; c += 2) {
            const float lo = f8_lo(acc[c / 2]), hi = f8_hi(acc[c / 2]);
            const float other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            if (in && c + odd < n) *reinterpret_cast<uint32_t *>(y) = odd ? bf16x2_bits(other, hi) : bf16x2_bits(lo, other);
            y += 2 * a.out;
        }
    } else {
        bf16 *y = static_cast<bf16 *>(a.y) + t0 * a.out + o;
        if (in && o < a.out)
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                if (c < n) *y = __float2bfloat16_rn(c & 1 ? f8_hi(acc[c / 2]) : f8_lo(acc[c / 2]));
                y += a.out;
            }
    }
}

// SPLIT: the cluster's CTAs share a tile, each a run of blocks.
template <int N, bool SPLIT>
__global__ void __launch_bounds__(kF8Threads, 1) linear_f8_kernel(const __grid_constant__ LinearF8Args a,
                                                                  const __grid_constant__ CUtensorMap wmap,
                                                                  const __grid_constant__ CUtensorMap xmap, int ydt)
{
    using S = F8Shape<N>;
    extern __shared__ char f8_smem[];
    __shared__ uint64_t full[kF8Stages], empty[kF8Stages], tfull[S::NB], tempty[S::NB], drain;
    __shared__ uint32_t tmem_hold;
    __shared__ int gave_up;
    char *ring = f8_smem + (1024 - s32(f8_smem) % 1024) % 1024;
    float *scales = reinterpret_cast<float *>(ring + kF8Ring + 16384);
    const int wbytes = a.rows * 128, bytes = 2 * (wbytes + N * 128);  // of a stage: two blocks of W, two of x
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = SPLIT ? (int)cl.block_rank() : 0, ctas = SPLIT ? (int)cl.num_blocks() : 1;
    const int kb0 = SPLIT ? (int)((int64_t)a.nkb * rank / ctas) : 0, kb1 = SPLIT ? (int)((int64_t)a.nkb * (rank + 1) / ctas) : a.nkb;
    const int64_t first = SPLIT ? blockIdx.x / ctas : blockIdx.x, step = SPLIT ? gridDim.x / ctas : gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < S::NB; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 8);
        mbar_init(&drain, 1);
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&tmem_hold)), "n"(S::COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_hold;
    pdl_wait();
    pdl_trigger();

    // The loading and the multiplying warp walk and wait whole and one lane issues: code that the compiler knows to be
    // uniform keeps the descriptors in uniform registers.
    uint32_t issued = 0;  // ring items of the loading warp
    if (warp == 8) {
        const uint32_t ring0 = s32(ring), issuer = f8_elect();
        uint32_t st = 0, phase = 1;
        bool good = true;
        for (int64_t tile = first; tile < a.tiles && good; tile += step) {
            const int64_t mt = tile / a.nt;
            const int o0 = (int)(mt * a.rows), t0 = (int)(tile - mt * a.nt) * N;
            for (int kb = kb0; kb < kb1; kb += 2) {
                if (!f8_wait(&empty[st], phase, a.status, kWaitRingEmpty)) {
                    good = false;
                    break;
                }
                if (issuer) {
                    const uint32_t w = ring0 + st * bytes, x = w + 2 * wbytes;
                    const int n = min(2, kb1 - kb);
                    mbar_expect_tx(&full[st], n * (bytes / 2));
                    for (int i = 0; i < n; ++i) {
                        tma_load_2d_u32(w + i * wbytes, &wmap, (kb + i) * 128, o0, &full[st]);
                        tma_load_2d_u32(x + i * N * 128, &xmap, (kb + i) * 128, t0, &full[st]);
                    }
                }
                __syncwarp();
                ++issued;
                if (++st == a.stages) st = 0, phase ^= 1;
            }
        }
        if (!good || !f8_ring_tail(empty, a.stages, st, phase, a.status)) gave_up = 1;
    } else if (warp == 9) {
        const uint32_t ring0 = s32(ring), issuer = f8_elect();
        uint32_t st = 0, st_phase = 0, buf = 0, buf_phase = 1;
        bool good = true;
        for (int64_t tile = first; tile < a.tiles && good; tile += step) {
            for (int kb = kb0; kb < kb1; kb += 2) {
                if (!f8_wait(&tempty[buf], buf_phase, a.status, kWaitRingEmpty) || !f8_wait(&full[st], st_phase, a.status, kWaitRingFull)) {
                    good = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = sdesc(ring0 + st * bytes), db = sdesc(ring0 + st * bytes + 2 * wbytes);
                if (issuer) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f8_mma(tmem + buf * 2 * N, da + 2 * j, db + 2 * j, f8_idesc(128, N), j > 0);
                    if (kb + 1 < kb1) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f8_mma(tmem + buf * 2 * N + N, da + wbytes / 16 + 2 * j, db + N * 8 + 2 * j, f8_idesc(128, N), j > 0);
                    }
                    umma_commit(&tfull[buf]);
                    umma_commit(&empty[st]);
                }
                __syncwarp();
                if (++st == a.stages) st = 0, st_phase ^= 1;
                if (++buf == S::NB) buf = 0, buf_phase ^= 1;
            }
        }
        if (!good) {
            gave_up = 1;
            if (issuer) umma_commit(&drain);
            f8_wait(&drain, 0, a.status, kWaitDrain);
        }
    } else {
        const int half = warp / 4, quarter = warp % 4;
        float *mine = scales + warp * 8 * S::HALF;
        constexpr int C = S::HALF < 16 ? 8 : 16;         // columns of a tensor-memory load
        static_assert(S::HALF <= 32, "a lane has one token's scales");
        uint32_t blk = 0;
        bool good = true;
        for (int64_t tile = first; tile < a.tiles && good; tile += step) {
            const int64_t mt = tile / a.nt;
            const int64_t t0 = (tile - mt * a.nt) * N + half * S::HALF;
            uint64_t acc[S::HALF / 2];
#pragma unroll
            for (int i = 0; i < S::HALF / 2; ++i) acc[i] = 0;
            // A tile lies in one or two rows of scales, o0 / 128 and the next: a warp keeps its tokens' scales times either,
            // and a lane reads those of its row of W.  They come four blocks at a time, a group ahead.
            float wn[4], vn[4], xn[4], f[4], g[4];
            const int64_t t = min(t0 + lane, a.T - 1), o0 = mt * a.rows, b0 = o0 / 128;
            const int next = b0 + 1 < a.ob, second = (int)((o0 + quarter * 32 + lane) / 128 - b0);
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t k = min(kb + i, kb1 - 1);
                    wn[i] = __ldg(a.ws + k * a.ob + b0), vn[i] = __ldg(a.ws + k * a.ob + b0 + next), xn[i] = __ldg(a.xs + k * a.T + t);
                }
            };
            fetch(kb0);
            for (int kb = kb0; kb < kb1; kb += 2, ++blk) {
                // two blocks' scales for either row of them: [block][row][token]
                float *s = mine + (blk & 1) * 4 * S::HALF;
                if (((kb - kb0) & 3) == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = wn[i] * xn[i], g[i] = vn[i] * xn[i];
                    if (kb + 4 < kb1) fetch(kb + 4);
                }
                if (lane < S::HALF) s[lane] = f[0], s[S::HALF + lane] = g[0], s[2 * S::HALF + lane] = f[1], s[3 * S::HALF + lane] = g[1];
                f[0] = f[2], f[1] = f[3], g[0] = g[2], g[1] = g[3];
                __syncwarp();
                s += second ? S::HALF : 0;
                const int buf = blk % S::NB;
                if (!f8_wait(&tfull[buf], (blk / S::NB) & 1, a.status, kWaitRingFull)) {
                    good = false;
                    break;
                }
                tc_fence_after();
                const bool two = kb + 1 < kb1;
                const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 2 * N + half * S::HALF;
#pragma unroll
                for (int c = 0; c < S::HALF; c += C) {
                    uint32_t d[C], e[C];
                    f8_tmem_ld<C>(at + c, d);
                    if (two) f8_tmem_ld<C>(at + N + c, e);
                    f8_tmem_wait<C>(d);
                    f8_tmem_wait<C>(e);
                    if (c + C == S::HALF) {
                        tc_fence_before();
                        if (lane == 0) mbar_arrive(&tempty[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < C; i += 4) {
                        const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(s + c + i);
                        fma2(acc[(c + i) / 2], d[i], d[i + 1], p.x);
                        fma2(acc[(c + i) / 2 + 1], d[i + 2], d[i + 3], p.y);
                        if (two) {
                            const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(s + 2 * S::HALF + c + i);
                            fma2(acc[(c + i) / 2], e[i], e[i + 1], q.x);
                            fma2(acc[(c + i) / 2 + 1], e[i + 2], e[i + 3], q.y);
                        }
                    }
                }
            }
            if (!good) break;
            if (!SPLIT) {
                f8_store<S::HALF>(a, ydt, t0, o0 + quarter * 32 + lane, quarter * 32 + lane < a.rows, acc);
            } else {
                // the ring is idle: all of this CTA's blocks have been multiplied
                float *part = reinterpret_cast<float *>(ring);
#pragma unroll
                for (int c = 0; c < S::HALF; ++c) part[(half * S::HALF + c) * 128 + quarter * 32 + lane] = c & 1 ? f8_hi(acc[c / 2]) : f8_lo(acc[c / 2]);
            }
        }
        if (!good && lane == 0) gave_up = 1;
    }
    __syncwarp();
    if (SPLIT) {
        cl.sync();
        // columns dealt out over the CTAs; contributions in CTA order
        const int64_t mt = first / a.nt, t0 = (first - mt * a.nt) * N;
        for (int i = threadIdx.x; i < (N + ctas - 1) / ctas * 128; i += kF8Threads) {
            const int c = i / 128 * ctas + rank, row = i % 128;
            const int64_t t = t0 + c, o = mt * 128 + row;
            if (c < N && t < a.T && o < a.out) {
                float v = 0.0f;
                for (int r = 0; r < ctas; ++r) v += cl.map_shared_rank(reinterpret_cast<float *>(ring), r)[c * 128 + row];
                store_out(a.y, ydt, t * a.out + o, v);
            }
        }
        cl.sync();
    }
    tc_fence_before();
    __syncthreads();
    if (gave_up && threadIdx.x == 256) {
        // copies in flight land before this CTA ends
        for (uint32_t i = issued > a.stages ? issued - a.stages : 0; i < issued; ++i)
            f8_wait(&full[i % a.stages], (i / a.stages) & 1, a.status, kWaitDrain);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::COLS));
}

template <int N, bool SPLIT>
static cudaError_t f8_launch(const LinearF8Args &a, const CUtensorMap &wmap, const CUtensorMap &xmap, int ydt, int ctas, unsigned grid,
                             cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(linear_f8_kernel<N, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, F8Shape<N>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kF8Threads);
    cfg.dynamicSmemBytes = F8Shape<N>::SMEM;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_f8_kernel<N, SPLIT>, a, wmap, xmap, ydt);
}

// A tile's height and the CTAs that share its sum, for tiles of n tokens: the least of waves of CTAs times what a CTA takes.
// A block takes 0.22 us (n = 16; 0.33 for 64), from about 75 rows on more by its bytes, a tile 0.8 us (1.2) beside (all measured).
// 128 rows of W for 21504 are 168 tiles, two waves in the second of which most SMs have nothing: 1 token, 5376 -> 21504
// takes 26.7 us with them and 22.1 with 72 rows, which fill both; 5376 -> 5376 11.6 with any height that fits one wave.
struct F8Tiles {
    int rows, ctas;
    double time;
};

static F8Tiles f8_plan(const LinearF8Args &a, int n, int sms)
{
    F8Tiles best{128, 1, 1e30};
    const int64_t nt = (a.T + n - 1) / n;
    for (int rows = 128; rows >= 32; rows -= 8)
        for (int ctas = 1; ctas <= (rows == 128 ? 8 : 1); ctas *= 2) {
            if (ctas > 1 && a.nkb < 2 * ctas) break;
            const int64_t waves = ((a.out + rows - 1) / rows * nt * ctas + sms - 1) / sms;
            if (ctas > 1 && waves > 1) break;
            const double least = 220 + 2.2 * (n - 16), bytes = 130 + 2.1 * (n - 16) + 1.2 * rows;
            const double time = (double)waves * (((a.nkb + ctas - 1) / ctas) * (bytes > least ? bytes : least) + 800 + 8.3 * (n - 16)) + (ctas > 1 ? 3000 : 0);
            if (time < best.time) best = F8Tiles{rows, ctas, time};
        }
    return best;
}

template <int N>
static wl_status f8_run(LinearF8Args a, const uint8_t *x, const uint8_t *W, int64_t in, int ydt, const DeviceInfo *di, cudaStream_t st)
{
    const F8Tiles p = f8_plan(a, N, di->sm_count);
    CUtensorMap wmap, xmap;
    wl_status s = tmap_rows_u8(W, in, a.out, p.rows, &wmap);
    if (s != WL_OK) return s;
    s = tmap_rows_u8(x, in, a.T, N, &xmap);
    if (s != WL_OK) return s;
    a.nt = (int)((a.T + N - 1) / N);
    a.rows = p.rows;
    a.stages = kF8Ring / ((p.rows + N) * 256);
    a.tiles = (a.out + p.rows - 1) / p.rows * a.nt;
    const int64_t grid = p.ctas > 1 ? a.tiles * p.ctas : a.tiles < di->sm_count ? a.tiles : di->sm_count;
    const cudaError_t e = p.ctas > 1 ? f8_launch<N, true>(a, wmap, xmap, ydt, p.ctas, (unsigned)grid, st)
                                     : f8_launch<N, false>(a, wmap, xmap, ydt, 1, (unsigned)grid, st);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_linear_f8 launch");
}

// ------------------------------------------------------------- many tokens --
// Tokens are M and 256 rows of W are N: a lane's sums belong to one token and a
// warp's to one row of W's scales, so a block is scaled by one number a lane.
// (With W as M the scales come by column, 512 bytes of shared-memory reads for
// 32 columns: a tile of 256 tokens took 1.39 us a block, bound by that memory.)
// Two SMs share a tile of 256 tokens by 256 rows: each loads its 128 tokens and
// half of the rows, one MMA of M = 256 reads both, and each SM holds its tokens'
// 128 x 256 sums; an SM so fetches 32 KB for a block where it would need 48 KB
// alone.  Warps 0-7 scale and store (a warp: 32 tokens by 128 rows), warp 8
// loads, warp 9 of the pair's first CTA multiplies.  What bounds it: a block's
// MMAs take 512 cycles, its way through one of the two accumulators (done,
// read, handed back) about 1000, so that a block takes 740 to 840.
struct F8Pair {
    static constexpr int XBYTES = 128 * 128;
    static constexpr int STAGE = 2 * XBYTES;
    static constexpr int NST = 6;
    // Two accumulators of 256 columns.  (Four of 128 read the tokens twice as often and were slower, 475 against 359 us.)
    static constexpr int NB = 2;
    static constexpr int THREADS = 384;
    static constexpr int SMEM = 1024 + NST * STAGE + 8 * 4096;
};

__device__ __forceinline__ uint32_t in_cta(const void *p, unsigned rank)  // the same place in another CTA of the cluster
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(s32(p)), "r"(rank));
    return r;
}

// Arrives on the barrier of the pair's first CTA.  Relaxed: what it tells is that this warp's tensor-memory loads are
// done, which the fence before it orders; a release to the cluster waits for all of the warp's memory traffic (pairs
// spent more than half of their time there: 826 -> 505 us for 4096 x 5376 -> 21504).
__device__ __forceinline__ void f8_arrive_first(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_cta(bar, 0)) : "memory");
}

__device__ __forceinline__ void f8_pair_load(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void f8_pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(f8_idesc(256, 256)), "r"(acc));
}

// Arrives on the barrier of both CTAs once all MMAs so far are complete.
__device__ __forceinline__ void f8_pair_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(s32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ uint64_t f8_both(float f)
{
    uint64_t s;
    asm("mov.b64 %0, {%1, %1};" : "=l"(s) : "r"(__float_as_uint(f)));
    return s;
}

// acc += d * s for 32 columns.
__device__ __forceinline__ void f8_scale32(uint64_t *acc, const uint32_t *d, uint64_t s)
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) fma2(acc[i / 2], d[i], d[i + 1], s);
}

// A lane's row of 64 outputs from place `at` of y on, the first n of them in the matrix.
__device__ __forceinline__ void f8_store_row(void *y, int ydt, int64_t at, int n, const uint64_t acc[32])
{
    if (ydt == WL_OUT_F32) {
        float *p = static_cast<float *>(y) + at;
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c < n) p[c] = c & 1 ? f8_hi(acc[c / 2]) : f8_lo(acc[c / 2]);
    } else {
        bf16 *p = static_cast<bf16 *>(y) + at;
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c < n) p[c] = __float2bfloat16_rn(c & 1 ? f8_hi(acc[c / 2]) : f8_lo(acc[c / 2]));
    }
}

// A warp's 32 tokens by 64 rows through its 4 KB of shared memory: boxes of 32 rows of 128 bytes, swizzled, stored by
// TMA while the warp goes on to the next tile (16 bytes of 32 rows at a time straight from registers took 7 us a tile).
// Boxes are clipped at the matrix's end; one that would begin there is left out.
template <bool F32>
__device__ __forceinline__ void f8_store_boxes(const CUtensorMap *map, char *stage, int64_t t0, int64_t o0, int64_t T, int64_t out,
                                               const uint64_t acc[32])
{
    const int lane = threadIdx.x % 32;
    constexpr int W = F32 ? 32 : 64;  // columns of a box
#pragma unroll
    for (int b = 0; b < 64 / W; ++b) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint4 w;
            if constexpr (F32) {
                const uint64_t p = acc[(b * W + 4 * i) / 2], q = acc[(b * W + 4 * i) / 2 + 1];
                w = make_uint4((uint32_t)p, (uint32_t)(p >> 32), (uint32_t)q, (uint32_t)(q >> 32));
            } else {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = bf16x2_bits(f8_lo(acc[(b * W + 8 * i) / 2 + k]), f8_hi(acc[(b * W + 8 * i) / 2 + k]));
                w = make_uint4(v[0], v[1], v[2], v[3]);
            }
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = w;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && t0 < T && o0 + b * W < out) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"((int)(o0 + b * W)), "r"((int)t0), "r"(s32(stage))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}

// Scales and stores a pair's tiles, 32 tokens by the 128 rows of W of one of its SMs a warp.
__device__ __forceinline__ bool f8_pair_tiles(const LinearF8Args &a, const CUtensorMap &ymap, int ydt, int boxes, char *ring, uint32_t tmem,
                                              uint64_t *tfull, uint64_t *tempty, int rank, int64_t first, int64_t step)
{
    using S = F8Pair;
    constexpr int CTAS = 2;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = warp / 4, quarter = warp % 4;
    char *stage = ring + S::NST * S::STAGE + warp * 4096;
    uint32_t blk = 0;
    bool good = true;
    // Scales come four blocks at a time, a group ahead (one block ahead, waiting for them was most of a block's time; ahead
    // over the end of a tile too cost more in registers than the wait at a tile's begin: 351 against 340 us).
    float wn[4], xn[4], f[4];
    const float *wsp, *xsp;
    auto place = [&](int64_t tile, const float *&w, const float *&x) {  // of a tile's scales (a division: once a tile)
        const int64_t mt = tile / a.nt, t = (tile - mt * a.nt) * 128 * CTAS + rank * 128 + quarter * 32 + lane;
        w = a.ws + min(mt * 2 + half, (int64_t)a.ob - 1), x = a.xs + min(t, a.T - 1);
    };
    auto fetch = [&](const float *w, const float *x, int kb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = min(kb + i, a.nkb - 1);
            wn[i] = __ldg(w + k * a.ob), xn[i] = __ldg(x + k * a.T);
        }
    };
    for (int64_t tile = first; tile < a.tiles && good; tile += step) {
        const int64_t mt = tile / a.nt;
        const int64_t o0 = mt * 256 + half * 128, t = (tile - mt * a.nt) * 128 * CTAS + rank * 128 + quarter * 32 + lane;
        place(tile, wsp, xsp);
        fetch(wsp, xsp, 0);
        uint64_t acc[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0;
#pragma unroll 1
        for (int kb = 0; kb < a.nkb; ++kb, ++blk) {
            if ((kb & 3) == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = wn[i] * xn[i];
                fetch(wsp, xsp, kb + 4);
            }
            const uint64_t s = f8_both(f[0]);
            f[0] = f[1], f[1] = f[2], f[2] = f[3];
            const int buf = blk % S::NB;
            if (!f8_wait(&tfull[buf], (blk / S::NB) & 1, a.status, kWaitRingFull)) {
                good = false;
                break;
            }
            tc_fence_after();
            const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 256 + half * 128;
            // two loads of 32 columns in flight; the accumulator is free once the last two have arrived
            uint32_t d0[32], d1[32];
            f8_tmem_ld<32>(at, d0);
            f8_tmem_ld<32>(at + 32, d1);
            f8_tmem_wait<32>(d0);
            f8_tmem_wait<32>(d1);
            f8_scale32(acc, d0, s);
            f8_tmem_ld<32>(at + 64, d0);
            f8_scale32(acc + 16, d1, s);
            f8_tmem_ld<32>(at + 96, d1);
            f8_tmem_wait<32>(d0);
            f8_tmem_wait<32>(d1);
            tc_fence_before();
            if (lane == 0) f8_arrive_first(&tempty[buf]);
            f8_scale32(acc + 32, d0, s);
            f8_scale32(acc + 48, d1, s);
        }
        if (!good) break;
        // one branch for both halves: with a branch each ptxas gave the loop above other registers and 8 % more time
        if (boxes && ydt == WL_OUT_F32) {
            f8_store_boxes<true>(&ymap, stage, t - lane, o0, a.T, a.out, acc);
            f8_store_boxes<true>(&ymap, stage, t - lane, o0 + 64, a.T, a.out, acc + 32);
        } else if (boxes) {
            f8_store_boxes<false>(&ymap, stage, t - lane, o0, a.T, a.out, acc);
            f8_store_boxes<false>(&ymap, stage, t - lane, o0 + 64, a.T, a.out, acc + 32);
        } else if (t < a.T) {  // rows that are not 16 bytes apart
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (o0 + 64 * h < a.out)
                    f8_store_row(a.y, ydt, t * a.out + o0 + 64 * h, (int)min((int64_t)64, a.out - o0 - 64 * h), acc + 32 * h);
        }
    }
    return good;
}

__global__ void __launch_bounds__(F8Pair::THREADS, 1) linear_f8_pair_kernel(const __grid_constant__ LinearF8Args a,
                                                                                 const __grid_constant__ CUtensorMap wmap,
                                                                                 const __grid_constant__ CUtensorMap xmap,
                                                                                 const __grid_constant__ CUtensorMap ymap, int ydt,
                                                                                 int boxes)
{
    using S = F8Pair;
    extern __shared__ char f8_smem[];
    __shared__ uint64_t full[S::NST], empty[S::NST], tfull[S::NB], tempty[S::NB], drain;
    __shared__ uint32_t tmem_hold;
    __shared__ int gave_up;
    char *ring = f8_smem + (1024 - s32(f8_smem) % 1024) % 1024;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    constexpr int CTAS = 2;
    const int64_t first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::NST; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < S::NB; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 8 * CTAS);
        mbar_init(&drain, 1);
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&tmem_hold)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cl.sync();
    tc_fence_after();
    const uint32_t tmem = tmem_hold;
    pdl_wait();
    pdl_trigger();

    uint32_t issued = 0;  // ring items of the loading thread
    if (warp >= 8) {
        // the third warpgroup gives registers to the other two: 384 x 168 = 128 x 40 + 256 x 232
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 8) {
            const uint32_t ring0 = s32(ring), issuer = f8_elect(), bar0 = in_cta(&full[0], 0);
            uint32_t st = 0, phase = 1;
            bool good = true;
            for (int64_t tile = first; tile < a.tiles && good; tile += step) {
                const int64_t mt = tile / a.nt;
                const int o0 = (int)(mt * 256) + rank * 128, t0 = (int)(tile - mt * a.nt) * 128 * CTAS + rank * 128;
                for (int kb = 0; kb < a.nkb; ++kb) {
                    if (!f8_wait<true>(&empty[st], phase, a.status, kWaitRingEmpty)) {
                        good = false;
                        break;
                    }
                    if (issuer) {
                        const uint32_t p = ring0 + st * S::STAGE, bar = bar0 + st * 8;
                        if (rank == 0) mbar_expect_tx(&full[st], CTAS * S::STAGE);  // both CTAs' bytes
                        f8_pair_load(p, &xmap, kb * 128, t0, bar);
                        f8_pair_load(p + S::XBYTES, &wmap, kb * 128, o0, bar);
                    }
                    __syncwarp();
                    ++issued;
                    if (++st == S::NST) st = 0, phase ^= 1;
                }
            }
            if (!good || !f8_ring_tail<true>(empty, S::NST, st, phase, a.status)) gave_up = 1;
        } else if (warp == 9 && rank == 0) {
            // The whole warp walks and waits, one lane issues: code that the compiler knows to be uniform keeps the
            // descriptors in uniform registers (one lane alone took 630 cycles a block for MMAs of 512).
            const uint32_t ring0 = s32(ring), issuer = f8_elect();
            uint32_t st = 0, st_phase = 0, buf = 0, buf_phase = 1;
            bool good = true;
            for (int64_t tile = first; tile < a.tiles && good; tile += step) {
                for (int kb = 0; kb < a.nkb; ++kb) {
                    if (!f8_wait<true>(&tempty[buf], buf_phase, a.status, kWaitRingEmpty) ||
                        !f8_wait<true>(&full[st], st_phase, a.status, kWaitRingFull)) {
                        good = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = sdesc(ring0 + st * S::STAGE), db = sdesc(ring0 + st * S::STAGE + S::XBYTES);
                    if (issuer) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) f8_pair_mma(tmem + buf * 256, da + 2 * j, db + 2 * j, j > 0);
                        f8_pair_commit(&tfull[buf]);
                        f8_pair_commit(&empty[st]);
                    }
                    __syncwarp();
                    if (++st == S::NST) st = 0, st_phase ^= 1;
                    buf ^= 1;
                    if (buf == 0) buf_phase ^= 1;
                }
            }
            if (!good) {
                gave_up = 1;
                if (issuer) f8_pair_commit(&drain);
                f8_wait<true>(&drain, 0, a.status, kWaitDrain);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const bool good = f8_pair_tiles(a, ymap, ydt, boxes, ring, tmem, tfull, tempty, rank, first, step);
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // before the memory they read goes
        if (!good && lane == 0) gave_up = 1;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (gave_up && threadIdx.x == 256 && rank == 0) {
        // copies in flight (both CTAs') land before a CTA ends
        for (uint32_t i = issued > S::NST ? issued - S::NST : 0; i < issued; ++i)
            f8_wait<true>(&full[i % S::NST], (i / S::NST) & 1, a.status, kWaitDrain);
    }
    cl.sync();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

static wl_status f8_run_pair(LinearF8Args a, const uint8_t *x, const uint8_t *W, int64_t in, int ydt, const DeviceInfo *di,
                             cudaStream_t st)
{
    using S = F8Pair;
    constexpr int CTAS = 2;
    CUtensorMap wmap, xmap, ymap = {};
    wl_status s = tmap_rows_u8(W, in, a.out, 128, &wmap);
    if (s != WL_OK) return s;
    s = tmap_rows_u8(x, in, a.T, 128, &xmap);
    if (s != WL_OK) return s;
    const bool f32 = ydt == WL_OUT_F32, boxes = a.out % (f32 ? 4 : 8) == 0;  // a map's rows are 16 bytes apart
    if (boxes) {
        s = f32 ? tmap_2d_f32(a.y, a.out, a.T, 32, 32, &ymap) : tmap_2d_bf16(a.y, a.out, a.T, a.out, 64, 32, &ymap);
        if (s != WL_OK) return s;
    }
    a.nt = (int)((a.T + 128 * CTAS - 1) / (128 * CTAS));
    a.tiles = (a.out + 255) / 256 * a.nt;
    cudaError_t e = cudaFuncSetAttribute(linear_f8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return cuda_fail(e, "wl_linear_f8 attributes");
    const int64_t most = di->sm_count / CTAS, groups = a.tiles < most ? a.tiles : most;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CTAS;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CTAS * groups));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, linear_f8_pair_kernel, a, wmap, xmap, ymap, ydt, (int)boxes);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_linear_f8 launch");
}

// ------------------------------------------------------------- 33 to 128 tokens --
// W's bytes are the time, and each is read once: tokens are M (rows of the tile
// past them hold whatever the ring holds: their sums are not stored), `rows` rows
// of W are N, chosen so that the tiles fill whole waves of SMs.  A tile so begins
// at any multiple of 64 and crosses from one row of scales to the next at most
// once in a warp's columns.
struct F8Few {
    int rows, xrows;   // rows of W of a tile; rows of the token box: T up to a multiple of 8
    int stages, stage; // of the ring, bytes of one
    int cols, bufs;    // accumulators: 64, 128 or 256 columns, 512 in all
    int half;          // columns of a side
};

constexpr int kFewThreads = 384;
constexpr int kFewStages = 14;  // at most: tiles of 64 rows by 40 tokens

// 32 tokens (t0: the first) by 32 rows of W through the warp's shared memory.
template <bool F32>
__device__ __forceinline__ void f8_store_box32(const CUtensorMap *map, char *stage, int t0, int64_t o, const uint64_t acc[16])
{
    const int lane = threadIdx.x % 32;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
        if constexpr (F32) {
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4((uint32_t)acc[2 * i], (uint32_t)(acc[2 * i] >> 32), (uint32_t)acc[2 * i + 1], (uint32_t)(acc[2 * i + 1] >> 32));
        } else {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = bf16x2_bits(f8_lo(acc[4 * i + k]), f8_hi(acc[4 * i + k]));
            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"((int)o), "r"(t0), "r"(s32(stage))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// The lane's 16 outputs from place `at` of y on, the first n of them in the matrix (rows that are not 16 bytes apart).
__device__ __forceinline__ void f8_store16(void *y, int ydt, int64_t at, int n, const uint64_t acc[8])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) store_out(y, ydt, at + i, i & 1 ? f8_hi(acc[i / 2]) : f8_lo(acc[i / 2]));
}

__device__ __forceinline__ void f8_scale16(uint64_t *acc, const uint32_t *d, uint64_t s)
{
#pragma unroll
    for (int i = 0; i < 16; i += 2) fma2(acc[i / 2], d[i], d[i + 1], s);
}

__global__ void __launch_bounds__(kFewThreads, 1) linear_f8_few_kernel(const __grid_constant__ LinearF8Args a, const __grid_constant__ F8Few p,
                                                                       const __grid_constant__ CUtensorMap wmap,
                                                                       const __grid_constant__ CUtensorMap xmap,
                                                                       const __grid_constant__ CUtensorMap ymap, int ydt, int boxes)
{
    extern __shared__ char f8_smem[];
    __shared__ uint64_t full[kFewStages], empty[kFewStages], tfull[8], tempty[8], drain;
    __shared__ uint32_t tmem_hold;
    __shared__ int gave_up;
    char *ring = f8_smem + (1024 - s32(f8_smem) % 1024) % 1024;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < p.bufs; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 8);
        mbar_init(&drain, 1);
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&tmem_hold)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_hold;
    pdl_wait();
    pdl_trigger();

    uint32_t issued = 0;  // ring items of the loading warp
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");  // as in the pairs' kernel
        if (warp == 8) {
            const uint32_t ring0 = s32(ring), issuer = f8_elect();
            uint32_t st = 0, phase = 1;
            bool good = true;
            for (int64_t tile = blockIdx.x; tile < a.tiles && good; tile += gridDim.x) {
                const int o0 = (int)(tile * p.rows);
                for (int kb = 0; kb < a.nkb; ++kb) {
                    if (!f8_wait(&empty[st], phase, a.status, kWaitRingEmpty)) {
                        good = false;
                        break;
                    }
                    if (issuer) {
                        const uint32_t at = ring0 + st * p.stage;
                        mbar_expect_tx(&full[st], p.stage);
                        tma_load_2d_u32(at, &wmap, kb * 128, o0, &full[st]);
                        tma_load_2d_u32(at + p.rows * 128, &xmap, kb * 128, 0, &full[st]);
                    }
                    __syncwarp();
                    ++issued;
                    if (++st == p.stages) st = 0, phase ^= 1;
                }
            }
            if (!good || !f8_ring_tail(empty, p.stages, st, phase, a.status)) gave_up = 1;
        } else if (warp == 9) {
            const uint32_t ring0 = s32(ring), issuer = f8_elect(), idesc = f8_idesc(128, p.rows);
            uint32_t st = 0, st_phase = 0, buf = 0, buf_phase = 1;
            bool good = true;
            for (int64_t tile = blockIdx.x; tile < a.tiles && good; tile += gridDim.x) {
                for (int kb = 0; kb < a.nkb; ++kb) {
                    if (!f8_wait(&tempty[buf], buf_phase, a.status, kWaitRingEmpty) || !f8_wait(&full[st], st_phase, a.status, kWaitRingFull)) {
                        good = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t db = sdesc(ring0 + st * p.stage), da = sdesc(ring0 + st * p.stage + p.rows * 128);
                    if (issuer) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) f8_mma(tmem + buf * p.cols, da + 2 * j, db + 2 * j, idesc, j > 0);
                        umma_commit(&tfull[buf]);
                        umma_commit(&empty[st]);
                    }
                    __syncwarp();
                    if (++st == p.stages) st = 0, st_phase ^= 1;
                    if (++buf == p.bufs) buf = 0, buf_phase ^= 1;
                }
            }
            if (!good) {
                gave_up = 1;
                if (issuer) umma_commit(&drain);
                f8_wait(&drain, 0, a.status, kWaitDrain);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int side = warp / 4, quarter = warp % 4, t = quarter * 32 + lane;
        const int c0 = side * p.half, chunks = p.half / 16;  // columns of the warp, in 16s: 2, 4, 6 or 8
        const bool mine = quarter * 32 < a.T;
        char *stage = ring + p.stages * p.stage + warp * 4096;
        uint32_t buf = 0, phase = 0;
        bool good = true;
        for (int64_t tile = blockIdx.x; tile < a.tiles && good; tile += gridDim.x) {
            const int64_t o0 = tile * p.rows + c0, b0 = o0 / 128;
            const int cut = (int)((b0 + 1) * 128 - o0) / 16;  // the chunk where the next row of scales begins
            const float *wsp = a.ws + min(b0, (int64_t)a.ob - 1), *xsp = a.xs + min((int64_t)t, a.T - 1);
            const int next = b0 + 1 < a.ob;
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            // scales come two blocks at a time, a group ahead
            float wn[2], vn[2], xn[2], f[2], g[2];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t k = min(kb + i, a.nkb - 1);
                    wn[i] = __ldg(wsp + k * a.ob), vn[i] = __ldg(wsp + k * a.ob + next), xn[i] = __ldg(xsp + k * a.T);
                }
            };
            if (mine) fetch(0);
#pragma unroll 1
            for (int kb = 0; kb < a.nkb; ++kb) {
                if (mine && (kb & 1) == 0) {
                    f[0] = wn[0] * xn[0], f[1] = wn[1] * xn[1], g[0] = vn[0] * xn[0], g[1] = vn[1] * xn[1];
                    fetch(kb + 2);
                }
                if (!f8_wait(&tfull[buf], phase, a.status, kWaitRingFull)) {
                    good = false;
                    break;
                }
                if (mine) {
                    tc_fence_after();
                    const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * p.cols + c0;
                    const uint64_t s0 = f8_both(f[0]), s1 = f8_both(g[0]);
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        if (c < chunks) {
                            uint32_t d0[16], d1[16];
                            f8_tmem_ld<16>(at + 16 * c, d0);
                            f8_tmem_ld<16>(at + 16 * c + 16, d1);
                            f8_tmem_wait<16>(d0);
                            f8_tmem_wait<16>(d1);
                            f8_scale16(acc + 8 * c, d0, c < cut ? s0 : s1);
                            f8_scale16(acc + 8 * c + 8, d1, c + 1 < cut ? s0 : s1);
                        }
                    }
                    tc_fence_before();
                    f[0] = f[1], g[0] = g[1];
                }
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == p.bufs) buf = 0, phase ^= 1;
            }
            if (!good) break;
            if (!mine) continue;
            if (boxes) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (2 * b < chunks && o0 + 32 * b < a.out) {
                        if (ydt == WL_OUT_F32) f8_store_box32<true>(&ymap, stage, quarter * 32, o0 + 32 * b, acc + 16 * b);
                        else f8_store_box32<false>(&ymap, stage, quarter * 32, o0 + 32 * b, acc + 16 * b);
                    }
            } else if (t < a.T) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < chunks && o0 + 16 * c < a.out)
                        f8_store16(a.y, ydt, t * a.out + o0 + 16 * c, (int)min((int64_t)16, a.out - o0 - 16 * c), acc + 8 * c);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // before the memory they read goes
        if (!good && lane == 0) gave_up = 1;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (gave_up && threadIdx.x == 256) {
        for (uint32_t i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
            f8_wait(&full[i % p.stages], (i / p.stages) & 1, a.status, kWaitDrain);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

// The tile height for 33 to 128 tokens and what it is thought to take: waves of tiles, a block's and a tile's time as
// measured (96 tokens, 1152 -> 262144: 58.7 us with 256 rows, 65 with 192; 128 tokens, 5376 -> 21504: 26.5 with 192, 42 with 128).
static double f8_few_plan(int64_t T, int64_t out, int nkb, int sms, F8Few *p)
{
    double best = 1e30;
    p->xrows = (int)(T + 7) / 8 * 8;
    for (int rows = 64; rows <= 256; rows += 64) {
        const int64_t waves = ((out + rows - 1) / rows + sms - 1) / sms;
        const double time = (double)waves * (nkb * (300 + 1.35 * rows) + 10.5 * rows);
        if (time < best) best = time, p->rows = rows;
    }
    p->half = p->rows / 2;  // a multiple of 32: boxes of 32 rows of W
    p->stage = (p->rows + p->xrows) * 128;
    p->stages = kF8Ring / p->stage;
    p->cols = p->rows <= 64 ? 64 : p->rows <= 128 ? 128 : 256;
    p->bufs = 512 / p->cols;
    return best;
}

static wl_status f8_run_few(LinearF8Args a, const F8Few &p, const uint8_t *x, const uint8_t *W, int64_t in, int ydt, const DeviceInfo *di,
                            cudaStream_t st)
{
    CUtensorMap wmap, xmap, ymap = {};
    wl_status s = tmap_rows_u8(W, in, a.out, p.rows, &wmap);
    if (s != WL_OK) return s;
    s = tmap_rows_u8(x, in, a.T, p.xrows, &xmap);
    if (s != WL_OK) return s;
    const bool f32 = ydt == WL_OUT_F32, boxes = a.out % (f32 ? 4 : 8) == 0;
    if (boxes) {
        s = f32 ? tmap_2d_f32(a.y, a.out, a.T, 32, 32, &ymap) : tmap_2d_bf16_swz(a.y, a.out, a.T, a.out, 32, 32, 64, &ymap);
        if (s != WL_OK) return s;
    }
    a.tiles = (a.out + p.rows - 1) / p.rows;
    const int smem = 1024 + p.stages * p.stage + 8 * 4096;
    cudaError_t e = cudaFuncSetAttribute(linear_f8_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kF8Ring + 8 * 4096);
    if (e != cudaSuccess) return cuda_fail(e, "wl_linear_f8 attributes");
    const int64_t grid = a.tiles < di->sm_count ? a.tiles : di->sm_count;
    e = launch_dependent(linear_f8_few_kernel, dim3((unsigned)grid), kFewThreads, (size_t)smem, st, a, p, wmap, xmap, ymap, ydt, (int)boxes);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_linear_f8 launch");
}

wl_status launch_linear_f8(const uint8_t *x, const float *x_scale, const uint8_t *W, const float *w_scale, void *y, int64_t T,
                           int64_t in, int64_t out, int ydt, const DeviceInfo *di, cudaStream_t st)
{
    const LinearF8Args a{x_scale, w_scale, y, T, out, (int)((in + 127) / 128), (int)((out + 127) / 128), 0, 128, 0, 0, di->status};
    if (T > 32) {
        // The least of what the kernels are thought to take: pairs 0.46 us a block and 2.5 us a tile (measured), the others above.
        F8Few p;
        const int64_t pairs = (out + 255) / 256 * ((T + 255) / 256), at_once = di->sm_count / 2;
        const double pair = (double)((pairs + at_once - 1) / at_once) * (a.nkb * 460.0 + 2500.0) + 1000.0;
        const double few = T <= 128 ? f8_few_plan(T, out, a.nkb, di->sm_count, &p) : 1e30, split = f8_plan(a, 64, di->sm_count).time;
        if (pair <= few && pair <= split) return f8_run_pair(a, x, W, in, ydt, di, st);
        if (few <= split) return f8_run_few(a, p, x, W, in, ydt, di, st);
    }
    if (T <= 16) return f8_run<16>(a, x, W, in, ydt, di, st);
    if (T <= 32) return f8_run<32>(a, x, W, in, ydt, di, st);
    return f8_run<64>(a, x, W, in, ydt, di, st);
}

}  // namespace wl
