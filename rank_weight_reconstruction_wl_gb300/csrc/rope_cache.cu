// rope_cache.cu -- rotary positions with the quantising cache write, and the
// cache read.
#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace wl {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;  // rows of a lane group in flight

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

// 8 elements as they are loaded: 16 bytes of bf16 or 32 of fp32.
template <typename X>
struct Raw8 {
    uint4 w[sizeof(X) / 2];
    __device__ __forceinline__ void load(const X *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ Raw8 from(int lane, int width) const
    {
        Raw8 o;
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i)
            o.w[i] = make_uint4(__shfl_sync(0xffffffffu, w[i].x, lane, width), __shfl_sync(0xffffffffu, w[i].y, lane, width),
                                __shfl_sync(0xffffffffu, w[i].z, lane, width), __shfl_sync(0xffffffffu, w[i].w, lane, width));
        return o;
    }
    __device__ __forceinline__ void values(float v[8]) const
    {
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[sizeof(X) / 2 - 1].x, w[sizeof(X) / 2 - 1].y, w[sizeof(X) / 2 - 1].z, w[sizeof(X) / 2 - 1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sizeof(X) == 4 ? __uint_as_float(u[j]) : (j & 1) ? bf_hi(u[j / 2]) : bf_lo(u[j / 2]);
    }
};

// One CTA per token.  `width` lanes share a row (one head of q, k or v), 8
// elements each; a lane group has kRopeRows rows in flight.
//   angle = frac(position * phase / 2^64) turns, from the wrapped 64-bit
//   product, so no position loses accuracy in a range reduction (fp32: 2^-26 turn);
//   (a, b) -> A (a cos - b sin, a sin + b cos);
//   k, v: e = row exponent of max|x|, code = e4m3(x 2^-e), scale = 2^e.
// All heads of the token share its angles (formed once, while the rows load)
// and its place in the cache.  kHalves: pairs (i, i + rot/2) whose partners
// are whole 8-element chunks away, so that they come by shuffle; otherwise
// pairs are neighbours (interleaved, within the lane) or the row is staged in
// shared memory.  A row is read once and written once, but what bounds a
// prompt is instruction issue, at three quarters of its rate, with the chain
// of loads to a token's place between (4096 tokens of 32 + 16 + 16 bf16 heads of
// 128 into an e4m3 cache: 31.9 us, 3.7 TB/s; the bytes alone would take 17.6).
// Angles whose lanes read 64 bytes apart cost 2.7 us more, two rows in flight
// 2 us, CTAs that walk several tokens and look ahead 5 us (spilled registers).
// One token takes 5.5 us, launch and two chained loads.
template <typename X, bool kE4M3, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads, sizeof(X) == 2 ? 4 : 2) rope_append_kernel(const __grid_constant__ RopeArgs a)
{
    // cos, sin of pair p; kHalves: at (p % 8) * 17 + p / 8, so that the lanes of
    // a row, 8 pairs apart, read neighbouring words
    __shared__ float2 trig[kHalves ? 8 * 17 : 128];
    __shared__ float row_buf[kHalves ? 1 : kRopeThreads * 8];
    const CacheArgs &c = a.c;
    const int tok = blockIdx.x, b = tok / c.n, i = tok - b * c.n;
    const int w = a.width, g = threadIdx.x / w, ngroups = kRopeThreads / w, sub = threadIdx.x % w;
    const int e0 = sub * 8, half = a.rot / 2;
    const bool mine = e0 < c.dim;
    const int rows = a.q_heads + 2 * c.kv_heads, first_v = a.q_heads + c.kv_heads;
    Raw8<X> raw[kRopeRows];
    const X *qp = static_cast<const X *>(a.q) + tok * a.q_stride + e0;
    const X *kp = static_cast<const X *>(a.k) + tok * a.k_stride - (int64_t)a.q_heads * c.dim + e0;
    const X *vp = static_cast<const X *>(a.v) + tok * a.v_stride - (int64_t)first_v * c.dim + e0;
    auto load = [&](int r0) {
#pragma unroll
        for (int p = 0; p < kRopeRows; ++p) {
            const int r = r0 + p * ngroups + g;
            raw[p].zero();
            if (r < rows && mine) raw[p].load((r < a.q_heads ? qp : r < first_v ? kp : vp) + r * c.dim);
        }
    };
    pdl_wait();
    pdl_trigger();  // only now: a kernel after this one may rely on all before it
    load(0);
    const int len = seq_len(c, b);
    const bool live = i < seq_count(c, b);
    const int64_t at0 = live ? cache_row(c, b, 0, len + i) : -1;  // row of head 0; head h is h * page_size on
    if (live && threadIdx.x < half) {
        const int pos = a.positions ? a.positions[tok] : len + i;
        const uint64_t turn = (uint64_t)(int64_t)pos * a.phase[threadIdx.x];
        float s, co;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // 2^-31: half turns
        trig[kHalves ? (threadIdx.x & 7) * 17 + (threadIdx.x >> 3) : threadIdx.x] = make_float2(co * a.amplitude, s * a.amplitude);
    }
    if (live && at0 < 0 && threadIdx.x == 0) atomicOr(c.status, kStatusPage);
    __syncthreads();
    float *buf = row_buf + (kHalves ? 0 : g * w * 8);
    const bool upper = e0 >= half, turns = live && e0 < a.rot;
    const int partner = !turns ? sub : upper ? sub - half / 8 : sub + half / 8;
    float2 t[8];  // this lane's angles; the sine's sign is that of its side of the pair
    if (kHalves) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            t[j] = turns ? trig[j * 17 + (upper ? e0 - half : e0) / 8] : make_float2(0.0f, 0.0f);
            if (!upper) t[j].y = -t[j].y;
        }
    }
    const int last = (threadIdx.x | 31) / w;  // the warp's last lane group
    bf16 *qo = a.q_out + (int64_t)tok * a.q_heads * c.dim + e0;
    for (int r0 = 0; r0 < rows; r0 += kRopeRows * ngroups) {
        if (r0 > 0) load(r0);
#pragma unroll
        for (int p = 0; p < kRopeRows; ++p) {
            if (r0 + p * ngroups >= rows) break;  // (the same for all)
            const int r = r0 + p * ngroups + g;
            const bool isv = r >= first_v, on = r < rows && mine;
            float v[8];
            raw[p].values(v);
            if (kHalves) {
                float o[8];
                raw[p].from(partner, w).values(o);
                if (!isv && turns) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = fmaf(o[j], t[j].y, v[j] * t[j].x);
                }
            } else {
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
            }
            if (r0 + p * ngroups + last >= a.q_heads) {  // some row of the warp goes to the cache
                uint32_t amax = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
                for (int d = w / 2; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                if (on && r >= a.q_heads && at0 >= 0) {
                    const int64_t at = at0 + (int64_t)(isv ? r - first_v : r - a.q_heads) * c.page_size;
                    // a NaN or an infinity in the row, or what rounds to an infinity of bf16
                    const bool bad = amax >= (kE4M3 ? 0x7f800000u : 0x7f7f8000u);
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
            if (on && r < a.q_heads) {
                if (!live)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
                store8(qo + r * c.dim, v);
            }
        }
    }
}

template <bool kE4M3, bool kHalves>
static cudaError_t rope_launch(const RopeArgs &a, int xdt, int64_t tokens, cudaStream_t st)
{
    if (xdt == WL_OUT_F32)
        return launch_dependent(rope_append_kernel<float, kE4M3, kHalves>, dim3((unsigned)tokens), kRopeThreads, 0, st, a);
    else
        return launch_dependent(rope_append_kernel<bf16, kE4M3, kHalves>, dim3((unsigned)tokens), kRopeThreads, 0, st, a);
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
    const bool e4 = cache.format == WL_CACHE_E4M3, halves = !rope.interleaved && rope.rot % 16 == 0;
    const int64_t tokens = seqs.batch * seqs.n;
    const cudaError_t e = halves ? (e4 ? rope_launch<true, true>(a, xdt, tokens, st) : rope_launch<false, true>(a, xdt, tokens, st))
                                 : (e4 ? rope_launch<true, false>(a, xdt, tokens, st) : rope_launch<false, false>(a, xdt, tokens, st));
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_rope_append launch");
}

// ------------------------------------------------------------------ read --
// 16 codes as loaded, and their values.
template <bool kE4M3>
struct Codes16 {
    uint4 w[kE4M3 ? 1 : 2];
    __device__ __forceinline__ void load(const char *p)
    {
#pragma unroll
        for (int i = 0; i < (kE4M3 ? 1 : 2); ++i) w[i] = ld_stream16(p + 16 * i);
    }
    __device__ __forceinline__ void values(float v[16], float scale) const
    {
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[kE4M3 ? 0 : 1].x, w[kE4M3 ? 0 : 1].y, w[kE4M3 ? 0 : 1].z, w[kE4M3 ? 0 : 1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = kE4M3 ? e4m3x2_f32((u[j / 2] >> (16 * (j & 1))) & 0xffffu) : make_float2(bf_lo(u[j]), bf_hi(u[j]));
            v[2 * j] = f.x * scale;
            v[2 * j + 1] = f.y * scale;
        }
    }
};

// A thread decodes 16 consecutive codes of a row of k and of the same row of v
// (one lookup, two independent loads).  `per` such items a token, `tokens`
// tokens a CTA.  Bound by DRAM bytes; the divisions that find an item's place
// are multiplications (64-bit ones took as long as the bytes: 39 us for 190 MB;
// now 35.4 us, 5.4 TB/s: four prompts of up to 4096 tokens, 16 heads of 128).
constexpr int kReadThreads = 256;

template <typename Y, bool kE4M3>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheArgs c, Y *k_out, Y *v_out,
                                                                  FastDiv per, FastDiv chunks, FastDiv n, int tokens, int all)
{
    pdl_wait();
    pdl_trigger();  // only now: a kernel after this one may rely on all before it
    const int tok0 = blockIdx.x * tokens, end = min(tokens, all - tok0) * (int)per.d;
    for (int e = threadIdx.x; e < end; e += kReadThreads) {
        const int t = per.div(e), in = e - t * (int)per.d, h = chunks.div(in), ch = in - h * (int)chunks.d;
        const int tok = tok0 + t, b = n.div(tok), i = tok - b * (int)n.d;
        const int64_t o = ((int64_t)tok * c.kv_heads + h) * c.dim + ch * 16;
        float v[16] = {}, u[16] = {};
        if (i < seq_count(c, b)) {
            const int64_t at = cache_row(c, b, h, seq_len(c, b) + i);
            if (at < 0) {
                if (ch == 0) atomicOr(c.status, kStatusPage);
            } else {
                const int64_t from = (at * c.dim + ch * 16) * (kE4M3 ? 1 : 2);
                Codes16<kE4M3> ck, cv;
                ck.load(c.k + from);
                cv.load(c.v + from);
                const float ks = __ldg(c.k_scale + at), vs = __ldg(c.v_scale + at);
                ck.values(v, ks);
                cv.values(u, vs);
            }
        }
        store8(k_out + o, v);
        store8(k_out + o + 8, v + 8);
        store8(v_out + o, u);
        store8(v_out + o + 8, u + 8);
    }
}

wl_status launch_cache_read(const wl_cache &cache, const wl_seqs &seqs, void *k_out, void *v_out, int dt,
                            const DeviceInfo *di, cudaStream_t st)
{
    const CacheArgs c = cache_args(cache, seqs, di->status);
    const int64_t chunk = cache.dim / 16, per = cache.kv_heads * chunk, all = seqs.batch * seqs.n;
    // one item per thread where a token has fewer than a CTA's worth
    const int tokens = (int)(per >= kReadThreads ? 1 : kReadThreads / per);
    const unsigned grid = (unsigned)((all + tokens - 1) / tokens);
    const FastDiv dp = fast_div(per), dc = fast_div(chunk), dn = fast_div(seqs.n);
    const bool e4 = cache.format == WL_CACHE_E4M3;
    cudaError_t e;
    if (dt == WL_OUT_F32)
        e = launch_dependent(e4 ? cache_read_kernel<float, true> : cache_read_kernel<float, false>, dim3(grid), kReadThreads, 0, st, c,
                             static_cast<float *>(k_out), static_cast<float *>(v_out), dp, dc, dn, tokens, (int)all);
    else
        e = launch_dependent(e4 ? cache_read_kernel<bf16, true> : cache_read_kernel<bf16, false>, dim3(grid), kReadThreads, 0, st, c,
                             static_cast<bf16 *>(k_out), static_cast<bf16 *>(v_out), dp, dc, dn, tokens, (int)all);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_cache_read launch");
}

}  // namespace wl
