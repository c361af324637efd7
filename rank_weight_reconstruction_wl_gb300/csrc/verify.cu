// verify.cu -- drafted tokens accepted or rejected against the model's
// distribution, and the token after them, from given random numbers.
//
//     w_i = 2^((l_i - max l) log2(e) / t),  R = w,  S = sum R
//     child c of node u, token k:  accepted if  r_c q_k S < R_k,  else R = max(R - S q, 0)
//     next: lowest i with R_i > 0 and R_0 + ... + R_i > r_0 S
//
// Only the rows of accepted nodes are read: a cluster owns a sequence and walks
// down its tree, one pass over a row (split over the cluster's warps) per node.
// Bound by HBM where the batch fills the GPU, by the chain of passes (load,
// reduction, cluster barrier) where it does not.
//
// Decisions.  A random number closer to a border between two tokens than the
// sums' rounding would give another token than exact arithmetic does, and a
// vocabulary has 10^5 borders.  So the sums that decide are made of weights held
// as two floats (about 2^-31 of each weight), and the sums of the fast pass
// decide only where their error (kTol of the row's sum) cannot matter.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace cg = cooperative_groups;

namespace wl {

constexpr int kVerThreads = 1024;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCtas = 16;  // CTAs of a cluster at most
constexpr double kTol = 5e-6; // fast sums are right to this part of the row's sum

// 2^(j/128) as two floats.
__constant__ float2 kExp2Table[128] = {
    {0x1.0p+0f, 0x0.0p+0f}, {0x1.0163dap+0f, 0x1.3f6666p-25f}, {0x1.02c9a4p+0f, -0x1.887fap-28f},
    {0x1.04315ep+0f, 0x1.0dcffp-25f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0706b2p+0f, 0x1.3bbedcp-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.09e3ecp+0f, 0x1.58de7p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.0cc922p+0f, 0x1.6e48fep-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f}, {0x1.0fb66ap+0f, 0x1.ffda64p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.12abdcp+0f, 0x1.b0c73p-30f}, {0x1.1429aap+0f, 0x1.d525bcp-25f},
    {0x1.15a98cp+0f, 0x1.14b1cap-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.18af94p+0f, -0x1.dcdc86p-26f},
    {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1bbe08p+0f, 0x1.011734p-26f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.1ed502p+0f, 0x1.7e6c8ep-27f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f}, {0x1.21f49ap+0f, -0x1.d0446ep-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.251ce4p+0f, 0x1.f654c8p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f},
    {0x1.284dfep+0f, 0x1.f5638p-28f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f}, {0x1.2b87fep+0f, -0x1.e4a4cep-25f},
    {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.2ecafap+0f, 0x1.27c5eap-25f}, {0x1.306fep+0f, 0x1.4636e2p-25f},
    {0x1.32171p+0f, -0x1.d993e8p-27f}, {0x1.33c08cp+0f, -0x1.b37d2p-25f}, {0x1.356c56p+0f, -0x1.b5803cp-30f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.38cae6p+0f, 0x1.a0bb0cp-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f},
    {0x1.3c32dcp+0f, 0x1.89d472p-27f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.3fa45p+0f, 0x1.2b2006p-26f},
    {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.431f5ep+0f, -0x1.abd5dap-26f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.46a41ep+0f, 0x1.a3a00ap-25f}, {0x1.486a2cp+0f, -0x1.47d866p-25f}, {0x1.4a32bp+0f, -0x1.e50584p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4dcb2ap+0f, -0x1.8088bcp-26f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f},
    {0x1.516daap+0f, 0x1.67b32p-27f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.551a4cp+0f, 0x1.4bb242p-25f},
    {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.58d12ep+0f, -0x1.6d07p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.5c9268p+0f, 0x1.4b28d6p-25f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f}, {0x1.605e1cp+0f, -0x1.a248fep-26f},
    {0x1.6247ecp+0f, -0x1.f8b55p-25f}, {0x1.643464p+0f, -0x1.66679cp-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f},
    {0x1.68155ep+0f, -0x1.766ad2p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.6c0128p+0f, -0x1.5e84a8p-25f},
    {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.6ff7ep+0f, -0x1.ab9aep-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.73f9a4p+0f, 0x1.14b02ep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f}, {0x1.780694p+0f, 0x1.fbcba8p-25f},
    {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.7c1edp+0f, 0x1.30c132p-28f}, {0x1.7e2f34p+0f, -0x1.261634p-25f},
    {0x1.804276p+0f, -0x1.783cbep-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8471a4p+0f, 0x1.88f1ecp-26f},
    {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.88ac7ep+0f, -0x1.9d665ap-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.8cf322p+0f, -0x1.29576ep-25f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f}, {0x1.9145bp+0f, 0x1.723ff8p-25f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.95a44cp+0f, 0x1.790a42p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f},
    {0x1.9a0f18p+0f, -0x1.e6bf08p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.9e8632p+0f, -0x1.873738p-26f},
    {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a309bep+0f, 0x1.8945a6p-25f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.a799e2p+0f, -0x1.99e994p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f}, {0x1.ac36bcp+0f, -0x1.606432p-31f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b0e072p+0f, 0x1.31b6ccp-25f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f},
    {0x1.b59728p+0f, 0x1.bcab28p-25f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.ba5b04p+0f, -0x1.ebdf36p-25f},
    {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.bf2c26p+0f, -0x1.0a387ep-26f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.c40ab6p+0f, -0x1.7c2c98p-39f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f}, {0x1.c8f6dap+0f, -0x1.7f230ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.cdf0b6p+0f, -0x1.54478p-25f}, {0x1.d072d4p+0f, 0x1.40f13p-25f},
    {0x1.d2f87p+0f, 0x1.01b13ep-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.d80e32p+0f, -0x1.26cf8ep-25f},
    {0x1.da9e6p+0f, 0x1.ed9942p-27f}, {0x1.dd322p+0f, -0x1.9fc974p-25f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.e26462p+0f, -0x1.614bdap-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f}, {0x1.e7a52p+0f, -0x1.0e2cep-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.ecf482p+0f, 0x1.b1ccfep-25f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f},
    {0x1.f252b4p+0f, -0x1.1288aep-25f}, {0x1.f50766p+0f, -0x1.246ebp-26f}, {0x1.f7bfdap+0f, 0x1.b397c2p-25f},
    {0x1.fa7c18p+0f, 0x1.9e90d8p-28f}, {0x1.fd3c22p+0f, 0x1.71ee3ep-25f}};

// ------------------------------------------------------------ two floats --
struct FF {
    float h, l;
};

__device__ __forceinline__ FF ff_add(FF a, FF b)
{
    const float s = a.h + b.h, t = s - a.h;
    const float e = (a.h - (s - t)) + (b.h - t);  // Knuth's two-sum: exact
    return FF{s, e + (a.l + b.l)};
}

__device__ __forceinline__ double ff_double(FF a) { return (double)a.h + (double)a.l; }
__device__ __forceinline__ FF ff_of(double d)
{
    const float h = (float)d;
    return FF{h, (float)(d - (double)h)};
}

// 2^((l - m) c), l <= m, right to about 2^-31 of itself; 0 below 2^-100 and where l is -infinity (rows with a NaN do not
// come here).  h has the table's bits, l is up to 2^-8 of h.
__device__ __forceinline__ FF weight(float l, float m, FF c, const float2 *table)
{
    const float d = l - m, t = d - l;
    const float dl = (l - (d - t)) - (m + t);  // what d has lost
    const float y = fmaxf(d * c.h, -128.0f);
    const float yl = fmaf(dl, c.h, fmaf(d, c.l, fmaf(d, c.h, -y)));
    // y + yl = k/128 + f, |f| <= 1/256
    const float magic = 12582912.0f;  // 1.5 * 2^23
    const float z = fmaf(y, 128.0f, magic);
    const float f = fmaf(z - magic, -0.0078125f, y) + yl;
    // 2^f - 1 = f ln2 + (f ln2)^2 / 2 + (f ln2)^3 / 6, the next term below 2^-38
    const float g = f * fmaf(f, fmaf(f, 0x1.c6b08ep-5f, 0x1.ebfbep-3f), 0x1.62e43p-1f);
    const float2 T = table[__float_as_int(z) & 127];
    // 2^k by its bits: z's integer part from bit 7 on
    const float s = __int_as_float(((__float_as_int(z) & ~127) << 16) + 0x3f800000);
    return y > -100.0f ? FF{T.x * s, fmaf(T.x, g, T.y) * s} : FF{0.0f, 0.0f};
}

// max(R - S q, 0)
__device__ __forceinline__ FF residual(FF R, float q, FF S)
{
    const float p = q * S.h;
    const float pl = fmaf(q, S.h, -p) + q * S.l;
    const float s = R.h - p, t = s - R.h;
    const float e = (R.h - (s - t)) - (p + t) + (R.l - pl);
    const float h = s + e;
    return h > 0.0f ? FF{h, e - (h - s)} : FF{0.0f, 0.0f};
}

// --------------------------------------------------------------- helpers --
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return bf2f(v); }

// A row seen as 16-byte vectors of E elements; the first and last may stick out.
template <typename T>
struct RowVecs {
    static constexpr int E = 16 / (int)sizeof(T);
    const T *row;
    int n, mis, nv;
    __device__ __forceinline__ RowVecs(const T *r, int len) : row(r), n(len)
    {
        mis = (int)(reinterpret_cast<uintptr_t>(r) % 16 / sizeof(T));
        nv = (mis + n + E - 1) / E;
    }
    __device__ __forceinline__ int first(int v) const { return v * E - mis; }
    // Elements of vector v; `fill` outside the row.
    __device__ __forceinline__ void load(int v, float fill, float x[E]) const
    {
        const int e0 = first(v);
        if (v < nv && e0 >= 0 && e0 + E <= n) {
            const uint4 u = ld_stream16(row + e0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < E; ++i)
                x[i] = sizeof(T) == 4 ? __uint_as_float(w[i % 4]) : (i & 1) ? bf_hi(w[i / 2 % 4]) : bf_lo(w[i / 2 % 4]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = e0 + i >= 0 && e0 + i < n ? to_f(row[e0 + i]) : fill;
        }
    }
};

// E consecutive elements from `at` on (any alignment), 0 outside the row.
template <typename T, int E>
__device__ __forceinline__ void load_at(const T *row, int at, int n, float x[E])
{
    if (at >= 0 && at + E <= n && reinterpret_cast<uintptr_t>(row + at) % 16 == 0 && E * sizeof(T) % 16 == 0) {
#pragma unroll
        for (int v = 0; v < (int)(E * sizeof(T) / 16); ++v) {
            const uint4 u = ld_stream16(reinterpret_cast<const char *>(row + at) + 16 * v);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 16 / (int)sizeof(T); ++i)
                x[v * 16 / (int)sizeof(T) + i] = sizeof(T) == 4 ? __uint_as_float(w[i % 4]) : (i & 1) ? bf_hi(w[i / 2 % 4]) : bf_lo(w[i / 2 % 4]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = at + i >= 0 && at + i < n ? to_f(row[at + i]) : 0.0f;
    }
}

struct VerPart {  // a CTA's share of a row's statistics
    float m, s;
    int idx;
};

enum VerCode { kAccept, kPass, kEnd };

struct VerShared {
    // the sequence, as CTA 0 read it
    int parent[kMaxTree], token[kMaxTree];
    float draw[kMaxTree];
    int count, greedy, valid;
    FF c;
    // what the current node's row and draft row hold at its children's tokens, as CTA 0 read them
    float child_l[2][kMaxTree], child_q[2][kMaxTree];
    // the CTAs' shares of a row's maximum and sum, and of a pass's sum
    VerPart part[2][kVerCtas];
    double total[2][kVerCtas];
    // within the CTA
    VerPart warp_part[kVerWarps];
    FF warp_total[kVerWarps];
    FF S[kMaxTree];  // sum of R before rejection j
    int excluded[kMaxTree], nex, rejected;
    float2 table[128];
    int path[kMaxTree];
    float m;          // the row's maximum ...
    int best;         // ... and its place, -1 for a row without a distribution
    int code, node, current;
    double sum, base;
    int sel;
};

// One row of logits and its share of this warp.
template <typename L>
struct VerRow {
    RowVecs<L> vecs;
    int v0, v1;  // the warp's vectors
    __device__ __forceinline__ VerRow(const L *row, int vocab, int rank, int ctas) : vecs(row, vocab)
    {
        const int per = (vecs.nv + ctas * kVerWarps - 1) / (ctas * kVerWarps);
        v0 = min((rank * kVerWarps + (int)threadIdx.x / 32) * per, vecs.nv);
        v1 = min(v0 + per, vecs.nv);
    }
};

// This warp's share of another row, which begins at `next`, into L2.
template <typename T, typename L>
__device__ __forceinline__ void prefetch_row(const T *next, const VerRow<L> &r)
{
    constexpr int LINE = 128 / (int)sizeof(T);
    const int e1 = min(r.vecs.first(r.v1), r.vecs.n);
    for (int e = max(r.vecs.first(r.v0), 0) + (int)threadIdx.x % 32 * LINE; e < e1; e += 32 * LINE)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(next + e));
}

__device__ __forceinline__ VerPart join(VerPart a, float c)  // over the warp
{
    float top = a.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int first = (int)__reduce_min_sync(0xffffffffu, (unsigned)(a.m == top ? a.idx : 0x7fffffff));
    float s = a.m > -CUDART_INF_F ? a.s * ex2((a.m - top) * c) : a.m == a.m ? 0.0f : a.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return VerPart{top, s, first};
}

// The lane's share of a row's maximum and its place (greedy) or sum.
template <typename L>
__device__ __forceinline__ VerPart row_part(const VerRow<L> &r, bool greedy, float c)
{
    constexpr int E = RowVecs<L>::E, U = 4;
    float m = -CUDART_INF_F, s = 0.0f, sl = 0.0f;
    int best = 0x7fffffff;
    for (int v = r.v0 + (int)threadIdx.x % 32; v < r.v1; v += 32 * U) {
        float x[U][E];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (v + 32 * j < r.v1) {
                r.vecs.load(v + 32 * j, -CUDART_INF_F, x[j]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) x[j][i] = -CUDART_INF_F;
            }
        }
        if (greedy) {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (x[j][i] > m) best = r.vecs.first(v + 32 * j) + i;
                    m = max_nan(m, x[j][i]);
                }
            continue;
        }
        float top = x[0][0];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) top = max_nan(top, x[j][i]);
        if (!(top <= m)) {
            const float now = max_nan(m, top);
            const float f = m > -CUDART_INF_F ? ex2((m - now) * c) : 0.0f;
            s *= f, sl *= f, m = now;
        }
        if (m == -CUDART_INF_F) continue;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float w = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) w += ex2((x[j][i] - m) * c);
            const float t = s + w, z = t - s;
            sl += (s - (t - z)) + (w - z);
            s = t;
        }
    }
    return VerPart{m, s + sl, best};
}

// R of the E elements from vector v on: after `rejected` rejections (draft), or without the excluded tokens (no draft).
template <typename L, typename Q, bool DRAFT>
__device__ __forceinline__ void residuals(const VerShared &sh, const VerRow<L> &r, const Q *qrow, int vocab, int v, int rejected, int nex,
                                          FF R[RowVecs<L>::E])
{
    constexpr int E = RowVecs<L>::E;
    float x[E], q[E];
    const int e0 = r.vecs.first(v);
    r.vecs.load(v, -CUDART_INF_F, x);
    if (DRAFT && rejected > 0) load_at<Q, E>(qrow, e0, vocab, q);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        R[i] = weight(x[i], sh.m, sh.c, sh.table);
        if (DRAFT) {
            for (int j = 0; j < rejected; ++j) R[i] = residual(R[i], q[i], sh.S[j]);
        } else {
            for (int j = 0; j < nex; ++j)
                if (sh.excluded[j] == e0 + i) R[i] = FF{0.0f, 0.0f};
        }
    }
}

// The sum of a vector's numbers: what of them is a multiple of 2^-14 adds up without rounding, the rest is below 2^-14.
template <int E>
__device__ __forceinline__ FF vec_sum(const FF R[E])
{
    FF s{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float h = (R[i].h + 768.0f) - 768.0f;  // 1.5 * 2^9: its last place is 2^-14
        s.h += h, s.l += (R[i].h - h) + R[i].l;
    }
    return s;
}

__device__ __forceinline__ FF ff_warp_sum(FF a)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) a = ff_add(a, FF{__shfl_xor_sync(0xffffffffu, a.h, d), __shfl_xor_sync(0xffffffffu, a.l, d)});
    return a;
}

// Sum of R over the row, by all threads of the cluster: sh.sum, the CTAs' shares in sh.total[turn], the warps' in sh.warp_total.
template <typename L, typename Q, bool DRAFT>
__device__ __forceinline__ void sum_pass(VerShared &sh, cg::cluster_group &cl, const VerRow<L> &r, const Q *qrow, int vocab, int turn)
{
    constexpr int E = RowVecs<L>::E;
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks(), lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int rejected = sh.rejected;
    int nex = 0;  // excluded tokens, where any is among this warp's elements
    for (int j = 0; j < sh.nex; ++j)
        if (sh.excluded[j] >= r.vecs.first(r.v0) && sh.excluded[j] < r.vecs.first(r.v1)) nex = sh.nex;
    FF acc{0.0f, 0.0f};
    for (int v = r.v0 + lane; v < r.v1; v += 32) {
        FF R[E];
        residuals<L, Q, DRAFT>(sh, r, qrow, vocab, v, rejected, nex, R);
        acc = ff_add(acc, vec_sum<E>(R));
    }
    acc = ff_warp_sum(acc);
    if (lane == 0) sh.warp_total[warp] = acc;
    __syncthreads();
    if (warp == 0) {
        double t = lane < kVerWarps ? ff_double(sh.warp_total[lane]) : 0.0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (lane < ctas) cl.map_shared_rank(&sh, lane)->total[turn][rank] = t;
    }
    cl.sync();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int i = 0; i < ctas; ++i) t += sh.total[turn][i];
        sh.sum = t;
    }
    __syncthreads();
}

// The token that the draw falls on: the CTA, then its warp, then the element, by running sums.
template <typename L, typename Q, bool DRAFT>
__device__ __forceinline__ void choose(VerShared &sh, int rank, int ctas, const VerRow<L> &r, const Q *qrow, int vocab, int turn,
                                       int32_t *next)
{
    constexpr int E = RowVecs<L>::E;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const double target = (double)sh.draw[0] * sh.sum;
    if (warp == 0) {
        double before = 0.0, base = 0.0;
        int sel = -1, last = 0;
        for (int i = 0; i < ctas; ++i) {
            const double t = sh.total[turn][i];
            if (t > 0.0) {
                last = i;
                if (sel < 0) base = before;
                if (sel < 0 && before + t > target) sel = i;
            }
            before += t;
        }
        int w = -1;
        if ((sel < 0 ? last : sel) == rank) {
            const double mine = lane < kVerWarps ? ff_double(sh.warp_total[lane]) : 0.0;
            double upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
            const unsigned over = __ballot_sync(0xffffffffu, mine > 0.0 && base + upto > target);
            w = over ? __ffs((int)over) - 1 : 31 - __clz((int)some);
            if (lane == w) sh.base = base + (upto - mine);
        }
        if (lane == 0) sh.sel = w;
    }
    __syncthreads();
    if (warp != sh.sel) return;
    double base = sh.base;
    int last = 0;
    for (int v0 = r.v0; v0 < r.v1; v0 += 32) {
        FF R[E];
        if (v0 + lane < r.v1) {
            residuals<L, Q, DRAFT>(sh, r, qrow, vocab, v0 + lane, sh.rejected, sh.nex, R);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) R[i] = FF{0.0f, 0.0f};
        }
        const FF acc = vec_sum<E>(R);
        const int e0 = r.vecs.first(v0 + lane);
        int top = -1;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (R[i].h > 0.0f) top = e0 + i;
        top = __reduce_max_sync(0xffffffffu, top);
        if (top >= 0) last = top;
        const double tile = ff_double(ff_warp_sum(acc));
        if (base + tile > target) {
            double upto = ff_double(acc);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            double run = base + __shfl_up_sync(0xffffffffu, upto, 1);
            if (lane == 0) run = base;
            unsigned hit = 0x7fffffffu;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                run += ff_double(R[i]);
                if (R[i].h > 0.0f && run > target) hit = min(hit, (unsigned)(e0 + i));
            }
            hit = __reduce_min_sync(0xffffffffu, hit);
            if (hit != 0x7fffffffu) {
                last = (int)hit;
                break;
            }
        }
        base += tile;
    }
    if (lane == 0) *next = last;
}

template <typename L, typename Q, bool DRAFT>
__global__ void __launch_bounds__(kVerThreads, 1) verify_kernel(const __grid_constant__ VerifyArgs a)
{
    __shared__ VerShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int b = (int)blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t row0 = (int64_t)b * a.n;
    if (tid < 128) sh.table[tid] = kExp2Table[tid];
    cl.sync();  // from here on peers write into this CTA's memory
    pdl_wait();
    pdl_trigger();

    // CTA 0 reads the sequence for all, so that all decide from the same numbers and take the same way
    if (rank == 0) {
        if (tid < a.n) {
            const int parent = a.mask ? 63 - __clzll((long long)(a.mask[row0 + tid] & ((1ull << tid) - 1))) : tid - 1;
            const int token = a.tokens[row0 + tid];
            const float draw = a.uniforms[row0 + tid];
            for (int r = 0; r < ctas; ++r) {
                VerShared *p = cl.map_shared_rank(&sh, r);
                p->parent[tid] = parent, p->token[tid] = token, p->draw[tid] = draw;
            }
        }
        if (tid == kMaxTree) {
            const int count = a.count ? min(max(a.count[b], 0), a.n) : a.n;
            const float t = a.temperatures ? a.temperatures[b] : a.temperature;
            const FF c = ff_of(1.4426950408889634 / (double)fminf(t, 1e30f));
            for (int r = 0; r < ctas; ++r) {
                VerShared *p = cl.map_shared_rank(&sh, r);
                p->count = count, p->greedy = t < 1e-6f, p->valid = t == t, p->c = c;
            }
        }
    }
    cl.sync();
    if (sh.count == 0) {
        if (rank == 0 && tid < a.n) a.path[row0 + tid] = -1;
        if (rank == 0 && tid == 0) a.accepted[b] = 0, a.next[b] = -1;
        return;
    }

    const bool greedy = sh.greedy;
    int node = 0, level = 0, turn = 0;
    for (;;) {
        const VerRow<L> row(static_cast<const L *>(a.logits) + (row0 + node) * a.logits_stride, a.vocab, rank, ctas);
        const Q *qrow = DRAFT ? static_cast<const Q *>(a.draft) + (row0 + node) * a.draft_stride : nullptr;
        const int side = level & 1;
        if (tid == 0) sh.path[level] = node;
        if (rank == 0 && tid >= kMaxTree && tid < kMaxTree + a.n) {
            const int i = tid - kMaxTree, k = sh.token[i];
            if (i < sh.count && i > node && sh.parent[i] == node) {
                const bool in = k >= 0 && k < a.vocab;
                const float l = in ? to_f(row.vecs.row[k]) : -CUDART_INF_F;
                const float q = DRAFT ? (in ? to_f(qrow[k]) : 0.0f) : 1.0f;
                for (int r = 0; r < ctas; ++r) {
                    VerShared *p = cl.map_shared_rank(&sh, r);
                    p->child_l[side][i] = l, p->child_q[side][i] = q;
                }
            }
        }
        if (a.n > 1) {
            // the first child's row is the likeliest next one: towards L2 while this one is read
            const unsigned lo = __ballot_sync(0xffffffffu, lane < sh.count && lane > node && sh.parent[lane] == node);
            const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < sh.count && lane + 32 > node && sh.parent[lane + 32] == node);
            const int kid = lo ? __ffs((int)lo) - 1 : hi ? 31 + __ffs((int)hi) : 0;
            if (kid) prefetch_row(static_cast<const L *>(a.logits) + (row0 + kid) * a.logits_stride, row);
        }
        const VerPart mine = join(row_part(row, greedy, sh.c.h), sh.c.h);
        if (lane == 0) sh.warp_part[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const VerPart p = join(lane < kVerWarps ? sh.warp_part[lane] : VerPart{-CUDART_INF_F, 0.0f, 0x7fffffff}, sh.c.h);
            if (lane < ctas) cl.map_shared_rank(&sh, lane)->part[turn][rank] = p;
        }
        cl.sync();

        // The children, in order, by warp 0 of every CTA alike.  A pass over R is asked for where a test is too close
        // for the fast sum, and where a rejection (draft) changes all of R.
        double S = 0.0, S0 = 0.0;
        bool exact = false;
        uint64_t kids = 0;
        int k = 0, nex = 0;
        FF R[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // of nodes lane and lane + 32
        if (warp == 0) {
            const VerPart p = join(lane < ctas ? sh.part[turn][lane] : VerPart{-CUDART_INF_F, 0.0f, 0x7fffffff}, sh.c.h);
            const bool valid = sh.valid && p.m > -CUDART_INF_F && p.m < CUDART_INF_F;
            S = S0 = p.s;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = lane + 32 * h;
                const bool kid = valid && i < sh.count && i > node && sh.parent[i] == node;
                kids |= (uint64_t)__ballot_sync(0xffffffffu, kid) << (32 * h);
                if (kid && !greedy) R[h] = weight(sh.child_l[side][i], p.m, sh.c, sh.table);
            }
            if (lane == 0) sh.m = p.m, sh.best = valid ? p.idx : -1, sh.nex = 0, sh.rejected = 0;
            if (lane == 0 && valid && !greedy) sh.best = 0;
            __syncwarp();
        }
        turn ^= 1;
        for (;;) {
            if (warp == 0) {
                int code = kEnd, to = node;
                while (kids) {
                    const int i = __ffsll((long long)kids) - 1;
                    if (greedy) {
                        if (sh.token[i] == sh.best) {
                            code = kAccept, to = i;
                            break;
                        }
                        kids &= kids - 1;
                        continue;
                    }
                    const FF Ri{__shfl_sync(0xffffffffu, i < 32 ? R[0].h : R[1].h, i % 32), __shfl_sync(0xffffffffu, i < 32 ? R[0].l : R[1].l, i % 32)};
                    const double have = ff_double(Ri), want = (double)sh.draw[i] * (double)sh.child_q[side][i] * S;
                    const bool yes = want < have;
                    if (!exact && ((have > 0.0 && fabs(want - have) <= kTol * S0) || (DRAFT && !yes))) {
                        code = kPass;
                        break;
                    }
                    if (yes) {
                        code = kAccept, to = i;
                        break;
                    }
                    kids &= kids - 1;
                    if (DRAFT) {
                        const FF f = ff_of(S);
                        if (lane == 0) sh.S[k] = f;
                        ++k;
#pragma unroll
                        for (int h = 0; h < 2; ++h) R[h] = residual(R[h], sh.child_q[side][lane + 32 * h], f);
                        code = kPass;
                        break;
                    }
                    // the token leaves the row, for later siblings too
                    const int token = sh.token[i];
                    if (have > 0.0) {
                        S -= have;
                        if (lane == 0) sh.excluded[nex] = token;
                        ++nex;
                        exact = false;  // the last pass's shares no longer hold
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (sh.token[lane + 32 * h] == token) R[h] = FF{0.0f, 0.0f};
                }
                if (lane == 0) sh.code = code, sh.node = to, sh.rejected = k, sh.nex = nex, sh.current = exact;
            }
            __syncthreads();
            if (sh.code != kPass) break;
            if (DRAFT && sh.rejected == 0) prefetch_row(qrow, row);  // wanted if the child is rejected, as it nearly is
            sum_pass<L, Q, DRAFT>(sh, cl, row, qrow, a.vocab, turn);
            turn ^= 1;
            if (warp == 0) S = sh.sum, exact = true;
        }
        if (sh.code == kAccept) {
            node = sh.node;
            ++level;
            continue;
        }

        if (greedy || sh.best < 0) {
            if (rank == 0 && tid == 0) a.next[b] = sh.best;
        } else {
            if (!sh.current) {
                sum_pass<L, Q, DRAFT>(sh, cl, row, qrow, a.vocab, turn);
                turn ^= 1;
            }
            if (!(sh.sum > 0.0)) {  // nothing is left: from the row itself
                __syncthreads();
                if (tid == 0) sh.rejected = 0, sh.nex = 0;
                __syncthreads();
                sum_pass<L, Q, DRAFT>(sh, cl, row, qrow, a.vocab, turn);
                turn ^= 1;
            }
            choose<L, Q, DRAFT>(sh, rank, ctas, row, qrow, a.vocab, turn ^ 1, a.next + b);
        }
        break;
    }
    if (rank == 0) {
        if (tid < a.n) a.path[row0 + tid] = tid <= level ? sh.path[tid] : -1;
        if (tid == 0) a.accepted[b] = level + 1;
    }
}

template <typename L, typename Q, bool DRAFT>
static cudaError_t verify_launch(const VerifyArgs &a, int ctas, cudaStream_t st)
{
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.batch * ctas));
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(verify_kernel<L, Q, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, verify_kernel<L, Q, DRAFT>, a);
}

template <typename L>
static cudaError_t verify_draft(const VerifyArgs &a, int ddt, int ctas, cudaStream_t st)
{
    if (!a.draft) return verify_launch<L, float, false>(a, ctas, st);
    return ddt == WL_OUT_F32 ? verify_launch<L, float, true>(a, ctas, st) : verify_launch<L, bf16, true>(a, ctas, st);
}

wl_status launch_verify(const VerifyArgs &a, int ldt, int ddt, const DeviceInfo *di, cudaStream_t st)
{
    // A sequence's CTAs: as many as fill the GPU, at most one for 8192 tokens of the vocabulary.
    int ctas = kVerCtas;
    while (ctas > 1 && ((int64_t)a.batch * ctas > di->sm_count || (int64_t)a.vocab < 8192 * (ctas / 2))) ctas /= 2;
    const cudaError_t e = ldt == WL_OUT_F32 ? verify_draft<float>(a, ddt, ctas, st) : verify_draft<bf16>(a, ddt, ctas, st);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_verify launch");
}

}  // namespace wl
