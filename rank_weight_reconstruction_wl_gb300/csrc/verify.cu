// verify.cu -- drafted tokens accepted or rejected against the model's
// distribution, and the token after them, from given random numbers.
//
//     w_i = 2^((l_i - max l) log2(e) / t),  R = w,  S = sum R
//     child c of node u, token k:  accepted if  r_c q_k S < R_k,  else R = max(R - S q, 0)
//     next: lowest i with R_i > 0 and R_0 + ... + R_i > r_0 S
//
// Only the rows of accepted nodes are read: a cluster owns a sequence and walks
// down its tree, one pass over a row (split over the cluster's warps) per node.
// Bound by the chain of passes (load, reductions, cluster barrier): 4 us a node
// for a vocabulary of 262144, 7 where 32 sequences fill the GPU.  Sampling one
// such token 11 us, 32 drafted trees of 24 62 to 68, 16 chains of 8 with draft
// rows 98.5 (two exact passes after the walk); the trees with draft rows 215 to
// 273.  Statistics of all rows first and a walk after would read 6 times the bytes
// for those trees and 20 times for wide greedy ones; for chains, most of whose
// rows are walked, 1.8 times, which has not been tried.
//
// Decisions.  A random number closer to a border between two tokens than the
// sums' rounding would give another token than exact arithmetic does, and a
// vocabulary has 10^5 borders.  So the sums that decide are made of weights held
// as two floats (two_float.h), and the sums of the fast pass decide only where
// their error (a few 10^-6 of the row's sum) cannot matter.
//
// How near a border may be.  Weights and sums are off by e = 2^-36 of themselves
// (weights below 2^-32 by more, but all of them weigh 2^-8 at most).  A border
// among plain weights moves by 2 u (1 - u) e of the row's sum S: what is off by
// the same on both sides cancels.  After j rejections against q a token has
// w_i - q_i (S_0 + ... + S_{j-1}).  Let A_j be the error of that sum: S_j, the
// sum over the tokens left, is off by D - Q A_j, |D| <= e S, Q <= 1 their mass in
// q, so A_{j+1} = (1 - Q) A_j + D, |A_j| <= j e S, and the errors of all R add up
// to (j + 1) e S at most: 2^-30 of S for 63 rejections.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <atomic>

#include "cache_row.cuh"
#include "dec_ptx.cuh"
#include "two_float.h"

namespace cg = cooperative_groups;

namespace wl {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCtas = 16;  // CTAs of a cluster at most
constexpr float kTolSum = 6e-7f, kTolBit = 1.3e-7f;
// A fast sum is right to kTolSum + kTolBit log2(vocab) of the row's sum: 2^-22 for ex2, three roundings of 2^-24 in a
// vector's sum, and three of y = (l - max) c, each |y| 2^-24 ln2 of the weight, whose sum over the row is at most
// log2(vocab) 2^-24 ln2 of its sum (the entropy of the weights is at most log2(vocab)).

// --------------------------------------------------------------- helpers --
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest of the warp; NaN if one is.
__device__ __forceinline__ float warp_max_nan(float a)
{
    float y;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(a));
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
    // Vector v as loaded; -infinity outside the row (v < v1, the end of a share).
    __device__ __forceinline__ uint4 raw(int v, int v1) const
    {
        const int e0 = first(v);
        if (v < v1 && e0 >= 0 && e0 + E <= n) return ld_stream16(row + e0);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
        if (v < v1) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (e0 + i >= 0 && e0 + i < n) {
                    if constexpr (sizeof(T) == 4) {
                        w[i % 4] = __float_as_uint(row[e0 + i]);
                    } else {
                        const uint32_t u = __float_as_uint(to_f(row[e0 + i])) >> 16;
                        w[i / 2 % 4] = i & 1 ? (w[i / 2 % 4] & 0xffffu) | u << 16 : (w[i / 2 % 4] & 0xffff0000u) | u;
                    }
                }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void unpack(const uint4 &u, float x[E])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < E; ++i)
            x[i] = sizeof(T) == 4 ? __uint_as_float(w[i % 4]) : (i & 1) ? bf_hi(w[i / 2 % 4]) : bf_lo(w[i / 2 % 4]);
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

__device__ __forceinline__ FF ff_warp_sum(FF a)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) a = ff_add(a, FF{__shfl_xor_sync(0xffffffffu, a.h, d), __shfl_xor_sync(0xffffffffu, a.l, d)});
    return a;
}

struct VerPart {  // a share of a row: its largest logit, the first place of it, the sum of the weights relative to it
    float m;
    FF s;
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
    FF total[2][kVerCtas];
    // within the CTA
    VerPart warp_part[32];  // empty past kVerWarps, as the two below
    FF warp_total[32];
    FF S[kMaxTree];  // sum of R before rejection j
    int excluded[kMaxTree], nex, rejected;
    float out_w[kMaxTree];  // weights of the excluded
    float table[64];
    int path[kMaxTree];
    float part_sum;   // the row's sum by the fast pass
    float m;          // the row's maximum ...
    int best;         // ... and its place, -1 for a row without a distribution
    int code, node, current;
    FF sum, base, target;
    FF tile_sum[32], tile_base;
    int sel, sure, again, tile, over;
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

// A share's sum relative to a larger maximum.
__device__ __forceinline__ FF rescaled(const VerPart &a, float top, const VerShared &sh)
{
    if (!(a.m > -CUDART_INF_F)) return FF{a.m == a.m ? 0.0f : a.m, 0.0f};
    return ff_norm(ff_mul(a.s, weight(a.m, top, sh.c, sh.table)));
}

// Shares of the warp's lanes together: the maximum with its place (greedy) or with the sum.
__device__ __forceinline__ VerPart join(const VerPart &a, const VerShared &sh)
{
    const float top = warp_max_nan(a.m);
    if (sh.greedy) return VerPart{top, {0.0f, 0.0f}, (int)__reduce_min_sync(0xffffffffu, (unsigned)(a.m == top ? a.idx : 0x7fffffff))};
    return VerPart{top, ff_norm(ff_warp_sum(rescaled(a, top, sh))), 0};
}

// The lane's share of a row's maximum and its place (greedy) or sum.
template <typename L>
__device__ __forceinline__ VerPart row_part(const VerShared &sh, const VerRow<L> &r, bool greedy)
{
    const float c = sh.c.h;
    constexpr int E = RowVecs<L>::E, U = 8;
    float m = -CUDART_INF_F, s = 0.0f, sl = 0.0f;
    int best = 0x7fffffff;
    uint4 ahead[U];  // the next vectors, under way while these are summed
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < U; ++j) ahead[j] = r.vecs.raw(r.v0 + lane + 32 * j, r.v1);
    for (int v = r.v0 + lane; v < r.v1; v += 32 * U) {
        uint4 now[U];
        float x[E], top = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < U; ++j) now[j] = ahead[j];
#pragma unroll
        for (int j = 0; j < U; ++j) ahead[j] = r.vecs.raw(v + 32 * (U + j), r.v1);
        if (greedy) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                RowVecs<L>::unpack(now[j], x);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (x[i] > m) best = r.vecs.first(v + 32 * j) + i;
                    m = max_nan(m, x[i]);
                }
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            RowVecs<L>::unpack(now[j], x);
#pragma unroll
            for (int i = 0; i < E; ++i) top = max_nan(top, x[i]);
        }
        if (!(top <= m)) {
            const float next = max_nan(m, top);
            const FF f = m > -CUDART_INF_F ? ff_mul(FF{s, sl}, weight(m, next, sh.c, sh.table)) : FF{0.0f, 0.0f};
            s = f.h, sl = f.l, m = next;
        }
        if (m == -CUDART_INF_F) continue;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            RowVecs<L>::unpack(now[j], x);
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = ex2((x[i] - m) * c);
#pragma unroll
            for (int d = 1; d < E; d *= 2)
#pragma unroll
                for (int i = 0; i < E; i += 2 * d) x[i] += x[i + d];
            const float w = x[0], t = s + w, z = t - s;
            sl += (s - (t - z)) + (w - z);
            s = t;
        }
    }
    return VerPart{m, ff_norm(FF{s, sl}), best};
}

// f(i, R_i) for the elements of a vector as loaded, from element e0 on: R after `rejected` rejections (draft), or without
// the excluded tokens (no draft).  A word at a time, not unrolled: this code runs a few times in a launch, and unrolled
// it took longer to be fetched than to run (5 us of 14 for a vocabulary of 1000).
template <typename L, bool DRAFT, typename F>
__device__ __forceinline__ void each_R(const VerShared &sh, uint4 w, const float *qs, int e0, int rejected, int nex, F f)
{
    constexpr int E = RowVecs<L>::E, P = E / 4;  // elements of a word
    float q[E];
    if (DRAFT) {
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = qs[i];
    }
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const int i = e0 + k * P + h;
            FF R = weight(P == 1 ? __uint_as_float(w.x) : h ? bf_hi(w.x) : bf_lo(w.x), sh.m, sh.c, sh.table);
            if (DRAFT) {
#pragma unroll 1
                for (int j = 0; j < rejected; ++j) R = residual(R, q[h], sh.S[j]);
            } else {
#pragma unroll 1
                for (int j = 0; j < nex; ++j)
                    if (sh.excluded[j] == i) R = FF{0.0f, 0.0f};
            }
            f(i, R);
        }
        w.x = w.y, w.y = w.z, w.z = w.w;
        if (DRAFT) {
#pragma unroll
            for (int i = 0; i + P < E; ++i) q[i] = q[i + P];
        }
    }
}

// The sum of a vector's R.  Every addition keeps what it rounds off: many light tokens of equal weight would add up the
// same rounding each.
template <typename L, bool DRAFT>
__device__ __forceinline__ FF vec_sum(const VerShared &sh, const uint4 &w, const float *q, int e0, int rejected, int nex)
{
    FF s{0.0f, 0.0f};
    each_R<L, DRAFT>(sh, w, q, e0, rejected, nex, [&](int, FF R) { s = ff_add(s, R); });
    return s;
}

// Sum of R over the row, by all threads of the cluster: sh.sum, the CTAs' shares in sh.total[turn], the warps' in sh.warp_total.
template <typename L, typename Q, bool DRAFT>
__device__ __noinline__ void sum_pass(VerShared &sh, cg::cluster_group &cl, const VerRow<L> &r, const Q *qrow, int vocab, int turn)
{
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks(), lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int rejected = sh.rejected;
    int nex = 0;  // excluded tokens, where any is among this warp's elements
    for (int j = 0; j < sh.nex; ++j)
        if (sh.excluded[j] >= r.vecs.first(r.v0) && sh.excluded[j] < r.vecs.first(r.v1)) nex = sh.nex;
    FF acc{0.0f, 0.0f};
    // the next vectors, of the draft row too, are under way while these are summed
    constexpr int E = RowVecs<L>::E;
    uint4 ahead[2] = {r.vecs.raw(r.v0 + lane, r.v1), r.vecs.raw(r.v0 + lane + 32, r.v1)};
    float q[E], qa[E];
    if (DRAFT && rejected > 0) load_at<Q, E>(qrow, r.vecs.first(r.v0 + lane), vocab, qa);
    for (int v = r.v0 + lane; v < r.v1; v += 32) {
        const uint4 raw = ahead[0];
        ahead[0] = ahead[1], ahead[1] = r.vecs.raw(v + 64, r.v1);
        if (DRAFT && rejected > 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = qa[i];
            load_at<Q, E>(qrow, r.vecs.first(v + 32), vocab, qa);
        }
        acc = ff_sum(acc, vec_sum<L, DRAFT>(sh, raw, q, r.vecs.first(v), rejected, nex));
    }
    acc = ff_norm(ff_warp_sum(acc));
    if (lane == 0) sh.warp_total[warp] = acc;
    __syncthreads();
    if (warp == 0) {
        const FF t = ff_norm(ff_warp_sum(sh.warp_total[lane]));
        if (lane < ctas) cl.map_shared_rank(&sh, lane)->total[turn][rank] = t;
    }
    cl.sync();
    if (warp == 0) {
        const FF t = ff_norm(ff_warp_sum(lane < ctas ? sh.total[turn][lane] : FF{0.0f, 0.0f}));
        if (lane == 0) sh.sum = t;
    }
    __syncthreads();
}

// Inclusive running sums over the warp.
__device__ __forceinline__ FF ff_warp_scan(FF a)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const FF o{__shfl_up_sync(0xffffffffu, a.h, d), __shfl_up_sync(0xffffffffu, a.l, d)};
        if ((int)threadIdx.x % 32 >= d) a = ff_norm(ff_add(a, o));
    }
    return a;
}

// The first lane whose running sum of `mine` from `base` on passes target, or the last with any; *before: the sum up to
// it; *end: the sum of all; false where none passes.
__device__ __forceinline__ bool pick(FF mine, FF base, FF target, int *at, FF *before, FF *end)
{
    const int lane = threadIdx.x % 32;
    const FF upto = ff_norm(ff_add(base, ff_warp_scan(mine)));
    const unsigned some = __ballot_sync(0xffffffffu, mine.h > 0.0f), over = __ballot_sync(0xffffffffu, mine.h > 0.0f && ff_less(target, upto));
    const int i = over ? __ffs((int)over) - 1 : some ? 31 - __clz((int)some) : -1;
    FF b{__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
    if (lane == 0) b = base;
    *before = FF{__shfl_sync(0xffffffffu, b.h, i & 31), __shfl_sync(0xffffffffu, b.l, i & 31)};
    *end = FF{__shfl_sync(0xffffffffu, upto.h, 31), __shfl_sync(0xffffffffu, upto.l, 31)};
    *at = i;
    return over != 0;
}

// What the fast pass has of a share of the row, without the excluded tokens in its vectors [v0, v1).
template <typename L>
__device__ __forceinline__ FF fast_share(const VerShared &sh, const VerPart &p, const VerRow<L> &r, int v0, int v1)
{
    FF s = rescaled(p, sh.m, sh);
    for (int j = 0; j < sh.nex; ++j)
        if (sh.excluded[j] >= r.vecs.first(v0) && sh.excluded[j] < r.vecs.first(v1)) s = ff_norm(ff_add(s, FF{-sh.out_w[j], 0.0f}));
    return s.h > 0.0f ? s : FF{0.0f, 0.0f};
}

// The token that the draw falls on: the CTA, its warp, of that warp's elements the tile (all warps of the CTA sum one
// each), then the element, by running sums.  fast: CTA and warp by the sums of the fast pass, which are `tol` off at most;
// sh.sure tells (in the CTA that has the token) whether that decides it.  Else by those of sum_pass.
template <typename L, typename Q, bool DRAFT>
__device__ __noinline__ void choose(VerShared &sh, int rank, int ctas, const VerRow<L> &r, const Q *qrow, int vocab, int turn, bool fast,
                                    float tol, int32_t *next)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int per = (r.vecs.nv + ctas * kVerWarps - 1) / (ctas * kVerWarps);
    if (warp == 0) {
        FF mine{0.0f, 0.0f}, base, end, sum = sh.sum;
        if (lane < ctas) mine = fast ? fast_share(sh, sh.part[turn][lane], r, lane * kVerWarps * per, (lane + 1) * kVerWarps * per) : sh.total[turn][lane];
        if (fast) sum = ff_norm(ff_warp_sum(mine));
        const FF target = ff_mul(sum, sh.draw[0]);
        int cta, w = -1;
        pick(mine, FF{0.0f, 0.0f}, target, &cta, &base, &end);
        if (max(cta, 0) == rank) {
            const int g = rank * kVerWarps + lane;
            pick(fast ? fast_share(sh, sh.warp_part[lane], r, g * per, (g + 1) * per) : sh.warp_total[lane], base, target, &w, &base, &end);
            w = max(w, 0);
        }
        if (lane == 0) sh.sel = w, sh.base = base, sh.target = target, sh.sure = 0;
    }
    __syncthreads();
    if (sh.sel < 0) return;
    const FF target = sh.target;
    const int v0 = min((rank * kVerWarps + sh.sel) * per, r.vecs.nv), v1 = min(v0 + per, r.vecs.nv);
    int tile = -1;
    constexpr int E = RowVecs<L>::E;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float q[E];
    FF mine{0.0f, 0.0f};
#pragma unroll 1
    for (int t0 = 0; v0 + 32 * t0 < v1; t0 += kVerWarps) {
        const int v = v0 + 32 * (t0 + warp) + lane;
        raw = r.vecs.raw(v, v1);
        if (DRAFT && sh.rejected > 0) load_at<Q, E>(qrow, r.vecs.first(v), vocab, q);
        mine = vec_sum<L, DRAFT>(sh, raw, q, r.vecs.first(v), sh.rejected, sh.nex);
        const FF s = ff_norm(ff_warp_sum(mine));
        if (lane == 0) sh.tile_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            FF before, end;
            int at;
            const bool over = pick(sh.tile_sum[lane], sh.base, target, &at, &before, &end);
            __syncwarp();
            if (lane == 0) {
                sh.over = over;
                if (at >= 0) sh.tile = t0 + at, sh.tile_base = before;
                else if (t0 == 0) sh.tile = 0, sh.tile_base = before;
                sh.base = end;
            }
        }
        __syncthreads();
        tile = sh.tile;
        if (sh.over) break;
    }
    if (warp != tile % kVerWarps) return;
    const int v = v0 + 32 * tile + lane, e0 = r.vecs.first(v);
    if (!sh.over) {  // the last tile with any, perhaps not of the last round
        raw = r.vecs.raw(v, v1);
        if (DRAFT && sh.rejected > 0) load_at<Q, E>(qrow, e0, vocab, q);
        mine = vec_sum<L, DRAFT>(sh, raw, q, e0, sh.rejected, sh.nex);
    }
    const FF upto = ff_norm(ff_add(sh.tile_base, ff_warp_scan(ff_norm(mine))));
    FF run{__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
    if (lane == 0) run = sh.tile_base;
    int top = -1;
    unsigned hit = 0x7fffffffu;
    bool clear = false;
    each_R<L, DRAFT>(sh, raw, q, e0, sh.rejected, sh.nex, [&](int i, FF R) {
        const FF was = run;
        run = ff_norm(ff_add(run, R));
        if (R.h > 0.0f) top = i;
        if (hit == 0x7fffffffu && R.h > 0.0f && ff_less(target, run)) {
            hit = (unsigned)i;
            clear = target.h - was.h > tol && run.h - target.h > tol;
        }
    });
    const unsigned first = __reduce_min_sync(0xffffffffu, hit);
    top = __reduce_max_sync(0xffffffffu, top);
    const bool sure = __any_sync(0xffffffffu, first != 0x7fffffffu && hit == first && clear);
    if (lane == 0) {
        sh.sure = sure;
        if (!fast || sure) *next = first != 0x7fffffffu ? (int)first : max(top, 0);
    }
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
    if (tid < 32) {
        sh.warp_part[tid] = VerPart{-CUDART_INF_F, {0.0f, 0.0f}, 0x7fffffff};
        sh.warp_total[tid] = sh.tile_sum[tid] = FF{0.0f, 0.0f};
    }
    if (tid < 64) sh.table[tid] = tid < 32 ? kExp2High[tid] : kExp2Low[tid - 32];
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
            const double t = a.temperatures ? (double)a.temperatures[b] : a.temperature;
            const FF c = ff_of(1.4426950408889634 / fmin(t, 1e30));
            for (int r = 0; r < ctas; ++r) {
                VerShared *p = cl.map_shared_rank(&sh, r);
                p->count = count, p->greedy = t < 1e-6, p->valid = t == t, p->c = c;
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
    const float tol = kTolSum + kTolBit * (float)(32 - __clz(a.vocab));
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
        const VerPart mine = join(row_part(sh, row, greedy), sh);
        if (lane == 0) sh.warp_part[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const VerPart p = join(lane < kVerWarps ? sh.warp_part[lane] : VerPart{-CUDART_INF_F, {0.0f, 0.0f}, 0x7fffffff}, sh);
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
            const VerPart p = join(lane < ctas ? sh.part[turn][lane] : VerPart{-CUDART_INF_F, {0.0f, 0.0f}, 0x7fffffff}, sh);
            const bool valid = sh.valid && p.m > -CUDART_INF_F && p.m < CUDART_INF_F;
            S = S0 = ff_double(p.s);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = lane + 32 * h;
                const bool kid = valid && i < sh.count && i > node && sh.parent[i] == node;
                kids |= (uint64_t)__ballot_sync(0xffffffffu, kid) << (32 * h);
                if (kid && !greedy) R[h] = weight(sh.child_l[side][i], p.m, sh.c, sh.table);
            }
            if (lane == 0) sh.part_sum = p.s.h;
            if (lane == 0) sh.m = p.m, sh.best = valid ? p.idx : -1, sh.nex = 0, sh.rejected = 0;
            if (lane == 0 && valid && !greedy) sh.best = 0;
            __syncwarp();
        }
        const int fast_turn = turn;
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
                    const double have = ff_double(Ri), rq = (double)sh.draw[i] * (double)sh.child_q[side][i], want = rq * S;
                    const bool yes = want < have;
                    if (!exact && ((have > 0.0 && fabs(want - have) <= fabs(rq) * tol * S0) || (DRAFT && !yes))) {
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
                        if (lane == 0) sh.excluded[nex] = token, sh.out_w[nex] = (float)have;
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
            if (warp == 0) S = ff_double(sh.sum), exact = true;
        }
        if (sh.code == kAccept) {
            node = sh.node;
            ++level;
            continue;
        }

        if (greedy || sh.best < 0) {
            if (rank == 0 && tid == 0) a.next[b] = sh.best;
        } else {
            bool done = false;
            if (!sh.current && sh.rejected == 0) {
                // by the fast sums, where no border is near; the CTA that has the token tells the others
                if (tid == 0) sh.again = 0;
                cl.sync();
                // Off are the draw's target, by tol of the part u of the sum that it is, and the sum before its token: no
                // more than tol of the whole, nor than 5e-6 of itself (|y| up to 32), and 1e-9 for all smaller weights.
                const float u = fminf(fmaxf(sh.draw[0], 0.0f), 1.0f), off = u * tol + fminf(tol, sh.nex > 0 ? tol : 5e-6f * u) + 1e-9f;
                choose<L, Q, DRAFT>(sh, rank, ctas, row, qrow, a.vocab, fast_turn, true, off * sh.part_sum, a.next + b);
                __syncthreads();
                if (sh.sel >= 0 && !sh.sure && tid < ctas) cl.map_shared_rank(&sh, tid)->again = 1;
                cl.sync();
                done = !sh.again;
            }
            if (!done) {
                if (!sh.current) {
                    sum_pass<L, Q, DRAFT>(sh, cl, row, qrow, a.vocab, turn);
                    turn ^= 1;
                }
                if (!(sh.sum.h > 0.0f)) {  // nothing is left: from the row itself
                    __syncthreads();
                    if (tid == 0) sh.rejected = 0, sh.nex = 0;
                    __syncthreads();
                    sum_pass<L, Q, DRAFT>(sh, cl, row, qrow, a.vocab, turn);
                    turn ^= 1;
                }
                choose<L, Q, DRAFT>(sh, rank, ctas, row, qrow, a.vocab, turn ^ 1, false, 0.0f, a.next + b);
            }
        }
        break;
    }
    if (rank == 0) {
        if (tid < a.n) a.path[row0 + tid] = tid <= level ? sh.path[tid] : -1;
        if (tid == 0) a.accepted[b] = level + 1;
    }
}

template <typename L, typename Q, bool DRAFT>
static cudaError_t verify_launch(const VerifyArgs &a, const DeviceInfo *di, cudaStream_t st)
{
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = st;
    cfg.attrs = at;
    // A sequence's CTAs: as many as let the clusters of all sequences run at once (a second wave doubles the time: 16
    // sequences on clusters of 8, of which fewer fit the GPU's partitions than its SMs would hold, took 118 us where
    // clusters of 7 take 96), one for 4096 tokens of the vocabulary at most.  How many clusters run at once is asked once a device.
    static std::atomic<int> at_once[64][kVerCtas + 1];
    static const int sizes[] = {16, 12, 8, 7, 6, 5, 4, 3, 2, 1};
    for (const int *size = sizes;; ++size) {
        const int ctas = *size;
        at[1].val.clusterDim.x = (unsigned)ctas;
        cfg.gridDim = dim3((unsigned)(a.batch * ctas));
        if (ctas == 1) break;
        if ((int64_t)a.vocab < 4096 * ctas || (int64_t)a.batch * ctas > di->sm_count) continue;
        std::atomic<int> *known = di->device < 64 ? &at_once[di->device][ctas] : nullptr;
        int n = known ? known->load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            cfg.numAttrs = 2;
            cudaError_t e = ctas > 8 ? cudaFuncSetAttribute(verify_kernel<L, Q, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
            if (e == cudaSuccess) {
                cudaLaunchConfig_t ask = cfg;
                ask.attrs = at + 1;
                ask.numAttrs = 1;
                e = cudaOccupancyMaxActiveClusters(&n, verify_kernel<L, Q, DRAFT>, &ask);
            }
            if (e != cudaSuccess) return e;
            n = n > 0 ? n : -1;
            if (known) known->store(n, std::memory_order_relaxed);
        }
        if (a.batch <= n) break;
    }
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<L, Q, DRAFT>, a);
}

template <typename L>
static cudaError_t verify_draft(const VerifyArgs &a, int ddt, const DeviceInfo *di, cudaStream_t st)
{
    if (!a.draft) return verify_launch<L, float, false>(a, di, st);
    return ddt == WL_OUT_F32 ? verify_launch<L, float, true>(a, di, st) : verify_launch<L, bf16, true>(a, di, st);
}

wl_status launch_verify(const VerifyArgs &a, int ldt, int ddt, const DeviceInfo *di, cudaStream_t st)
{
    const cudaError_t e = ldt == WL_OUT_F32 ? verify_draft<float>(a, ddt, di, st) : verify_draft<bf16>(a, ddt, di, st);
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_verify launch");
}

}  // namespace wl
