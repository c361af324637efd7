// tree_attention.cu -- attention of a tree of new tokens over a paged cache,
// on the fifth-generation tensor cores.
//
//     S^T = K Q^T        [128 positions x rows]      rows: (new token, query head) pairs of one kv head
//     x   = S scale log2(e) k_scale + log2(v_scale)  -inf where the row does not see the position
//     w   = 2^(x - m),   l += w / v_scale            m: running reference of the row
//     O^T += V^T w^T     [dim x rows]                out = O / l
//
// Both products take the cache's rows as they lie: K tiles are the K-major A
// operand of the first, V tiles (rows = positions) the MN-major A operand of
// the second, and the weights are written position by position as its MN-major
// B operand, so nothing is transposed.  The rows are the N dimension: a single
// token with 4 query heads costs N = 16 or 32, not a padded M = 128.
//
// e4m3 caches are multiplied without decoding.  The other operand keeps bf16's
// 8 bits as two e4m3 parts side by side in N, x = hi + lo / 32: a bf16 number
// is exactly two 4-bit parts, so an element of q loses nothing down to 2^-14 of
// the largest that shares its power of two: that of the row tile, or of the row
// where rows lie kTaSpread powers of two apart; below that it loses what lies
// under 2^-22 of it.  The weights of v are folded with the row scales
// (w = p * v_scale).  The largest weight of a row is 2^5 or more, the finest
// step 2^-14: a weight keeps 8 bits down to 2^-11 of the largest, and what lies
// below 2^-20 of it is dropped.  Every kTaFlush tiles the sums go to fp32 and
// the references start anew, so at most 8192 * 2^-20 = 0.8 % can be lost that
// way, and only if every position but one lies just below that line.
// bf16 caches take q as it is and a weight as two bf16 parts, 16 bits: with 8
// the weights' rounding adds as much to the result as its own rounding to bf16
// does (1.4 times the error; a lone heavy weight, 2.5 times).
//
// Work: (sequence, kv head, row tile) units of ceil(positions / 128) tiles are
// laid end to end and cut into one equal range per CTA (one CTA per SM), so
// ragged lengths balance; a unit cut by a range is joined from fp32 partials by
// tree_join_kernel, in a fixed order.
//
// Measured on e4m3 caches (median of calls, L2 flushed).  Bound by HBM where a
// kv head has few rows: one token on each of 32 contexts of 4224 to 8192
// positions, 16 kv heads of 128 with 2 query heads each, 839 MB: 135 us, 6.2
// TB/s (boxes of 8 KB at random pages read 6.4); 16 trees of 10 to 16 tokens on a
// bf16 cache, 419 MB: 77 us, 5.5 TB/s.  Bound by the softmax warps'
// instructions where it has many: 8 trees of 20 to 32 tokens, 4 query heads on
// one kv head of 256, 18000 to 32000 positions: 53 us for 104 MB and 22 GFLOP;
// 8 of 39 to 61 tokens, 16 heads on 4, 3375 to 6000 positions: 77 us, 32 GFLOP.
// One token on 1001 positions: 11.5 us and 6.5 us for the join, latency.
#include <atomic>
#include <type_traits>

#include "cache_row.cuh"
#include "dec_ptx.cuh"
#include "tc_ptx.cuh"
#include "tree_shape.h"

namespace wl {

constexpr int kTaMaxCtas = 152;
constexpr int kTaThreads = 512;  // warps 0-7 softmax, 8 MMA (9-11 idle), 12-15 cache loads
// Registers: the block is launched with 512 x 128; the softmax warps take 168
// each and the others keep 88 (256 x 168 + 256 x 88 = 512 x 128).
constexpr int kTaRegsSoftmax = 168, kTaRegsOther = 88;
static_assert(kTaRegsSoftmax + kTaRegsOther == 2 * 128, "register split");
constexpr int kTaSpread = 4;       // powers of two between query rows from which on each has a scale of its own
constexpr float kTaZero = 64.0f;    // scale of a row of zeros in v, as far as weights go: 2^-kTaZero
constexpr float kTaNone = -3.0e38f;  // reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;

struct TaArgs {
    CUtensorMap kmap, vmap;  // the codes as [rows, row bytes], boxes of `box` rows x 128 bytes, zero past a row's end
    int box;                 // rows of a box: a run of positions that lies in one page; 0: no box copies
    const bf16 *q;
    const uint64_t *mask;
    bf16 *out;
    float *part;   // [2 * ctas][RT][DP] partial sums
    float2 *ml;    // [2 * ctas][RT] reference and sum of each row
    int4 *desc;    // [ctas] unit that CTA c begins and others finish: sequence (-1: none), unit, place of its last tile, cost of all
    int q_heads, group, rtiles;
    uint32_t group_inv;  // ceil(2^32 / group), 0 for 1
    float scale;
    CacheArgs c;
};

// ---------------------------------------------------------------- helpers --
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Shared-memory matrix descriptor: lbo, sbo in bytes; sw: 2, 4, 6 for a 128-,
// 64-, 32-byte swizzle span.
__device__ __forceinline__ uint64_t ta_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, int sw)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)sw << 61);
}

__device__ __forceinline__ void tmem_ld16_nw(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// C (a multiple of 16) consecutive columns of this thread's lane: the load,
// and the wait that makes the registers valid (one wait covers all loads).
template <int C>
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t (&r)[C])
{
#pragma unroll
    for (int i = 0; i < C; i += 16) tmem_ld16_nw(taddr + i, r + i);
}
template <int C>
__device__ __forceinline__ void tmem_got(uint32_t (&r)[C])
{
#pragma unroll
    for (int i = 0; i < C; i += 16) tmem_wait16(r + i);
}
__device__ __forceinline__ void load16(const float *p, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(p)[i];
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 numbers in one register pair, with the packed operations.
__device__ __forceinline__ uint64_t f2(float lo, float hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ uint64_t u2(uint32_t lo, uint32_t hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two halves as e4m3 codes.
__device__ __forceinline__ uint32_t half2_e4m3(__half2 h)
{
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(v) : "r"(*reinterpret_cast<const uint32_t *>(&h)));
    return v;
}

__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return *reinterpret_cast<const __half2 *>(&h);
}

// Barrier `id` of `n` threads that also tells whether any of them brought true.
template <int n>
__device__ __forceinline__ bool bar_or(int id, bool in)
{
    uint32_t o;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(o)
        : "r"((uint32_t)in), "r"(id), "n"(n)
        : "memory");
    return o != 0;
}
template <int n>
__device__ __forceinline__ void bar_n(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(n) : "memory");
}
template <int n>
__device__ __forceinline__ void bar_arrive_n(int id)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(n) : "memory");
}

// Reduction of v[CW] over the warp: the result of column lane % CW.
template <int CW, typename Op>
__device__ __forceinline__ float warp_columns(float (&v)[CW], Op op)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d >= CW; d >>= 1)
#pragma unroll
        for (int i = 0; i < CW; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], d));
#pragma unroll
    for (int d = CW / 2; d > 0; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const float send = up ? v[i] : v[i + d], keep = up ? v[i + d] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, d));
        }
    }
    return v[0];
}

// A bounded wait that gives up at once when the CTA is winding down; true if
// what it waits for has come.  A wait that gives up sets the abort flag.  Every
// role then runs through its loops, so that barriers of threads stay matched,
// but a role whose wait gave up copies, multiplies and signals no more: a ring
// slot's barriers go on telling the truth, and what is still in flight can be
// waited for at the end.  (Softmax warps go on; what they write is in bounds.)
__device__ __forceinline__ bool ta_wait(uint64_t *bar, unsigned parity, unsigned *status, unsigned site, volatile int *abort_flag)
{
    if (mbar_test(bar, parity)) return true;
    const long long t0 = wait_clock();
    while (!*abort_flag) {
        if (mbar_test(bar, parity)) return true;
        if (wait_clock() - t0 > kWaitLimitCycles) {
            atomicOr(status, kStatusTimeout | site);
            *abort_flag = 1;
        }
    }
    return false;
}

// A last wait, for MMAs or copies in flight, also when the CTA is winding down.
__device__ __forceinline__ void ta_drain(uint64_t *bar, unsigned parity, unsigned *status)
{
    const long long t0 = wait_clock();
    while (!mbar_test(bar, parity)) {
        if (wait_clock() - t0 > kWaitLimitCycles) {
            atomicOr(status, kStatusTimeout | kWaitDrain);
            return;
        }
    }
}

// New token of row g of a kv head: g / group.  g < 64 group and group <= 4096,
// so the product with the rounded-up reciprocal is exact.
__device__ __forceinline__ int ta_token(const TaArgs &a, int g) { return a.group == 1 ? g : (int)__umulhi((uint32_t)g, a.group_inv); }

// ------------------------------------------------------------------ range --
// Walks a CTA's range of the tiles of all units, unit by unit.
// A unit change costs a CTA about as much as kTaSwitch tiles (its pipeline
// drains, the sums leave, queries are set up), so a unit counts that many more
// when the ranges are cut: without it the CTAs with more units finish last
// (8 trees of up to 61 tokens: SMs busy for 130 thousand cycles, the last for
// 165).  With
// fewer than that many tiles a CTA the ranges are cut by tiles alone.
constexpr int kTaSwitch = 4;

struct TaWalk {
    int total, start, left;  // cost of all units; place of the next segment in it; cost left
    int b, u, tile, ntiles, len, cnt, change;  // change: cost of a unit beside its tiles
};

__device__ __forceinline__ int ta_tiles(const CacheArgs &c, int b, int &len, int &cnt)
{
    len = seq_len(c, b);
    cnt = seq_count(c, b);
    return cnt > 0 ? (len + cnt + kTaTile - 1) / kTaTile : 1;
}

// Settles on a segment: a range that ends within a unit's change has none of
// its tiles.
__device__ __forceinline__ void ta_settle(TaWalk &w, int skip)
{
    // skip: how much of the change lies before the range
    const int pay = w.change - skip;
    if (pay > 0) {
        w.start += pay;
        w.left = max(w.left - pay, 0);
    }
}

// Called by whole warps.  The first total % ctas ranges are one longer.
__device__ __forceinline__ TaWalk ta_walk(const CacheArgs &c, int units)
{
    const int lane = threadIdx.x & 31;
    TaWalk w;
    int len, cnt;
    unsigned sum = 0;
    for (int b = lane; b < c.batch; b += 32) sum += (unsigned)ta_tiles(c, b, len, cnt);
    sum = __reduce_add_sync(0xffffffffu, sum);
    w.change = sum * units >= kTaSwitch * gridDim.x ? kTaSwitch : 0;
    w.total = ((int)sum + c.batch * w.change) * units;
    const int ctas = min((int)gridDim.x, w.total), each = w.total / ctas, more = w.total - each * ctas, id = blockIdx.x;
    w.start = id * each + min(id, more);
    w.left = id < ctas ? each + (id < more) : 0;
    w.b = w.u = w.tile = w.ntiles = w.len = w.cnt = 0;
    if (w.left == 0) return w;
    int base = 0;
    for (int b0 = 0; b0 < c.batch; b0 += 32) {
        const int mine = b0 + lane < c.batch ? (ta_tiles(c, b0 + lane, len, cnt) + w.change) * units : 0;
        int incl = mine;
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > w.start);
        if (past) {
            const int l = __ffs(past) - 1, off = w.start - (base + __shfl_sync(0xffffffffu, incl - mine, l));
            w.b = b0 + l;
            w.ntiles = ta_tiles(c, w.b, w.len, w.cnt);
            const int cost = w.ntiles + w.change, in = off % cost;
            w.u = off / cost;
            w.tile = max(in - w.change, 0);
            ta_settle(w, in);
            return w;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.left = 0;
    return w;
}

// The segment's end tile; then on to the next unit.
__device__ __forceinline__ int ta_end(const TaWalk &w) { return min(w.ntiles, w.tile + w.left); }
__device__ __forceinline__ void ta_next(TaWalk &w, const CacheArgs &c, int units)
{
    const int t1 = ta_end(w);
    w.left -= t1 - w.tile;
    w.start += t1 - w.tile;
    w.tile = t1;
    if (t1 == w.ntiles && w.left > w.change) {
        w.tile = 0;
        if (++w.u == units) {
            w.u = 0;
            ++w.b;
            w.ntiles = ta_tiles(c, w.b, w.len, w.cnt);
        }
        ta_settle(w, 0);
    } else if (t1 == w.ntiles) {
        w.left = 0;
    }
}

// A position's place in the cache, in two steps so that neither waits for the
// other's load: the table's page (-1 past the end and past the table; nothing is
// done with it yet, which would wait), then the row of the codes and scales, ~0
// where there is none.
__device__ __forceinline__ int ta_page(const CacheArgs &c, int b, int j, int end)
{
    if (j >= end) return -1;
    const int p = c.page_shift >= 0 ? j >> c.page_shift : j / c.page_size;
    return p < c.max_pages ? __ldg(c.pages + (int64_t)b * c.max_pages + p) : -1;
}
__device__ __forceinline__ uint32_t ta_row(const CacheArgs &c, int page, int hk, int j)
{
    const int off = c.page_shift >= 0 ? j & (c.page_size - 1) : j % c.page_size;
    return page < 0 || page >= c.npages ? ~0u : ((uint32_t)page * c.kv_heads + hk) * c.page_size + off;
}

// ------------------------------------------------------------------ kernel --
template <bool kE4M3, int DP, int RT>
__global__ void __launch_bounds__(kTaThreads, 1) tree_attention_kernel(const __grid_constant__ TaArgs a)
{
    using Z = TaShape<kE4M3, DP, RT>;
    constexpr int N = Z::N, CW = Z::CW, SLOTS = Z::SLOTS;
    extern __shared__ __align__(1024) char smem_raw[];
    // The whole limit is used, so there is no room to align by hand.
    if (s32(smem_raw) & 1023u) {
        pdl_wait();
        if (threadIdx.x == 0) {
            atomicOr(a.c.status, kStatusAlign);
            a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        return;
    }
    char *smem = smem_raw;
    char *sq = smem, *sp = sq + Z::QB, *ring = sp + 2 * Z::PB, *misc = ring + SLOTS * Z::SLOT;
    uint64_t *smask = reinterpret_cast<uint64_t *>(misc);            // [RT]
    float *red = reinterpret_cast<float *>(misc + 512);              // [2][4][32]
    float *nms = reinterpret_cast<float *>(misc + 1792);             // [2][32] minus the references of the columns
    uint32_t *rowtab = reinterpret_cast<uint32_t *>(misc + 2048);    // [4][2][32] rows of two tiles
    uint64_t *bars = reinterpret_cast<uint64_t *>(misc + 1536);
    uint64_t *full = bars, *empty = full + SLOTS, *s_full = empty + SLOTS, *s_empty = s_full + 2, *p_full = s_full + 4,
             *pv_done = s_full + 6, *q_ready = s_full + 8, *drain = s_full + 9;
    uint32_t *tmem_hold = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_hold + 1);
    uint8_t *qexp = reinterpret_cast<uint8_t *>(misc + Z::QEXP);     // [RT]

    const CacheArgs &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = c.kv_heads * a.rtiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], a.box ? 1 : 4);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], Z::PP ? 4 : 8);
            mbar_init(&p_full[i], Z::PP ? 4 : 8);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_ready, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(tmem_hold)),
                     "n"(Z::COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    TaWalk w = ta_walk(c, units);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_hold;
    pdl_trigger();

    if (warp >= 12) {
        // ------------------------------------------------ cache loads
        // Ring items in the order the MMAs take them: K0, K1, V0, K2, V1, ...
        // Two tiles ahead a page is looked up, one tile ahead it becomes a
        // row: no copy waits for a lookup.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTaRegsOther));
        int item = 0;
        bool live = true;  // no wait has given up
        if (a.box == 0) {
            // 16-byte copies: warp pw takes rows 32 pw .. of a tile; zeros
            // where there is no row
            const int pw = warp - 12;
            constexpr int LPR = Z::SLOTROW / 16, RPP = 32 / LPR;  // lanes per row, rows per pass
            const int ch = lane % LPR, sub = lane / LPR;
            uint32_t *tab = rowtab + pw * 64;  // rows of the even and odd tile
            const uint32_t to = (uint32_t)((ch >> 3) * (kTaTile * 128) + (pw * 32 + sub) * 128);
            const uint32_t sw = (uint32_t)(((ch & 7) ^ sub) << 4);  // the row's low bits are sub and those of the pass
            const uint32_t rowb = (uint32_t)(c.dim * Z::ES);
            auto copy = [&](const char *base, const uint32_t *tb) {
#pragma unroll
                for (int s = 0; s < Z::NS; ++s, ++item) {
                    const int slot = item % SLOTS;
                    const uint32_t dst = s32(ring + slot * Z::SLOT) + to, col = s * Z::SLOTROW + ch * 16;
                    const bool in = col < rowb;
                    const char *src = in ? base + col : base;
                    live = __all_sync(0xffffffffu, ta_wait(&empty[slot], (unsigned)(((item / SLOTS) & 1) ^ 1), c.status, kWaitRingEmpty, abort_flag)) && live;
                    if (!live) continue;
#pragma unroll 4
                    for (int p = 0; p < 32 / RPP; ++p) {
                        const uint32_t r = tb[p * RPP + sub];
                        const bool ok = in && r != ~0u;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         dst + p * (RPP * 128) + (sw ^ (((p * RPP) & 7) << 4))),
                                     "l"(src + (ok ? (uint64_t)r * rowb : 0ull)), "r"(ok ? 16 : 0));
                    }
                    cp_async_wait_all();
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[slot]);
                }
            };
            while (w.left > 0) {
                const int t1 = ta_end(w), hk = w.u / a.rtiles, end = min(w.cnt > 0 ? w.len + w.cnt : 0, t1 * kTaTile);
                int j = w.tile * kTaTile + pw * 32 + lane;
                auto place = [&](int t, int pg, int j) {
                    const uint32_t row = ta_row(c, pg, hk, j);
                    if (row == ~0u && j < end) atomicOr(c.status, kStatusPage);
                    __syncwarp();  // the tile that had this table has been issued
                    tab[(t & 1) * 32 + lane] = row;
                    __syncwarp();
                };
                int pg = ta_page(c, w.b, j, end), pg1 = ta_page(c, w.b, j + kTaTile, end);
                place(w.tile, pg, j);
                for (int t = w.tile; t < t1; ++t, j += kTaTile) {
                    pg = pg1;
                    pg1 = ta_page(c, w.b, j + 2 * kTaTile, end);
                    copy(c.k, tab + (t & 1) * 32);
                    if (t > w.tile) copy(c.v, tab + ((t - 1) & 1) * 32);
                    place(t + 1, pg, j + kTaTile);
                }
                copy(c.v, tab + ((t1 - 1) & 1) * 32);
                ta_next(w, c, units);
            }
        } else if (warp < 14) {
            // Boxes: warp 12 brings K, warp 13 V.  Lane r looks up run r of
            // a.box positions; one lane copies them all.  A run at the end
            // brings what its page holds beyond; what no box brings stays as
            // it was: scores there are masked, and the softmax warps zero the
            // rows of V that a segment's last tile lacks.  A run whose page
            // is not valid, which any tile may have, gets a box before V's first
            // row, which brings zeros.
            // Z::PACED: where a segment ends, K waits until V's last boxes have
            // been issued, and V until K has issued the boxes that come before
            // V's next ones, so that the parity of an empty slot is that of the
            // round before (barriers 4 and 5; the ring's order is the same, and
            // neither waits for what the other would issue later).
            const bool isv = warp == 13;
            const CUtensorMap *map = isv ? &a.vmap : &a.kmap;
            const int runs = kTaTile / a.box;
            const uint32_t bytes = (uint32_t)(a.box * Z::SLOTROW);
            uint32_t *tab = rowtab + isv * 64;
            const uint32_t ahead = (uint32_t)-a.box;
            int items = 0, last = -1;  // last: lane s's: the last item copied to slot s
            while (w.left > 0) {
                const int t1 = ta_end(w), n = t1 - w.tile, hk = w.u / a.rtiles;
                const int end = lane < runs ? min(w.cnt > 0 ? w.len + w.cnt : 0, t1 * kTaTile) : 0;
                int j = w.tile * kTaTile + lane * a.box;
                int pg = ta_page(c, w.b, j, end), pg1 = ta_page(c, w.b, j + kTaTile, end);
                if (Z::PACED && isv) bar_n<64>(5);
                if (Z::PACED && !isv && items > 0) bar_n<64>(4);
                for (int r = 0; r < n; ++r, j += kTaTile) {
                    uint32_t row = ta_row(c, pg, hk, j);
                    if (row == ~0u && j < end) {
                        atomicOr(c.status, kStatusPage);
                        if (isv) row = ahead;
                    }
                    tab[(r & 1) * 32 + lane] = row;  // the other half may still be read
                    pg = pg1;
                    pg1 = ta_page(c, w.b, j + 2 * kTaTile, end);
                    const uint32_t have = __ballot_sync(0xffffffffu, row != ~0u);
                    item = items + Z::NS * ta_item(r, n, isv);
                    __syncwarp();
#pragma unroll
                    for (int s = 0; s < Z::NS; ++s, ++item) {
                        const int slot = item % SLOTS;
                        live = __all_sync(0xffffffffu, ta_wait(&empty[slot], (unsigned)(((item / SLOTS) & 1) ^ 1), c.status, kWaitRingEmpty, abort_flag)) && live;
                        if (live && lane == slot) last = item;
                        if (live && elect_one()) {
                            mbar_expect_tx(&full[slot], (uint32_t)__popc(have) * bytes);
                            char *dst = ring + slot * Z::SLOT;
                            const uint32_t *tb = tab + (r & 1) * 32;
#pragma unroll 1
                            for (int k = 0; k < runs; ++k, dst += a.box * 128) {
                                const uint32_t at = tb[k];
                                if (at == ~0u) continue;
#pragma unroll
                                for (int h = 0; h < Z::SLOTROW / 128; ++h)
                                    tma_load_2d(dst + h * (kTaTile * 128), map, s * Z::SLOTROW + h * 128, (int)at, &full[slot]);
                            }
                        }
                        __syncwarp();
                    }
                    if (Z::PACED && !isv && r == min(n, 2) - 1) bar_arrive_n<64>(5);
                }
                items += 2 * Z::NS * n;
                ta_next(w, c, units);
                if (Z::PACED && isv && w.left > 0) bar_arrive_n<64>(4);
            }
            tab[lane] = (uint32_t)last;
        }
    } else if (warp >= 8) {
        // ------------------------------------------------ MMA issuer
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTaRegsOther));
        // One elected thread: inside a branch the compiler knows to be taken
        // by one thread an MMA issues in its own time (56, 70, 98 cycles at
        // N = 32, 64, 128); under a plain lane == 0 test each takes 120.
        if (warp == 8 && elect_one()) {
            constexpr uint32_t kType = kE4M3 ? 0u : (1u << 7) | (1u << 10);
            constexpr uint32_t kId = (1u << 4) | kType | ((uint32_t)(N >> 3) << 17) | (8u << 24);
            constexpr uint32_t kIdPV = kId | (3u << 15);  // both operands MN-major
            const uint32_t bq = s32(sq), bp = s32(sp), br = s32(ring);
            const uint32_t ocol = tmem + 2 * N;
            int item = 0, it = 0, seg = 0;
            bool live = true;  // no wait has given up
            auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t acc) {
                if (!live) return;
                if constexpr (kE4M3)
                    umma_f8(d, da, db, id, acc);
                else
                    umma(d, da, db, id, acc);
            };
            auto take = [&](int &slot) {
                slot = item % SLOTS;
                live = ta_wait(&full[slot], (unsigned)((item / SLOTS) & 1), c.status, kWaitRingFull, abort_flag) && live;
                ++item;
            };
            auto scores = [&](int i) {
                live = ta_wait(&s_empty[i & 1], (unsigned)(((i >> 1) & 1) ^ 1), c.status, kWaitRingEmpty, abort_flag) && live;
                tc_fence_after();
                const uint32_t d = tmem + (i & 1) * N;
#pragma unroll
                for (int s = 0; s < Z::NS; ++s) {
                    int slot;
                    take(slot);
                    const uint32_t ak = br + slot * Z::SLOT;
#pragma unroll
                    for (int k = 0; k < Z::SLOTROW / 32; ++k) {
                        const int gk = s * (Z::SLOTROW / 32) + k;
                        mma(d, ta_desc(ak + (k / 4) * (kTaTile * 128) + (k % 4) * 32, 16, 1024, 2),
                            ta_desc(bq + (gk / 4) * (N * 128) + (gk % 4) * 32, 16, 1024, 2), kId, gk > 0 ? 1u : 0u);
                    }
                    if (live) umma_commit(&empty[slot]);
                }
                if (live) umma_commit(&s_full[i & 1]);
            };
            auto values = [&](int i, bool first) {
                live = ta_wait(&p_full[i & 1], (unsigned)((i >> 1) & 1), c.status, kWaitRingFull, abort_flag) && live;
                tc_fence_after();
                const uint32_t pb = bp + (i & 1) * Z::PB;
#pragma unroll
                for (int s = 0; s < Z::NS; ++s) {
                    int slot;
                    take(slot);
                    const uint32_t av = br + slot * Z::SLOT;
                    constexpr int MS = Z::MT / Z::NS;  // M tiles of a slot
#pragma unroll
                    for (int m = 0; m < MS; ++m)
#pragma unroll
                        for (int h = 0; h < Z::PB / Z::PB1; ++h)
#pragma unroll
                            for (int k = 0; k < kTaTile / Z::KSTEP; ++k)
                                mma(ocol + ((Z::PP ? (i & 1) * Z::MT : 0) + s * MS + m) * N,
                                    ta_desc(av + m * Z::ES * (kTaTile * 128) + k * Z::KSTEP * 128, kTaTile * 128, 1024, 2),
                                    ta_desc(pb + h * Z::PB1 + k * Z::KSTEP * Z::PW, 8 * Z::PW, 8 * Z::PW, Z::SWP), kIdPV,
                                    (first && h + k == 0) ? 0u : 1u);
                    if (live) umma_commit(&empty[slot]);
                }
                if (live) umma_commit(&pv_done[i & 1]);
            };
            while (w.left > 0) {
                const int t1 = ta_end(w);
                live = ta_wait(q_ready, (unsigned)(seg & 1), c.status, kWaitRingFull, abort_flag) && live;
                tc_fence_after();
                for (int t = w.tile; t < t1; ++t, ++it) {
                    scores(it);
                    if (t > w.tile) values(it - 1, (t - 1 - w.tile) % kTaFlush < (Z::PP ? 2 : 1));
                }
                values(it - 1, (t1 - 1 - w.tile) % kTaFlush < (Z::PP ? 2 : 1));
                ++seg;
                ta_next(w, c, units);
            }
            umma_commit(drain);
            ta_drain(drain, 0, c.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax
        // A thread is one position of a tile (lane of S^T).  RT = 64: both
        // warpgroups work on every tile, half the columns each.  RT <= 32:
        // warpgroup wg takes the tiles of buffer wg, all columns, with sums
        // and references of its own, so that two tiles are in hand at once.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTaRegsSoftmax));
        const int wg = warp >> 2, tk = threadIdx.x & 127, col0 = Z::PP ? 0 : wg * CW;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        float *wred = red + wg * 128;
        float *fac = reinterpret_cast<float *>(sp);  // [3][64] factors of both streams and of flushed sums, when the buffers are idle
        int it = 0, items = 0;  // tiles and ring items of earlier segments
        if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
        while (w.left > 0) {
            const int t0 = w.tile, t1 = ta_end(w), total = w.cnt > 0 ? w.len + w.cnt : 0;
            const int hk = w.u / a.rtiles, row0 = (w.u - hk * a.rtiles) * RT, rows = min(RT, c.n * a.group - row0);
            constexpr int STEP = Z::PP ? 2 : 1;
            // scales of this thread's position, loaded a tile ahead
            const int tf = t0 + (Z::PP ? (it ^ wg) & 1 : 0);  // this warpgroup's first tile
            const int end = min(total, t1 * kTaTile);
            int pg1;
            uint32_t at;
            float ks, vs;
            {
                const int j = tf * kTaTile + tk;
                at = ta_row(c, ta_page(c, w.b, j, end), hk, j);
                pg1 = ta_page(c, w.b, j + STEP * kTaTile, end);
                ks = at != ~0u ? __ldg(c.k_scale + at) : 0.0f;
                vs = at != ~0u ? __ldg(c.v_scale + at) : 1.0f;
            }
            // nm: minus the references of the columns (the same for all threads,
            // so in shared memory), l: this position's sums, as pairs; unset:
            // columns that have seen nothing yet and have no reference.
            float *nm = nms + wg * 32;
            uint64_t l[CW / 2];
            uint32_t unset;
            auto fresh = [&]() {
                // a column beyond the rows never counts and never moves
                if (tk < CW) nm[tk] = col0 + tk < rows ? 0.0f : kTaNone;
#pragma unroll
                for (int i = 0; i < CW / 2; ++i) l[i] = 0ull;
                const int nc = min(max(rows - col0, 0), CW);
                unset = nc == 32 ? ~0u : (1u << nc) - 1;
            };
            fresh();
            // ---- the segment's queries: rows of the B operand
            float qscale = a.scale * kLog2e;
            int spread = 0;  // where rows have exponents of their own (qexp): the one that qscale stands for
            {
                // A lane has 8 elements of a row, a warp RPW rows at a time.
                constexpr int CH = DP / 8, RPW = 32 / CH, PER = RT / (8 * RPW);
                const int ck = lane % CH, d = ck * 8;
                const bf16 *base = a.q + ((int64_t)w.b * c.n * a.q_heads + hk * a.group) * c.dim + d;
                // where row `lane` (of 32, and of the next 32) lies; -1: zeros
                auto where = [&](int r) -> int {
                    const int tok = ta_token(a, row0 + r);
                    return r < rows && tok < w.cnt ? (tok * a.q_heads + row0 + r - tok * a.group) * c.dim : -1;
                };
                const int off0 = where(lane), off1 = RT > 32 ? where(lane + 32) : -1;
                uint4 raw[PER];  // all rows of a lane are in flight at once
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int r = (i * 8 + warp) * RPW + lane / CH;
                    int off = __shfl_sync(0xffffffffu, off0, r & 31);
                    if (RT > 32) {
                        const int up = __shfl_sync(0xffffffffu, off1, r & 31);
                        off = r < 32 ? off : up;
                    }
                    raw[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (off >= 0 && d < c.dim) raw[i] = *reinterpret_cast<const uint4 *>(base + off);
                }
                if (threadIdx.x < RT) {
                    const int g = row0 + threadIdx.x, i = ta_token(a, g);
                    uint64_t m = 0;
                    if ((int)threadIdx.x < rows && i < w.cnt) {
                        m = a.mask ? a.mask[(int64_t)w.b * c.n + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
                        if (w.cnt < 64) m &= (1ull << w.cnt) - 1;
                    }
                    smask[threadIdx.x] = m;
                }
                // e4m3: a power of two brings the largest |q| of the tile into
                // [128, 256), and the parts keep 8 bits of what lies up to 2^14
                // below it.  Where a row's largest lies 2^kTaSpread or more
                // below the tile's, each row has a power of two of its own, and
                // the scores take the difference back.
                int be = 0;        // biased exponent of the tile's largest
                bool odd = false;  // a NaN or an infinity among this lane's
                if (kE4M3) {
                    // largest |q|, and the least (less 1) that is not zero of the
                    // largest in each 16 elements of a row, as bits of bf16
                    uint32_t mx = 0, mn = ~0u;
#pragma unroll
                    for (int i = 0; i < PER; i += 2) {
                        uint32_t two[2] = {0u, 0u};  // two rows of 8 elements
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (i + k < PER) {
                                const uint4 &v = raw[i + k < PER ? i + k : i];
                                two[k] = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                            }
                        uint32_t top = __vmaxu2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[0], two[1], 0x7632));
                        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        const uint32_t a = top & 0xffffu, b = top >> 16;
                        mx = max(mx, max(a, b));
                        mn = min(mn, min(a - 1, b - 1));
                    }
                    odd = mx >= 0x7f80u;
                    // largest |element| of 8, as bits of bf16, but for NaN and infinity
                    auto top8 = [](const uint4 &v) {
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                        uint32_t top = 0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t h = (u[k / 2] >> (16 * (k & 1))) & 0x7fffu;
                            top = max(top, h < 0x7f80u ? h : 0u);
                        }
                        return top;
                    };
                    if (__builtin_expect(odd, 0)) {  // the largest of the others
                        mx = 0;
#pragma unroll
                        for (int i = 0; i < PER; ++i) mx = max(mx, top8(raw[i]));
                    }
                    mx = __reduce_max_sync(0xffffffffu, mx);
                    mn = __reduce_min_sync(0xffffffffu, mn);
                    if (lane == 0) reinterpret_cast<uint2 *>(red)[warp] = make_uint2(mx, mn);
                    bar_n<256>(3);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint2 o = reinterpret_cast<const uint2 *>(red)[i];
                        mx = max(mx, o.x);
                        mn = min(mn, o.y);
                    }
                    be = max((int)(mx >> 7), 14);
                    auto least = [&]() { return min(max((int)((min(mn, 0x7f7eu) + 1) >> 7), 14), be); };
                    // (no 16 elements far below the tile's largest: no row either)
                    if (__builtin_expect(be - least() >= kTaSpread, 0)) {
                        mn = ~0u;
                        // once more row by row, from memory: it is rare, and what is unrolled here slows the rest
#pragma unroll 1
                        for (int i = 0; i < PER; ++i) {
                            const int r = (i * 8 + warp) * RPW + lane / CH, off = where(r);
                            uint32_t top = off >= 0 && d < c.dim ? top8(*reinterpret_cast<const uint4 *>(base + off)) : 0u;
#pragma unroll 1
                            for (int x = CH / 2; x > 0; x >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
                            if (ck == 0) qexp[r] = (uint8_t)(top ? max(top >> 7, 14u) : 0u);
                            mn = min(mn, top - 1);
                        }
                        mn = __reduce_min_sync(0xffffffffu, mn);
                        bar_n<256>(3);
                        if (lane == 0) reinterpret_cast<uint32_t *>(red)[warp] = mn;
                        bar_n<256>(3);
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) mn = min(mn, reinterpret_cast<const uint32_t *>(red)[i]);
                        // the common exponent: 2^7 if rows lie on both sides of it, so that
                        // neither it nor a row's distance from it leaves fp32's range
                        if (be - least() >= kTaSpread) spread = be = min(max(134, least()), be);
                        // (a row of zeros takes the common one: its distance from a row's may be any)
                        if (ck == 0)
#pragma unroll 1
                            for (int r = warp * RPW + lane / CH; r < RT; r += 8 * RPW)
                                if (!qexp[r]) qexp[r] = (uint8_t)be;
                        __syncwarp();
                    }
                    qscale *= __uint_as_float((uint32_t)(be - 7) << 23);  // 2^(be - 134)
                }
                // K-major rows of 128-byte chunks, 16-byte units swizzled by the row
                char *o0 = sq + (kE4M3 ? (ck / 16) * (N * 128) + (ck & 1) * 8 : (ck / 8) * (N * 128));
                const int c16 = kE4M3 ? (ck / 2) & 7 : ck & 7;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int r = (i * 8 + warp) * RPW + lane / CH;
                    const uint4 v = raw[i];
                    char *o = o0 + r * 128 + ((c16 ^ (r & 7)) << 4);
                    if (kE4M3) {
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                        uint32_t hi[4], lo[4];
                        const float up = __uint_as_float((uint32_t)(261 - (spread ? qexp[r] : be)) << 23);  // brings the largest into [128, 256)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2 x = __floats2half2_rn(bf_lo(u[k]) * up, bf_hi(u[k]) * up);  // exact: 8 bits, below 256
                            hi[k] = half2_e4m3(x);
                            lo[k] = half2_e4m3(__hmul2(__hsub2(x, e4m3x2_half2(hi[k])), __float2half2_rn(32.0f)));
                        }
                        if (__builtin_expect(odd, 0)) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((u[k] & 0x7fffu) >= 0x7f80u) hi[k] |= 0x7fu;  // NaN, infinity: a NaN code
                                if ((u[k] >> 16 & 0x7fffu) >= 0x7f80u) hi[k] |= 0x7f00u;
                            }
                        }
                        *reinterpret_cast<uint2 *>(o) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                        *reinterpret_cast<uint2 *>(o + RT * 128) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                    } else {
                        *reinterpret_cast<uint4 *>(o) = v;
                    }
                }
                fence_async_smem();
                bar_n<256>(3);  // the masks too
                if (lane == 0) mbar_arrive(q_ready);
            }
            const int slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
            const bool whole = t0 == 0 && t1 == w.ntiles;
            bool flushed = false, some = false;  // some: this warpgroup has sums in tensor memory
            // Two copies of the tile loop, as rows with exponents of their own
            // are rare: a branch around the factors in a single loop took the
            // second wide-tree case above from 76 to 80 us.
            auto tiles = [&](auto own) {
                constexpr bool kOwn = decltype(own)::value;
                for (int t = t0; t < t1; ++t, ++it) {
                    if (!Z::PP || (it & 1) == wg) {
                        const int j = t * kTaTile + tk;
                        const bool seen = at != ~0u;
                        const bool bad = vs != vs;
                        // w / v_scale of few rows below 2^-104 could pass fp32's range (w is up to 2^8): such
                        // rows, nothing in them above 448 * 2^-104, count as if their scale were that
                        const float v1 = fmaxf(vs, 4.93038066e-32f);
                        // log2 of the scale, to 2^-22 of itself, and the reciprocal, exact for a power
                        // of two: a weight and its share of the sum are off alike, by 3.3e-6 at a scale
                        // of 2^-20.  (The exponent apart, exactly: 76.8 us instead of 76.0 in the second
                        // wide-tree case.)
                        const float lv = bad ? vs : __log2f(v1), iv = bad ? 1.0f : rcp_approx(v1);
                        const uint64_t cs2 = f2(ks * qscale, ks * qscale), lv2 = f2(lv, lv);
                        uint64_t iv2 = f2(iv, iv);
                        at = ta_row(c, pg1, hk, j + STEP * kTaTile);
                        ks = at != ~0u ? __ldg(c.k_scale + at) : 0.0f;
                        vs = at != ~0u ? __ldg(c.v_scale + at) : 1.0f;
                        pg1 = ta_page(c, w.b, j + 2 * STEP * kTaTile, end);
                        ta_wait(&s_full[it & 1], (unsigned)((it >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                        tc_fence_after();
                        const uint32_t sc = tmem + lanes + (it & 1) * N + col0;
                        uint64_t y[CW / 2];
                        {
                            uint32_t x[CW], xl[kE4M3 ? CW : 16];
                            tmem_get(sc, x);
                            if (kE4M3) tmem_get(sc + RT, xl);
                            // the weights' buffer is free once tile it - 2 has been multiplied
                            if (it >= 2)
                                ta_wait(&pv_done[it & 1], (unsigned)(((it - 2) >> 1) & 1), c.status, kWaitRingEmpty, abort_flag);
                            tmem_got(x);
                            if (kE4M3) tmem_got(xl);
                            const uint64_t r32 = f2(0.03125f, 0.03125f);
#pragma unroll
                            for (int i = 0; i < CW / 2; ++i) {
                                y[i] = u2(x[2 * i], x[2 * i + 1]);
                                if (kE4M3) y[i] = fma2(u2(xl[2 * i], xl[2 * i + 1]), r32, y[i]);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[it & 1]);
                        if constexpr (kOwn) {
#pragma unroll
                            for (int i = 0; i < CW / 2; i += 2) {
                                const uint32_t e = *reinterpret_cast<const uint32_t *>(qexp + col0 + 2 * i);
                                auto f = [&](uint32_t own) { return (own + 127 - spread) << 23; };
                                y[i] = mul2(y[i], u2(f(e & 0xffu), f(e >> 8 & 0xffu)));
                                y[i + 1] = mul2(y[i + 1], u2(f(e >> 16 & 0xffu), f(e >> 24)));
                            }
                        }
                        // y = x - m
#pragma unroll
                        for (int i = 0; i < CW / 2; ++i) y[i] = add2(fma2(y[i], cs2, lv2), *reinterpret_cast<const uint64_t *>(nm + 2 * i));
                        if (__builtin_expect(!__all_sync(0xffffffffu, seen && j < w.len && (!kE4M3 || iv != 1.0f)), 0)) {
                            if (kE4M3 && __any_sync(0xffffffffu, seen && iv == 1.0f)) {
                                // A row of zeros has scale 1, which may lie far above the others': its
                                // weight, which V's product does not need, would take their bits.  It
                                // counts as if its scale were 2^-kTaZero.  (The wait is sound in any tile:
                                // an operand is one slot of at least three.)
                                static_assert(!kE4M3 || (Z::NS == 1 && SLOTS >= 3), "a wait for V");
                                const int v0 = items + ta_item(t - t0, t1 - t0, true), slot = v0 % SLOTS;
                                ta_wait(&full[slot], (unsigned)((v0 / SLOTS) & 1), c.status, kWaitRingFull, abort_flag);
                                const char *row = ring + slot * Z::SLOT + tk * 128;
                                bool zero = seen && iv == 1.0f;
#pragma unroll 1
                                for (int h = 0; zero && h < Z::SLOTROW / 16; ++h) {
                                    const uint4 u = *reinterpret_cast<const uint4 *>(row + (h / 8) * (kTaTile * 128) + (((h ^ tk) & 7) << 4));
                                    zero = ((u.x | u.y | u.z | u.w) & 0x7f7f7f7fu) == 0;
                                }
                                __syncwarp();
                                const uint64_t less = f2(zero ? -kTaZero : 0.0f, zero ? -kTaZero : 0.0f);
#pragma unroll
                                for (int i = 0; i < CW / 2; ++i) y[i] = add2(y[i], less);
                                if (zero) iv2 = f2(exp2_int((int)kTaZero), exp2_int((int)kTaZero));
                            }
                            const int bit = j - w.len;
#pragma unroll
                            for (int i = 0; i < CW / 2; ++i) {
                                float p = f2_lo(y[i]), q = f2_hi(y[i]);
                                if (!seen || (bit >= 0 && !((smask[col0 + 2 * i] >> bit) & 1))) p = -INFINITY;
                                if (!seen || (bit >= 0 && !((smask[col0 + 2 * i + 1] >> bit) & 1))) q = -INFINITY;
                                y[i] = f2(p, q);
                            }
                        }
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < CW / 2; ++i) top = max3(top, f2_lo(y[i]), f2_hi(y[i]));
                        // Weights up to 2^kTop stay as they are; only a position
                        // above that moves its column's reference, to kGap below.
                        if (__builtin_expect(bar_or<128>(1 + wg, top > Z::kTop || unset), 0)) {
                            {
                                float v[CW];
#pragma unroll
                                for (int i = 0; i < CW / 2; ++i) v[2 * i] = f2_lo(y[i]), v[2 * i + 1] = f2_hi(y[i]);
                                const float cm = warp_columns<CW>(v, [](float p, float q) { return fmaxf(p, q); });
                                if (lane < CW) wred[(warp & 3) * 32 + lane] = cm;
                            }
                            bar_n<128>(1 + wg);
                            // one warp decides: how far each column's exponents move
                            // (also those about to reach the limit), the factor of its sums
                            if (tk < 32) {
                                const float mx = lane < CW ? fmaxf(fmaxf(wred[lane], wred[32 + lane]), fmaxf(wred[64 + lane], wred[96 + lane])) : -INFINITY;
                                const bool first = (unset >> lane) & 1 && mx > -INFINITY, move = first || mx > Z::kTop - Z::kNear;
                                const uint32_t set = __ballot_sync(0xffffffffu, move);
                                const float d = move ? Z::kTop - Z::kGap - mx : 0.0f;
                                wred[lane] = d;
                                wred[32 + lane] = first ? 1.0f : ex2(d);  // nothing to scale in a first one: its sums are zero
                                if (move) nm[lane] += d;
                                if (lane == 0) reinterpret_cast<uint2 *>(wred)[32] = make_uint2(unset & ~set, set);
                            }
                            bar_n<128>(1 + wg);
                            const uint2 state = reinterpret_cast<const uint2 *>(wred)[32];
                            unset = state.x;
#pragma unroll
                            for (int i = 0; i < CW; i += 8) {
                                if (!((state.y >> i) & 0xffu)) continue;
#pragma unroll
                                for (int k = i / 2; k < i / 2 + 4; ++k) {
                                    y[k] = add2(y[k], *reinterpret_cast<const uint64_t *>(wred + 2 * k));
                                    l[k] = mul2(l[k], *reinterpret_cast<const uint64_t *>(wred + 32 + 2 * k));
                                }
                            }
                            if (some) {
                                if (!Z::PP) {  // (else the sums' last tile is it - 2: waited for above)
                                    ta_wait(&pv_done[(it - 1) & 1], (unsigned)(((it - 1) >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                                    tc_fence_after();
                                }
                                constexpr int P = Z::MT * Z::PARTS;
#pragma unroll 1
                                for (int i = 0; i < CW; i += 8) {
                                    if (!((state.y >> i) & 0xffu)) continue;
                                    const uint32_t ad = tmem + lanes + 2 * N + (Z::PP ? wg * Z::MT * N : 0) + col0 + i;
                                    uint32_t o[P][8];
                                    float f[8];
#pragma unroll
                                    for (int p = 0; p < P; ++p) tmem_ld8_nw(ad + p * RT, o[p]);
#pragma unroll
                                    for (int k = 0; k < 8; ++k) f[k] = wred[32 + i + k];
#pragma unroll
                                    for (int p = 0; p < P; ++p) tmem_wait_ld8(o[p]);
#pragma unroll
                                    for (int p = 0; p < P; ++p) {
                                        float x[8];
#pragma unroll
                                        for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[p][k]) * f[k];
                                        tmem_st8(ad + p * RT, x);
                                    }
                                }
                                tmem_wait_st();
                            }
                        }
                        // weights: w = 2^(x - m) = p * v_scale
                        char *pr = sp + (it & 1) * Z::PB;
                        const uint32_t rowb = tk * Z::PW, sw = ((rowb >> 7) & (Z::PW / 16 - 1)) << 4;
#pragma unroll
                        for (int i = 0; i < CW; i += 16) {
                            uint32_t hi[4], lo[4], bw[8], bl[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float p = ex2(f2_lo(y[i / 2 + k])), q = ex2(f2_hi(y[i / 2 + k]));
                                l[i / 2 + k] = fma2(f2(p, q), iv2, l[i / 2 + k]);
                                if constexpr (kE4M3) {
                                    // 11 bits of the weight, cut into 4 + 4
                                    const __half2 h = __floats2half2_rn(p, q);
                                    const uint32_t c8 = half2_e4m3(h);
                                    const __half2 rest = __hmul2(__hsub2(h, e4m3x2_half2(c8)), __float2half2_rn(32.0f));
                                    const uint32_t l8 = half2_e4m3(rest);
                                    if (k & 1) {
                                        hi[k / 2] |= c8 << 16;
                                        lo[k / 2] |= l8 << 16;
                                    } else {
                                        hi[k / 2] = c8;
                                        lo[k / 2] = l8;
                                    }
                                } else {
                                    bw[k] = bf16x2_bits(p, q);
                                    bl[k] = bf16x2_bits(p - bf_lo(bw[k]), q - bf_hi(bw[k]));
                                }
                            }
                            if constexpr (kE4M3) {
                                *reinterpret_cast<uint4 *>(pr + ((rowb + col0 + i) ^ sw)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                                *reinterpret_cast<uint4 *>(pr + ((rowb + RT + col0 + i) ^ sw)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                            } else {
                                char *o0 = pr + ((rowb + 2 * (col0 + i)) ^ sw), *o1 = pr + ((rowb + 2 * (col0 + i) + 16) ^ sw);
                                *reinterpret_cast<uint4 *>(o0) = make_uint4(bw[0], bw[1], bw[2], bw[3]);
                                *reinterpret_cast<uint4 *>(o1) = make_uint4(bw[4], bw[5], bw[6], bw[7]);
                                *reinterpret_cast<uint4 *>(o0 + Z::PB1) = make_uint4(bl[0], bl[1], bl[2], bl[3]);
                                *reinterpret_cast<uint4 *>(o1 + Z::PB1) = make_uint4(bl[4], bl[5], bl[6], bl[7]);
                            }
                        }
                        if (__builtin_expect(a.box && t + 1 == t1 && !__all_sync(0xffffffffu, seen), 0)) {
                            // rows of V that are not there: weight 0 must meet a number
                            // (only in a last tile: of an earlier one the wait below
                            // could take the round of its slot before for its own)
                            const int n = t1 - t0, r = t - t0, v0 = items + Z::NS * ta_item(r, n, true);
                            for (int s = 0; s < Z::NS; ++s) {
                                const int vs = (v0 + s) % SLOTS;
                                const bool here = ta_wait(&full[vs], (unsigned)(((v0 + s) / SLOTS) & 1), c.status, kWaitRingFull, abort_flag);
                                if (here && !seen && (Z::PP || wg == 0))
                                    for (int h = 0; h < Z::SLOTROW / 16; ++h)
                                        *reinterpret_cast<uint4 *>(ring + vs * Z::SLOT + (h / 8) * (kTaTile * 128) + tk * 128 + (h % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        some = true;
                        fence_async_smem();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[it & 1]);
                    }
                    const bool last = t + 1 == t1;
                    if (!last && (t + 1 - t0) % kTaFlush != 0) continue;
                    // ---- the sums leave tensor memory
                    {
                        float v[CW];
#pragma unroll
                        for (int i = 0; i < CW / 2; ++i) v[2 * i] = f2_lo(l[i]), v[2 * i + 1] = f2_hi(l[i]);
                        const float ls = warp_columns<CW>(v, [](float p, float q) { return p + q; });
                        bar_n<128>(1 + wg);  // the last event's factors have been read
                        if (lane < CW) wred[(warp & 3) * CW + lane] = ls;
                        if (tk < CW && (unset >> tk) & 1) nm[tk] = -kTaNone;
                        const int own = it - (Z::PP ? (it ^ wg) & 1 : 0);  // this warpgroup's last tile, if it had one
                        if (some) ta_wait(&pv_done[own & 1], (unsigned)((own >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                        tc_fence_after();
                        bar_n<256>(3);
                        float top_r = kTaNone, sum = 0.0f;
                        if ((int)threadIdx.x < rows) {
                            const int r = threadIdx.x;
                            float f[3] = {1.0f, 0.0f, 0.0f};
                            auto side = [&](int g, int col, float &mr, float &sr) {
                                const float *o = red + g * 128;
                                mr = -nms[g * 32 + col];
                                sr = (o[col] + o[CW + col]) + (o[2 * CW + col] + o[3 * CW + col]);
                            };
                            if (Z::PP) {
                                float m0, m1, s0, s1;
                                side(0, r, m0, s0);
                                side(1, r, m1, s1);
                                top_r = fmaxf(m0, m1);
                                f[0] = ex2(m0 - top_r);
                                f[1] = ex2(m1 - top_r);
                                sum = s0 * f[0] + s1 * f[1];
                            } else {
                                side(r / CW, r % CW, top_r, sum);
                            }
                            if (flushed) {
                                const float2 o = a.ml[(int64_t)slot * RT + r];
                                const float mm = fmaxf(o.x, top_r), g = ex2(top_r - mm);
                                f[2] = ex2(o.x - mm);
                                f[0] *= g, f[1] *= g;
                                sum = sum * g + o.y * f[2];
                                top_r = mm;
                            }
                            if (last && whole) {
                                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                                for (int k = 0; k < 3; ++k) f[k] *= inv;
                            } else {
                                a.ml[(int64_t)slot * RT + r] = make_float2(top_r, sum);
                            }
#pragma unroll
                            for (int k = 0; k < 3; ++k) fac[k * 64 + r] = f[k];
                        }
                        bar_n<256>(3);
                        // which streams have sums: in a segment of one tile only one has
                        const int blk = (t - t0) % kTaFlush;  // tiles since the last flush, less one
                        const bool both = blk > 0;
                        const int lone = it & 1;
#pragma unroll 1
                        for (int q = wg; q < (RT / 16) * Z::MT; q += 2) {
                            const int i = (q % (RT / 16)) * 16, mt = q / (RT / 16), d = mt * 128 + tk;
                            if (i >= rows) continue;
                            float v[16] = {};
                            const int g0 = Z::PP && !both ? lone : 0, g1 = Z::PP && both ? 2 : g0 + 1;
#pragma unroll 1
                            for (int g = g0; g < g1; ++g) {
                                const uint32_t ad = tmem + lanes + 2 * N + (g * Z::MT + mt) * N + i;
                                uint32_t o[16], ol[16];
                                tmem_get(ad, o);
                                if (kE4M3) tmem_get(ad + RT, ol);
                                float f[16];
                                load16(fac + g * 64 + i, f);
                                tmem_got(o);
                                if (kE4M3) tmem_got(ol);
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    float x = __uint_as_float(o[k]);
                                    if (kE4M3) x = fmaf(__uint_as_float(ol[k]), 0.03125f, x);
                                    v[k] = fmaf(x, f[k], v[k]);
                                }
                            }
                            if (d >= c.dim) continue;
                            const int nr = min(16, rows - i);
                            float *pd = a.part + ((int64_t)slot * RT + i) * DP + d;
                            if (flushed) {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (k < nr) v[k] = fmaf(pd[k * DP], fac[128 + i + k], v[k]);
                            }
                            if (last && whole) {
                                int tok = ta_token(a, row0 + i), gi = row0 + i - tok * a.group;
                                bf16 *po = a.out + (((int64_t)w.b * c.n + tok) * a.q_heads + hk * a.group + gi) * c.dim + d;
                                const int64_t jump = (int64_t)(a.q_heads - a.group) * c.dim;
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    if (k < nr) *po = __float2bfloat16_rn(tok < w.cnt ? v[k] : 0.0f);
                                    po += c.dim;
                                    if (++gi == a.group) gi = 0, ++tok, po += jump;
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (k < nr) pd[k * DP] = v[k];
                            }
                        }
                        tc_fence_before();
                        flushed = true;
                        some = false;
                        fresh();
                        bar_n<256>(3);  // factors, masks and sums may be overwritten
                    }
                }
            };
            if constexpr (kE4M3) {
                if (__builtin_expect(spread, 0))
                    tiles(std::true_type{});
                else
                    tiles(std::false_type{});
            } else {
                tiles(std::false_type{});
            }
            if (threadIdx.x == 0 && t0 == 0 && !whole) {
                // (the place of the unit's last tile, and the cost of all)
                a.desc[blockIdx.x] = make_int4(w.b, w.u, w.start + w.ntiles - 1, w.total);
            }
            items += 2 * Z::NS * (t1 - t0);
            ta_next(w, c, units);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(*abort_flag && a.box, 0) && warp == 8) {
        // Boxes may be in flight: they land before the CTA's shared memory
        // goes.  In a slot only the last item copied can be, K's or V's (the
        // one before has been multiplied).
        if (lane < SLOTS) {
            const int last = max((int)rowtab[lane], (int)rowtab[64 + lane]);
            if (last >= 0) ta_drain(&full[lane], (unsigned)((last / SLOTS) & 1), c.status);
        }
        __syncwarp();
    }
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Z::COLS));
}

// Joins the partial sums of the unit that CTA blockIdx.x began and others
// finished.  A block has G groups of lanes that each cover a row; S of them
// share a row's contributors (few rows come with many contributors).  A lane
// takes references, sums and its 4 dims of a few contributors at a time, so
// that little lies between the first kernel's end and the stores but two
// round trips to L2; contributors are taken in a fixed order.
template <int DP, int RT, int S>
__global__ void __launch_bounds__(256, 6) tree_join_kernel(const __grid_constant__ TaArgs a)
{
    constexpr int L = DP / 4, G = 256 / L, R = G / S;  // 16-byte lanes of a row; rows of a block
    __shared__ float4 acc[G][L];
    __shared__ float2 mls[G];
    pdl_wait();
    pdl_trigger();  // only now: a kernel after this one may rely on all before it
    const int4 u = a.desc[blockIdx.x];
    if (u.x < 0) return;
    const CacheArgs &c = a.c;
    const int hk = u.y / a.rtiles, row0 = (u.y - hk * a.rtiles) * RT, t = threadIdx.x;
    const int grp = t / L, el = (t % L) * 4, part = grp % S, r = blockIdx.y * R + grp / S;
    const bool on = r < min(RT, c.n * a.group - row0);
    const int cnt = seq_count(c, u.x);
    // the CTA whose range has the unit's last tile (ranges as in ta_walk); contributors
    const int ctas = min((int)gridDim.x + 1, u.w), each = u.w / ctas, more = u.w - each * ctas, cut = more * (each + 1);
    const int n = (u.z < cut ? u.z / (each + 1) : more + (u.z - cut) / each) - (int)blockIdx.x + 1;
    float m = kTaNone, s = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int B = S > 1 ? 4 : 2;
    for (int k0 = part; on && k0 < n; k0 += B * S) {
        float2 ml[B];
        float4 v[B];
#pragma unroll
        for (int q = 0; q < B; ++q) {
            const int k = k0 + q * S;
            const int64_t at = (int64_t)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * RT + r;
            ml[q] = make_float2(kTaNone, 0.0f);
            v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < n) {
                ml[q] = a.ml[at];
                if (el < c.dim) v[q] = *reinterpret_cast<const float4 *>(a.part + at * DP + el);
            }
        }
        float top = m;
#pragma unroll
        for (int q = 0; q < B; ++q) top = fmaxf(top, ml[q].x);
        float f = ex2(m - top);
        m = top;
        s *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int q = 0; q < B; ++q) {
            f = ex2(ml[q].x - top);
            s = fmaf(ml[q].y, f, s);
            o.x = fmaf(v[q].x, f, o.x), o.y = fmaf(v[q].y, f, o.y), o.z = fmaf(v[q].z, f, o.z), o.w = fmaf(v[q].w, f, o.w);
        }
    }
    if (S > 1) {
        acc[grp][t % L] = o;
        if (t % L == 0) mls[grp] = make_float2(m, s);
        __syncthreads();
        if (part != 0) return;
        float top = m;
#pragma unroll
        for (int i = 1; i < S; ++i) top = fmaxf(top, mls[grp + i].x);
        float f = ex2(m - top);
        s *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int i = 1; i < S; ++i) {
            const float4 v = acc[grp + i][t % L];
            f = ex2(mls[grp + i].x - top);
            s = fmaf(mls[grp + i].y, f, s);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        }
    }
    if (!on || el >= c.dim) return;
    const int g = row0 + r, i = ta_token(a, g);
    const float f = s == 0.0f ? 0.0f : 1.0f / s;
    uint2 two = make_uint2(bf16x2_bits(o.x * f, o.y * f), bf16x2_bits(o.z * f, o.w * f));
    if (i >= cnt) two = make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(a.out + (((int64_t)u.x * c.n + i) * a.q_heads + hk * a.group + (g - i * a.group)) * c.dim + el) = two;
}

// -------------------------------------------------------------------- host --
// Row tile: the smallest of 16, 32, 64 that holds the rows of a kv head, and
// tiles of 64 above that.  The loads of a tile cost the same for any of them,
// and a smaller one has fewer columns to turn into weights and less to join.
// Above 64 rows the cache is read once per tile, from L2 after the first.
static int ta_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

static size_t ta_part_bytes(int RT, int DP) { return (size_t)2 * kTaMaxCtas * RT * DP * sizeof(float); }
static size_t ta_ml_bytes(int RT) { return (size_t)2 * kTaMaxCtas * RT * sizeof(float2); }

size_t tree_attention_workspace_bytes(int64_t, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim)
{
    const int RT = ta_rows(n * (q_heads / kv_heads)), DP = dim <= 128 ? 128 : 256;
    return (ta_part_bytes(RT, DP) + ta_ml_bytes(RT) + kTaMaxCtas * sizeof(int4) + 255) / 256 * 256;
}

template <bool kE4M3, int DP, int RT>
static cudaError_t ta_launch(const TaArgs &a, int ctas, int device, cudaStream_t st)
{
    using Z = TaShape<kE4M3, DP, RT>;
    // once per device (setting it twice is harmless)
    static std::atomic<uint64_t> set{0};
    cudaError_t e;
    if (!((set.load(std::memory_order_relaxed) >> device) & 1)) {
        e = cudaFuncSetAttribute(tree_attention_kernel<kE4M3, DP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
        if (e != cudaSuccess) return e;
        set.fetch_or((uint64_t)1 << device, std::memory_order_relaxed);
    }
    e = launch_dependent(tree_attention_kernel<kE4M3, DP, RT>, dim3(ctas), kTaThreads, Z::SMEM, st, a);
    if (e != cudaSuccess || ctas == 1) return e;
    // the join may become resident early; it waits for the whole first kernel
    constexpr int G = 1024 / DP, S = RT == 16 ? G : 1, R = G / S;
    const int rows = a.c.n * a.group < RT ? a.c.n * a.group : RT;
    return launch_dependent(tree_join_kernel<DP, RT, S>, dim3(ctas - 1, (rows + R - 1) / R), 256, 0, st, a);
}

wl_status launch_tree_attention(const bf16 *q, int64_t q_heads, const uint64_t *mask, float scale, const wl_cache &cache,
                                const wl_seqs &seqs, bf16 *out, void *ws, const DeviceInfo *di, cudaStream_t st)
{
    const int group = (int)(q_heads / cache.kv_heads), DP = cache.dim <= 128 ? 128 : 256;
    const int64_t rows = seqs.n * group;
    const int RT = ta_rows(rows);
    if (cache.pages * cache.kv_heads * cache.page_size >= (int64_t)0xffffffff)
        return fail(WL_ERR_UNSUPPORTED, "wl_tree_attention: pages * kv_heads * page_size must be below 2^32 - 1");
    TaArgs a;
    a.q = q, a.mask = mask, a.out = out;
    a.part = static_cast<float *>(ws);
    a.ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + ta_part_bytes(RT, DP));
    a.desc = reinterpret_cast<int4 *>(reinterpret_cast<char *>(a.ml) + ta_ml_bytes(RT));
    a.q_heads = (int)q_heads, a.group = group, a.rtiles = (int)((rows + RT - 1) / RT);
    a.group_inv = group > 1 ? (uint32_t)(((1ull << 32) + group - 1) / group) : 0u;
    a.scale = scale;
    a.c = cache_args(cache, seqs, di->status);
    // Runs of positions that never cross a page: the largest power of two that
    // divides the page size, 128 at most.  Under 8 rows a box would start
    // inside an 8-row swizzle group, so such pages go by 16-byte copies of four
    // warps, as do caches of more rows than a box can address (the cases at the
    // top: 143, 89, 75 and 112 us by copies when boxes took 144, 83, 64 and 88;
    // the copies share the softmax warps' load and store unit).
    const int64_t rowb = cache.dim * (cache.format == WL_CACHE_E4M3 ? 1 : 2), nrows = cache.pages * cache.kv_heads * cache.page_size;
    a.box = (int)(cache.page_size & -cache.page_size);
    if (a.box > kTaTile) a.box = kTaTile;
    if (a.box < 8 || nrows > 0x7fffffff) a.box = 0;
    if (a.box > 0) {
        wl_status s = tmap_rows_u8(cache.k, rowb, nrows, a.box, &a.kmap);
        if (s == WL_OK) s = tmap_rows_u8(cache.v, rowb, nrows, a.box, &a.vmap);
        if (s != WL_OK) return s;
    }
    // at most one CTA per tile that the table can hold
    const int64_t tiles = seqs.batch * cache.kv_heads * a.rtiles * ((seqs.max_pages * cache.page_size + seqs.n + kTaTile - 1) / kTaTile);
    int ctas = di->sm_count < kTaMaxCtas ? di->sm_count : kTaMaxCtas;
    if (tiles + seqs.batch * cache.kv_heads * a.rtiles * kTaSwitch > 0x7fffffff)
        return fail(WL_ERR_UNSUPPORTED, "wl_tree_attention: batch * kv_heads * positions of the page table / 128 must be below 2^31");
    if (tiles < ctas) ctas = (int)tiles;
    cudaError_t e;
    if (cache.format == WL_CACHE_E4M3) {
        if (DP == 128)
            e = RT == 16 ? ta_launch<true, 128, 16>(a, ctas, di->device, st) : RT == 32 ? ta_launch<true, 128, 32>(a, ctas, di->device, st) : ta_launch<true, 128, 64>(a, ctas, di->device, st);
        else
            e = RT == 16 ? ta_launch<true, 256, 16>(a, ctas, di->device, st) : RT == 32 ? ta_launch<true, 256, 32>(a, ctas, di->device, st) : ta_launch<true, 256, 64>(a, ctas, di->device, st);
    } else {
        if (DP == 128)
            e = RT == 16 ? ta_launch<false, 128, 16>(a, ctas, di->device, st) : RT == 32 ? ta_launch<false, 128, 32>(a, ctas, di->device, st) : ta_launch<false, 128, 64>(a, ctas, di->device, st);
        else
            e = RT == 16 ? ta_launch<false, 256, 16>(a, ctas, di->device, st) : RT == 32 ? ta_launch<false, 256, 32>(a, ctas, di->device, st) : ta_launch<false, 256, 64>(a, ctas, di->device, st);
    }
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_tree_attention launch");
}

}  // namespace wl
