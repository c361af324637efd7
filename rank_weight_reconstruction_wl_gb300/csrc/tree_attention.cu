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
// is exactly two 4-bit parts, so q loses nothing but what lies 2^-22 below the
// largest |q| of the tile.  The weights of v are folded with the row scales
// (w = p * v_scale); a weight keeps 8 bits down to 2^-18 of the largest and is
// dropped below 2^-22 of it.  Sums over more than kTaFlush tiles are therefore
// flushed to fp32, which bounds what a CTA can drop by 8192 * 2^-22 = 0.2 %.
// bf16 caches take one bf16 part.
//
// Work: (sequence, kv head, row tile) units of ceil(positions / 128) tiles are
// laid end to end and cut into one equal range per CTA (one CTA per SM), so
// ragged lengths balance; a unit cut by a range is joined from fp32 partials by
// tree_join_kernel, in a fixed order.
#include "cache_row.cuh"
#include "dec_ptx.cuh"
#include "tc_ptx.cuh"

namespace wl {

constexpr int kTaMaxCtas = 152;
constexpr int kTaThreads = 512;  // warps 0-7 softmax, 8 MMA (9-11 idle), 12-15 cache loads
// Registers: the block is launched with 512 x 128; the softmax warps take 168
// each and the others keep 88 (256 x 168 + 256 x 88 = 512 x 128).
constexpr int kTaRegsSoftmax = 168, kTaRegsOther = 88;
static_assert(kTaRegsSoftmax + kTaRegsOther == 2 * 128, "register split");
constexpr int kTaTile = 128;     // positions per tile
constexpr int kTaFlush = 64;     // tiles summed in tensor memory before the sums move to fp32 partials
constexpr float kTaNone = -3.0e38f;  // reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;

struct TaArgs {
    const bf16 *q;
    const uint64_t *mask;
    bf16 *out;
    float *part;   // [2 * ctas][RT][DP] partial sums
    float2 *ml;    // [2 * ctas][RT] reference and sum of each row
    int4 *desc;    // [ctas] unit that CTA c begins and others finish: sequence, unit, last CTA (sequence -1: none)
    int q_heads, group, rtiles;
    float scale;
    CacheArgs c;
};

template <bool kE4M3, int DP, int RT>
struct TaShape {
    static constexpr int ES = kE4M3 ? 1 : 2;
    static constexpr int PARTS = kE4M3 ? 2 : 1;
    static constexpr int N = PARTS * RT;             // columns of both products
    static constexpr int ROWB = DP * ES;             // bytes of a cache row
    static constexpr int SLOTROW = ROWB < 256 ? ROWB : 256;
    static constexpr int NS = ROWB / SLOTROW;        // ring slots per K or V tile
    static constexpr int SLOT = kTaTile * SLOTROW;
    static constexpr int QB = N * ROWB;
    static constexpr int PW = 2 * RT;                // bytes of a position's weights
    static constexpr int PB = kTaTile * PW;
    static constexpr int MISC = 2048;
    static constexpr int ROOM = (232448 - 1024 - MISC - QB - 2 * PB) / SLOT;
    static constexpr int SLOTS = ROOM < 12 ? ROOM : 12;
    static constexpr int SMEM = 1024 + MISC + QB + 2 * PB + SLOTS * SLOT;
    static constexpr int MT = DP / 128;              // M tiles of the second product
    static constexpr int COLS = (2 + MT) * N <= 64 ? 64 : (2 + MT) * N <= 128 ? 128 : (2 + MT) * N <= 256 ? 256 : 512;
    static constexpr int KSTEP = 32 / ES;            // contraction elements per MMA: 32 bytes of a K-major row
    static constexpr int CW = RT / 2;                // columns per softmax warpgroup
    static constexpr int SWP = PW == 128 ? 2 : PW == 64 ? 4 : 6;  // swizzle code of the weights' rows
    static_assert(SLOTS >= 4 && SMEM <= 232448 && (2 + MT) * N <= 512, "tile shape");
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

// CW consecutive columns of this thread's lane, waited for.
template <int CW>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, float (&v)[CW])
{
    uint32_t r[CW];
    if constexpr (CW == 8) {
        tmem_ld8_nw(taddr, r);
        tmem_wait_ld8(r);
    } else {
#pragma unroll
        for (int i = 0; i < CW; i += 16) tmem_ld16_nw(taddr + i, r + i);
#pragma unroll
        for (int i = 0; i < CW; i += 16) tmem_wait16(r + i);
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// A bounded wait that gives up at once when the CTA is winding down.  A wait
// that gives up sets the abort flag; every role then runs through its loops
// without waiting, copying or issuing, so barriers stay matched.
__device__ __forceinline__ void ta_wait(uint64_t *bar, unsigned parity, unsigned *status, unsigned site, volatile int *abort_flag)
{
    if (mbar_test(bar, parity)) return;
    const long long t0 = wait_clock();
    while (!*abort_flag && !mbar_test(bar, parity)) {
        if (wait_clock() - t0 > kWaitLimitCycles) {
            atomicOr(status, kStatusTimeout | site);
            *abort_flag = 1;
        }
    }
}

// The last wait, for MMAs in flight, also when the CTA is winding down.
__device__ __forceinline__ void ta_drain(uint64_t *bar, unsigned *status)
{
    const long long t0 = wait_clock();
    while (!mbar_test(bar, 0)) {
        if (wait_clock() - t0 > kWaitLimitCycles) {
            atomicOr(status, kStatusTimeout | kWaitDrain);
            return;
        }
    }
}

// ------------------------------------------------------------------ range --
// Walks a CTA's range of the tiles of all units, unit by unit.
struct TaWalk {
    int64_t total, start, left;  // all tiles; first tile of the next segment; tiles left
    int b, u, tile, ntiles, len, cnt, ctas;  // ctas: CTAs with work (no more than tiles)
};

__device__ __forceinline__ int ta_tiles(const CacheArgs &c, int b, int &len, int &cnt)
{
    len = seq_len(c, b);
    cnt = seq_count(c, b);
    return cnt > 0 ? (len + cnt + kTaTile - 1) / kTaTile : 1;
}

// Called by whole warps.
__device__ __forceinline__ TaWalk ta_walk(const CacheArgs &c, int units)
{
    const int lane = threadIdx.x & 31;
    TaWalk w;
    int len, cnt;
    int64_t sum = 0;
    for (int b = lane; b < c.batch; b += 32) sum += ta_tiles(c, b, len, cnt);
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    w.total = sum * units;
    w.ctas = (int)min((int64_t)gridDim.x, w.total);
    w.start = (int64_t)blockIdx.x * w.total / w.ctas;
    w.left = (int)blockIdx.x < w.ctas ? ((int64_t)blockIdx.x + 1) * w.total / w.ctas - w.start : 0;
    w.b = w.u = w.tile = w.ntiles = w.len = w.cnt = 0;
    if (w.left == 0) return w;
    int64_t base = 0;
    for (int b0 = 0; b0 < c.batch; b0 += 32) {
        int64_t mine = b0 + lane < c.batch ? (int64_t)ta_tiles(c, b0 + lane, len, cnt) * units : 0;
        int64_t incl = mine;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > w.start);
        if (past) {
            const int l = __ffs(past) - 1;
            const int64_t off = w.start - (base + __shfl_sync(0xffffffffu, incl - mine, l));
            w.b = b0 + l;
            w.ntiles = ta_tiles(c, w.b, w.len, w.cnt);
            w.u = (int)(off / w.ntiles);
            w.tile = (int)(off - (int64_t)w.u * w.ntiles);
            return w;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.left = 0;
    return w;
}

// The segment's end tile; then on to the next unit.
__device__ __forceinline__ int ta_end(const TaWalk &w) { return (int)min((int64_t)w.ntiles, w.tile + w.left); }
__device__ __forceinline__ void ta_next(TaWalk &w, const CacheArgs &c, int units)
{
    const int t1 = ta_end(w);
    w.left -= t1 - w.tile;
    w.start += t1 - w.tile;
    w.tile = t1;
    if (t1 == w.ntiles && w.left > 0) {
        w.tile = 0;
        if (++w.u == units) {
            w.u = 0;
            ++w.b;
            w.ntiles = ta_tiles(c, w.b, w.len, w.cnt);
        }
    }
}

// ------------------------------------------------------------------ kernel --
template <bool kE4M3, int DP, int RT>
__global__ void __launch_bounds__(kTaThreads, 1) tree_attention_kernel(const __grid_constant__ TaArgs a)
{
    using Z = TaShape<kE4M3, DP, RT>;
    constexpr int N = Z::N, CW = Z::CW, SLOTS = Z::SLOTS;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (s32(smem_raw) & 1023u)) & 1023u);
    char *sq = smem, *sp = sq + Z::QB, *ring = sp + 2 * Z::PB, *misc = ring + SLOTS * Z::SLOT;
    uint64_t *smask = reinterpret_cast<uint64_t *>(misc);            // [RT]
    float *red = reinterpret_cast<float *>(misc + 512);              // [2][4][32]
    float *qmax = reinterpret_cast<float *>(misc + 2016);            // [8]
    uint64_t *bars = reinterpret_cast<uint64_t *>(misc + 1536);
    uint64_t *full = bars, *empty = full + SLOTS, *s_full = empty + SLOTS, *s_empty = s_full + 2, *p_full = s_full + 4,
             *pv_done = s_full + 6, *q_ready = s_full + 8, *drain = s_full + 9;
    uint32_t *tmem_hold = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_hold + 1);
    static_assert((2 * 12 + 11) * 8 <= 2016 - 1536, "barriers");

    const CacheArgs &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = c.kv_heads * a.rtiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 8);
            mbar_init(&p_full[i], 8);
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
    TaWalk w = ta_walk(c, units);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_hold;
    pdl_trigger();

    if (warp >= 12) {
        // ------------------------------------------------ cache loads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTaRegsOther));
        // Ring items in the order the MMAs take them: K0, K1, V0, K2, V1, ...
        // Warp pw holds rows 32 pw .. of a tile: a lane looks up one row's
        // place, then the lanes of a row copy 16 bytes each.
        const int pw = warp - 12;
        constexpr int LPR = Z::SLOTROW / 16, RPP = 32 / LPR;  // lanes per row, rows per pass
        const int ch = lane % LPR, sub = lane / LPR;
        int item = 0;
        auto place = [&](int j, int total, int hk) -> int64_t {
            if (j >= total) return -1;
            const int64_t row = cache_row(c, w.b, hk, j);
            if (row < 0) atomicOr(c.status, kStatusPage);
            return row;
        };
        auto copy = [&](const char *base, int64_t row) {
#pragma unroll
            for (int s = 0; s < Z::NS; ++s, ++item) {
                const int slot = item % SLOTS;
                ta_wait(&empty[slot], (unsigned)(((item / SLOTS) & 1) ^ 1), c.status, kWaitRingEmpty, abort_flag);
                if (*abort_flag) continue;
                const uint32_t dst = s32(ring + slot * Z::SLOT);
                const int col = s * Z::SLOTROW + ch * 16;
                const bool in = col < c.dim * Z::ES;
#pragma unroll
                for (int p = 0; p < 32 / RPP; ++p) {
                    const int r = p * RPP + sub, t = pw * 32 + r;
                    const int64_t at = __shfl_sync(0xffffffffu, row, r);
                    const bool ok = in && at >= 0;
                    const char *src = ok ? base + at * (c.dim * Z::ES) + col : base;
                    const uint32_t d = dst + (uint32_t)((ch >> 3) * (kTaTile * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(ok ? 16 : 0) : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s32(&full[slot])) : "memory");
            }
        };
        while (w.left > 0) {
            const int t1 = ta_end(w), total = w.cnt > 0 ? w.len + w.cnt : 0, hk = w.u / a.rtiles;
            int64_t prev = -1, next = place(w.tile * kTaTile + pw * 32 + lane, total, hk);
            for (int t = w.tile; t < t1; ++t) {
                const int64_t row = next;
                if (t + 1 < t1) next = place((t + 1) * kTaTile + pw * 32 + lane, total, hk);
                copy(c.k, row);
                if (t > w.tile) copy(c.v, prev);
                prev = row;
            }
            copy(c.v, prev);
            ta_next(w, c, units);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
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
            auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t acc) {
                if constexpr (kE4M3)
                    umma_f8(d, da, db, id, acc);
                else
                    umma(d, da, db, id, acc);
            };
            auto take = [&](int &slot) {
                slot = item % SLOTS;
                ta_wait(&full[slot], (unsigned)((item / SLOTS) & 1), c.status, kWaitRingFull, abort_flag);
                fence_async_smem();  // the copies were ordinary shared-memory writes
                ++item;
            };
            auto scores = [&](int i) {
                ta_wait(&s_empty[i & 1], (unsigned)(((i >> 1) & 1) ^ 1), c.status, kWaitRingEmpty, abort_flag);
                tc_fence_after();
                const uint32_t d = tmem + (i & 1) * N;
#pragma unroll
                for (int s = 0; s < Z::NS; ++s) {
                    int slot;
                    take(slot);
                    if (*abort_flag) continue;
                    const uint32_t ak = br + slot * Z::SLOT;
#pragma unroll
                    for (int k = 0; k < Z::SLOTROW / 32; ++k) {
                        const int gk = s * (Z::SLOTROW / 32) + k;
                        mma(d, ta_desc(ak + (k / 4) * (kTaTile * 128) + (k % 4) * 32, 16, 1024, 2),
                            ta_desc(bq + (gk / 4) * (N * 128) + (gk % 4) * 32, 16, 1024, 2), kId, gk > 0 ? 1u : 0u);
                    }
                    umma_commit(&empty[slot]);
                }
                umma_commit(&s_full[i & 1]);
            };
            auto values = [&](int i, bool first) {
                ta_wait(&p_full[i & 1], (unsigned)((i >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                tc_fence_after();
                const uint32_t pb = bp + (i & 1) * Z::PB;
#pragma unroll
                for (int s = 0; s < Z::NS; ++s) {
                    int slot;
                    take(slot);
                    if (*abort_flag) continue;
                    const uint32_t av = br + slot * Z::SLOT;
                    constexpr int MS = Z::MT / Z::NS;  // M tiles of a slot
#pragma unroll
                    for (int m = 0; m < MS; ++m)
#pragma unroll
                        for (int k = 0; k < kTaTile / Z::KSTEP; ++k)
                            mma(ocol + (s * MS + m) * N,
                                ta_desc(av + m * Z::ES * (kTaTile * 128) + k * Z::KSTEP * 128, kTaTile * 128, 1024, 2),
                                ta_desc(pb + k * Z::KSTEP * Z::PW, 8 * Z::PW, 8 * Z::PW, Z::SWP), kIdPV, (first && k == 0) ? 0u : 1u);
                    umma_commit(&empty[slot]);
                }
                umma_commit(&pv_done[i & 1]);
            };
            while (w.left > 0) {
                const int t1 = ta_end(w);
                ta_wait(q_ready, (unsigned)(seg & 1), c.status, kWaitRingFull, abort_flag);
                tc_fence_after();
                for (int t = w.tile; t < t1; ++t, ++it) {
                    scores(it);
                    if (t > w.tile) values(it - 1, (t - 1 - w.tile) % kTaFlush == 0);
                }
                values(it - 1, (t1 - 1 - w.tile) % kTaFlush == 0);
                ++seg;
                ta_next(w, c, units);
            }
            umma_commit(drain);
            ta_drain(drain, c.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax
        // Warpgroup wg takes columns wg * CW ..; a thread is one position of
        // a tile (lane of S^T) and, at the end, one dim of each M tile.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTaRegsSoftmax));
        const int wg = warp >> 2, tk = threadIdx.x & 127, col0 = wg * CW;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        float *wred = red + wg * 128;
        int it = 0;
        if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
        while (w.left > 0) {
            const int t0 = w.tile, t1 = ta_end(w), total = w.cnt > 0 ? w.len + w.cnt : 0;
            const int hk = w.u / a.rtiles, row0 = (w.u - hk * a.rtiles) * RT, rows = min(RT, c.n * a.group - row0);
            // place and scales of this thread's position, loaded a tile ahead
            auto place = [&](int t) -> int64_t {
                const int j = t * kTaTile + tk;
                return j < total ? cache_row(c, w.b, hk, j) : -1;
            };
            int64_t at = place(t0), at1 = t0 + 1 < t1 ? place(t0 + 1) : -1;
            float ks = at >= 0 ? __ldg(c.k_scale + at) : 0.0f, vs = at >= 0 ? __ldg(c.v_scale + at) : 1.0f;
            bar_n<256>(3);  // both warpgroups are done with the previous segment's masks
            // ---- the segment's queries: rows of the B operand
            float qscale = a.scale * kLog2e;
            {
                constexpr int CH = DP / 8, PER = RT * CH / 256;  // 8-element chunks of a row, per thread
                uint4 qv[PER];
                uint32_t amax = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = threadIdx.x + i * 256, r = e / CH, d = (e % CH) * 8, g = row0 + r;
                    qv[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < rows && d < c.dim && g / a.group < w.cnt) {
                        const int64_t tok = (int64_t)w.b * c.n + g / a.group;
                        qv[i] = *reinterpret_cast<const uint4 *>(a.q + (tok * a.q_heads + hk * a.group + g % a.group) * c.dim + d);
                    }
                    if (kE4M3) {
                        const uint32_t u[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t lo = u[j] & 0x7fffu, hi = (u[j] >> 16) & 0x7fffu;
                            amax = max(amax, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                        }
                    }
                }
                if (threadIdx.x < RT) {
                    const int g = row0 + threadIdx.x, i = g / a.group;
                    uint64_t m = 0;
                    if ((int)threadIdx.x < rows && i < w.cnt) {
                        m = a.mask ? a.mask[(int64_t)w.b * c.n + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
                        if (w.cnt < 64) m &= (1ull << w.cnt) - 1;
                    }
                    smask[threadIdx.x] = m;
                }
                float up = 1.0f;
                if (kE4M3) {
                    // one power of two brings the largest |q| of the tile into [128, 256)
                    amax = __reduce_max_sync(0xffffffffu, amax);
                    if (lane == 0) qmax[warp] = __uint_as_float(amax << 16);
                    bar_n<256>(3);
                    float mx = 0.0f;
                    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, qmax[i]);
                    const int be = max((int)(__float_as_uint(mx) >> 23), 14);
                    up = __uint_as_float((uint32_t)(261 - be) << 23);  // 2^(134 - be)
                    qscale *= __uint_as_float((uint32_t)(be - 7) << 23);
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = threadIdx.x + i * 256, r = e / CH, ck = e % CH;
                    if (kE4M3) {
                        const uint32_t u[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                        uint32_t hi[2] = {}, lo[2] = {};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = bf_lo(u[j]) * up, y = bf_hi(u[j]) * up;
                            uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
                            const float2 b = e4m3x2_f32(h);
                            const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2((x - b.x) * 32.0f, (y - b.y) * 32.0f), __NV_SATFINITE, __NV_E4M3);
                            if ((u[j] & 0x7fffu) >= 0x7f80u) h |= 0x7fu;  // NaN, infinity: a NaN code
                            if ((u[j] >> 16 & 0x7fffu) >= 0x7f80u) h |= 0x7f00u;
                            hi[j / 2] |= h << (16 * (j & 1));
                            lo[j / 2] |= l << (16 * (j & 1));
                        }
                        const int cc = ck / 16, c16 = (ck / 2) & 7, half = (ck & 1) * 8;
                        char *o = sq + cc * (N * 128) + half;
                        *reinterpret_cast<uint2 *>(o + r * 128 + ((c16 ^ (r & 7)) << 4)) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2 *>(o + (RT + r) * 128 + ((c16 ^ (r & 7)) << 4)) = make_uint2(lo[0], lo[1]);
                    } else {
                        *reinterpret_cast<uint4 *>(sq + (ck / 8) * (N * 128) + r * 128 + (((ck & 7) ^ (r & 7)) << 4)) = qv[i];
                    }
                }
                fence_async_smem();
                bar_n<256>(3);  // the masks too
                if (lane == 0) mbar_arrive(q_ready);
            }
            float m[CW], l[CW];
#pragma unroll
            for (int i = 0; i < CW; ++i) m[i] = kTaNone, l[i] = 0.0f;
            const int slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
            const bool whole = t0 == 0 && t1 == w.ntiles;
            bool flushed = false;
            for (int t = t0; t < t1; ++t, ++it) {
                const int j = t * kTaTile + tk;
                const bool seen = at >= 0;
                const float cs = ks * qscale, lv = log2f(vs), iv = vs == vs ? 1.0f / vs : 1.0f;
                at = at1;
                if (t + 1 < t1) {
                    ks = at >= 0 ? __ldg(c.k_scale + at) : 0.0f;
                    vs = at >= 0 ? __ldg(c.v_scale + at) : 1.0f;
                    at1 = t + 2 < t1 ? place(t + 2) : -1;
                }
                float x[CW];
                ta_wait(&s_full[it & 1], (unsigned)((it >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                tc_fence_after();
                const uint32_t sc = tmem + lanes + (it & 1) * N + col0;
                tmem_cols<CW>(sc, x);
                if (kE4M3) {
#pragma unroll
                    for (int i = 0; i < CW; i += 8) {
                        float lo[8];
                        tmem_cols<8>(sc + RT + i, lo);
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[i + k] = fmaf(lo[k], 0.03125f, x[i + k]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[it & 1]);
                float top = -INFINITY;
                if (!seen) {
#pragma unroll
                    for (int i = 0; i < CW; ++i) x[i] = -INFINITY;
                } else if (j < w.len) {
#pragma unroll
                    for (int i = 0; i < CW; ++i) {
                        x[i] = fmaf(x[i], cs, lv);
                        top = fmaxf(top, x[i] - m[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < CW; ++i) {
                        x[i] = (smask[col0 + i] >> (j - w.len)) & 1 ? fmaf(x[i], cs, lv) : -INFINITY;
                        top = fmaxf(top, x[i] - m[i]);
                    }
                }
                // Weights up to 2^8 are held as they are; only a position above
                // that moves its row's reference (to 2^7 below it).
                if (bar_or<128>(1 + wg, top > 8.0f)) {
#pragma unroll
                    for (int i = 0; i < CW; i += 8) {
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = x[i + k];
                        const float cm = warp_columns<8>(y, [](float p, float q) { return fmaxf(p, q); });
                        if (lane < 8) wred[(warp & 3) * 32 + i + lane] = cm;
                    }
                    bar_n<128>(1 + wg);
                    const bool sums = (t - t0) % kTaFlush != 0;  // sums of earlier tiles are in tensor memory
                    if (sums) {
                        ta_wait(&pv_done[(it - 1) & 1], (unsigned)(((it - 1) >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                        tc_fence_after();
                    }
#pragma unroll
                    for (int i = 0; i < CW; i += 8) {
                        float f[8];
                        bool any = false;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float mx = fmaxf(fmaxf(wred[i + k], wred[32 + i + k]), fmaxf(wred[64 + i + k], wred[96 + i + k]));
                            f[k] = 1.0f;
                            if (mx - m[i + k] > 8.0f) {
                                f[k] = ex2(m[i + k] - (mx - 7.0f));
                                m[i + k] = mx - 7.0f;
                                l[i + k] *= f[k];
                                any = true;
                            }
                        }
                        if (!any || !sums) continue;
#pragma unroll
                        for (int p = 0; p < Z::MT * Z::PARTS; ++p) {
                            const uint32_t ad = tmem + lanes + 2 * N + p * RT + col0 + i;
                            float o[8];
                            tmem_cols<8>(ad, o);
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] *= f[k];
                            tmem_st8(ad, o);
                        }
                    }
                    if (sums) tmem_wait_st();
                    bar_n<128>(1 + wg);  // wred is free again
                }
                // weights: w = 2^(x - m) = p * v_scale
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    x[i] = ex2(x[i] - m[i]);
                    l[i] = fmaf(x[i], iv, l[i]);
                }
                if (it >= 2)
                    ta_wait(&pv_done[it & 1], (unsigned)(((it - 2) >> 1) & 1), c.status, kWaitRingEmpty, abort_flag);
                char *pr = sp + (it & 1) * Z::PB;
                const uint32_t rowb = tk * Z::PW, sw = ((rowb >> 7) & (Z::PW / 16 - 1)) << 4;
                if constexpr (kE4M3) {
                    uint32_t hi[CW / 4], lo[CW / 4];
#pragma unroll
                    for (int i = 0; i < CW / 4; ++i) {
                        uint32_t hh[2], ll[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float p = x[4 * i + 2 * k], q = x[4 * i + 2 * k + 1];
                            hh[k] = __nv_cvt_float2_to_fp8x2(make_float2(p, q), __NV_SATFINITE, __NV_E4M3);
                            const float2 b = e4m3x2_f32(hh[k]);
                            ll[k] = __nv_cvt_float2_to_fp8x2(make_float2((p - b.x) * 32.0f, (q - b.y) * 32.0f), __NV_SATFINITE, __NV_E4M3);
                        }
                        hi[i] = hh[0] | (hh[1] << 16);
                        lo[i] = ll[0] | (ll[1] << 16);
                    }
                    if constexpr (CW == 8) {
                        *reinterpret_cast<uint2 *>(pr + ((rowb + col0) ^ sw)) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2 *>(pr + ((rowb + RT + col0) ^ sw)) = make_uint2(lo[0], lo[1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < CW / 16; ++i) {
                            *reinterpret_cast<uint4 *>(pr + ((rowb + col0 + 16 * i) ^ sw)) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                            *reinterpret_cast<uint4 *>(pr + ((rowb + RT + col0 + 16 * i) ^ sw)) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < CW / 8; ++i)
                        *reinterpret_cast<uint4 *>(pr + ((rowb + 2 * (col0 + 8 * i)) ^ sw)) =
                            make_uint4(bf16x2_bits(x[8 * i], x[8 * i + 1]), bf16x2_bits(x[8 * i + 2], x[8 * i + 3]),
                                       bf16x2_bits(x[8 * i + 4], x[8 * i + 5]), bf16x2_bits(x[8 * i + 6], x[8 * i + 7]));
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[it & 1]);

                const bool last = t + 1 == t1;
                if (!last && (t + 1 - t0) % kTaFlush != 0) continue;
                // ---- the sums leave tensor memory
                ta_wait(&pv_done[it & 1], (unsigned)((it >> 1) & 1), c.status, kWaitRingFull, abort_flag);
                tc_fence_after();
                const float ls = warp_columns<CW>(l, [](float p, float q) { return p + q; });
                if (lane < CW) wred[(warp & 3) * 32 + lane] = ls;
                bar_n<128>(1 + wg);
#pragma unroll
                for (int i = 0; i < CW; i += 8) {
                    float f0[8], f1[8];  // factors of these sums and of those flushed before
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = col0 + i + k;
                        float sum = (wred[i + k] + wred[32 + i + k]) + (wred[64 + i + k] + wred[96 + i + k]);
                        float top_r = m[i + k];
                        f0[k] = 1.0f, f1[k] = 0.0f;
                        if (flushed) {
                            const float2 o = a.ml[(int64_t)slot * RT + r];
                            top_r = fmaxf(o.x, top_r);
                            f0[k] = ex2(m[i + k] - top_r);
                            f1[k] = ex2(o.x - top_r);
                            sum = sum * f0[k] + o.y * f1[k];
                        }
                        if (last && whole) {
                            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                            f0[k] *= inv, f1[k] *= inv;
                        }
                        m[i + k] = top_r;
                        l[i + k] = sum;
                    }
#pragma unroll
                    for (int mt = 0; mt < Z::MT; ++mt) {
                        const int d = mt * 128 + tk;
                        const uint32_t ad = tmem + lanes + 2 * N + mt * N + col0 + i;
                        float o[8];
                        tmem_cols<8>(ad, o);
                        if (kE4M3) {
                            float lo[8];
                            tmem_cols<8>(ad + RT, lo);
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = fmaf(lo[k], 0.03125f, o[k]);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = col0 + i + k;
                            if (r >= rows || d >= c.dim) continue;
                            float *pd = a.part + ((int64_t)slot * RT + r) * DP + d;
                            float v = o[k] * f0[k];
                            if (flushed) v = fmaf(*pd, f1[k], v);
                            if (last && whole) {
                                const int g = row0 + r, tokn = g / a.group;
                                a.out[(((int64_t)w.b * c.n + tokn) * a.q_heads + hk * a.group + g % a.group) * c.dim + d] =
                                    __float2bfloat16_rn(tokn < w.cnt ? v : 0.0f);
                            } else {
                                *pd = v;
                            }
                        }
                    }
                }
                bar_n<128>(1 + wg);  // every thread has read ml and wred
                if (!(last && whole) && tk == 0) {
#pragma unroll
                    for (int i = 0; i < CW; ++i) a.ml[(int64_t)slot * RT + col0 + i] = make_float2(m[i], l[i]);
                }
                tc_fence_before();
                bar_n<128>(1 + wg);
                flushed = true;
#pragma unroll
                for (int i = 0; i < CW; ++i) m[i] = kTaNone, l[i] = 0.0f;
            }
            if (threadIdx.x == 0 && t0 == 0 && !whole) {
                // unit ends at tile index e of all: CTA ceil(e * ctas / total) - 1 has its last tile
                const int64_t e = w.start + w.ntiles;
                a.desc[blockIdx.x] = make_int4(w.b, w.u, (int)((e * w.ctas + w.total - 1) / w.total) - 1, 0);
            }
            ta_next(w, c, units);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Z::COLS));
}

// Joins the partial sums of the unit that CTA blockIdx.x began and others
// finished; one block per row of it, contributors in CTA order.
template <int DP, int RT>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TaArgs a)
{
    constexpr int L = DP / 4, G = 256 / L;  // 16-byte lanes of a row; groups that share the contributors
    __shared__ float wgt[kTaMaxCtas + 1], redm[8], reds[8];
    __shared__ float4 acc[G][L];
    pdl_wait();
    const int4 u = a.desc[blockIdx.x];
    if (u.x < 0) return;
    const CacheArgs &c = a.c;
    const int r = blockIdx.y, hk = u.y / a.rtiles, g = (u.y - hk * a.rtiles) * RT + r;
    if (g >= c.n * a.group) return;
    const int n = u.z - (int)blockIdx.x + 1, t = threadIdx.x;  // contributors
    auto slot = [&](int k) -> int64_t { return (int64_t)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * RT + r; };
    float2 ml = make_float2(kTaNone, 0.0f);
    if (t < n) ml = a.ml[slot(t)];
    float m = ml.x;
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (t % 32 == 0) redm[t / 32] = m;
    __syncthreads();
    for (int i = 0; i < 8; ++i) m = fmaxf(m, redm[i]);
    const float f = t < n ? ex2(ml.x - m) : 0.0f;
    if (t < n) wgt[t] = f;
    float s = ml.y * f;
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (t % 32 == 0) reds[t / 32] = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < 8; ++i) s += reds[i];
    const int lane = t % L, grp = t / L;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (lane * 4 < c.dim) {
#pragma unroll 8
        for (int k = grp; k < n; k += G) {
            const float4 v = *reinterpret_cast<const float4 *>(a.part + slot(k) * DP + lane * 4);
            const float h = wgt[k];
            o.x = fmaf(v.x, h, o.x), o.y = fmaf(v.y, h, o.y), o.z = fmaf(v.z, h, o.z), o.w = fmaf(v.w, h, o.w);
        }
    }
    acc[grp][lane] = o;
    __syncthreads();
    if (grp != 0 || lane * 4 >= c.dim) return;
    for (int i = 1; i < G; ++i) {
        const float4 v = acc[i][lane];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    const int i = g / a.group;
    const float inv = i < seq_count(c, u.x) && s != 0.0f ? 1.0f / s : 0.0f;
    uint2 two = make_uint2(bf16x2_bits(o.x * inv, o.y * inv), bf16x2_bits(o.z * inv, o.w * inv));
    if (i >= seq_count(c, u.x)) two = make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(a.out + (((int64_t)u.x * c.n + i) * a.q_heads + hk * a.group + g % a.group) * c.dim + lane * 4) = two;
}

// -------------------------------------------------------------------- host --
// Row tile: the smallest of 16, 32, 64 that holds the rows of a kv head.  The
// loads of a tile cost the same for any of them, and a smaller one has fewer
// columns to turn into weights.
static int ta_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

static size_t ta_part_bytes(int RT, int DP) { return (size_t)2 * kTaMaxCtas * RT * DP * sizeof(float); }
static size_t ta_ml_bytes(int RT) { return (size_t)2 * kTaMaxCtas * RT * sizeof(float2); }

size_t tree_attention_workspace_bytes(int64_t, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim)
{
    const int RT = ta_rows(n * (q_heads / kv_heads)), DP = dim <= 128 ? 128 : 256;
    return (ta_part_bytes(RT, DP) + ta_ml_bytes(RT) + kTaMaxCtas * sizeof(int4) + 255) / 256 * 256;
}

template <bool kE4M3, int DP, int RT>
static cudaError_t ta_launch(const TaArgs &a, int ctas, cudaStream_t st)
{
    using Z = TaShape<kE4M3, DP, RT>;
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<kE4M3, DP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (e != cudaSuccess) return e;
    tree_attention_kernel<kE4M3, DP, RT><<<ctas, kTaThreads, Z::SMEM, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || ctas == 1) return e;
    // the join may become resident early; it waits for the whole first kernel
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int rows = a.c.n * a.group;
    cfg.gridDim = dim3(ctas - 1, rows < RT ? rows : RT);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<DP, RT>, a);
}

wl_status launch_tree_attention(const bf16 *q, int64_t q_heads, const uint64_t *mask, float scale, const wl_cache &cache,
                                const wl_seqs &seqs, bf16 *out, void *ws, const DeviceInfo *di, cudaStream_t st)
{
    const int group = (int)(q_heads / cache.kv_heads), DP = cache.dim <= 128 ? 128 : 256;
    const int64_t rows = seqs.n * group;
    const int RT = ta_rows(rows);
    TaArgs a;
    a.q = q, a.mask = mask, a.out = out;
    a.part = static_cast<float *>(ws);
    a.ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + ta_part_bytes(RT, DP));
    a.desc = reinterpret_cast<int4 *>(reinterpret_cast<char *>(a.ml) + ta_ml_bytes(RT));
    a.q_heads = (int)q_heads, a.group = group, a.rtiles = (int)((rows + RT - 1) / RT);
    a.scale = scale;
    a.c = cache_args(cache, seqs, di->status);
    // at most one CTA per tile that the table can hold
    const int64_t tiles = seqs.batch * cache.kv_heads * a.rtiles * ((seqs.max_pages * cache.page_size + seqs.n + kTaTile - 1) / kTaTile);
    int ctas = di->sm_count < kTaMaxCtas ? di->sm_count : kTaMaxCtas;
    if (tiles < ctas) ctas = (int)tiles;
    cudaError_t e;
    if (cache.format == WL_CACHE_E4M3) {
        if (DP == 128)
            e = RT == 16 ? ta_launch<true, 128, 16>(a, ctas, st) : RT == 32 ? ta_launch<true, 128, 32>(a, ctas, st) : ta_launch<true, 128, 64>(a, ctas, st);
        else
            e = RT == 16 ? ta_launch<true, 256, 16>(a, ctas, st) : RT == 32 ? ta_launch<true, 256, 32>(a, ctas, st) : ta_launch<true, 256, 64>(a, ctas, st);
    } else {
        if (DP == 128)
            e = RT == 16 ? ta_launch<false, 128, 16>(a, ctas, st) : RT == 32 ? ta_launch<false, 128, 32>(a, ctas, st) : ta_launch<false, 128, 64>(a, ctas, st);
        else
            e = RT == 16 ? ta_launch<false, 256, 16>(a, ctas, st) : RT == 32 ? ta_launch<false, 256, 32>(a, ctas, st) : ta_launch<false, 256, 64>(a, ctas, st);
    }
    return e == cudaSuccess ? WL_OK : cuda_fail(e, "wl_tree_attention launch");
}

}  // namespace wl
