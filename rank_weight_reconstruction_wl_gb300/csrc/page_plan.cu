// page_plan.cu -- page tables grown and shrunk on the GPU from the sequences'
// lengths, with the slots of their new tokens.
//
//     need = ceil((len + count) / page_size);  back = max(0, held - need);  want = max(0, need - held)
//     k-th page given back -> stack place top + sum(back) - 1 - k;   up = top + sum(back)
//     sequence fits where the inclusive sum of want up to it <= up;  k-th page taken <- stack place up - 1 - k
//
// Both k run over all sequences in order, so the places are prefix sums and
// every page is moved by a thread of its own.  One cluster: a CTA owns a run of
// sequences, the CTAs exchange their totals, and cluster barriers stand between
// the pages given back and those taken.  Bound by latency: the barriers and
// chains of two or three dependent loads; what scales with the work (page
// moves, slots) is spread over all threads.
#include <cooperative_groups.h>

#include "cache_row.cuh"
#include "dec_ptx.cuh"

namespace cg = cooperative_groups;

namespace wl {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 16;

struct PlanDevice {
    PlanArgs a;
    FastDiv by_page, by_n;
    int per;  // sequences of a CTA
};

__device__ __forceinline__ int64_t plan_len(const PlanArgs &a, int b) { return max(__ldg(a.len + b), 0); }
__device__ __forceinline__ int plan_count(const PlanArgs &a, int b)
{
    return a.count ? min(max(__ldg(a.count + b), 0), a.n) : a.n;
}

// Exclusive prefix sum of v over the CTA (all threads); *total: the sum.
__device__ int plan_scan(int v, int *red, int *total)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) red[warp] = s;
    __syncthreads();
    int w = red[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += o;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return s - v + (warp > 0 ? before : 0);
}

// The sequence of move x: the last j < n with first[j] <= x.
__device__ __forceinline__ int plan_find(const int *first, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int64_t plan_slot(const PlanDevice &p, int b, int64_t len, int room, int i)
{
    if (i >= room) return -1;
    const int j = (int)(len + i);  // room: within the table, below 2^30
    const int page = p.by_page.div(j);
    return (int64_t)p.a.pages[(int64_t)b * p.a.max_pages + page] * p.a.page_size + (j - page * p.a.page_size);
}

// Dynamic shared memory: first page given back, first taken, need and held of each of the CTA's sequences.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanDevice p, int inline_slots)
{
    extern __shared__ int plan_smem[];
    __shared__ int red[32];
    __shared__ int sums[2][kPlanCtas];
    const PlanArgs &a = p.a;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int b0 = rank * p.per, nb = max(0, min(p.per, a.batch - b0));
    cluster_arrive();  // waited for before the first store into a peer: until then it may not have begun
    int *back0 = plan_smem, *want0 = back0 + p.per, *need = want0 + p.per, *have = need + p.per;
    pdl_wait();
    const int top = min(max(__ldg(a.top), 0), a.pool);
    int backs = 0, wants = 0;
    for (int i0 = 0; i0 < nb; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int bk = 0, wt = 0;
        if (i < nb) {
            const int64_t end = plan_len(a, b0 + i) + plan_count(a, b0 + i);
            const int nd = (int)min((end + a.page_size - 1) / a.page_size, (int64_t)a.max_pages);
            const int hv = min(max(a.held[b0 + i], 0), a.max_pages);
            need[i] = nd, have[i] = hv;
            bk = max(0, hv - nd), wt = max(0, nd - hv);
        }
        int tb, tw;
        const int sb = plan_scan(bk, red, &tb);
        const int sw = plan_scan(wt, red, &tw);
        if (i < nb) back0[i] = backs + sb, want0[i] = wants + sw;
        backs += tb, wants += tw;
    }
    cluster_wait();
    if (threadIdx.x < ctas) {
        int *peer = cl.map_shared_rank(&sums[0][0], threadIdx.x);
        peer[rank] = backs;
        peer[kPlanCtas + rank] = wants;
    }
    cl.sync();
    int back_base = 0, want_base = 0, all_back = 0;
    for (int r = 0; r < ctas; ++r) {
        if (r < rank) back_base += sums[0][r], want_base += sums[1][r];
        all_back += sums[0][r];
    }
    const int up = min(top + all_back, a.pool);
    // Four moves of a thread at a time, so that their loads overlap (one at a time: 512 prompts' pages and back 43 us).
    constexpr int U = 4;
    for (int x0 = threadIdx.x; x0 < backs; x0 += U * kPlanThreads) {
        int32_t *entry[U];
        int32_t page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * kPlanThreads, i = plan_find(back0, nb, min(x, backs - 1));
            entry[u] = x < backs ? a.pages + (int64_t)(b0 + i) * a.max_pages + need[i] + (x - back0[i]) : nullptr;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) page[u] = entry[u] ? *entry[u] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (entry[u]) {
                const int place = up - 1 - (back_base + x0 + u * kPlanThreads);
                if (place >= 0) a.free_pages[place] = page[u];
                *entry[u] = -1;
            }
    }
    cl.sync();
    const int fitting = min(wants, up - want_base);  // moves of sequences past the pool's end are not looked at
    for (int x0 = threadIdx.x; x0 < fitting; x0 += U * kPlanThreads) {
        int32_t *entry[U];
        int32_t page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * kPlanThreads, i = plan_find(want0, nb, min(x, fitting - 1));
            const bool fits = x < fitting && want_base + want0[i] + need[i] - have[i] <= up;
            entry[u] = fits ? a.pages + (int64_t)(b0 + i) * a.max_pages + have[i] + (x - want0[i]) : nullptr;
            page[u] = fits ? __ldcg(a.free_pages + up - 1 - (want_base + x)) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (entry[u]) *entry[u] = page[u];
    }
    __syncthreads();  // below, have[] becomes the room
    int taken = 0;  // of the whole call, up to this thread's last sequence that fits
    for (int i = threadIdx.x; i < nb; i += kPlanThreads) {
        const int upto = want_base + want0[i] + max(0, need[i] - have[i]);
        const bool fits = upto <= up;
        const int now = fits ? need[i] : min(have[i], need[i]);
        if (fits) taken = max(taken, upto);
        a.held[b0 + i] = now;
        const int64_t len = plan_len(a, b0 + i);
        const int room = (int)min(max((int64_t)now * a.page_size - len, (int64_t)0), (int64_t)plan_count(a, b0 + i));
        a.room[b0 + i] = room;
        have[i] = room;
    }
    // the last sequence that fits: all before it that fit took theirs
    for (int d = 16; d > 0; d >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, d));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kPlanThreads / 32; ++w) taken = max(taken, red[w]);
        *cl.map_shared_rank(&sums[0][rank], 0) = taken;
    }
    cl.sync();
    if (rank == 0 && threadIdx.x == 0) {
        for (int r = 1; r < ctas; ++r) taken = max(taken, sums[0][r]);
        *a.top = up - taken;
    }
    pdl_trigger();
    if (inline_slots) {
        for (int x = threadIdx.x; x < nb * a.n; x += kPlanThreads) {
            const int i = p.by_n.div(x);
            a.slots[(int64_t)b0 * a.n + x] = plan_slot(p, b0 + i, plan_len(a, b0 + i), have[i], x - i * a.n);
        }
    }
}

__global__ void __launch_bounds__(256) page_slots_kernel(const __grid_constant__ PlanDevice p)
{
    pdl_wait();
    pdl_trigger();
    // a sequence's slots by a run of blocks: the length, the room and a page are looked up once for the slots that share them
    const int b = (int)blockIdx.x;
    const int64_t len = plan_len(p.a, b);
    const int room = __ldg(p.a.room + b);
    int64_t *out = p.a.slots + (int64_t)b * p.a.n;
    for (int i = (int)blockIdx.y * 256 + threadIdx.x; i < p.a.n; i += (int)gridDim.y * 256) out[i] = plan_slot(p, b, len, room, i);
}

wl_status launch_page_plan(const PlanArgs &args, const DeviceInfo *di, cudaStream_t st)
{
    PlanDevice p{args, fast_div(args.page_size), fast_div(args.n > 0 ? args.n : 1), 0};
    // One CTA has no cluster barriers to wait for; many sequences move many pages (512 prompts and back: 30.7 us with 16, 41.6 with 8).
    const int ctas = args.batch > 256 ? kPlanCtas : args.batch > 64 ? 8 : 1;
    p.per = (args.batch + ctas - 1) / ctas;
    const size_t smem = (size_t)p.per * 4 * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 131072);
    if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_fail(e, "wl_page_plan attributes");
    const bool slots = args.slots && args.n > 0;
    const bool inl = slots && (int64_t)args.batch * args.n <= 8192 * ctas;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, page_plan_kernel, p, (int)inl);
    if (e != cudaSuccess) return cuda_fail(e, "wl_page_plan launch");
    if (slots && !inl) {
        int64_t blocks = (args.n + 255) / 256;
        while (blocks > 1 && (blocks > 65535 || blocks * args.batch > 16 * di->sm_count)) blocks = (blocks + 1) / 2;
        e = launch_dependent(page_slots_kernel, dim3((unsigned)args.batch, (unsigned)blocks), 256, 0, st, p);
        if (e != cudaSuccess) return cuda_fail(e, "wl_page_plan slots launch");
    }
    return WL_OK;
}

}  // namespace wl
