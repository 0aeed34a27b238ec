// Pages, positions and slots of a step, built on the device from the
// sequences' lengths.
//
// Paged caches keep a sequence's tokens in fixed-size pages named by a table
// ("语言模型能自己决定该看哪里吗？", DA state machine section: vLLM's KV
// blocks).  For sequence b holding n_b tokens that gets a_b more (a_b = -1:
// it has ended):
//   held_b = ceil(n_b / P),  need_b = ceil((n_b + a_b) / P) - held_b
// The pages of ended sequences go onto a stack of free pages in (sequence,
// page) order, then the i-th page needed, counted in the same order, is the
// i-th from the top.  (A number that names no page is no page of the sequence:
// it stays off the stack, and the pages above it move down.)  Token i of the step belongs to the sequence b with
// cu_b <= i < cu_{b+1} (cu: prefix sums of a), has position n_b + i - cu_b and
// goes to slot page * P + position % P.
//
// One cluster: every CTA computes the prefix sums of all sequences for itself
// (a few KB of lengths), they push the freed pages, meet at one cluster
// barrier -- behind which the inputs may be overwritten, so lengths and the
// free count can be updated in place -- and then share the writing of tables
// and tokens.  Bound by latency: the dependent trips lengths -> scan -> stack
// -> table, about 16 bytes per token beside them.  Measured: 32 sequences of one
// token 4.4 us (one CTA), 256 sequences with up to 131072 tokens 10.3 us (0.5 us of
// it for the barrier behind which CTAs may tell each other of a number that is no
// page).
#include <cooperative_groups.h>

#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRows = 4;   // rows of 32 pages or tokens that a warp has in flight
constexpr int kPlanItems = kPlanMaxBatch / kPlanThreads;   // sequences per thread

struct Sums {
    long long tok, need, back;
};

__device__ __forceinline__ Sums plus(const Sums &x, const Sums &y)
{
    return {x.tok + y.tok, x.need + y.need, x.back + y.back};
}

// exclusive prefix over the block; `total` receives the block's sum
__device__ __forceinline__ Sums block_scan(Sums v, Sums *warp_sum, Sums &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums y = {__shfl_up_sync(~0u, inc.tok, o), __shfl_up_sync(~0u, inc.need, o),
                        __shfl_up_sync(~0u, inc.back, o)};
        if (lane >= o) inc = plus(inc, y);
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        Sums w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y = {__shfl_up_sync(~0u, w.tok, o), __shfl_up_sync(~0u, w.need, o),
                            __shfl_up_sync(~0u, w.back, o)};
            if (lane >= o) w = plus(w, y);
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    total = warp_sum[31];
    Sums r = {inc.tok - v.tok, inc.need - v.need, inc.back - v.back};
    if (warp > 0) r = plus(r, warp_sum[warp - 1]);
    return r;
}

// ONE: the cluster is this CTA alone, and its barrier the CTA's
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads) k_plan_append(const PlanArgs a)
{
    pdl_wait();
    pdl_trigger();
    namespace cg = cooperative_groups;
    extern __shared__ int plan_sm[];
    __shared__ Sums warp_sum[32];
    __shared__ int s_none, s_kept;   // whether a CTA was to push what is no page; how many pages the stack got
    const int B = a.B, P = 1 << a.Plog2, tid = threadIdx.x;
    int *s_old = plan_sm;            // [B] tokens held
    int *s_new = s_old + B;          // [B] tokens to come, -1 = ended
    int *s_need = s_new + B;         // [B] fresh pages of earlier sequences (of an ended one: freed pages)
    int *s_cu = s_need + B;          // [B + 1]
    const int rank = ONE ? 0 : (int)cg::this_cluster().block_rank(), ranks = ONE ? 1 : (int)cg::this_cluster().num_blocks();
    auto meet = [] {
        if (ONE) __syncthreads();
        else cg::this_cluster().sync();
    };
    auto tell = [&](int *mine, int value) {   // every CTA's copy of a shared variable, by one warp
        if (ONE) *mine = value;
        else if ((tid & 31) < ranks) *cg::this_cluster().map_shared_rank(mine, tid & 31) = value;
    };
    const long long Lcap = (long long)a.max_pages << a.Plog2;
    if (tid == 0) s_none = 0;
    if (!ONE) asm volatile("barrier.cluster.arrive;" ::: "memory");   // s_none may be written by the others

    // ---- lengths, and what they ask for
    Sums mine = {0, 0, 0};
    Sums part[kPlanItems];
    int bad = 0;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
        const int b = tid * kPlanItems + u;
        part[u] = mine;
        if (b >= B) continue;
        int old = a.sl[b], add = a.add[b];
        if (old < 0 || old > Lcap || add < -1 || (long long)old + add > Lcap) {
            if (rank == 0) fault(a.st, CHK_SEQ_LEN, old < 0 || old > Lcap ? old : add);
            bad = 1;
        }
        const long long held = ((long long)old + P - 1) >> a.Plog2;
        const long long then = ((long long)old + add + P - 1) >> a.Plog2;
        if (add < 0) mine.back += held;
        else mine.tok += add, mine.need += then - held;
        s_old[b] = old;
        s_new[b] = add;
    }
    bad = __syncthreads_or(bad);
    Sums all;
    const Sums before = block_scan(mine, warp_sum, all);
    const int count = *a.count;
    if (count < 0 || count > a.num_free) {
        if (rank == 0 && tid == 0) fault(a.st, CHK_COUNT, count);
        bad = 1;
    }
    if (!bad) {
        int chk = 0;
        long long what = 0;
        if (all.tok > a.max_tokens) chk = CHK_CAPACITY_TOKENS, what = all.tok;
        else if (count + all.back > a.num_free) chk = CHK_CAPACITY_PAGES, what = count + all.back;
        else if (all.need > count + all.back) chk = CHK_CAPACITY_PAGES, what = all.need;
        if (chk) {
            if (rank == 0 && tid == 0)
                record(a.st, SA_ERR_CAPACITY, chk, (int)(what > 0x7fffffff ? 0x7fffffff : what));
            bad = 1;
        }
    }
    // a step that cannot be taken changes nothing
    if (bad) all = {0, 0, 0};
    int top = count + (int)all.back;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
        const int b = tid * kPlanItems + u;
        if (b >= B) continue;
        const Sums x = plus(before, part[u]);
        s_cu[b] = bad ? 0 : (int)x.tok;
        s_need[b] = (int)(s_new[b] < 0 ? x.back : x.need);
    }
    if (tid == 0) s_cu[B] = (int)all.tok;
    __syncthreads();
    const int gtid = rank * kPlanThreads + tid, threads = ranks * kPlanThreads, lane = tid & 31;
    bool none = false;   // one that is no page
    if (!bad && all.back > 0) {
        // pages of ended sequences onto the stack, a warp a sequence
        for (int b = gtid >> 5; b < B; b += threads >> 5) {
            if (s_new[b] >= 0) continue;
            const int held = (s_old[b] + P - 1) >> a.Plog2;
            for (int p = lane; p < held; p += 32 * kRows) {
                int page[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    page[u] = p + 32 * u < held ? a.table[(size_t)b * a.max_pages + p + 32 * u] : 0;
#pragma unroll
                for (int u = 0; u < kRows; ++u) {
                    if (p + 32 * u >= held) break;
                    if (page[u] < 0 || page[u] >= a.num_pages) {
                        fault(a.st, CHK_PAGE, page[u]);
                        none = true;
                    }
                    a.free[count + s_need[b] + p + 32 * u] = page[u];
                }
            }
        }
    }
    if (!ONE) asm volatile("barrier.cluster.wait;" ::: "memory");
    if (__any_sync(~0u, none)) tell(&s_none, 1);
    meet();   // every CTA has read the inputs; the stack is whole
    if (__builtin_expect(s_none != 0, 0)) {   // (set in all CTAs or in none)
        if (gtid < 32) {
            int kept = 0;
            for (int i = lane; i - lane < (int)all.back; i += 32) {
                const int page = i < (int)all.back ? a.free[count + i] : -1;
                const bool fine = page >= 0 && page < a.num_pages;
                const unsigned m = __ballot_sync(~0u, fine);   // (and every lane has read its number)
                if (fine) a.free[count + kept + __popc(m & ((1u << lane) - 1))] = page;
                kept += __popc(m);
                __syncwarp();
            }
            tell(&s_kept, kept);
        }
        meet();
        top = count + s_kept;
        if (all.need > top) {   // not enough without them (and recorded already)
            bad = 1;
            all = {0, 0, 0};
            for (int b = tid; b <= B; b += kPlanThreads) s_cu[b] = 0;
            __syncthreads();
        }
    }

    // ---- lengths, prefix sums, fresh table entries
    for (int b = gtid; b < B; b += threads) {
        const int add = s_new[b];
        a.sl_out[b] = bad ? s_old[b] : add < 0 ? 0 : s_old[b] + add;
        a.cu[b] = s_cu[b];
    }
    if (gtid == 0) {
        a.cu[B] = (int)all.tok;
        *a.count_out = bad ? count : top - (int)all.need;
    }
    if (!bad) {
        for (int b = gtid >> 5; b < B; b += threads >> 5) {
            const int old = s_old[b], add = s_new[b];
            if (add <= 0) continue;
            const int held = (old + P - 1) >> a.Plog2, then = (old + add + P - 1) >> a.Plog2;
            const int *from = a.free + top - 1 - s_need[b] + held;
            for (int p = held + lane; p < then; p += 32 * kRows) {
                int page[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u) page[u] = p + 32 * u < then ? from[-(p + 32 * u)] : 0;
#pragma unroll
                for (int u = 0; u < kRows; ++u) {
                    if (p + 32 * u >= then) break;
                    if (page[u] < 0 || page[u] >= a.num_pages) {
                        fault(a.st, CHK_PAGE, page[u]);
                        page[u] = -1;
                    }
                    a.table[(size_t)b * a.max_pages + p + 32 * u] = page[u];
                }
            }
        }
    }
    // ---- tokens: a run of them per warp, so that the sequence is searched for
    // once, kRows rows at a time, so that the page lookups overlap
    const int total = (int)all.tok, warps = threads >> 5;
    const int run = (a.max_tokens + warps * 32 - 1) / (warps * 32) * 32;
    const int end = (int)min((long long)a.max_tokens, (long long)run * ((gtid >> 5) + 1));
    int seq = 0;
    {
        int lo = 0, hi = B - 1;   // the last b with cu_b <= i holds i (empty ones before it have the same cu)
        const int i = run * (gtid >> 5) + lane;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_cu[mid] <= i) lo = mid; else hi = mid - 1;
        }
        seq = lo;
    }
    for (int i0 = run * (gtid >> 5) + lane; i0 < end; i0 += 32 * kRows) {
        int pos[kRows], of[kRows], page[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = i0 + 32 * u;
            pos[u] = 0;
            of[u] = -1;
            page[u] = -1;
            if (i >= total || i >= end) continue;
            while (s_cu[seq + 1] <= i) ++seq;
            of[u] = seq;
            pos[u] = s_old[seq] + i - s_cu[seq];
            const int held = (s_old[seq] + P - 1) >> a.Plog2, p = pos[u] >> a.Plog2;
            page[u] = p < held ? a.table[(size_t)seq * a.max_pages + p] : a.free[top - 1 - (s_need[seq] + p - held)];
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = i0 + 32 * u;
            if (i >= end) break;
            long long slot = -1;
            if (of[u] >= 0) {
                if (page[u] < 0 || page[u] >= a.num_pages) fault(a.st, CHK_PAGE, page[u]);
                else slot = ((long long)page[u] << a.Plog2) + (pos[u] & (P - 1));
            }
            a.pos[i] = pos[u];
            a.slots[i] = slot;
            if (a.seq_ids) a.seq_ids[i] = of[u];
        }
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t s)
{
    // a step's few tokens need one CTA (4.4 us for 32); 131072 take 10.3 us with
    // 16 CTAs and 13.7 with 8
    const int ctas = a.max_tokens > 32 * kPlanThreads ? 16 : a.max_tokens > 4 * kPlanThreads || a.B > kPlanThreads ? 8 : 1;
    auto kern = ctas == 1 ? k_plan_append<true> : k_plan_append<false>;
    const size_t smem = (size_t)(4 * a.B + 1) * sizeof(int);
    if (smem > 40960) {   // (static shared memory comes on top, up to 48 KB together without asking)
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (4 * kPlanMaxBatch + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    if (ctas == 1) return launch_pdl(kern, dim3(1), dim3(kPlanThreads), smem, s, a);
    if (ctas > 8) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace sa
