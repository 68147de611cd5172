// q8_plan.cu -- the bookkeeping of a step on the device: from each sequence's tokens in the cache
// and new tokens, the pages that it takes from the free list, and every new token's row, position
// and slot.
//
// One launch.  Sequences are taken kThreads at a time: a scan over the CTA gives their first rows,
// a second one the pages before them; then each token finds its sequence by bisection of the first
// rows, and its page from the table (a page that the sequence had) or from the free list (a new
// one, whose rank among all new pages is known, so nothing waits for the table's update).  Bound by
// latency: 12 bytes written a token (on the device, after a flush of L2: 48 sequences of a token each 6 to 9 us; 300 of
// up to 400 tokens, 57,000 rows, 19, and 21 with one row of a thread at a time).  One CTA serves up to kFewTokens rows; more are spread over a
// cluster, whose CTAs scan alike and share the rows; its barrier also keeps apart the reading of
// the lengths and of the free count from their update in place.
#include "q8_dev.cuh"
#include "q8_internal.h"

namespace q8 {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int64_t kFewTokens = 4096;
constexpr int kBatch = 4;  // rows that a thread has under way

struct PlanParams {
    int32_t *table;
    const int32_t *lens, *fresh, *free_pages, *free_count;
    int32_t *starts, *positions, *lens_out, *free_left;
    int64_t *slots;
    uint32_t *status;
    int64_t T;
    int32_t batch, table_width, page_shift, pages, free_capacity;
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum of v over the threads before this one; `total` over all of them.
__device__ __forceinline__ int64_t scan_before(int64_t v, int64_t *s_part, int64_t &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t run = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += w;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = run;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_part[w];
        total += s_part[w];
    }
    return before + run - v;
}

template <int kCtas>
__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ int64_t s_part[kWarps];
    __shared__ int32_t s_start[kThreads], s_old[kThreads];  // of the sequences in hand: first row, tokens before
    __shared__ int64_t s_taken[kThreads];                   // new pages before theirs, less the entries they had
    const int tid = threadIdx.x;
    const uint32_t rank = kCtas > 1 ? cluster_ctarank() : 0u;
    const int page = 1 << p.page_shift;
    const int64_t room = static_cast<int64_t>(p.table_width) << p.page_shift;
    uint32_t flags = 0u;
    int64_t count = 0;
    if (p.free_pages) {
        const int32_t n = *p.free_count;
        count = min(max(n, 0), p.free_capacity);
        if (count != n) flags |= Q8_DEV_BAD_INDEX;
    }
    int64_t rows = 0, taken = 0;  // of the sequences before those in hand
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + tid;
        int64_t old = 0, want = 0;
        if (b < p.batch) {
            const int32_t l = p.lens[b], n = p.fresh[b];
            old = min(max(static_cast<int64_t>(l), int64_t{0}), room);
            want = min(max(static_cast<int64_t>(n), int64_t{0}), room - old);
            if (old != l || want != n) flags |= Q8_DEV_BAD_INDEX;
        }
        int64_t total;
        const int64_t before = rows + scan_before(want, s_part, total);
        const int64_t start = min(before, p.T), news = min(before + want, p.T) - start;
        if (news != want) flags |= Q8_DEV_BAD_INDEX;  // more rows than the call has
        rows += total;
        const int64_t had = (old + page - 1) >> p.page_shift;
        const int64_t need = p.free_pages ? ((old + news + page - 1) >> p.page_shift) - had : 0;
        const int64_t pages_before = taken + scan_before(need, s_part, total);
        taken += total;
        s_start[tid] = static_cast<int32_t>(b < p.batch ? start : p.T);
        s_old[tid] = static_cast<int32_t>(old);
        s_taken[tid] = pages_before - had;
        if (kCtas > 1) cluster_sync();  // every CTA has read these sequences' lengths
        __syncthreads();
        if (rank == 0 && b < p.batch) {
            p.lens_out[b] = static_cast<int32_t>(old + news);
            p.starts[b] = static_cast<int32_t>(start);
        }
        // their rows
        const int64_t first = s_start[0], last = min(rows, p.T);
        const int held = min(kThreads, p.batch - b0);
        // (kBatch rows of a thread at a time, so that their loads of pages are under way together)
        constexpr int64_t kRows = kCtas * kThreads;
        for (int64_t tb = first + rank * kThreads + tid; tb < last; tb += kBatch * kRows) {
            int32_t pos[kBatch], pg[kBatch], *at[kBatch];
            bool taken_now[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t t = tb + i * kRows;
                if (t >= last) break;
                int lo = 0, hi = held;  // the last sequence that begins at or before t
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_start[mid] <= t) lo = mid;
                    else hi = mid;
                }
                pos[i] = s_old[lo] + static_cast<int32_t>(t - s_start[lo]);
                const int32_t entry = pos[i] >> p.page_shift;
                const int32_t seq_had = (s_old[lo] + page - 1) >> p.page_shift;
                at[i] = p.table + static_cast<int64_t>(b0 + lo) * p.table_width + entry;
                taken_now[i] = entry >= seq_had && p.free_pages;
                const int64_t k = s_taken[lo] + entry;  // rank among the new pages
                if (!taken_now[i]) pg[i] = *at[i];
                else if (k < count) pg[i] = p.free_pages[count - 1 - k];
                else flags |= Q8_DEV_NO_PAGE, pg[i] = INT32_MIN;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t t = tb + i * kRows;
                if (t >= last) break;
                if (static_cast<uint32_t>(pg[i]) >= static_cast<uint32_t>(p.pages)) {
                    if (pg[i] != INT32_MIN || !taken_now[i]) flags |= Q8_DEV_BAD_INDEX;
                    pg[i] = -1;
                }
                const int32_t off = pos[i] & (page - 1);
                if (taken_now[i] && off == 0) *at[i] = pg[i];
                p.slots[t] = pg[i] < 0 ? -1 : (static_cast<int64_t>(pg[i]) << p.page_shift) + off;
                p.positions[t] = pos[i];
            }
        }
        __syncthreads();  // the sequences in hand give way to the next
    }
    rows = min(rows, p.T);
    for (int64_t t = rows + rank * kThreads + tid; t < p.T; t += kCtas * kThreads) {
        p.slots[t] = -1;
        p.positions[t] = 0;
    }
    if (kCtas > 1) cluster_sync();  // every CTA has read the free count
    __syncthreads();
    if (rank == 0 && tid == 0) {
        p.starts[p.batch] = static_cast<int32_t>(rows);
        if (p.free_pages && p.free_left) *p.free_left = static_cast<int32_t>(max(count - taken, int64_t{0}));
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && (tid & 31) == 0 && p.status) atomicOr(p.status, flags);
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

}  // namespace

q8_status launch_plan(const PlanArgs &a, uint32_t *dev_status, cudaStream_t stream) {
    PlanParams p = {a.table, a.lens, a.new_tokens, a.free_pages, a.free_count, a.starts, a.positions, a.lens_out, a.free_left,
                    a.slots, dev_status, a.T, a.batch, a.table_width, ilog2(a.page_size), a.pages, a.free_capacity};
    if (a.T <= kFewTokens) {
        plan_kernel<1><<<1, kThreads, 0, stream>>>(p);
        return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_kernel<kCluster>, p) == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
