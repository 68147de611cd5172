// q8_sample.cu -- draw the next token of each row of logits: temperature,
// top-k, top-p and min-p from a given uniform number, in one launch.
//
// Definition.  With m the row's largest logit, e_i = exp((l_i - m) / T) in
// binary32 (1 where l_i = m) and w_i = floor(e_i 2^40) a whole number: sums of
// w are exact in 64 bits, so they do not depend on the order of adding and
// every comparison below is decided the same way by any split of the work.
// Words are ranked by (logit descending, index ascending).  top-k keeps the
// first k; top-p, of those, the ones before which less than ceil(p * sum) lies;
// min-p, of those, the ones with e_i >= min_p.  With W the sum of what is left
// and r = floor(u W), the token is the first word in index order whose running
// sum passes r.  Words with w_i = 0 (below 2^-40 of the likeliest) cannot be
// drawn and are not counted.
//
// The row is not sorted: the words kept are a prefix of the ranking, and what
// is needed is where it ends.
//  - few words: the row is cut into 128 groups.  At least k words are no smaller than
//    the k-th largest group maximum, and few more are (top-k up to 96).  For more
//    words the rank among the maxima is where 1.5 k words (1400 for top-p alone) are
//    expected: with f of the groups above the bound, -log(1 - f) words a group.  From
//    256 words on the maxima are of every 4th word, which keeps f away from 1: the
//    number of words found then strays by an eighth or less.  The maxima come with
//    the row's largest logit, so one pass gathers the words above that bound and one
//    CTA sorts them and draws.  Whether they are enough is known exactly (top-k: their
//    number; top-p: their mass against that of the whole row, summed before they are
//    gathered, when every word's e takes its logit's place); where not, the searches
//    below follow.
//  - larger top-k: a histogram of counts over 2048 equal steps of the distance
//    from the largest logit (down to exp(-28) or the row's smallest logit) finds
//    the step that holds the k-th word.
//  - top-p without a small top-k: every word's e replaces its logit in shared
//    memory (if it has not yet) and the masses are summed.  Words below (1 - p) / V of that sum lie
//    past the end together, so only the others enter a histogram of masses by
//    e's leading bits, which finds the bin that holds the end.
// If the words up to the end of that step or bin are at most 2048, they are
// gathered and drawn from by one CTA.  Otherwise the words of that step alone are
// gathered and sorted to find the last one kept (their logits read again, since
// different logits may have equal e), and the draw is a pass over the row in
// index order.  A step that holds more than 2048 words (many equal logits) is
// searched digit by digit in the logits' 32-bit order keys.  Equal logits at the
// end of the prefix are kept in index order.
//
// A row belongs to a cluster of up to 16 CTAs; each keeps its slice of the row
// in shared memory, so the logits are read from memory once.  Bound: by
// latency for few rows (passes over shared memory with cluster barriers, about
// 1000 cycles each, between them), by the passes' instructions for many.
// Measured: one row of 262,144 words 12 us with top-k 50, 16 without a filter, 43
// with top-p 0.95 alone (13,823 words kept); 64 rows of 131,071 words 30, 45 and 113 us (9,032
// kept), 52 with mixed knobs.  A pass that weighs every word takes 70 instructions a word, the
// histogram of masses twice as many.
#include <cooperative_groups.h>

#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "q8_dev.cuh"
#include "q8_internal.h"

namespace cg = cooperative_groups;

namespace q8 {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;        // words one CTA sorts
constexpr int kPer = kList / kThreads;
constexpr int kMaxCluster = 16;
constexpr int kGroups = 128;       // of a row, for a bound on its k-th logit
// Top-k whose bound is the k-th largest group maximum: up to 3/4 of the groups, above which 1.4 k words
// are expected, as many as the rule for more words asks for.  With limits of 32, 64, 96 and 112, k = 65 takes
// 11.6, 11.8, 10.9 and 11.0 us (one row of 32,000 words), 11.8, 11.8, 11.4 and 11.3 (131,071), k = 112 13.1 to 13.4
// everywhere.
constexpr int kFewK = kGroups * 3 / 4;
// Top-k that is looked for through the list at all: 1.5 k words are asked for, and an eighth more still
// fit.  From 1050 to 1150 words: 131,071 words, one row 17.2 to 17.6 us and 23.7 through the histogram, 64 rows
// 41 to 43 and 62.5; 262,144 words 19 and 27.8, 81 to 85 and 132; 64 rows of 32,000 words, where the list does
// not do for one or the other, 32.2 and 26.5.  At 1200 it does not for one row of 262,144 either: 32.5 and 27.8.
constexpr int kManyK = kList * 9 / 16;
constexpr int kListP = 1400;       // words asked for where only top-p counts
constexpr int kCopies = 4;         // bulk copies of a slice
constexpr float kUnit = 1.0f / 1099511627776.0f;  // 2^-40

struct SampleParams {
    const void *logits;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *token, *kept;
    float *logprob;
    uint32_t *status;
    int64_t ld;
    int32_t V, slice;
    int32_t rows;  // to be put in order of what they take; 0: as they come
};

struct alignas(16) Shared {
    union {
        struct {
            uint32_t mass_lo[kBins], mass_hi[kBins];
        };
        unsigned long long list[kList];  // (key, index), in CTA 0; not while a histogram is in use
    };
    uint32_t count[kBins];
    alignas(16) float groups[kGroups];         // of all CTAs, written by each
    unsigned long long sub_mass[kMaxCluster];  // per CTA, written by each
    uint32_t sub_count[kMaxCluster];
    float maxima[kMaxCluster], minima[kMaxCluster];
    unsigned long long sub_above[kMaxCluster];
    unsigned long long warp_mass[kWarps], warp_above[kWarps];
    uint32_t warp_count[kWarps];
    float warp_min[kWarps], warp_max[kWarps];
    float thread_groups[kGroups];              // this CTA's, of at most 32 threads
    float bound;
    uint32_t enough;
    // what a search found, in the CTA that found it
    uint32_t digit, before_count, in_count;
    unsigned long long before_mass, in_mass;
    uint32_t last, ties, ranked;
    uint32_t listed;  // words in the list of CTA 0
    uint64_t bars[kCopies];
};

// Ascending order of this key is descending order of the value (-0 = +0).
__device__ __forceinline__ uint32_t rank_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float unkey(uint32_t key) { return __uint_as_float((key & 0x80000000u) ? key : ~key & 0x7FFFFFFFu); }

// e of a row's words.  A pass is bound by its instructions and branches, so the quotient (l - top) / T
// is made without either's slow parts: both are multiplied by a power of two that brings T into
// [1, 2) (exact), and with y = 1 / T rounded to nearest two corrections q + (d - q T) y of q = d y give
// d / T rounded to nearest (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  Below -2^40 e is 0; where d is small enough for a step to underflow, e is 1.
// Every step is monotone, expf too (looked at for all neighbouring floats from 0 to -104), so e
// ranks words as their logits do but where it is equal.
struct Row {
    float top, divisor, scale, rcp;  // divisor: T over the power of two, in [1, 2) (T itself where rare)
    bool rare;  // T has no such power, or is infinite
    __device__ __forceinline__ Row(float l, float t) {
        const uint32_t bits = __float_as_uint(t), exponent = bits >> 23;
        rare = exponent < 1 || exponent > 253;
        top = l;
        divisor = rare ? t : __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
        scale = rare ? 1.0f : __uint_as_float((254 - exponent) << 23);
        rcp = __frcp_rn(divisor);
    }
    __device__ __noinline__ float slow(float l) const { return l == top ? 1.0f : (l == -INFINITY ? 0.0f : expf(__fdiv_rn(l - top, divisor))); }
    __device__ __forceinline__ float weight(float l) const {
        if (rare) return slow(l);
        const float d = fmaxf((l - top) * scale, -0x1p40f);
        float q = d * rcp;
        q = fmaf(fmaf(-q, divisor, d), rcp, q);
        q = fmaf(fmaf(-q, divisor, d), rcp, q);
        const float e = expf(q);
        return l == top ? 1.0f : e;
    }
};
// floor(e 2^40) for 0 <= e <= 1 from e's own bits: 64-bit conversions are slow here (the pass
// over 16384 words took 20,000 cycles with two of them a word)
__device__ __forceinline__ unsigned long long mass_of(float e) {
    const uint32_t b = __float_as_uint(e), m = (b & 0x7FFFFFu) | 0x800000u;
    return (static_cast<unsigned long long>(m) << 17) >> min(127 - static_cast<int>(b >> 23), 63);  // e = m 2^(exponent - 150)
}

// Exclusive running sums of m and c over the threads of the CTA, and the totals.
__device__ void scan_cta(Shared &s, unsigned long long m, uint32_t c, unsigned long long &m_before, uint32_t &c_before,
                         unsigned long long &m_all, uint32_t &c_all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned long long mr = m;
    uint32_t cr = c;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long mv = __shfl_up_sync(0xffffffffu, mr, o);
        const uint32_t cv = __shfl_up_sync(0xffffffffu, cr, o);
        if (lane >= o) mr += mv, cr += cv;
    }
    __syncthreads();
    if (lane == 31) s.warp_mass[warp] = mr, s.warp_count[warp] = cr;
    __syncthreads();
    m_all = 0, c_all = 0;
    unsigned long long mb = 0;
    uint32_t cb = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) mb = m_all, cb = c_all;
        m_all += s.warp_mass[w];
        c_all += s.warp_count[w];
    }
    m_before = mr - m + mb, c_before = cr - c + cb;
}

// Ascending sort of n <= kList different words of s.list into kBins buckets by bin(word), which
// does not fall from one word to a larger one; within a bucket by counting.  (A bitonic sort
// of 2048 took 20,000 cycles and more.)  s.count is used.
template <typename Bin>
__device__ void sort_buckets(Shared &s, int n, Bin bin) {
    const int tid = threadIdx.x;
    unsigned long long x[kPer];
    int b[kPer];
    uint32_t at[kPer];
    for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kThreads;
        x[j] = i < n ? s.list[i] : 0ull;
        b[j] = i < n ? bin(x[j]) : -1;
        at[j] = b[j] >= 0 ? atomicAdd(&s.count[b[j]], 1u) : 0u;
    }
    __syncthreads();
    // where each bucket begins
    uint32_t c[kBins / kThreads], sum = 0, before, all;
    unsigned long long mb, ma;
#pragma unroll
    for (int j = 0; j < kBins / kThreads; ++j) c[j] = s.count[tid * (kBins / kThreads) + j], sum += c[j];
    scan_cta(s, 0ull, sum, mb, before, ma, all);
#pragma unroll
    for (int j = 0; j < kBins / kThreads; ++j) {
        s.count[tid * (kBins / kThreads) + j] = before;
        before += c[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (b[j] >= 0) s.list[s.count[b[j]] + at[j]] = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (b[j] < 0) continue;
        const uint32_t i0 = s.count[b[j]], i1 = b[j] + 1 < kBins ? s.count[b[j] + 1] : static_cast<uint32_t>(n);
        at[j] = i0;
        for (uint32_t i = i0; i < i1; ++i) at[j] += s.list[i] < x[j] ? 1u : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (b[j] >= 0) s.list[at[j]] = x[j];
    __syncthreads();
}

// log(w / all): through 1 - (all - w) / all where the word has most of the mass
__device__ __forceinline__ float log_share(unsigned long long w, unsigned long long all) {
    return 2 * w > all ? log1pf(-__fdiv_rn(static_cast<float>(all - w), static_cast<float>(all)))
                       : logf(__fdiv_rn(static_cast<float>(w), static_cast<float>(all)));
}
// The mass that is passed by the token drawn with u.
__device__ __forceinline__ unsigned long long place_of(float u, unsigned long long all) {
    const double x = floor(static_cast<double>(u) * static_cast<double>(all));
    const unsigned long long r = x > 0.0 ? static_cast<unsigned long long>(x) : 0ull;
    return r > all - 1 ? all - 1 : r;
}
// The mass that top-p asks for.
__device__ __forceinline__ unsigned long long mass_wanted(float top_p, unsigned long long total) {
    const double cut = ceil(static_cast<double>(top_p) * static_cast<double>(total));
    return cut < 1.0 ? 1ull : static_cast<unsigned long long>(cut);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    float *const buf = reinterpret_cast<float *>(smem + sizeof(Shared));
    using Elem = typename std::conditional<BF16, uint16_t, float>::type;
    constexpr int kVec = 16 / sizeof(Elem);
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // before any CTA writes into another's shared memory, both run
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int row = blockIdx.x / ranks;
    if (p.rows > 0) {  // the row at this place of the order: those that a list of few words will not do for, then the others
        bool more = false;
        if (tid < p.rows) {
            const int k = p.top_k ? p.top_k[tid] : 0;
            more = (k <= 0 || k > kManyK) && !(p.temperature && !(p.temperature[tid] > 0.0f));
        }
        const uint32_t vote = __ballot_sync(0xffffffffu, more);
        if (lane == 0) s.warp_count[warp] = __popc(vote);
        __syncthreads();
        int before = __popc(vote & ((1u << lane) - 1)), all = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s.warp_count[w] : 0;
            all += s.warp_count[w];
        }
        if (tid < p.rows && (more ? before : all + tid - before) == row) s.digit = tid;
        __syncthreads();
        row = s.digit;
    }
    const Elem *const logits = static_cast<const Elem *>(p.logits) + row * p.ld;
    // Slices begin on 16-byte boundaries of the row (rows need not), and words keep
    // their place within 16 bytes (of the input's type) in shared memory.
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(Elem));
    const int first = min(max(rank * p.slice - skew, 0), p.V), n = min((rank + 1) * p.slice - skew, p.V) - first;
    const int pad = rank == 0 ? skew : 0;
    const Elem *const mine = logits + first;
    float *const vals = buf + pad;  // logits, NaN as -inf; later e

    auto widen = [](Elem v) -> float {
        if constexpr (BF16)
            return __uint_as_float(static_cast<uint32_t>(v) << 16);
        else
            return v;
    };
    // a word's logit from memory, for the few that need it again
    auto logit = [&](int i) -> float {
        const float v = widen(mine[i]);
        return v != v ? -INFINITY : v;
    };

    // ---- the row's knobs, and which words the bound is made from ----------------------------
    float temp = p.temperature ? p.temperature[row] : 1.0f;
    int k = p.top_k ? p.top_k[row] : 0;
    float top_p = p.top_p ? p.top_p[row] : 1.0f;
    if (!(top_p < 1.0f)) top_p = 1.0f;  // all words
    const float min_p = p.min_p ? p.min_p[row] : 0.0f;
    const float u = p.u[row];
    if (!(temp > 0.0f)) temp = 1.0f, k = 1;
    if (k <= 0 || k > p.V) k = p.V;
    // words to gather; 0: no list
    const int list = k <= kFewK ? k : (k <= kManyK ? k + k / 2 : (k == p.V && top_p < 1.0f ? kListP : 0));
    const int every = list <= 2 * kGroups ? 1 : 4;

    // ---- the slice; the row's largest and smallest logits -----------------------------
    float top = -INFINITY, low = INFINITY, some = -INFINITY;  // some: of every 4th word
    bool nan = false;
    auto look = [&](float v) -> float {
        const bool bad = v != v;
        nan = nan || bad;
        v = bad ? -INFINITY : v;
        top = fmaxf(top, v);
        low = fminf(low, v == -INFINITY ? INFINITY : v);
        return v;
    };
    const int head = min((kVec - pad) % kVec, n), body = (n - head) / kVec;  // words, then runs of 16 bytes
    if (tid < 2 * kVec) {  // words before and after the whole runs
        const int i = tid < kVec ? tid : head + body * kVec + tid - kVec;
        if (tid < kVec ? i < head : i < n) vals[i] = look(widen(mine[i]));
    }
    if constexpr (BF16) {
        const uint4 *const src = reinterpret_cast<const uint4 *>(mine + head);
        float4 *const dst = reinterpret_cast<float4 *>(vals + head);
        for (int b0 = tid; b0 < body; b0 += 4 * kThreads) {
            uint4 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b0 + j * kThreads < body) q[j] = src[b0 + j * kThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = b0 + j * kThreads;
                if (b < body) {
                    const float4 v = make_float4(look(bf16lo_f32(q[j].x)), look(bf16hi_f32(q[j].x)), look(bf16lo_f32(q[j].y)),
                                                 look(bf16hi_f32(q[j].y)));
                    const float4 w = make_float4(look(bf16lo_f32(q[j].z)), look(bf16hi_f32(q[j].z)), look(bf16lo_f32(q[j].w)),
                                                 look(bf16hi_f32(q[j].w)));
                    dst[2 * b] = v, dst[2 * b + 1] = w;
                    some = fmaxf(some, fmaxf(v.x, w.x));
                }
            }
        }
    } else {
        auto part = [&](int c) { return static_cast<int>(static_cast<int64_t>(body) * c / kCopies); };
        if (tid == 0) {
            for (int c = 0; c < kCopies; ++c) mbar_init(&s.bars[c], 1);
            fence_mbar_init();
            for (int c = 0; c < kCopies; ++c) {
                const int b0 = part(c), bytes = (part(c + 1) - b0) * 16;
                mbar_arrive_expect_tx(&s.bars[c], bytes);
                if (bytes > 0) bulk_g2s(vals + head + b0 * kVec, mine + head + b0 * kVec, bytes, &s.bars[c]);
            }
        }
        __syncthreads();
        bool late = false;
        float4 *const run = reinterpret_cast<float4 *>(vals + head);
        for (int c = 0; c < kCopies; ++c) {
            late = !mbar_wait_bounded(&s.bars[c], 0) || late;
            const int b1 = part(c + 1);
#pragma unroll 4
            for (int b = part(c) + tid; b < b1; b += kThreads) {
                const float4 q = run[b];
                const float4 v = make_float4(look(q.x), look(q.y), look(q.z), look(q.w));
                if (q.x != q.x || q.y != q.y || q.z != q.z || q.w != q.w) run[b] = v;
                some = fmaxf(some, v.x);
            }
        }
        if (late) {
            if (p.status) atomicOr(p.status, Q8_DEV_TIMEOUT);
            drain_after_timeout();
        }
    }
    if (nan && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
    // the largest of each of this CTA's kGroups / ranks groups of 4 ranks threads, first of runs of
    // at most 32; the largest and smallest of all
    if (every == 1) some = top;
    const int part = min(4 * ranks, 32);
    for (int o = 1; o < part; o <<= 1) some = fmaxf(some, __shfl_xor_sync(0xffffffffu, some, o));
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if (tid % part == 0) s.thread_groups[tid / part] = some;
    if (lane == 0) s.warp_min[warp] = low, s.warp_max[warp] = top;
    if (tid == 0) s.listed = 0;
    cluster.barrier_wait();
    __syncthreads();
    if (tid < kGroups) {  // a thread writes one group's maximum to one CTA
        const int g = tid / ranks;
        some = s.thread_groups[4 * ranks > 32 ? 2 * g : g];
        if (4 * ranks > 32) some = fmaxf(some, s.thread_groups[2 * g + 1]);
        cluster.map_shared_rank(&s, tid % ranks)->groups[rank * (kGroups / ranks) + g] = some;
    } else if (warp == kGroups / 32) {
        low = s.warp_min[lane % kWarps], top = s.warp_max[lane % kWarps];
        for (int o = 16; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        }
        if (lane < ranks) {
            Shared *o = cluster.map_shared_rank(&s, lane);
            o->minima[rank] = low, o->maxima[rank] = top;
        }
    }
    cluster.sync();
    top = s.maxima[lane % ranks], low = s.minima[lane % ranks];
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }

    const Row r(top, temp);

    auto nothing = [&]() {
        if (rank == 0 && tid == 0) {
            p.token[row] = -1;
            if (p.logprob) p.logprob[row] = -INFINITY;
            if (p.kept) p.kept[row] = 0;
        }
    };
    if (top == -INFINITY) {
        nothing();
        return;
    }

    // CTA 0's list gets every word for which in(i) holds (those that fit; `listed` counts all).
    auto gather = [&](auto in, bool from_memory) {
        Shared *o = cluster.map_shared_rank(&s, 0);
        for (int i0 = tid; i0 - tid < n; i0 += 32 * kThreads) {
            uint32_t hits = 0;  // of this thread's next 32 words
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
                const int i = i0 + j * kThreads;
                if (i - tid >= n) break;
                hits |= i < n && in(i) ? 1u << j : 0u;
            }
            if (!__any_sync(0xffffffffu, hits != 0)) continue;
            uint32_t have = __popc(hits), at = have;
            for (int q = 1; q < 32; q <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, at, q);
                if (lane >= q) at += v;
            }
            uint32_t base = 0;
            if (lane == 31) base = atomicAdd(&o->listed, at);
            at += __shfl_sync(0xffffffffu, base, 31) - have;
            for (; hits != 0; hits &= hits - 1, ++at)
                if (at < kList) {
                    const int i = i0 + (__ffs(hits) - 1) * kThreads;
                    o->list[at] = static_cast<unsigned long long>(rank_key(from_memory ? logit(i) : vals[i])) << 32 |
                                  static_cast<uint32_t>(first + i);
                }
        }
        cluster.sync();
    };
    // Sorts the list of CTA 0 by (key, index).
    auto sort = [&](int count) {
        if (count <= 128) {  // each word's place is how many come before it
            unsigned long long x = 0;
            int at = 0;
            if (tid < count) x = s.list[tid];
            if (warp * 32 < count)
#pragma unroll 8
                for (int j = 0; j < count; ++j) at += s.list[j] < x ? 1 : 0;
            __syncthreads();
            if (tid < count) s.list[at] = x;
            __syncthreads();
            return;
        }
        // buckets by the distance from the list's largest logit
        float hi = -INFINITY, lo = INFINITY;
        for (int i = tid; i < count; i += kThreads) {
            const float l = unkey(static_cast<uint32_t>(s.list[i] >> 32));
            hi = fmaxf(hi, l), lo = fminf(lo, l);
        }
        for (int o = 16; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        }
        if (lane == 0) s.warp_max[warp] = hi, s.warp_min[warp] = lo;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) hi = fmaxf(hi, s.warp_max[w]), lo = fminf(lo, s.warp_min[w]);
        const float span = hi - lo, per = span > 0.0f && span < INFINITY ? __fdiv_rn(static_cast<float>(kBins - 1), span) : 0.0f;
        sort_buckets(s, count, [&](unsigned long long x) {
            const float l = unkey(static_cast<uint32_t>(x >> 32));
            return l == hi ? 0 : static_cast<int>(fminf((hi - l) * per, static_cast<float>(kBins - 1)));
        });
    };

    // The whole draw from the list of CTA 0: the row's first words, at least as many as can be
    // kept.  want = 0: the mass that top-p asks for is that of the first k of them.
    auto draw_from_list = [&](unsigned long long want) {
        const int count = static_cast<int>(s.listed);
        sort(count);
        if (count <= 128) {  // one warp, four words a lane
            if (warp == 0) {
                unsigned long long w[4], sum = 0;
                float e[4];
                uint32_t idx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = lane * 4 + j;
                    const unsigned long long x = i < count && i < k ? s.list[i] : ~0ull;
                    idx[j] = static_cast<uint32_t>(x);
                    e[j] = x != ~0ull ? r.weight(unkey(static_cast<uint32_t>(x >> 32))) : 0.f;
                    w[j] = mass_of(e[j]);
                    sum += w[j];
                }
                unsigned long long before = sum;
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long v = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += v;
                }
                if (top_p < 1.0f && want == 0) want = mass_wanted(top_p, __shfl_sync(0xffffffffu, before, 31));
                before -= sum;
                sum = 0;
                uint32_t words = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = w[j] != 0 && (!(top_p < 1.0f) || before < want) && e[j] >= min_p;
                    before += w[j];
                    // by index: 20 bits of index above 41 of mass
                    s.list[lane * 4 + j] = in ? static_cast<unsigned long long>(idx[j]) << 41 | w[j] : ~0ull;
                    sum += in ? w[j] : 0ull;
                    words += in ? 1u : 0u;
                }
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                words = __reduce_add_sync(0xffffffffu, words);
                if (lane == 0) s.warp_mass[0] = sum, s.warp_count[0] = words;
            }
            __syncthreads();
            const unsigned long long all = s.warp_mass[0], low41 = (1ull << 41) - 1;
            if (all == 0) {
                nothing();
            } else if (tid < count) {
                const unsigned long long x = s.list[tid], place = place_of(u, all);
                unsigned long long before = 0;
#pragma unroll 8
                for (int j = 0; j < count; ++j) {
                    const unsigned long long y = s.list[j];
                    before += y < x ? y & low41 : 0ull;
                }
                if (x != ~0ull && before <= place && place < before + (x & low41)) {
                    p.token[row] = static_cast<int32_t>(x >> 41);
                    if (p.logprob) p.logprob[row] = log_share(x & low41, all);
                    if (p.kept) p.kept[row] = static_cast<int32_t>(s.warp_count[0]);
                }
            }
            return;
        }
        unsigned long long w[kPer], sum = 0;
        float e[kPer];
        uint32_t idx[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            w[j] = 0, e[j] = 0.f, idx[j] = 0;
            if (i < count && i < k) {
                const unsigned long long x = s.list[i];
                idx[j] = static_cast<uint32_t>(x);
                e[j] = r.weight(unkey(static_cast<uint32_t>(x >> 32)));
                w[j] = mass_of(e[j]);
            }
            sum += w[j];
        }
        unsigned long long before = 0, total;
        uint32_t c0, c1;
        if (top_p < 1.0f) {
            scan_cta(s, sum, 0u, before, c0, total, c1);
            if (want == 0) want = mass_wanted(top_p, total);
        }
        unsigned long long kept = 0;
        uint32_t words = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const bool in = w[j] != 0 && (!(top_p < 1.0f) || before < want) && e[j] >= min_p;
            before += w[j];
            if (!in) w[j] = 0;
            kept += w[j];
            words += in ? 1u : 0u;
        }
        unsigned long long all;
        uint32_t all_words;
        scan_cta(s, kept, words, before, c0, all, all_words);
        if (all == 0) {
            nothing();
            return;
        }
        // the words kept, by index: 20 bits of index above 41 of mass
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (w[j] != 0) s.list[c0++] = static_cast<unsigned long long>(idx[j]) << 41 | w[j];
        __syncthreads();
        const unsigned long long place = place_of(u, all), low41 = (1ull << 41) - 1;
        auto give = [&](uint32_t word, unsigned long long mass) {
            p.token[row] = static_cast<int32_t>(word);
            if (p.logprob) p.logprob[row] = log_share(mass, all);
            if (p.kept) p.kept[row] = static_cast<int32_t>(all_words);
        };
        if (all_words <= 128) {
            if (tid < static_cast<int>(all_words)) {
                const unsigned long long x = s.list[tid];
                before = 0;
#pragma unroll 8
                for (int j = 0; j < static_cast<int>(all_words); ++j) {
                    const unsigned long long y = s.list[j];
                    before += y < x ? y & low41 : 0ull;
                }
                if (before <= place && place < before + (x & low41)) give(static_cast<uint32_t>(x >> 41), x & low41);
            }
            return;
        }
        const float per_word = __fdiv_rn(static_cast<float>(kBins), static_cast<float>(p.V));
        sort_buckets(s, static_cast<int>(all_words),
                     [&](unsigned long long x) { return min(static_cast<int>(static_cast<float>(x >> 41) * per_word), kBins - 1); });
        kept = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            w[j] = 0;
            if (i < static_cast<int>(all_words)) {
                const unsigned long long x = s.list[i];
                idx[j] = static_cast<uint32_t>(x >> 41);
                w[j] = x & low41;
            }
            kept += w[j];
        }
        scan_cta(s, kept, 0u, before, c0, total, c1);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (w[j] != 0 && before <= place && place < before + w[j]) give(idx[j], w[j]);
            before += w[j];
        }
    };

    // ---- a list of few words ----------------------------------------------------------------
    unsigned long long row_mass = 0;  // of all words, where their e are in place
    if (list > 0) {
        float bound = -INFINITY;
        if (p.V > kList) {
            // the wanted one in the ranking of the group maxima (equal ones by their place): four
            // threads count what comes before one maximum
            static_assert(kThreads == 4 * kGroups, "four threads a group");
            const int place = k <= kFewK ? k : min(kGroups, max(1, static_cast<int>(ceilf(kGroups * (1.0f - expf(-static_cast<float>(list) / (every * kGroups)))))));
            const int me = tid >> 2, j0 = (tid & 3) * (kGroups / 4);
            const float x = s.groups[me];
            int at = 0;
#pragma unroll
            for (int j = j0; j < j0 + kGroups / 4; j += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(&s.groups[j]);
                at += (y.x > x || (y.x == x && j < me)) + (y.y > x || (y.y == x && j + 1 < me)) +
                      (y.z > x || (y.z == x && j + 2 < me)) + (y.w > x || (y.w == x && j + 3 < me));
            }
            at += __shfl_xor_sync(0xffffffffu, at, 1);
            at += __shfl_xor_sync(0xffffffffu, at, 2);
            if (at == place - 1) s.bound = x;
            __syncthreads();
            bound = s.bound;
        }
        if (k == p.V && top_p < 1.0f) {
            // e in place of the logits, and whether the mass above the bound is what top-p asks for
            const float least = r.weight(bound);
            unsigned long long m = 0, a = 0;
            uint32_t c = 0;
            for (int j0 = tid; j0 < n; j0 += 4 * kThreads) {
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = r.weight(j0 + j * kThreads < n ? vals[j0 + j * kThreads] : -INFINITY);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j0 + j * kThreads < n) vals[j0 + j * kThreads] = e[j];
                    const unsigned long long w = mass_of(e[j]);
                    m += w;
                    if (e[j] >= least && e[j] > 0.f) a += w, ++c;
                }
            }
            for (int o = 16; o > 0; o >>= 1) {
                m += __shfl_xor_sync(0xffffffffu, m, o);
                a += __shfl_xor_sync(0xffffffffu, a, o);
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) s.warp_mass[warp] = m, s.warp_above[warp] = a, s.warp_count[warp] = c;
            __syncthreads();
            if (tid < ranks) {
                m = 0, a = 0, c = 0;
                for (int w = 0; w < kWarps; ++w) m += s.warp_mass[w], a += s.warp_above[w], c += s.warp_count[w];
                Shared *o = cluster.map_shared_rank(&s, tid);
                o->sub_mass[rank] = m, o->sub_above[rank] = a, o->sub_count[rank] = c;
            }
            cluster.sync();
            a = 0, c = 0;
            for (int o = 0; o < ranks; ++o) row_mass += s.sub_mass[o], a += s.sub_above[o], c += s.sub_count[o];
            const unsigned long long want = mass_wanted(top_p, row_mass);
            if (c <= kList && a >= want) {
                gather([&](int i) { return vals[i] >= least && vals[i] > 0.f; }, true);
                if (rank == 0) draw_from_list(want);
                return;
            }
        } else {
            gather([&](int i) { return vals[i] >= bound && vals[i] > -INFINITY; }, false);
            if (rank == 0) {  // are they enough?
                const uint32_t listed = s.listed;
                __syncthreads();  // before it may be set back below
                const bool enough = listed <= kList && (bound == -INFINITY || listed >= static_cast<uint32_t>(k));
                if (tid < ranks) cluster.map_shared_rank(&s, tid)->enough = enough ? 1u : 0u;
                if (!enough && tid == 0) s.listed = 0;
            }
            cluster.sync();
            if (s.enough) {
                if (rank == 0) draw_from_list(0ull);
                return;
            }
        }
    }

    // ---- searches over the whole row ------------------------------------------------------
    struct Place {
        uint32_t bin, before_count, in_count;
        unsigned long long before_mass, in_mass;
    };
    auto clear = [&]() {
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0, s.mass_lo[i] = 0, s.mass_hi[i] = 0;
        __syncthreads();
    };
    // One word a lane into the histogram (bin < 0: none).  A warp of equal bins (equal logits)
    // adds once.  64-bit sums are kept in two words: whoever carries the low one over adds that
    // to the high one.
    auto add_to = [&](int bin, unsigned long long w) {
        uint32_t one = 1;
        if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
            if (bin < 0) return;
            for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            one = 32;
            if (lane != 0) bin = -1;
        }
        if (bin >= 0) {
            atomicAdd(&s.count[bin], one);
            if (w != 0) {
                const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&s.mass_lo[bin], lo);
                const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
                if (hi != 0) atomicAdd(&s.mass_hi[bin], hi);
            }
        }
    };
    // The bin in which `want` (a count or a mass) is reached, adding to what f says came before;
    // false, for all threads, if it never is.
    auto locate = [&](int bins, bool by_mass, unsigned long long want, Place &f) -> bool {
        cluster.sync();
        // CTA `rank` adds up its share of the bins over all CTAs: several threads a bin where there are
        // enough (each takes some of the CTAs, the first of them the sum), up to four bins a thread where not
        const int share = bins / ranks, b0 = rank * share, each = (share + kThreads - 1) / kThreads;
        const int helpers = each > 1 ? 1 : min(4, kThreads / share), me = tid / helpers, sub = tid % helpers;
        uint32_t cnt[kBins / kThreads] = {};
        unsigned long long mas[kBins / kThreads] = {};
        uint32_t c_sum = 0;
        unsigned long long m_sum = 0;
#pragma unroll
        for (int j = 0; j < kBins / kThreads; ++j) {
            const int b = me * each + j;
            if (j < each && b < share) {
#pragma unroll 4
                for (int c = sub; c < ranks; c += helpers) {
                    const Shared *o = cluster.map_shared_rank(&s, c);
                    cnt[j] += o->count[b0 + b];
                    if (by_mass) mas[j] += static_cast<unsigned long long>(o->mass_hi[b0 + b]) << 32 | o->mass_lo[b0 + b];
                }
            }
        }
        for (int q = 1; q < helpers; q <<= 1) {  // then each > 1 does not hold: one bin a thread
            cnt[0] += __shfl_xor_sync(0xffffffffu, cnt[0], q);
            mas[0] += __shfl_xor_sync(0xffffffffu, mas[0], q);
        }
#pragma unroll
        for (int j = 0; j < kBins / kThreads; ++j) {
            if (sub != 0) cnt[j] = 0, mas[j] = 0;
            c_sum += cnt[j];
            m_sum += mas[j];
        }
        unsigned long long mb, m_all;
        uint32_t cb, c_all;
        scan_cta(s, m_sum, c_sum, mb, cb, m_all, c_all);
        if (tid < ranks) {
            Shared *o = cluster.map_shared_rank(&s, tid);
            o->sub_count[rank] = c_all;
            o->sub_mass[rank] = m_all;
        }
        cluster.sync();
        uint32_t c_total = f.before_count;
        unsigned long long m_total = f.before_mass;
        int owner = -1;
        for (int c = 0; c < ranks; ++c) {
            if (c == rank) cb += c_total, mb += m_total;
            c_total += s.sub_count[c];
            m_total += s.sub_mass[c];
            if (owner < 0 && (by_mass ? m_total : c_total) >= want) owner = c;
        }
        if (owner < 0) return false;
        if (rank == owner) {
#pragma unroll
            for (int j = 0; j < kBins / kThreads; ++j) {
                const unsigned long long have = by_mass ? mb : cb;
                const unsigned long long with = by_mass ? mb + mas[j] : static_cast<unsigned long long>(cb) + cnt[j];
                if (have < want && with >= want) {
                    s.digit = b0 + me * each + j;
                    s.before_count = cb, s.in_count = cnt[j];
                    s.before_mass = mb, s.in_mass = mas[j];
                }
                cb += cnt[j];
                mb += mas[j];
            }
        }
        cluster.sync();
        const Shared *o = cluster.map_shared_rank(&s, owner);
        f.bin = o->digit;
        f.before_count = o->before_count, f.in_count = o->in_count;
        f.before_mass = o->before_mass, f.in_mass = o->in_mass;
        return true;
    };

    uint32_t last = 0xFFFFFFFFu;  // the last key kept
    uint32_t ties = 0xFFFFFFFFu;  // how many words of that key, in index order
    bool ranked = false;          // fewer than there are

    // The last word kept, exactly, when `in` holds for the words of the step in which it lies.
    // weight(key): a word's share of `want`.
    auto end_in_step = [&](auto in, bool from_memory, unsigned long long before0, unsigned long long want, auto weight) {
        gather(in, from_memory);
        if (rank == 0) {
            const int count = min(static_cast<int>(s.listed), kList);
            sort(count);
            unsigned long long w[kPer], sum = 0, before, total;
            uint32_t c0, c1;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = tid * kPer + j;
                w[j] = i < count ? weight(static_cast<uint32_t>(s.list[i] >> 32)) : 0ull;
                sum += w[j];
            }
            scan_cta(s, sum, 0u, before, c0, total, c1);
            before += before0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = tid * kPer + j;
                if (w[j] != 0 && before < want && before + w[j] >= want) {
                    const uint32_t key = static_cast<uint32_t>(s.list[i] >> 32);
                    int b = i;
                    while (b > 0 && static_cast<uint32_t>(s.list[b - 1] >> 32) == key) --b;
                    s.last = key;
                    s.ties = static_cast<uint32_t>(i - b + 1);
                    s.ranked = i + 1 < count && static_cast<uint32_t>(s.list[i + 1] >> 32) == key ? 1u : 0u;
                }
                before += w[j];
            }
            if (tid == 0) s.listed = 0;
        }
        cluster.sync();
        const Shared *o = cluster.map_shared_rank(&s, 0);
        last = o->last, ties = o->ties, ranked = o->ranked != 0;
    };
    // The same by the digits of the order key (11, 11, 10 bits), for any number of equal words.
    auto end_by_digits = [&](auto in, bool from_memory, bool by_mass, unsigned long long before0, unsigned long long want, auto weight) {
        uint32_t prefix = 0;
        Place f = {};
        f.before_count = by_mass ? 0u : static_cast<uint32_t>(before0);
        f.before_mass = by_mass ? before0 : 0ull;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : kBins;
            const int above = pass == 1 ? 21 : 10;
            clear();
            for (int i0 = warp * 32; i0 < n; i0 += kThreads) {
                const int i = i0 + lane;
                int d = -1;
                unsigned long long w = 0;
                if (i < n && in(i)) {
                    const uint32_t key = rank_key(from_memory ? logit(i) : vals[i]);
                    if (pass == 0 || (key >> above) == prefix) {
                        d = static_cast<int>((key >> shift) & (bins - 1));
                        w = by_mass ? weight(key) : 0ull;
                    }
                }
                add_to(d, w);
            }
            locate(bins, by_mass, want, f);
            prefix = pass == 0 ? f.bin : (pass == 1 ? (prefix << 11) | f.bin : (prefix << 10) | f.bin);
        }
        last = prefix;
        if (by_mass) {
            const unsigned long long w = f.in_mass / f.in_count;
            ties = static_cast<uint32_t>((want - f.before_mass + w - 1) / w);
        } else {
            ties = static_cast<uint32_t>(want) - f.before_count;
        }
        ranked = ties < f.in_count;
        cluster.sync();  // everyone has read what was found
    };
    // Words with the last key that lie before this thread's first word, i0 .. i1 being its run.
    const int run = (n + kThreads - 1) / kThreads, i0 = min(tid * run, n), i1 = min(i0 + run, n);
    auto ties_before = [&](auto key_of) -> uint32_t {
        uint32_t c = 0, before, all;
        unsigned long long mb, ma;
        for (int i = i0; i < i1; ++i) c += key_of(i) == last ? 1u : 0u;
        scan_cta(s, 0ull, c, mb, before, ma, all);
        cluster.sync();
        if (tid < ranks) cluster.map_shared_rank(&s, tid)->sub_count[rank] = all;
        cluster.sync();
        for (int b = 0; b < rank; ++b) before += s.sub_count[b];
        cluster.sync();
        return before;
    };

    if (k < p.V) {
        // steps of the distance from the top: monotone in l, as a difference, a product and a
        // truncation are, each rounded one way.  Past 28 T words have no mass (exp(-28) < 2^-40)
        const float far = 28.0f * temp, range = fminf(far, top - low);
        const float per = range > 0.0f && range < INFINITY ? __fdiv_rn(static_cast<float>(kBins - 1), range) : 0.0f;
        auto step_of = [&](float l) -> int {
            const float d = top - l;
            const int b = d <= far && l > -INFINITY ? static_cast<int>(fminf(d * per, static_cast<float>(kBins - 1))) : -1;
            return l == top ? 0 : b;
        };
        clear();
        for (int w0 = warp * 32; w0 < n; w0 += kThreads * 4) {
            int b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = w0 + j * kThreads + lane;
                b[j] = i < n ? step_of(vals[i]) : -1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) add_to(b[j], 0ull);
        }
        Place f = {};
        const unsigned long long want = static_cast<unsigned long long>(k);
        if (locate(kBins, false, want, f)) {
            const int bin = static_cast<int>(f.bin);
            if (f.before_count + f.in_count <= kList) {
                gather([&](int i) { const int b = step_of(vals[i]); return b >= 0 && b <= bin; }, false);
                if (rank == 0) draw_from_list(0ull);
                return;
            }
            auto in = [&](int i) { return step_of(vals[i]) == bin; };
            if (f.in_count <= kList)
                end_in_step(in, false, f.before_count, want, [](uint32_t) { return 1ull; });
            else
                end_by_digits(in, false, false, f.before_count, want, [](uint32_t) { return 1ull; });
        }
    }

    // ---- e in place of the logits, 0 for words that top-k leaves out; with no filter they stay ----
    const bool all_words_in = k == p.V && !(top_p < 1.0f);
    unsigned long long total = 0;
    if (ranked) {
        uint32_t eq = ties_before([&](int i) { return rank_key(vals[i]); });
        for (int i = i0; i < i1; ++i) {
            const uint32_t key = rank_key(vals[i]);
            const float e = key < last || (key == last && eq < ties) ? r.weight(vals[i]) : 0.f;
            eq += key == last ? 1u : 0u;
            vals[i] = e;
            total += mass_of(e);
        }
        ranked = false;
    } else if (!all_words_in && row_mass == 0) {
        for (int w0 = tid; w0 < n; w0 += 4 * kThreads) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float l = w0 + j * kThreads < n ? vals[w0 + j * kThreads] : -INFINITY;
                e[j] = rank_key(l) <= last ? r.weight(l) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (w0 + j * kThreads < n) vals[w0 + j * kThreads] = e[j];
                total += mass_of(e[j]);
            }
        }
    }

    // ---- top-p ----------------------------------------------------------------------------
    uint32_t eq_before = 0;
    int end_bin = kBins;       // words past this bin are out
    bool edge = false;         // words of this bin are in up to `last`
    // bins of e, the largest first: its leading bits, as many as leave the least e a bin
    int shift = 23;
    auto bin_of = [&](float e) -> int { return e > 0.f ? static_cast<int>(min((0x3F800000u - __float_as_uint(e)) >> shift, kBins - 1u)) : kBins; };
    if (top_p < 1.0f) {
        clear();
        if (row_mass != 0) {
            total = row_mass;
        } else {
            unsigned long long mb, m_all;
            uint32_t cb, c_all;
            scan_cta(s, total, 0u, mb, cb, m_all, c_all);
            cluster.sync();
            if (tid < ranks) cluster.map_shared_rank(&s, tid)->sub_mass[rank] = m_all;
            cluster.sync();
            total = 0;
            for (int c = 0; c < ranks; ++c) total += s.sub_mass[c];
        }
        const unsigned long long want = mass_wanted(top_p, total);
        // words below this e have together less than total - want, or each no mass
        const float share = __fdiv_rn(static_cast<float>(total - min(want, total)), static_cast<float>(p.V));
        const float least = fmaxf(share * 0.999f, 1.0f) * kUnit;
        while (shift > 0 && (0x3F800000u - __float_as_uint(least)) >> (shift - 1) < static_cast<uint32_t>(kBins)) --shift;
        for (int w0 = warp * 32; w0 < n; w0 += kThreads * 4) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = w0 + j * kThreads + lane;
                e[j] = i < n ? vals[i] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = e[j] >= least;
                if (__any_sync(0xffffffffu, in)) add_to(in ? bin_of(e[j]) : -1, in ? mass_of(e[j]) : 0ull);
            }
        }
        Place f = {};
        if (locate(kBins, true, want, f)) {
            const int bin = static_cast<int>(f.bin);
            auto weight = [&](uint32_t key) { return mass_of(r.weight(unkey(key))); };
            if (f.before_count + f.in_count <= kList) {
                gather([&](int i) { return vals[i] >= least && bin_of(vals[i]) <= bin; }, true);
                if (rank == 0) k = p.V, draw_from_list(want);
                return;
            }
            auto in = [&](int i) { return vals[i] >= least && bin_of(vals[i]) == bin; };
            if (f.in_count <= kList)
                end_in_step(in, true, f.before_mass, want, weight);
            else
                end_by_digits(in, true, true, f.before_mass, want, weight);
            end_bin = bin, edge = true;
        }
        if (edge && ranked) eq_before = ties_before([&](int i) { return bin_of(vals[i]) == end_bin ? rank_key(logit(i)) : 0xFFFFFFFFu; });
    }
    auto keep = [&](int i, uint32_t eq) -> float {
        const float e = all_words_in ? r.weight(vals[i]) : vals[i];
        if (!edge) return e;
        const int b = bin_of(e);
        if (b != end_bin) return b < end_bin ? e : 0.f;
        const uint32_t key = rank_key(logit(i));
        return key < last || (key == last && eq < ties) ? e : 0.f;
    };
    unsigned long long sum = 0;  // of this thread's run
    uint32_t count = 0;
    auto tally = [&](float e) {
        const unsigned long long w = e >= min_p ? mass_of(e) : 0ull;
        sum += w;
        count += w != 0 ? 1u : 0u;
    };
    __syncthreads();
    if (edge && ranked) {
        uint32_t eq = eq_before;
        for (int i = i0; i < i1; ++i) {
            tally(keep(i, eq));
            if (bin_of(vals[i]) == end_bin) eq += rank_key(logit(i)) == last ? 1u : 0u;
        }
    } else {
        // each lane starts elsewhere in its run, so that a warp's reads hit all banks
        int j = run > 0 ? lane % run : 0;
        for (int q = 0; q < run; q += 4) {
            float e[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                e[h] = q + h < run && i0 + j < i1 ? keep(i0 + j, 0u) : 0.f;
                j = j + 1 == run ? 0 : j + 1;
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) tally(e[h]);
        }
    }

    // ---- the draw, in index order ------------------------------------------------------------
    unsigned long long before, cta_mass;
    uint32_t c_before, cta_count;
    scan_cta(s, sum, count, before, c_before, cta_mass, cta_count);
    cluster.sync();
    if (tid < ranks) {
        Shared *o = cluster.map_shared_rank(&s, tid);
        o->sub_mass[rank] = cta_mass;
        o->sub_count[rank] = cta_count;
    }
    cluster.sync();
    unsigned long long all = 0;
    uint32_t all_count = 0;
    for (int c = 0; c < ranks; ++c) {
        if (c == rank) before += all;
        all += s.sub_mass[c];
        all_count += s.sub_count[c];
    }
    if (all == 0) {
        nothing();
        return;
    }
    const unsigned long long place = place_of(u, all);
    const uint32_t owner = __ballot_sync(0xffffffffu, place >= before && place < before + sum);
    if (owner) {  // one warp of the row: its lanes walk the owner's run together
        const int src = __ffs(owner) - 1;
        before = __shfl_sync(0xffffffffu, before, src);
        uint32_t eq = __shfl_sync(0xffffffffu, eq_before, src);
        const int w0 = __shfl_sync(0xffffffffu, i0, src), w1 = __shfl_sync(0xffffffffu, i1, src);
        for (int b = w0; b < w1; b += 32) {
            const int i = b + lane;
            uint32_t my_eq = eq;
            if (edge && ranked) {
                const uint32_t same = __ballot_sync(0xffffffffu, i < w1 && bin_of(vals[i]) == end_bin && rank_key(logit(i)) == last);
                my_eq += __popc(same & ((1u << lane) - 1));
                eq += __popc(same);
            }
            const float e = i < w1 ? keep(i, my_eq) : 0.f;
            const unsigned long long w = e >= min_p ? mass_of(e) : 0ull;
            unsigned long long c = w;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, before + c > place);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    p.token[row] = first + i;
                    if (p.logprob) p.logprob[row] = log_share(w, all);
                    if (p.kept) p.kept[row] = static_cast<int32_t>(all_count);
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, c, 31);
        }
    }
}

constexpr int kSmem = 227 * 1024 - 1024;

int slice_of(int V, int ranks) { return ((V + 7 + ranks - 1) / ranks + 7) & ~7; }
bool fits(int V, int ranks) { return sizeof(Shared) + static_cast<size_t>(slice_of(V, ranks)) * 4 <= kSmem; }

// The largest cluster that the current device runs with as much shared memory as a row may take.  16 is more
// than every device promises, and a part of one may have no 16 free SMs in one place.  0: a CUDA call failed.
int largest_cluster(const DeviceInfo *di) {
    static std::atomic<int> found[64];
    int n = di->device < 64 ? found[di->device].load(std::memory_order_relaxed) : 0;
    for (int ranks = kMaxCluster; n == 0 && ranks >= 1; ranks /= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(kThreads);
        cfg.gridDim = dim3(ranks);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ranks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int active = 0;
        if (cudaOccupancyMaxActiveClusters(&active, sample_kernel<false>, &cfg) != cudaSuccess) return 0;
        if (active > 0) n = ranks;
    }
    if (n > 0 && di->device < 64) found[di->device].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

q8_status launch_sample(const SampleArgs &a, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (di->device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        for (auto *f : {sample_kernel<false>, sample_kernel<true>})
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
                cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return Q8_ERR_CUDA;
        ready.fetch_or(bit);
    }
    SampleParams p = {a.logits, a.temperature, a.top_p, a.min_p, a.u, a.top_k, a.token, a.kept, a.logprob, dev_status,
                      a.ld, a.V, 0, 0};
    int most = largest_cluster(di);
    if (most == 0) return Q8_ERR_CUDA;
    // Q8_SAMPLE_CLUSTER = 1, 2, 4 or 8 asks for at most that many CTAs a row (as on a device that runs no
    // more); it never changes the results
    if (const char *e = std::getenv("Q8_SAMPLE_CLUSTER")) {
        const int ask = std::atoi(e);
        if (ask == 1 || ask == 2 || ask == 4 || ask == 8) most = ask < most ? ask : most;
    }
    if (!fits(a.V, most)) return Q8_ERR_UNSUPPORTED;
    // CTAs per row: slices of at most 8192 words while all rows' CTAs find an SM of their own, else
    // of 16384 (two CTAs an SM) where that is possible with half as many.  Clusters of 16 need 16
    // free SMs of one GPC, so they find fewer.  With top-k 50, in us: 131071 words, 16 CTAs and 8: 11.2 and
    // 12.8 for one row, 20.1 and 15.7 for 16, 50 and 30 for 64.  32000 words, 4 and 2: 11.3 and 12.3 for 16
    // rows, 13.9 and 12.9 for 64, 26 and 16 for 128 (8 CTAs: 10.9 for one row, but top-p alone 24 in place
    // of 19).  262144 words, 16 and 8: 12.8 and 15.3 for one row, 59 and 60 for 64.
    int ranks = 1;
    while (ranks < most && a.V > 8192 * ranks) ranks *= 2;
    const int64_t places = ranks == kMaxCluster ? di->sm_count * 2 / 3 : di->sm_count;
    if (ranks > 1 && a.rows * int64_t{ranks} > places && a.V <= 8192 * ranks) ranks /= 2;
    // Rows with knobs of their own, more than run at once: those that take longer begin first (64 rows of
    // 131071 words with mixed knobs: 72 us as they come, 53 so; 64 alike: 30.4 and 30.9).
    p.rows = a.top_k && a.rows <= kThreads && a.rows * int64_t{ranks} > di->sm_count ? a.rows : 0;
    p.slice = slice_of(a.V, ranks);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + static_cast<size_t>(p.slice) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * ranks);
    return cudaLaunchKernelEx(&cfg, a.bf16 ? sample_kernel<true> : sample_kernel<false>, p) == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
