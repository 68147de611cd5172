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
// No sort: the words kept are a prefix of the ranking, so what is needed is
// its last word -- the k-th for top-k, the one that reaches the mass for top-p.
// The 32-bit order key of the logit is searched digit by digit (11, 11, 10
// bits): a histogram of counts and masses per digit, a scan to the bin that
// holds the place looked for, then only words of that bin.  Equal logits at
// the place are kept in index order, counted by division (equal logits have
// equal masses).
//
// A row belongs to a cluster of up to 8 CTAs; each keeps its slice of the row
// in shared memory, so the logits are read from memory once.  Bound: by
// latency for few rows (a handful of passes over shared memory, each with
// cluster barriers), by the passes' instructions for many.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "q8_dev.cuh"
#include "q8_internal.h"

namespace cg = cooperative_groups;

namespace q8 {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr float kOne = 1099511627776.0f;  // 2^40

struct SampleParams {
    const void *logits;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *token, *kept;
    float *logprob;
    uint32_t *status;
    int64_t ld;
    int32_t V, slice, bf16, resident;
};

struct Shared {
    unsigned long long mass[kBins];
    uint32_t count[kBins];
    unsigned long long sub_mass[kMaxCluster];  // per CTA, written by all of them
    uint32_t sub_count[kMaxCluster];
    float maxima[kMaxCluster];
    unsigned long long warp_mass[kWarps];
    uint32_t warp_count[kWarps];
    float warp_max[kWarps];
    // what a search found, written by the CTA that found it
    uint32_t digit;
    uint32_t before_count;
    unsigned long long before_mass;
    uint32_t in_count;
    unsigned long long in_mass;
};

// Ascending order of this key is descending order of the value (-0 = +0).
__device__ __forceinline__ uint32_t rank_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}

struct Row {
    float top, temp;
    __device__ __forceinline__ float weight(float l) const { return l == top ? 1.0f : expf(__fdiv_rn(l - top, temp)); }
    // e below 2^-40 has no mass: nothing to compute below exp(-28)
    __device__ __forceinline__ unsigned long long mass(float l, float &e) const {
        e = 0.f;
        if (l == -INFINITY || l - top < -28.0f * temp) return 0ull;
        e = weight(l);
        return static_cast<unsigned long long>(e * kOne);
    }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }

__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    float *const vals = reinterpret_cast<float *>(smem + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int row = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = min(rank * p.slice, p.V), n = min(p.slice, p.V - first);
    const int64_t at = row * p.ld + first;

    auto global_value = [&](int i) {
        float v = p.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p.logits)[at + i]) << 16)
                         : static_cast<const float *>(p.logits)[at + i];
        return v != v ? -INFINITY : v;
    };
    auto value = [&](int i) { return p.resident ? vals[i] : global_value(i); };

    // ---- the slice and the row's largest logit ---------------------------------------
    float top = -INFINITY;
    bool nan = false;
    for (int i0 = tid; i0 < n; i0 += kThreads * 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kThreads;
            v[j] = -INFINITY;
            if (i < n)
                v[j] = p.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p.logits)[at + i]) << 16)
                              : static_cast<const float *>(p.logits)[at + i];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kThreads;
            if (v[j] != v[j]) v[j] = -INFINITY, nan = true;
            if (i < n && p.resident) vals[i] = v[j];
            top = fmaxf(top, v[j]);
        }
    }
    if (nan && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s.warp_max[warp] = top;
    __syncthreads();
    if (warp == 0) {
        top = s.warp_max[lane];
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane < ranks) cluster.map_shared_rank(&s, lane)->maxima[rank] = top;
    }
    cluster.sync();
    for (int c = 0; c < ranks; ++c) top = fmaxf(top, s.maxima[c]);

    Row r;
    r.top = top;
    r.temp = p.temperature ? p.temperature[row] : 1.0f;
    int64_t k = p.top_k ? p.top_k[row] : 0;
    if (!(r.temp > 0.0f)) r.temp = 1.0f, k = 1;
    if (k <= 0 || k > p.V) k = p.V;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f, min_p = p.min_p ? p.min_p[row] : 0.0f;

    // ---- the place in the ranking where `want_count` words, or `want_mass`, are reached --
    // Finds the key of the word there, and what lies before that key.
    struct Found {
        uint32_t key, before_count, in_count;
        unsigned long long before_mass, in_mass;  // in_*: of the words with that key
    };
    auto search = [&](bool by_mass, unsigned long long want, uint32_t last, Found &f) -> bool {
        // words with keys above `last` are out; false if fewer than wanted are there
        uint32_t prefix = 0, before_count = 0;
        unsigned long long before_mass = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : kBins;
            const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const float l = value(i);
                const uint32_t key = rank_key(l);
                if (key > last || (pass > 0 && (key >> above) != prefix)) continue;
                float e;
                const unsigned long long w = r.mass(l, e);
                if (w == 0) continue;
                const uint32_t d = (key >> shift) & (bins - 1);
                atomicAdd(&s.count[d], 1u);
                atomicAdd(&s.mass[d], w);
            }
            cluster.sync();
            // CTA `rank` adds up its share of the bins over all CTAs
            const int share = bins / ranks, b0 = rank * share;
            uint32_t c_sum = 0;
            unsigned long long m_sum = 0;
            uint32_t my_count[2] = {0, 0};
            unsigned long long my_mass[2] = {0, 0};
            for (int j = 0; j < 2; ++j) {
                const int b = tid * 2 + j;  // two neighbouring bins a thread
                if (b < share)
                    for (int c = 0; c < ranks; ++c) {
                        const Shared *o = cluster.map_shared_rank(&s, c);
                        my_count[j] += o->count[b0 + b];
                        my_mass[j] += o->mass[b0 + b];
                    }
            }
            // inclusive scan over the CTA's threads
            c_sum = my_count[0] + my_count[1];
            m_sum = my_mass[0] + my_mass[1];
            uint32_t c_run = c_sum;
            unsigned long long m_run = m_sum;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t cv = __shfl_up_sync(0xffffffffu, c_run, o);
                const unsigned long long mv = __shfl_up_sync(0xffffffffu, m_run, o);
                if (lane >= o) c_run += cv, m_run += mv;
            }
            if (lane == 31) s.warp_count[warp] = c_run, s.warp_mass[warp] = m_run;
            __syncthreads();
            uint32_t c_all = 0;
            unsigned long long m_all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) c_run += c_all, m_run += m_all;
                c_all += s.warp_count[w];
                m_all += s.warp_mass[w];
            }
            if (tid < ranks) {
                Shared *o = cluster.map_shared_rank(&s, tid);
                o->sub_count[rank] = c_all;
                o->sub_mass[rank] = m_all;
            }
            cluster.sync();
            uint32_t c_before = before_count, c_total = before_count;
            unsigned long long m_before = before_mass, m_total = before_mass;
            for (int c = 0; c < ranks; ++c) {
                if (c == rank) c_before = c_total, m_before = m_total;
                c_total += s.sub_count[c];
                m_total += s.sub_mass[c];
            }
            if (by_mass ? m_total < want : c_total < want) return false;  // the same for all threads
            // the bin in which the wanted place lies: before it less than wanted, with it enough
            uint32_t cb = c_before + c_run - c_sum;
            unsigned long long mb = m_before + m_run - m_sum;
            for (int j = 0; j < 2; ++j) {
                const unsigned long long have = by_mass ? mb : cb;
                const unsigned long long with = by_mass ? mb + my_mass[j] : static_cast<unsigned long long>(cb) + my_count[j];
                if (have < want && with >= want) {
                    for (int c = 0; c < ranks; ++c) {
                        Shared *o = cluster.map_shared_rank(&s, c);
                        o->digit = b0 + tid * 2 + j;
                        o->before_count = cb;
                        o->before_mass = mb;
                        o->in_count = my_count[j];
                        o->in_mass = my_mass[j];
                    }
                }
                cb += my_count[j];
                mb += my_mass[j];
            }
            cluster.sync();
            prefix = pass == 0 ? s.digit : (pass == 1 ? (prefix << 11) | s.digit : (prefix << 10) | s.digit);
            before_count = s.before_count;
            before_mass = s.before_mass;
        }
        f.key = prefix;
        f.before_count = before_count, f.before_mass = before_mass;
        f.in_count = s.in_count, f.in_mass = s.in_mass;
        return true;
    };

    uint32_t last = 0xFFFFFFFFu;   // the last key kept
    uint32_t ties = 0xFFFFFFFFu;   // how many words of that key, in index order
    bool ranked = false;           // fewer than there are
    unsigned long long total = 0;  // mass of the words kept so far
    bool have_total = false;
    Found f;
    if (k < p.V && search(false, static_cast<unsigned long long>(k), last, f)) {
        last = f.key;
        ties = static_cast<uint32_t>(k) - f.before_count;
        ranked = ties < f.in_count;
        total = f.before_mass + f.in_mass / f.in_count * ties;
        have_total = true;
    }
    if (top_p < 1.0f) {
        if (!have_total) {
            unsigned long long m = 0;
            for (int i = tid; i < n; i += kThreads) {
                float e;
                m += r.mass(value(i), e);
            }
            m = warp_sum(m);
            if (lane == 0) s.warp_mass[warp] = m;
            __syncthreads();
            if (warp == 0) {
                m = warp_sum(s.warp_mass[lane]);
                if (lane < ranks) cluster.map_shared_rank(&s, lane)->sub_mass[rank] = m;
            }
            cluster.sync();
            for (int c = 0; c < ranks; ++c) total += s.sub_mass[c];
            cluster.sync();
        }
        const double cut = ceil(static_cast<double>(top_p) * static_cast<double>(total));
        const unsigned long long want = cut < 1.0 ? 1ull : static_cast<unsigned long long>(cut);
        // words before which less than `want` lies: up to the one that reaches it
        if (search(true, want, last, f)) {
            const unsigned long long w = f.in_mass / f.in_count;
            const uint32_t t = static_cast<uint32_t>((want - f.before_mass + w - 1) / w);
            last = f.key;
            ties = t;
            ranked = ties < f.in_count;
        }
    }

    // ---- the draw: sums in index order, a contiguous run of words per warp ---------------
    const int run = (n + kWarps - 1) / kWarps, w0 = min(warp * run, n), w1 = min(w0 + run, n);
    uint32_t eq_before = 0;  // words with the last key before this warp's
    if (ranked) {
        uint32_t c = 0;
        for (int i = w0 + lane; i < w1; i += 32) c += rank_key(value(i)) == last ? 1u : 0u;
        c = warp_sum(c);
        if (lane == 0) s.warp_count[warp] = c;
        __syncthreads();
        uint32_t all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) eq_before = all;
            all += s.warp_count[w];
        }
        if (tid < ranks) cluster.map_shared_rank(&s, tid)->sub_count[rank] = all;
        cluster.sync();
        for (int c2 = 0; c2 < rank; ++c2) eq_before += s.sub_count[c2];
        cluster.sync();
    }
    // mass of word i if it is kept; eq: words with the last key before i
    auto kept_mass = [&](float l, uint32_t eq) -> unsigned long long {
        const uint32_t key = rank_key(l);
        if (key > last || (key == last && eq >= ties)) return 0ull;
        float e;
        const unsigned long long w = r.mass(l, e);
        return e >= min_p ? w : 0ull;
    };
    unsigned long long sum = 0;
    uint32_t count = 0;
    {
        uint32_t eq = eq_before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const float l = i < w1 ? value(i) : -INFINITY;
            uint32_t mine = eq;
            if (ranked) {
                const uint32_t same = __ballot_sync(0xffffffffu, i < w1 && rank_key(l) == last);
                mine += __popc(same & ((1u << lane) - 1));
                eq += __popc(same);
            }
            const unsigned long long w = i < w1 ? kept_mass(l, ranked ? mine : 0u) : 0ull;
            sum += w;
            count += w != 0 ? 1u : 0u;
        }
    }
    sum = warp_sum(sum);
    count = warp_sum(count);
    __syncthreads();
    if (lane == 0) s.warp_mass[warp] = sum, s.warp_count[warp] = count;
    __syncthreads();
    unsigned long long cta_mass = 0, before = 0;
    uint32_t cta_count = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = cta_mass;
        cta_mass += s.warp_mass[w];
        cta_count += s.warp_count[w];
    }
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
        if (rank == 0 && tid == 0) {
            p.token[row] = -1;
            if (p.logprob) p.logprob[row] = -INFINITY;
            if (p.kept) p.kept[row] = 0;
        }
        return;
    }
    const double x = floor(static_cast<double>(p.u[row]) * static_cast<double>(all));
    unsigned long long rr = x > 0.0 ? static_cast<unsigned long long>(x) : 0ull;
    if (rr > all - 1) rr = all - 1;
    if (rr >= before && rr < before + sum) {  // this warp's run holds the token
        uint32_t eq = eq_before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const float l = i < w1 ? value(i) : -INFINITY;
            uint32_t mine = eq;
            if (ranked) {
                const uint32_t same = __ballot_sync(0xffffffffu, i < w1 && rank_key(l) == last);
                mine += __popc(same & ((1u << lane) - 1));
                eq += __popc(same);
            }
            const unsigned long long w = i < w1 ? kept_mass(l, ranked ? mine : 0u) : 0ull;
            unsigned long long c = w;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, before + c > rr);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    p.token[row] = first + i;
                    // log(w / all): through 1 - (all - w) / all where the word has most of the mass
                    if (p.logprob)
                        p.logprob[row] = 2 * w > all ? log1pf(-__fdiv_rn(static_cast<float>(all - w), static_cast<float>(all)))
                                                     : logf(__fdiv_rn(static_cast<float>(w), static_cast<float>(all)));
                    if (p.kept) p.kept[row] = static_cast<int32_t>(all_count);
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, c, 31);
        }
    }
}

constexpr int kSmem = 227 * 1024 - 1024;

}  // namespace

q8_status launch_sample(const SampleArgs &a, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (di->device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
            return Q8_ERR_CUDA;
        ready.fetch_or(bit);
    }
    SampleParams p = {a.logits, a.temperature, a.top_p, a.min_p, a.u, a.top_k, a.token, a.kept, a.logprob, dev_status,
                      a.ld, a.V, 0, a.bf16, 0};
    // CTAs per row: slices of at least 4096 words, at most 8 (a portable cluster)
    int ranks = 1;
    while (ranks < kMaxCluster && a.V > 4096 * ranks) ranks *= 2;
    p.slice = (a.V + ranks - 1) / ranks;
    const size_t bytes = static_cast<size_t>(p.slice) * 4;
    p.resident = bytes + sizeof(Shared) <= static_cast<size_t>(kSmem) ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + (p.resident ? bytes : 0);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * ranks);
    return cudaLaunchKernelEx(&cfg, sample_kernel, p) == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
