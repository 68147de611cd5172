// q8_attn.cu -- attention of one new token per sequence over a paged Q8_0
// key-value cache, split over the cache's length and joined in one launch.
//
// Mathematics.  With s_t = scale * q . k_t and any m, out = (sum_t 2^(s'_t - m)
// v_t) / (sum_t 2^(s'_t - m)), s' = s log2(e).  A warp walks tokens keeping
// (m, l, O) = (reference, sum, weighted sum); two such triples join
// into (max m, l1 2^(m1 - m) + l2 2^(m2 - m), ...), which is how the warps of
// a CTA and the CTAs of a sequence are put together, in a fixed order.  The
// reference is set 11 below the largest score, so that weights use binary16's range
// downwards, and is moved only when a score passes it by 15 (a vote, no shuffles
// otherwise): any m gives the same quotient.  (From 2^23 on, where scores are 1 apart
// and more, it is the largest score itself: rounded, 15 could become 16.)
//
// Scores: keys' codes are exact in binary16, and each query head is scaled by
// a power of two so that its largest value lies in [2^14, 2^15): the bf16
// query is then exact in binary16 down to 2^-31 of that value, and off by at most 2^-39 of it below.  A warp MMA
// (m16n8k16) multiplies 16 tokens x 32 codes by 8 query heads; the block's
// scale multiplies its fp32 result, as in the matmuls.
// Weighted sum: O^T = V^T P, 16 dimensions x 16 tokens by 8 heads, sums in fp32.
// Two roundings to binary16, for one MMA a tile, against 2^-8 of the bf16 result: the value
// s * code by 2^-11 of itself at most, the weight by 2^-11 of itself down to 2^-25 of the
// warp's largest and by 2^-36 of that below, which for 2^18 tokens makes 2^-18.
// (With the largest at 1, weights lost digits from 2^-14 on and vanished at 2^-25, out of
// O but not out of l.)
// Value scales from 512 on could overflow s * code: their tokens are added in a turn
// of their own, with s 2^-9 and O 2^-9, both exact.
//
// Bound: bytes of the cache, 2.125 per dimension and token, each read once
// for up to 16 query heads; beyond 8 query heads to a key head by latency: 2 CTAs an
// SM find room in shared memory, whose 8 warps issue in 42 % of the slots.  Measured: 262,144
// tokens of 8 key heads (128 dimensions, 64 query heads) 96.5 us, 5.9 TB/s; 48 sequences of 0 to
// 6000 tokens, 32 / 8 heads, 64.9 us, 5.35 TB/s; the loads alone take 93 and 61.  One sequence of
// 200 tokens: 7.9 us, the list, one tile's latency and the join.
//
// Split: every warp is its own pipeline over 16-token tiles (a tile lies in
// one page, so its codes and scales are four contiguous runs), filled by
// 16-byte asynchronous copies; a warp waits for nobody until its item ends.
// Work is cut into units of kWarps tiles (the sequences' lengths are read on
// the device); CTA c takes units [c * per, (c + 1) * per) of the list of all
// (sequence, key head, group of query heads) items, so CTAs carry the same
// load whatever the lengths.  An item within one CTA is finished there; the
// others leave (m, l, O) in the workspace, where they are joined in CTA order, in
// bunches and then the bunches, each by the last CTA to arrive.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>

#include "q8_async.cuh"
#include "q8_dev.cuh"
#include "q8_internal.h"

namespace q8 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnitTokens = kWarps * 16;
constexpr int kMaxGrid = 1024;    // CTAs a launch may have (sizes the workspace)
constexpr size_t kTicketBytes = Q8_ATTN_ZEROED_BYTES;
static_assert(kTicketBytes == size_t{4} * kMaxGrid * 4, "the tickets");
constexpr int kMinUnits = 2;      // units a CTA takes at least; 3 and 4 gain in one short case what they lose in another
constexpr float kLift = 11.0f;    // log2 of the largest weight when the reference is set
constexpr float kTop = 15.0f;     // and of the largest that leaves it: 2^15 (2^15.5, rounded) is within binary16
constexpr float kLiftEnd = 0x1p23f;  // magnitude of a score from which on there is neither
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
    const int8_t *kq, *vq;
    const uint16_t *ks, *vs;
    const uint16_t *q;
    const int32_t *table, *lens;
    uint16_t *out;
    float *lse;
    uint32_t *tickets;  // [2][2 * kMaxGrid]: by the first part of a bunch, of an item
    float *parts;       // [2 * kMaxGrid][HG * (D + 2)]
    uint32_t *status;
    int64_t ldq;
    int32_t batch, q_heads, kv_heads, group, splits;  // splits: runs of HG heads in a group
    int32_t table_width, pages, page_shift, window;
    float scale, softcap;
};

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t *p, uint32_t v) {
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The token (0 .. 7) that MMA row f stands for; rows f + 8 stand for token
// + 8.  Chunks of 16 bytes are stored at chunk ^ (128-byte line & 7); these
// orders make both access patterns hit all banks once: keys (rows f = 0..3
// and 4..7, two chunks each) and values (rows 0, 2, 4, 6 and 1, 3, 5, 7, two
// neighbouring lanes' chunks each).
template <int D>
__device__ __forceinline__ int token_of(int f) {
    constexpr uint32_t order = D == 64 ? 0x37265140u : (D == 128 ? 0x57136420u : 0x67453210u);
    return (order >> (4 * f)) & 7;
}
// Byte offset of 16-byte chunk c of a tile's token r.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    const uint32_t m = r * (D / 16) + c;
    return (m ^ ((m >> 3) & 7)) * 16;
}

// The NB scales of a token: as pairs, and widened.
template <int NB>
__device__ __forceinline__ void raw_scales(uint32_t at, uint32_t (&w)[NB / 2]) {
    if constexpr (NB == 8) {
        const uint4 v = lds128(at);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (NB == 4) {
        const uint2 v = lds64(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = lds32(at);
    }
}
template <int NB>
__device__ __forceinline__ void token_scales(uint32_t at, float (&f)[NB]) {
    uint32_t w[NB / 2];
    raw_scales<NB>(at, w);
#pragma unroll
    for (int b = 0; b < NB / 2; ++b) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[b]));
        f[2 * b] = v.x, f[2 * b + 1] = v.y;
    }
}

// N codes of one token, as offsets from -128.
template <int N>
__device__ __forceinline__ void run_codes(uint32_t at, uint32_t (&w)[N / 4]) {
    if constexpr (N == 16) {
        const uint4 v = lds128(at);
        w[0] = v.x ^ 0x80808080u, w[1] = v.y ^ 0x80808080u, w[2] = v.z ^ 0x80808080u, w[3] = v.w ^ 0x80808080u;
    } else {
        const uint2 v = lds64(at);
        w[0] = v.x ^ 0x80808080u, w[1] = v.y ^ 0x80808080u;
    }
}

// Where a CTA is in the list of items.
struct Walk {
    int b, unit, units;      // units of this sequence's items
    int kvh, run;            // the item: key head, and run of its query heads
    int len, first;          // tokens, and the first one seen
    int base;                // first token of unit 0 (a multiple of 16)
};

__device__ __forceinline__ int seq_len(const AttnParams &p, int b, bool flag) {
    const int n = p.lens[b], top = p.table_width << p.page_shift;
    const int c = min(max(n, 0), top);
    if (flag && c != n && p.status) atomicOr(p.status, Q8_DEV_BAD_INDEX);
    return c;
}
__device__ __forceinline__ int seq_first(const AttnParams &p, int len) {
    return p.window > 0 ? max(0, len - p.window) : 0;
}
__device__ __forceinline__ int seq_units(const AttnParams &p, int len) {
    const int base = seq_first(p, len) & ~15;
    return (len - base + kUnitTokens - 1) / kUnitTokens;
}
__device__ __forceinline__ void enter(const AttnParams &p, Walk &w) {
    w.len = seq_len(p, w.b, false);
    w.first = seq_first(p, w.len);
    w.base = w.first & ~15;
    w.units = seq_units(p, w.len);
}
// The next unit of the list (the caller knows that there is one).
__device__ __forceinline__ void advance(const AttnParams &p, Walk &w) {
    if (++w.unit < w.units) return;
    w.unit = 0;
    if (++w.run < p.splits) return;
    w.run = 0;
    if (++w.kvh < p.kv_heads) return;
    w.kvh = 0;
    do {
        ++w.b;
        enter(p, w);
    } while (w.units == 0 && w.b + 1 < p.batch);
}

template <int D, int NT>
struct Cfg {
    static constexpr int HG = 8 * NT;              // query heads of an item
    static constexpr int kCodes = 16 * D;          // bytes of a tile's key (or value) codes
    static constexpr int kScales = D;              // bytes of its scales: 16 * (D / 32) * 2
    static constexpr int kStage = 2 * (kCodes + kScales);
    // as deep as the CTAs that registers allow leave room for; a stage more or fewer is within 3 % (66.4 us
    // with 4 for 48 ragged sequences, 65.2 with 3, which leave room for 3 CTAs in place of 2), but for 16
    // heads of 128 dimensions (28.4 us with 4, 30.4 with 3)
    static constexpr int kStages = D == 256 ? 2 : (D == 128 && NT == 1 ? 3 : 4);
    static constexpr int kCtas = D == 256 ? 2 : 3;  // CTAs an SM that registers must allow
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kOPitch = D + 8;
    static constexpr int kJoin = (HG * kOPitch + 2 * kWarps * HG + 2 * HG) * 4;
    static constexpr int kSmem = kRing + kJoin;
    static constexpr int kPart = HG * (D + 2);     // floats of one partial result
    // What ending an item (joining the warps, leaving a part or the answer) takes, in units' time.
    // With 0, 2, 4, 6, 8 units 48 ragged sequences (8 heads, 128 dimensions) take 71, 65.7, 64.2, 64.9, 66.2
    // us; with 2, 4, 6, 8 others with 16 heads 104, 86.1, 82.6, 83.4.
    static constexpr int kEndUnits = NT == 1 ? 4 : 6;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas) attn_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<D, NT>;
    constexpr int NB = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ uint32_t s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    float *const s_o = reinterpret_cast<float *>(smem + C::kRing);
    float *const s_m = s_o + C::HG * C::kOPitch;  // [kWarps][HG]
    float *const s_l = s_m + kWarps * C::HG;
    float *const s_mm = s_l + kWarps * C::HG;     // [HG] joined
    float *const s_ll = s_mm + C::HG;

    // ---- the list: an item takes its units and kEndUnits; how long that is, and where this CTA begins ----
    const int heads = p.kv_heads * p.splits;
    long long total = 0;
    for (int b = tid; b < p.batch; b += kThreads) {
        const int n = seq_units(p, seq_len(p, b, blockIdx.x == 0));
        total += n > 0 ? n + C::kEndUnits : 0;
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) s_scan[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += s_scan[w];
    total *= heads;
    const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinUnits));
    const long long u0 = per * blockIdx.x, u1 = min(u0 + per, total);

    // sequences of no tokens have no units: write their answer
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        if (seq_len(p, b, false) > 0) continue;
        for (int i = tid; i < p.q_heads * D / 8; i += kThreads)
            reinterpret_cast<uint4 *>(p.out)[static_cast<int64_t>(b) * p.q_heads * (D / 8) + i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = tid; i < p.q_heads; i += kThreads) p.lse[static_cast<int64_t>(b) * p.q_heads + i] = -INFINITY;
    }
    if (u0 >= u1) return;

    // the sequence at place u0 of the list: each warp scans for itself, 32 at a time
    Walk wk;
    long long left = u1 - u0;  // of this CTA's stretch of the list, from its next unit on
    long long item0;           // where the item begins
    {
        long long before = 0;
        int b0 = 0;
        while (true) {
            const int b = b0 + lane;
            const int units = b < p.batch ? seq_units(p, seq_len(p, b, false)) : 0;
            const long long n = units > 0 ? static_cast<long long>(units + C::kEndUnits) * heads : 0;
            long long run = n;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, before + run > u0);
            if (hit) {
                const int src = __ffs(hit) - 1;
                before += __shfl_sync(0xffffffffu, run - n, src);
                wk.b = b0 + src;
                break;
            }
            before += __shfl_sync(0xffffffffu, run, 31);
            b0 += 32;
        }
        enter(p, wk);
        const long long in = u0 - before;
        const int cost = wk.units + C::kEndUnits, item = static_cast<int>(in / cost);
        wk.kvh = item / p.splits, wk.run = item - wk.kvh * p.splits;
        wk.unit = static_cast<int>(in - static_cast<long long>(item) * cost);
        item0 = u0 - wk.unit;
        if (wk.unit >= wk.units) {  // at the end of an item that others work on: begin with the next
            left -= cost - wk.unit;
            item0 += cost;
            if (left <= 0) return;
            wk.unit = wk.units - 1;
            advance(p, wk);
        }
    }

    // ---- this warp's pipeline ------------------------------------------------------
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStage;
    Walk ld = wk;              // the next unit to load
    long long ld_left = left;
    int ld_slot = 0;
    int ld_page = -1;          // page of the tile to load next, read one step ahead
    uint32_t held = 0;         // bit i: slot i holds a tile
    const int page_mask = (1 << p.page_shift) - 1;
    auto tile_of = [&](const Walk &w) { return w.base + w.unit * kUnitTokens + warp * 16; };
    auto fetch_page = [&]() {
        ld_page = -1;
        if (ld_left > 0) {
            const int tok = tile_of(ld);
            if (tok < ld.len) ld_page = p.table[static_cast<int64_t>(ld.b) * p.table_width + (tok >> p.page_shift)];
        }
    };
    // 16-byte chunk m of a tile lies at m ^ ((m >> 3) & 7): for this lane's chunks lane + 32 i,
    // one place for even i and one for odd
    const uint32_t even = (lane ^ (lane >> 3)) * 16, odd = even ^ 64;
    auto load = [&]() {
        if (ld_left > 0) {
            const int tok = tile_of(ld);
            const bool ok = tok < ld.len && static_cast<uint32_t>(ld_page) < static_cast<uint32_t>(p.pages);
            held = (held & ~(1u << ld_slot)) | (static_cast<uint32_t>(ok) << ld_slot);
            // a page outside the cache: its tokens are left out
            if (!ok && tok < ld.len && lane == 0 && p.status) atomicOr(p.status, Q8_DEV_BAD_INDEX);
            if (ok) {
                const int64_t row = ((static_cast<int64_t>(ld_page) * p.kv_heads + ld.kvh) << p.page_shift) + (tok & page_mask);
                const uint32_t st = ring + ld_slot * C::kStage;
                const int8_t *kc = p.kq + row * D + lane * 16, *vc = p.vq + row * D + lane * 16;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t to = st + ((i & 1) ? odd : even) + i * 512;
                    cp_async16(to, kc + i * 512);
                    cp_async16(to + C::kCodes, vc + i * 512);
                }
                if (lane < D / 8) {
                    const bool is_v = lane >= D / 16;
                    const uint8_t *src = reinterpret_cast<const uint8_t *>(is_v ? p.vs : p.ks) + row * (NB * 2) + (is_v ? lane - D / 16 : lane) * 16;
                    cp_async16(st + 2 * C::kCodes + lane * 16, src);
                }
            }
            ld_left -= ld.unit + 1 < ld.units ? 1 : 1 + C::kEndUnits;
            if (ld_left > 0) advance(p, ld);
            fetch_page();
        }
        ld_slot = ld_slot + 1 == C::kStages ? 0 : ld_slot + 1;
        cp_async_commit();
    };
    fetch_page();
    for (int i = 0; i < C::kStages - 1; ++i) load();

    // ---- where this lane reads in a tile ----------------------------------------------
    // keys: tokens r0 and r0 + 8, 8 codes of each block; values: of tokens ra, rb, ra + 8, rb + 8 the
    // dimensions kRun g .. kRun (g + 1) - 1 of each kRun * 8, which lie in one block
    const int r0 = token_of<D>(g), ra = token_of<D>(2 * t), rb = token_of<D>(2 * t + 1);
    constexpr int kRun = D == 64 ? 8 : 16, kRuns = D / (8 * kRun);
    constexpr uint32_t kEight = 8 * D;  // bytes from a token to the eighth after it (the same place modulo 8 lines)
    uint32_t key_at[NB], va_at[kRuns], vb_at[kRuns];
#pragma unroll
    for (int b = 0; b < NB; ++b) key_at[b] = chunk_at<D>(r0, 2 * b + (t >> 1)) + (t & 1) * 8;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const int d = kRun * (8 * k + g);
        va_at[k] = C::kCodes + chunk_at<D>(ra, d / 16) + d % 16;
        vb_at[k] = C::kCodes + chunk_at<D>(rb, d / 16) + d % 16;
    }
    const int vs_at = (kRun * g / 32) * 2;  // bytes to the scale of a token's first run; the next is kRun * 8 / 32 on
    constexpr uint32_t kFlip = D == 64 ? 64u : 0u;  // at 64 dimensions 8 tokens are 4 lines: the chunk's place changes

    // ---- items ---------------------------------------------------------------------
    int slot = 0;
    while (left > 0) {
        const int seg_first = wk.unit;
        const int seg = static_cast<int>(min(left, static_cast<long long>(wk.units - wk.unit)));
        const int head0 = wk.kvh * p.group + wk.run * C::HG;    // first query head of the item
        const int nheads = min(C::HG, p.group - wk.run * C::HG);
        // this lane's query fragments: head g (+ 8 per n-tile), 8 dimensions of each block
        uint32_t qf[NT][NB][4];
        float fac[NT][2];  // scores of head 2t, 2t + 1: MMA result -> log2 units (or softcap's argument)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + g;
            uint4 raw[NB];
            float amax = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                raw[b] = h < nheads ? *reinterpret_cast<const uint4 *>(p.q + wk.b * p.ldq + static_cast<int64_t>(head0 + h) * D +
                                                                       32 * b + 8 * t)
                                    : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16lo_f32(w[i])), fabsf(bf16hi_f32(w[i]))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^e with amax * 2^e in [2^14, 2^15); exponents kept where 2^e and 2^-e are normal
            int ex = static_cast<int>(__float_as_uint(amax) >> 23);
            ex = min(max(ex, 30), 254);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[n][b][i] = f32x2_to_f16x2(bf16lo_f32(w[i]) * up, bf16hi_f32(w[i]) * up);
            }
            float f = p.scale * down;
            f = p.softcap > 0.f ? f / p.softcap : f * kLog2e;
            f = fmaxf(fminf(f, FLT_MAX), -FLT_MAX);  // a score of zero stays one
            fac[n][0] = __shfl_sync(0xffffffffu, f, (2 * t) * 4);
            fac[n][1] = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
        }
        float m[NT][2], l[NT][2], o[NT][D / 16][4];
        float ref[NT][2], top[NT][2];  // m, or 0 where nothing was seen; the score that moves it
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = top[n][0] = top[n][1] = -INFINITY;
            ref[n][0] = ref[n][1] = 0.f;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }

        for (int s = 0; s < seg; ++s) {
            const int tok = wk.base + (seg_first + s) * kUnitTokens + warp * 16;
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            const bool live = (held >> slot) & 1;
            load();  // into the slot that the step before this one read
            const uint32_t st = ring + slot * C::kStage;
            if (live) {
                // ---- scores: 16 tokens x 8 NT heads
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                const uint32_t sk = st + 2 * C::kCodes, sv = sk + C::kScales;
                float s0[NB], s1[NB];
                token_scales<NB>(sk + r0 * NB * 2, s0);
                token_scales<NB>(sk + (r0 + 8) * NB * 2, s1);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint2 w0 = lds64(st + key_at[b]);
                    const uint2 w1 = lds64(st + ((key_at[b] + kEight) ^ kFlip));
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    codes4_to_f16x2(w0.x, a0, a2);
                    codes4_to_f16x2(w1.x, a1, a3);
                    codes4_to_f16x2(w0.y, b0, b2);
                    codes4_to_f16x2(w1.y, b1, b3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d0, d1, d2, d3;
                        mma_f16_16816_new(d0, d1, d2, d3, a0, a1, a2, a3, qf[n][b][0], qf[n][b][1]);
                        mma_f16_16816(d0, d1, d2, d3, b0, b1, b2, b3, qf[n][b][2], qf[n][b][3]);
                        acc[n][0] = fmaf(s0[b], d0, acc[n][0]);
                        acc[n][1] = fmaf(s0[b], d1, acc[n][1]);
                        acc[n][2] = fmaf(s1[b], d2, acc[n][2]);
                        acc[n][3] = fmaf(s1[b], d3, acc[n][3]);
                    }
                }
                // value scales of tokens (ra, rb) and (ra + 8, rb + 8), as pairs
                uint32_t s01[kRuns], s89[kRuns];
#pragma unroll
                for (int k = 0; k < kRuns; ++k) {
                    const uint32_t from = sv + vs_at + k * (kRun * 8 / 32) * 2;
                    s01[k] = lds16(from + ra * NB * 2) | lds16(from + rb * NB * 2) << 16;
                    s89[k] = lds16(from + (ra + 8) * NB * 2) | lds16(from + (rb + 8) * NB * 2) << 16;
                }
                // ---- weights
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] *= fac[n][i & 1];
                if (p.softcap > 0.f) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] = p.softcap * kLog2e * tanhf(acc[n][i]);
                }
                if (tok < wk.first || tok + 16 > wk.len) {  // some tokens are not seen: no weight, and no value
                    auto seen = [&](int r) { return tok + r >= wk.first && tok + r < wk.len; };
                    const bool in0 = seen(r0), in1 = seen(r0 + 8);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] = (i < 2 ? in0 : in1) ? acc[n][i] : -INFINITY;
                    const uint32_t m01 = (seen(ra) ? 0xFFFFu : 0u) | (seen(rb) ? 0xFFFF0000u : 0u);
                    const uint32_t m89 = (seen(ra + 8) ? 0xFFFFu : 0u) | (seen(rb + 8) ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int k = 0; k < kRuns; ++k) s01[k] &= m01, s89[k] &= m89;
                }
                bool grows = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) grows = grows || fmaxf(acc[n][j], acc[n][2 + j]) > top[n][j];
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float y = fmaxf(acc[n][j], acc[n][2 + j]);
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                            y = fmaxf(y - (fabsf(y) < kLiftEnd ? kLift : 0.f), m[n][j]);
                            const float f = m[n][j] == -INFINITY ? 0.f : ex2(m[n][j] - y);
                            m[n][j] = y;
                            ref[n][j] = y == -INFINITY ? 0.f : y;
                            top[n][j] = y + (fabsf(y) < kLiftEnd ? kTop : 0.f);
                            l[n][j] *= f;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) o[n][i][j] *= f, o[n][i][2 + j] *= f;
                        }
                }
                // a scale of 512 or more in either half (of any sign, though the quantizer makes none below zero)
                uint32_t most = 0x5FFF5FFFu;
#pragma unroll
                for (int k = 0; k < kRuns; ++k) most = __vmaxu2(most, __vmaxu2(s01[k] & 0x7FFF7FFFu, s89[k] & 0x7FFF7FFFu));
                const bool big = __any_sync(0xffffffffu, most != 0x5FFF5FFFu);
                uint32_t pf[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = ex2(acc[n][i] - ref[n][i & 1]);
                    l[n][0] += w[0] + w[2];
                    l[n][1] += w[1] + w[3];
                    pf[n][0] = movmatrix(f32x2_to_f16x2(w[0], w[1]));
                    pf[n][1] = movmatrix(f32x2_to_f16x2(w[2], w[3]));
                }
                // ---- weighted values: MMA rows g and g + 8 of tile q are this lane's dimensions 2 q and
                // 2 q + 1 of its run
                auto add_values = [&](const uint32_t (&t01)[kRuns], const uint32_t (&t89)[kRuns]) {
#pragma unroll
                    for (int k = 0; k < kRuns; ++k) {
                        uint32_t wa[kRun / 4], wb[kRun / 4], wc[kRun / 4], wd[kRun / 4];
                        run_codes<kRun>(st + va_at[k], wa);
                        run_codes<kRun>(st + vb_at[k], wb);
                        run_codes<kRun>(st + ((va_at[k] + kEight) ^ kFlip), wc);
                        run_codes<kRun>(st + ((vb_at[k] + kEight) ^ kFlip), wd);
#pragma unroll
                        for (int q = 0; q < kRun / 2; ++q) {
                            const uint32_t y = __byte_perm(wa[q / 2], wb[q / 2], (q & 1) ? 0x7362 : 0x5140);
                            const uint32_t z = __byte_perm(wc[q / 2], wd[q / 2], (q & 1) ? 0x7362 : 0x5140);
                            const uint32_t k1152 = 0x64806480u;
                            const uint32_t a0 = hmul2(hsub2(__byte_perm(y, 0x64646464u, 0x4140), k1152), t01[k]);
                            const uint32_t a1 = hmul2(hsub2(__byte_perm(y, 0x64646464u, 0x4342), k1152), t01[k]);
                            const uint32_t a2 = hmul2(hsub2(__byte_perm(z, 0x64646464u, 0x4140), k1152), t89[k]);
                            const uint32_t a3 = hmul2(hsub2(__byte_perm(z, 0x64646464u, 0x4342), k1152), t89[k]);
                            constexpr int kTiles = kRun / 2;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16_16816(o[n][k * kTiles + q][0], o[n][k * kTiles + q][1], o[n][k * kTiles + q][2],
                                              o[n][k * kTiles + q][3], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                        }
                    }
                };
                if (big) {  // the tokens of large scales by themselves, then the others (one loop around both took 3 % more)
                    auto scale_o = [&](float f) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) o[n][i][0] *= f, o[n][i][1] *= f, o[n][i][2] *= f, o[n][i][3] *= f;
                    };
                    uint32_t t01[kRuns], t89[kRuns];
#pragma unroll
                    for (int k = 0; k < kRuns; ++k) {
                        const uint32_t m01 = __vcmpgeu2(s01[k] & 0x7FFF7FFFu, 0x60006000u), m89 = __vcmpgeu2(s89[k] & 0x7FFF7FFFu, 0x60006000u);
                        t01[k] = hmul2(s01[k] & m01, 0x18001800u);  // 2^-9
                        t89[k] = hmul2(s89[k] & m89, 0x18001800u);
                        s01[k] &= ~m01, s89[k] &= ~m89;
                    }
                    scale_o(0x1p-9f);
                    add_values(t01, t89);
                    scale_o(0x1p9f);
                }
                add_values(s01, s89);
            }
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
        }

        // ---- join the warps -------------------------------------------------------------
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[n][j];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                l[n][j] = x;
                if (g == 0) {
                    s_m[warp * C::HG + n * 8 + 2 * t + j] = m[n][j];
                    s_l[warp * C::HG + n * 8 + 2 * t + j] = x;
                }
            }
        __syncthreads();
        if (tid < C::HG) {
            float mm = -INFINITY, ll = 0.f;
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * C::HG + tid]);
            for (int w = 0; w < kWarps; ++w) {
                const float mw = s_m[w * C::HG + tid];
                ll += mw == -INFINITY ? s_l[w * C::HG + tid] : s_l[w * C::HG + tid] * ex2(mw - mm);
            }
            s_mm[tid] = mm;
            s_ll[tid] = ll;
        }
        // each warp adds its sums to one quarter of the dimensions after another, beginning with its
        // own: quarter q takes warps q, q + 1, ... in that order
        float f[NT][2];
#pragma unroll 1
        for (int turn = 0; turn < kWarps; ++turn) {
            __syncthreads();
            if (turn == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) f[n][j] = m[n][j] == -INFINITY ? 1.f : ex2(m[n][j] - s_mm[n * 8 + 2 * t + j]);
            }
            const int quarter = (warp + kWarps - turn) % kWarps;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                if (i / (D / 64) != quarter) continue;
                const int d = kRun * (8 * (i / (kRun / 2)) + g) + 2 * (i % (kRun / 2));
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float2 *at = reinterpret_cast<float2 *>(s_o + (n * 8 + 2 * t + j) * C::kOPitch + d);
                        float2 v = make_float2(o[n][i][j] * f[n][j], o[n][i][2 + j] * f[n][j]);
                        if (turn > 0) {
                            const float2 old = *at;
                            v.x += old.x;
                            v.y += old.y;
                        }
                        *at = v;
                    }
            }
        }
        __syncthreads();

        // ---- give the item's answer, or leave a part of it --------------------------------
        auto answer = [&](int h, int d, float mm, float ll, float4 v) {  // four dimensions of a head
            const float r = ll == 0.f ? 0.f : 1.f / ll;
            const __nv_bfloat162 x = __floats2bfloat162_rn(v.x * r, v.y * r);
            const __nv_bfloat162 y = __floats2bfloat162_rn(v.z * r, v.w * r);
            const int64_t row = static_cast<int64_t>(wk.b) * p.q_heads + head0 + h;
            *reinterpret_cast<uint2 *>(p.out + row * D + d) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
            if (p.lse && d == 0) p.lse[row] = ll == 0.f ? -INFINITY : fmaf(mm + kLift, 0.69314718055994531f, logf(ll * 0x1p-11f));
        };
        const int quads = nheads * (D / 4);
        auto own = [&](int h, int d) { return *reinterpret_cast<const float4 *>(s_o + h * C::kOPitch + d); };
        if (seg == wk.units) {
            for (int i = tid; i < quads; i += kThreads) {
                const int h = i / (D / 4), d = i % (D / 4) * 4;
                answer(h, d, s_mm[h], s_ll[h], own(h, d));
            }
        } else {
            // CTAs c0 .. c1 have a part each.  The last of a bunch of neighbours joins theirs into one, the
            // last bunch of the item those: with all of them left to the item's last CTA, 57 parts took
            // 20 us at the end of a long sequence.
            const int c0 = static_cast<int>(item0 / per), c1 = static_cast<int>((item0 + wk.units - 1) / per);
            auto slot_of = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };
            auto part = [&](int c) { return p.parts + static_cast<int64_t>(slot_of(c)) * C::kPart; };
            auto leave = [&](float *to, int h, int d, float mm, float ll, float4 v) {
                __stcg(reinterpret_cast<float4 *>(to + h * D + d), v);
                if (d == 0) __stcg(reinterpret_cast<float2 *>(to + C::HG * D) + h, make_float2(mm, ll));
            };
            // counts this CTA in; true for the last of n (one thread's fence, after the barrier: a fence
            // waits for the copies its thread has under way)
            auto last_of = [&](uint32_t *ticket, int n) -> bool {
                __syncthreads();
                if (tid == 0) {
                    s_last = atomic_add_acq_rel(ticket, 1u) == static_cast<uint32_t>(n - 1) ? 1u : 0u;
                    if (s_last) *ticket = 0u;
                }
                __syncthreads();
                return s_last != 0;
            };
            // the parts of CTAs a, a + step, ... (n of them) joined in that order, eight under way at a time
            auto join = [&](int a, int step, int n, int h, int d, float &mm, float &ll, float4 &v) {
                mm = -INFINITY, ll = 0.f, v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int c = 0; c < n; c += 8) {
                    float2 ml[8];
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float *from = part(a + min(c + k, n - 1) * step);
                        ml[k] = __ldcg(reinterpret_cast<const float2 *>(from + C::HG * D) + h);
                        x[k] = __ldcg(reinterpret_cast<const float4 *>(from + h * D + d));
                    }
                    float top = mm;
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
                    auto weight = [&](float m1) { return m1 == -INFINITY ? (top == -INFINITY ? 1.f : 0.f) : ex2(m1 - top); };
                    const float f0 = weight(mm);
                    ll *= f0, v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (c + k >= n) continue;
                        const float f1 = weight(ml[k].x);
                        ll = fmaf(ml[k].y, f1, ll);
                        v.x = fmaf(x[k].x, f1, v.x), v.y = fmaf(x[k].y, f1, v.y);
                        v.z = fmaf(x[k].z, f1, v.z), v.w = fmaf(x[k].w, f1, v.w);
                    }
                    mm = top;
                }
            };
            const int c = static_cast<int>(blockIdx.x), n = c1 - c0 + 1;
            int bunch = 8;
            while (bunch * bunch < n) bunch *= 2;  // 1024 CTAs at most: 32
            const int first = c0 + (c - c0) / bunch * bunch, in_bunch = min(bunch, c1 - first + 1);
            const int bunches = (n + bunch - 1) / bunch;
            for (int i = tid; i < quads; i += kThreads) {
                const int h = i / (D / 4), d = i % (D / 4) * 4;
                leave(part(c), h, d, s_mm[h], s_ll[h], own(h, d));
            }
            if (last_of(p.tickets + slot_of(first), in_bunch)) {
                for (int i = tid; i < quads; i += kThreads) {
                    const int h = i / (D / 4), d = i % (D / 4) * 4;
                    float mm, ll;
                    float4 v;
                    join(first, 1, in_bunch, h, d, mm, ll, v);
                    if (bunches == 1) {
                        answer(h, d, mm, ll, v);
                    } else {
                        // it goes to the first part's place, once every thread has read that
                        *reinterpret_cast<float4 *>(s_o + h * C::kOPitch + d) = v;
                        if (d == 0) s_mm[h] = mm, s_ll[h] = ll;
                    }
                }
                if (bunches > 1) {
                    __syncthreads();
                    for (int i = tid; i < quads; i += kThreads) {
                        const int h = i / (D / 4), d = i % (D / 4) * 4;
                        leave(part(first), h, d, s_mm[h], s_ll[h], own(h, d));
                    }
                    if (last_of(p.tickets + 2 * kMaxGrid + slot_of(c0), bunches)) {
                        for (int i = tid; i < quads; i += kThreads) {
                            const int h = i / (D / 4), d = i % (D / 4) * 4;
                            float mm, ll;
                            float4 v;
                            join(c0, bunch, bunches, h, d, mm, ll, v);
                            answer(h, d, mm, ll, v);
                        }
                    }
                }
            }
        }
        __syncthreads();

        left -= seg + C::kEndUnits;
        item0 += wk.units + C::kEndUnits;
        if (left > 0) {
            wk.unit = wk.units - 1;
            advance(p, wk);
        }
    }
    cp_async_wait<0>();
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

// Query heads that share one pass over the keys and values: 8, or 16 where a group has more than
// 8 and the cache is long (`units` of 64 tokens, over all sequences, key heads and 16 heads).  Then
// half as many bytes count; in a short one more items of half the work do.  At 256 dimensions 16
// heads' sums would not fit the registers.  With 16 and 8, 64 / 4 heads of 128 dimensions: 86 and 97 us
// for 48 sequences (36,000 units), 70.6 and 74.7 for 16 (24,000), 41 and 40 (12,000), 28.5 and 25.5
// (6,000), 17.5 and 13.9 for two (400).
int tiles_of(int group, int head_dim, int64_t units) { return head_dim <= 128 && group > 8 && units > 10000 ? 2 : 1; }

template <int D, int NT>
q8_status launch(const AttnParams &p, int64_t most_units, const DeviceInfo *di, cudaStream_t stream) {
    using C = Cfg<D, NT>;
    static std::atomic<int> per_sm[64];
    int n = di->device < 64 ? per_sm[di->device].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kernel<D, NT>, kThreads, C::kSmem) != cudaSuccess)
            return Q8_ERR_CUDA;
        if (n < 1) return Q8_ERR_UNSUPPORTED;
        if (di->device < 64) per_sm[di->device].store(n, std::memory_order_relaxed);
    }
    int64_t grid = static_cast<int64_t>(n) * di->sm_count;
    if (grid > kMaxGrid) grid = kMaxGrid;
    const int64_t need = (most_units + kMinUnits - 1) / kMinUnits;
    if (grid > need) grid = need;
    if (grid < 1) grid = 1;
    attn_kernel<D, NT><<<static_cast<unsigned>(grid), kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace

// Counters, then two partial results per CTA.
size_t attn_workspace(int q_heads, int kv_heads, int head_dim) {
    const int hg = 8 * tiles_of(q_heads / kv_heads, head_dim, INT64_MAX);
    return kTicketBytes + static_cast<size_t>(2) * kMaxGrid * hg * (head_dim + 2) * 4;
}

q8_status launch_attn(const q8_kv_cache &c, const AttnArgs &a, void *ws, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    const WsRange counters = {0, kTicketBytes};
    const WsRange data = {kTicketBytes, attn_workspace(a.q_heads, c.kv_heads, c.head_dim) - kTicketBytes};
    const q8_status st = claim_workspace(ws, &counters, 1, &data, 1, stream);
    if (st != Q8_OK) return st;
    AttnParams p = {};
    p.kq = c.kq, p.vq = c.vq, p.ks = c.ks, p.vs = c.vs;
    p.q = a.q, p.table = a.table, p.lens = a.lens, p.out = a.out, p.lse = a.lse;
    p.tickets = static_cast<uint32_t *>(ws);
    p.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kTicketBytes);
    p.status = dev_status;
    p.ldq = a.ldq;
    p.batch = a.batch, p.q_heads = a.q_heads, p.kv_heads = c.kv_heads;
    p.group = a.q_heads / c.kv_heads;
    p.table_width = a.table_width, p.pages = c.pages, p.page_shift = ilog2(c.page_size);
    // c tanh(s / c) is s (1 - (s / c)^2 / 3 + ...): from c = 2^40 on s itself for every score that binary32 can
    // tell from its neighbours by less than 2^4 (and c log2(e) would overflow near the end of the range)
    p.window = a.window, p.scale = a.scale, p.softcap = a.softcap < 0x1p40f ? a.softcap : 0.f;
    int64_t span = static_cast<int64_t>(a.table_width) * c.page_size;
    const int64_t reach = int64_t{a.window} + 15;  // a window may begin anywhere in a tile
    if (a.window > 0 && span > reach) span = reach;
    const int64_t units = (span + kUnitTokens - 1) / kUnitTokens * a.batch * p.kv_heads;
    const int nt = tiles_of(p.group, c.head_dim, units * ((p.group + 15) / 16));
    p.splits = (p.group + 8 * nt - 1) / (8 * nt);
    const int64_t most = units * p.splits;
    if (c.head_dim == 64) return nt == 1 ? launch<64, 1>(p, most, di, stream) : launch<64, 2>(p, most, di, stream);
    if (c.head_dim == 128) return nt == 1 ? launch<128, 1>(p, most, di, stream) : launch<128, 2>(p, most, di, stream);
    return launch<256, 1>(p, most, di, stream);
}

}  // namespace q8
