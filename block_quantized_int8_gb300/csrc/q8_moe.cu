// q8_moe.cu -- a mixture-of-experts layer for a few tokens (T <= 32) in one
// kernel: routing, gate and up products with SwiGLU, down products, and the
// weighted sum over each token's experts.
//
// Mathematics.  Token t takes the top_k experts of largest logit (ties: the
// lower index), w_j = exp(l_j - l_max) / z with z summed over the chosen (or
// all) experts; y_t = sum_j w_j W2_e(silu(W1_e x_t) * (W3_e x_t)).
//
// Bound: the chosen experts' weights, 1.0625 bytes each, read once for all
// tokens that chose them (for up to 16; an expert with more is read again,
// from L2).  Both products are streams of 16-row weight tiles against a few
// tokens' vectors: m16n8k16 warp MMAs of 16 weight rows by 8 tokens, one block
// of 32 columns at a time, whose fp32 result is multiplied by the block's
// scale as in the matmuls.  Measured: 32 tokens, 8 of 128 experts of 2048 x 1024,
// 147 us (748 MB, 5.1 TB/s; the product loops run at 6); 7 tokens, 6 of 64 of 2048 x
// 1376, 69 us (286 MB); one token, 2 of 16 of 1536 x 4096, 21 us (40 MB), most of it
// the routing, the vectors and the waits between products.
//
// One CTA of 16 warps per SM.  The tokens' vectors of an expert lie in shared
// memory as binary16 for as long as the CTA works on it; weights come through
// a ring of each warp's own (16-byte asynchronous copies of 16 rows x 128
// columns), so warps wait for one another only where the CTA moves on past
// the experts it has in shared memory.  (A first form with the vectors in the
// ring, and so a CTA barrier per 128 columns, took 2.4 times as long.)  The host
// does not know which experts are chosen: every CTA works the routing out for
// itself from the logits and cuts the same lists of tasks into equal runs.  Between
// the products, and before the sum, all CTAs wait for one another (a cooperative
// launch): as three kernels the call took 157 us in place of 152 for 32 tokens, most
// of the difference each kernel's own beginning.  (Waiting only for the neighbours that
// made a CTA's hidden units was slower, 153 us against 149: CTAs that are ahead take
// bandwidth from those behind.)
// Where a CTA's tasks do not fill its warps evenly, 2, 4 or 8 warps share one,
// each a range of its columns.
//
// gate/up: a task is 8 hidden units of one expert: MMA rows 0..7 are
// their gate rows, 8..15 their up rows, so a thread holds both factors of its
// unit and SwiGLU needs no exchange.  x (bf16) is scaled by a power of two per
// token to a largest value in [2^14, 2^15): exact in binary16 down to 2^-31 of it, and off by at
// most 2^-39 of it below.
// Hidden units go to the workspace in fp32.
// down: a task is 16 output rows of one expert over a segment of its hidden
// units.  The hidden units, scaled likewise per token and segment,
// are taken as the sum of two binary16 values (22 bits), so fp32 outputs keep
// their digits.  Each task leaves its tokens' rows in the workspace, and
// they are added up in the order of the token's experts and segments.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "q8_async.cuh"
#include "q8_dev.cuh"
#include "q8_internal.h"

namespace q8 {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxT = 32;
constexpr int kMaxE = 512;
constexpr int kMaxPairs = kMaxT * 16;  // tokens x chosen experts
constexpr int kGroup = 16;             // most tokens of an entry: an expert with more is listed again
constexpr int kNT = kGroup / 8;        // MMA tiles of 8 tokens
constexpr int kMaxEntries = kMaxE + kMaxPairs / 8;
constexpr int kChunk = 128;            // columns of a stage
constexpr int kBlocks = kChunk / 32;
constexpr int kTile = 16 * kChunk;     // bytes of a warp's codes in a stage
constexpr int kScalePitch = 16;        // a row's scales take up to 12 bytes
constexpr int kStage = kTile + 16 * kScalePitch;
constexpr int kMaxStages = 8;
constexpr int kSmem = 227 * 1024 - 7 * 1024;  // beside the routing
constexpr int kJoin = kWarps * 32 * 4 * kNT * 4;  // sums of warps that share a task
// What the vectors of one entry may take: two stages of every warp stay beside them.
constexpr int kMostX = kSmem - kWarps * 2 * kStage;

struct MoeParams {
    const uint16_t *x;      // bf16 [T][ldx]
    const float *logits;    // [T][ldl]
    const int8_t *q13, *q2;
    const uint16_t *s13, *s2;
    float *y;               // [T][ldy]
    int32_t *ids;           // [T][top_k] or null
    float *weights;         // [T][top_k] or null
    float *hidden;          // [pairs][F]
    float *z;               // [segments][pairs][H]: the experts' outputs
    uint32_t *counters;     // CTAs that have made their hidden units, and their outputs
    uint32_t *status;
    int64_t ldx, ldl, ldy;
    int32_t T, E, H, F, top_k, renorm;
    int32_t cap;            // tokens of an entry: 8 or 16
};

// The routing: entries of an expert and up to `cap` of its tokens, by expert,
// then token; a pair is a token of an entry.
struct alignas(16) Routing {
    uint16_t expert[kMaxEntries];
    uint16_t base[kMaxEntries + 1];  // first pair of each entry
    uint8_t token[kMaxPairs];        // the pairs' tokens
    int16_t pair[kMaxPairs];         // [T][top_k]: the pair of each choice, -1 for none
    float w[kMaxPairs];              // [T][top_k]: its weight
    int32_t used;                    // entries
    int32_t most;                    // tokens of the largest
};
// What only making it needs; lies where the ring comes later.
struct Making {
    uint32_t mask[kMaxE];    // tokens that chose the expert
    uint16_t first[kMaxE];   // first pair of the expert
    int16_t id[kMaxPairs];   // [T][top_k]
};

// A total order of floats as unsigned integers; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

// One warp's token: its top_k experts by repeated maximum of NK keys a lane (v: the logits of
// experts lane, lane + 32, ...; -inf past the last).
template <int NK>
__device__ void route_token(const MoeParams &p, Routing &r, Making &mk, int t, const float (&v)[NK], bool report) {
    const int lane = threadIdx.x & 31;
    uint32_t key[NK];
    bool nan = false;
    // this lane's best: the largest key, the lowest index of equal ones
    uint32_t m = 0;
    int mi = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        nan = nan || v[i] != v[i];
        key[i] = order_key(v[i]);
        if (key[i] > m) m = key[i], mi = lane + 32 * i;
    }
    if (report && __any_sync(0xffffffffu, nan) && lane == 0 && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
    uint32_t got = 0;  // lane j: the j-th choice
    int id = -1;
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, m);
        if (best <= kKeyNegInf) break;  // nothing left to choose
        const uint32_t who = __ballot_sync(0xffffffffu, m == best);
        int e;
        if (who & (who - 1))  // equal logits in several lanes
            e = __reduce_min_sync(0xffffffffu, m == best ? mi : kMaxE);
        else
            e = __shfl_sync(0xffffffffu, mi, __ffs(who) - 1);
        if (lane == j) got = best, id = e;
        if (m == best && mi == e) {  // its lane takes it out
            m = 0;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                if (lane + 32 * i == e) key[i] = 0;
                if (key[i] > m) m = key[i], mi = lane + 32 * i;
            }
        }
    }
    const float l = __uint_as_float((got & 0x80000000u) ? got ^ 0x80000000u : ~got);
    const float top = __shfl_sync(0xffffffffu, l, 0);
    const float mine = id < 0 ? 0.f : (l == top ? 1.f : expf(l - top));
    float z = mine;
    if (!p.renorm) {
        z = 0.f;
#pragma unroll
        for (int i = 0; i < NK; ++i)
            if (lane + 32 * i < p.E && v[i] == v[i]) z += v[i] == top ? 1.f : expf(v[i] - top);
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane < p.top_k) {
        mk.id[t * p.top_k + lane] = static_cast<int16_t>(id);
        r.w[t * p.top_k + lane] = id < 0 ? 0.f : __fdiv_rn(mine, z);
        if (id >= 0) atomicOr(&mk.mask[id], 1u << t);
    }
}

template <int NK>
__device__ void route_tokens(const MoeParams &p, Routing &r, Making &mk, bool report) {
    static_assert(kMaxT <= 2 * kWarps, "a warp routes at most two tokens");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v[2][NK];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < NK; ++i)
            v[q][i] = warp + q * kWarps < p.T && lane + 32 * i < p.E ? p.logits[(warp + q * kWarps) * p.ldl + lane + 32 * i] : -INFINITY;
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
        if (warp + q * kWarps >= p.T) break;
        route_token<NK>(p, r, mk, warp + q * kWarps, v[0], report);
#pragma unroll
        for (int i = 0; i < NK; ++i) v[0][i] = v[1][i];
    }
}

__device__ void route(const MoeParams &p, Routing &r, Making &mk, bool report) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < p.E; e += kThreads) mk.mask[e] = 0;
    __syncthreads();
    if (p.E <= 32)
        route_tokens<1>(p, r, mk, report);
    else if (p.E <= 128)
        route_tokens<4>(p, r, mk, report);
    else
        route_tokens<kMaxE / 32>(p, r, mk, report);
    __syncthreads();
    if (warp == 0) {  // a lane takes `each` neighbouring experts
        const int each = (p.E + 31) / 32, e0 = lane * each, e1 = min(e0 + each, p.E);
        int n = 0, parts = 0, most = 0;
        for (int e = e0; e < e1; ++e) {
            const int k = __popc(mk.mask[e]);
            n += k, parts += (k + p.cap - 1) / p.cap, most = max(most, min(k, p.cap));
        }
        int run = n, erun = parts;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o), ev = __shfl_up_sync(0xffffffffu, erun, o);
            if (lane >= o) run += v, erun += ev;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 31) {
            r.base[erun] = static_cast<uint16_t>(run);
            r.used = erun;
            r.most = most;
        }
        int at = erun - parts, pair = run - n;
        for (int e = e0; e < e1; ++e) {
            const int k = __popc(mk.mask[e]);
            mk.first[e] = static_cast<uint16_t>(pair);
            for (int i = 0; i < k; i += p.cap, ++at) {
                r.expert[at] = static_cast<uint16_t>(e);
                r.base[at] = static_cast<uint16_t>(pair + i);
            }
            pair += k;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * p.top_k; i += kThreads) {
        const int e = mk.id[i], t = i / p.top_k;
        int at = -1;
        if (e >= 0) {
            at = mk.first[e] + __popc(mk.mask[e] & ((1u << t) - 1));
            r.token[at] = static_cast<uint8_t>(t);
        }
        r.pair[i] = static_cast<int16_t>(at);
    }
    __syncthreads();
}

// Chunk c (16 bytes) of a weight tile's row r: placed so that the MMA operand
// reads hit every bank once.
__device__ __forceinline__ uint32_t weight_at(int r, int c) { return (r * 8 + (c ^ ((r & 3) << 1))) * 16; }
// Bytes from one token's vector to the next, for the same reason: 64 past a multiple of 128
// for 2-byte values, 16 past one for the two parts of a value (4 bytes).
template <bool DOWN>
__device__ __forceinline__ int pitch_of(int columns) {
    return DOWN ? columns * 4 + 16 : columns * 2 + ((columns * 2) % 128 == 0 ? 64 : 0);
}

// A warp's weight tiles as they come: 16 rows (8 from row0, 8 from row8) of a
// [rows][K] matrix, 128 columns at a time.  Pointers move with the columns.
struct TileLoad {
    const int8_t *a, *b;   // this lane's place in rows 0..7 and 8..15
    const uint16_t *s;     // this lane's row of scales (lanes 0..15), at the stage's columns
    int64_t row0, row8;
    int col;

    __device__ __forceinline__ void begin(const int8_t *q, const uint16_t *sc, int64_t r0, int64_t r8, int K, int c0, int lane) {
        row0 = r0, row8 = r8, col = c0;
        a = q + (r0 + (lane >> 3)) * K + c0 + (lane & 7) * 16;
        b = q + (r8 + (lane >> 3)) * K + c0 + (lane & 7) * 16;
        s = sc + (lane < 8 ? r0 + lane : r8 + (lane & 7)) * (K >> 5) + (c0 >> 5);
    }
    // codes: this lane's first chunk in the stage; scales: the warp's
    __device__ __forceinline__ void load(uint32_t codes, uint32_t scales, const uint16_t *sc, int K, int lane) {
        if (col + (lane & 7) * 16 < K) {
            cp_async16(codes, a);
            cp_async16(codes + 4 * kChunk, a + 4 * K);
            cp_async16(codes + 8 * kChunk, b);
            cp_async16(codes + 12 * kChunk, b + 4 * K);
        }
        if ((K & (kChunk - 1)) == 0) {
            if (lane < 16) cp_async8(scales + lane * kScalePitch, s);
        } else {
            // rows of scales start at any 2-byte offset: take the aligned words
            // that hold this chunk's (the array ends on a word: rows % 32 == 0)
            constexpr int kWords = kBlocks / 2 + 1;
            const int nb = K >> 5, words = min(kWords, (min(kBlocks, nb - (col >> 5)) + 2) >> 1);
#pragma unroll
            for (int i = 0; i < (16 * kWords + 31) / 32; ++i) {
                const int j = i * 32 + lane;
                const int r = j / kWords, wd = j - r * kWords;
                if (r < 16 && wd < words) {
                    const int64_t row = r < 8 ? row0 + r : row8 + (r - 8);
                    const int64_t at = (row * nb + (col >> 5)) & ~int64_t(1);
                    if (at + wd * 2 < (row + 1) * nb) cp_async4(scales + r * kScalePitch + wd * 4, sc + at + wd * 2);
                }
            }
        }
        a += kChunk, b += kChunk, s += kBlocks, col += kChunk;
    }
};

// The scales of a row's chunk, as pairs.
struct Scales {
    uint32_t w[kBlocks / 2];
    __device__ __forceinline__ void get(uint32_t at, bool odd) {
        const uint4 a = lds128(at);
        w[0] = odd ? __funnelshift_r(a.x, a.y, 16) : a.x;
        w[1] = odd ? __funnelshift_r(a.y, a.z, 16) : a.y;
    }
    __device__ __forceinline__ float of(int b) const {
        const __half2 h = *reinterpret_cast<const __half2 *>(&w[b >> 1]);
        return (b & 1) ? __high2float(h) : __low2float(h);
    }
};

// Waits until at most n (below kMaxStages) of this thread's last groups of copies are under way.
__device__ __forceinline__ void wait_but(int n) {
    switch (n) {
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    case 6: cp_async_wait<6>(); break;
    case 7: cp_async_wait<7>(); break;
    default: cp_async_wait<0>();
    }
}

constexpr int kRow8 = 8 * kChunk;  // from a tile's row g to row g + 8
// 16 rows x 32 columns of codes as two binary16 MMA operands (8 columns a lane).
struct Codes {
    uint32_t a[4], b[4];
    __device__ __forceinline__ void get(uint32_t at) {
        const uint2 w0 = lds64(at), w1 = lds64(at + kRow8);
        codes4_to_f16x2(w0.x, a[0], a[2]);
        codes4_to_f16x2(w1.x, a[1], a[3]);
        codes4_to_f16x2(w0.y, b[0], b[2]);
        codes4_to_f16x2(w1.y, b[1], b[3]);
    }
    // d = (these codes) x, x this lane's 8 values
    __device__ __forceinline__ void mul(float *d, const uint4 &x) const {
        mma_f16_16816_new(d[0], d[1], d[2], d[3], a[0], a[1], a[2], a[3], x.x, x.y);
        mma_f16_16816(d[0], d[1], d[2], d[3], b[0], b[1], b[2], b[3], x.z, x.w);
    }
    // the same with x in two parts: values 0..3 (high, low), then 4..7
    __device__ __forceinline__ void mul2(float *d, const uint4 &x, const uint4 &y) const {
        float l[4];
        mma_f16_16816_new(d[0], d[1], d[2], d[3], a[0], a[1], a[2], a[3], x.x, x.y);
        mma_f16_16816_new(l[0], l[1], l[2], l[3], a[0], a[1], a[2], a[3], x.z, x.w);
        mma_f16_16816(d[0], d[1], d[2], d[3], b[0], b[1], b[2], b[3], y.x, y.y);
        mma_f16_16816(l[0], l[1], l[2], l[3], b[0], b[1], b[2], b[3], y.z, y.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += l[i];
    }
};
// 2^(14 - e) and 2^(e - 14) for a largest magnitude m of exponent e: m goes to [2^14, 2^15)
// (zero, subnormal and non-finite m keep factors in range)
__device__ __forceinline__ int scale_exponent(float m) { return min(max(static_cast<int>(__float_as_uint(m) >> 23), 30), 254); }
__device__ __forceinline__ float scale_up(int ex) { return __uint_as_float(static_cast<uint32_t>(268 - ex) << 23); }
__device__ __forceinline__ float scale_down(int ex) { return __uint_as_float(static_cast<uint32_t>(ex - 14) << 23); }


// A stage: acc += (tile) x for N MMA tiles of tokens; x is this lane's place in the vectors (token
// g, its 8 of each block's columns), tok8 on for token g + 8.  ALL: the stage holds kBlocks blocks
// (no test in the way of overlapping them).
template <bool DOWN, int N, bool ALL>
__device__ __forceinline__ void stage_product(uint32_t codes, const uint32_t (&code_at)[kBlocks], const Scales &s0, const Scales &s1,
                                              int nb, uint32_t x, int tok8, float (&acc)[kNT][4]) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        if (!ALL && b >= nb) break;
        Codes w;
        w.get(codes + code_at[b]);
        const float f0 = s0.of(b), f1 = s1.of(b);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float d[4];
            const uint32_t from = x + b * (DOWN ? 128 : 64) + i * tok8;
            if constexpr (DOWN)
                w.mul2(d, lds128(from), lds128(from + 16));
            else
                w.mul(d, lds128(from));
            acc[i][0] = fmaf(f0, d[0], acc[i][0]);
            acc[i][1] = fmaf(f0, d[1], acc[i][1]);
            acc[i][2] = fmaf(f1, d[2], acc[i][2]);
            acc[i][3] = fmaf(f1, d[3], acc[i][3]);
        }
    }
}

// A token's x in shared memory, bf16 as copied there, to binary16 of x 2^(14 - e) in place (a
// warp's work; loops are kept short: this code runs once, and what it costs is fetching it).
__device__ int scale_x(uint32_t at, int n) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;  // the largest magnitude's bits, in either half
#pragma unroll 2
    for (int c = lane; c < n / 8; c += 32) {
        const uint4 v = lds128(at + c * 16);
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    }
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    const int e = scale_exponent(__uint_as_float(m << 16));
    const float up = scale_up(e);
#pragma unroll 2
    for (int c = lane; c < n / 8; c += 32) {
        const uint4 v = lds128(at + c * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f32x2_to_f16x2(bf16lo_f32(w[i]) * up, bf16hi_f32(w[i]) * up);
        sts128(at + c * 16, make_uint4(h[0], h[1], h[2], h[3]));
    }
    return e;
}
// Hidden units likewise: four fp32 values become their four high parts and four low parts.
__device__ int scale_hidden(uint32_t at, int n) {
    const int lane = threadIdx.x & 31;
    float m = 0.f;
#pragma unroll 2
    for (int c = lane; c < n / 4; c += 32) {
        const uint4 v = lds128(at + c * 16);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))),
                           fmaxf(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w)))));
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = scale_exponent(m);
    const float up = scale_up(e);
#pragma unroll 2
    for (int c = lane; c < n / 4; c += 32) {
        const uint4 v = lds128(at + c * 16);
        const float x[4] = {__uint_as_float(v.x) * up, __uint_as_float(v.y) * up, __uint_as_float(v.z) * up, __uint_as_float(v.w) * up};
        uint32_t h[2], l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[i] = f32x2_to_f16x2(x[2 * i], x[2 * i + 1]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            l[i] = f32x2_to_f16x2(x[2 * i] - f.x, x[2 * i + 1] - f.y);
        }
        sts128(at + c * 16, make_uint4(h[0], h[1], l[0], l[1]));
    }
    return e;
}

// Hidden units of a segment of the down product: F in equal parts (of whole chunks) of at most
// 1024, or 512 where an entry has more than 8 tokens (whose vectors take twice the room); up
// to 1536 units are one segment.  At 1376 units one takes 71.7 us and two 74.7 (7 tokens, 6
// of 64 experts); at 4096, where more rows of vectors are waited for at once, parts of 1024
// take 59.3 and of 1408 61.1, of 2048 65 (32 tokens, 2 of 8); parts of 512 were 4 to 12 % slower
// than of 1024 everywhere.
__device__ __forceinline__ int segment_of(int most, int F) {
    const int n = most > 8 ? (F + 511) / 512 : (F <= 1536 ? 1 : (F + 1023) / 1024);
    return ((F + n - 1) / n + kChunk - 1) / kChunk * kChunk;
}

// One of the two products.  `ready` is called, by every thread, once the first weights are on
// their way, and says whether what the vectors are made of is there (false: give up).
template <bool DOWN, typename Ready>
__device__ __forceinline__ bool phase(const MoeParams &p, const Routing &r, int (&s_ex)[2][kGroup], uint8_t *smem, Ready ready) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // ---- the list of tasks: group (an entry, for DOWN with a segment) major, then tiles of rows --
    const int K = DOWN ? p.F : p.H;                          // columns of the weights
    const int rows8 = (r.most + 7) & ~7;
    const int seg = DOWN ? segment_of(r.most, K) : K;        // columns of a group
    const int nseg = (K + seg - 1) / seg;
    const int tiles = DOWN ? p.H / 16 : p.F / 8;
    const int groups = r.used * nseg;
    const uint32_t tasks = static_cast<uint32_t>(groups) * tiles;
    const uint32_t run = tasks / gridDim.x, more = tasks - run * gridDim.x;  // the first `more` CTAs take one more
    const uint32_t t0 = run * blockIdx.x + min(blockIdx.x, more), t1 = t0 + run + (blockIdx.x < more ? 1 : 0);
    if (t0 >= t1) return ready();
    const int mine = static_cast<int>(t1 - t0);

    // ---- shared memory: one or two groups' vectors, the ring, sums of warps that share ------------
    const int pitch = pitch_of<DOWN>(DOWN ? seg : K), tok8 = 8 * pitch, x_bytes = rows8 * pitch;
    // warps to a task: what makes the rounds of tasks shortest, a chunk's time for joining included
    // (one token, 2 of 16 experts of 1536 x 4096: 22.6 us, and 25.0 with one warp to a task)
    int share = 1;
    {
        const int chunks = (min(seg, K) + kChunk - 1) / kChunk;
        int best = (mine + kWarps - 1) / kWarps * chunks;
        for (int s = 2; s <= 8; s *= 2) {
            const int cost = (mine * s + kWarps - 1) / kWarps * ((chunks + s - 1) / s + 1);
            if (cost < best && x_bytes + kJoin + kWarps * 2 * kStage <= kSmem) best = cost, share = s;
        }
    }
    const int teams = kWarps / share, team = warp / share, part = warp - team * share;
    const int join = share > 1 ? kJoin : 0;
    const int busy = min(mine, teams) * share;
    // two groups' vectors where the ring keeps three stages: half as many waits for the whole CTA (7
    // tokens, 6 of 64 experts: 75 us and with one 83; 32 tokens, 8 of 128: 151 and 162)
    const int bufs = 2 * x_bytes + join + busy * 3 * kStage <= kSmem ? 2 : 1;
    const int stages = min((kSmem - bufs * x_bytes - join) / (busy * kStage), kMaxStages);
    const uint32_t xs = smem_addr(smem), ring = xs + bufs * x_bytes + warp * stages * kStage, ring_end = ring + stages * kStage;
    float *const s_join = reinterpret_cast<float *>(smem + bufs * x_bytes + busy * stages * kStage);
    const bool works = team < mine;

    // ---- this warp's weights: tasks team, team + teams, ...; of each group's columns its share ----
    auto chunk0 = [&](int columns) { return (columns + kChunk - 1) / kChunk * part / share; };
    auto chunk1 = [&](int columns) { return (columns + kChunk - 1) / kChunk * (part + 1) / share; };
    struct At {
        int task;          // of this CTA
        int group, tile;
    };
    auto enter = [&](At &a) {
        const uint32_t n = t0 + a.task;
        a.group = static_cast<int>(n / tiles);
        a.tile = static_cast<int>(n - a.group * tiles);
    };
    auto next = [&](At &a) {
        a.task += teams;
        a.tile += teams;
        while (a.tile >= tiles) a.tile -= tiles, ++a.group;
    };
    auto columns_of = [&](int group) { return DOWN ? min(seg, K - group % nseg * seg) : K; };
    At ld = {team, 0, 0};
    if (works) enter(ld);
    TileLoad tile;
    int ld_left = 0;  // chunks of the task still to load; 0: begin the next
    uint32_t ld_at = ring;
    const uint32_t code_to = weight_at(lane >> 3, lane & 7);
    const int8_t *const q = DOWN ? p.q2 : p.q13;
    const uint16_t *const sc = DOWN ? p.s2 : p.s13;
    auto load = [&]() {
        while (ld_left == 0 && ld.task < mine) {
            const int cols = columns_of(ld.group), c0 = chunk0(cols);
            ld_left = chunk1(cols) - c0;
            const int64_t e = r.expert[DOWN ? ld.group / nseg : ld.group];
            const int from = (DOWN ? ld.group % nseg * seg : 0) + c0 * kChunk;
            if constexpr (DOWN) {
                const int64_t row = e * p.H + ld.tile * 16;
                tile.begin(q, sc, row, row + 8, K, from, lane);
            } else {
                const int64_t row = e * 2 * p.F + ld.tile * 8;
                tile.begin(q, sc, row, row + p.F, K, from, lane);
            }
            next(ld);
        }
        if (ld_left > 0) {
            tile.load(ld_at + code_to, ld_at + kTile, sc, K, lane);
            --ld_left;
        }
        ld_at = ld_at + kStage == ring_end ? ring : ld_at + kStage;
        cp_async_commit();
    };
    auto begin = [&]() {
        if (works)
#pragma unroll 1
            for (int i = 0; i < stages - 1; ++i) load();
    };

    uint32_t code_at[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) code_at[b] = weight_at(g, 2 * b + (t >> 1)) + (t & 1) * 8;
    // rows of a tile start at even places, so the parity of a row's first scale is that of g
    const bool odd = ((K >> 5) & 1) != 0 && (g & 1);
    uint32_t at = ring;
    At now = {team, 0, 0};
    enter(now);
    const int g_first = static_cast<int>(t0 / tiles), g_last = static_cast<int>((t1 - 1) / tiles);
    for (int gb = g_first; gb <= g_last; gb += bufs) {
        // ---- the vectors of groups gb .. gb + bufs - 1, a warp a token -----------------------------
        if (gb != g_first) __syncthreads();  // nobody reads the ones before any more
        if (DOWN && gb == g_first) {  // weights first: these vectors are not there yet
            begin();
            if (!ready()) {
                cp_async_wait<0>();
                return false;
            }
        }
        auto vectors = [&](auto take) {
#pragma unroll 1
            for (int i = warp; i < bufs * rows8; i += kWarps) {
                const int buf = i >= rows8 ? 1 : 0, k = i - buf * rows8, group = gb + buf;
                if (group > g_last) break;
                const int entry = DOWN ? group / nseg : group, base = r.base[entry];
                if (k < r.base[entry + 1] - base) take(buf, k, group, base + k, xs + buf * x_bytes + k * pitch);
            }
        };
        vectors([&](int, int, int group, int pr, uint32_t to) {
            const void *from;
            int n;  // 16-byte copies
            if constexpr (DOWN) {
                from = p.hidden + static_cast<int64_t>(pr) * p.F + group % nseg * seg;
                n = columns_of(group) / 4;
            } else {
                from = p.x + r.token[pr] * p.ldx;
                n = p.H / 8;
            }
#pragma unroll 1
            for (int c = lane; c < n; c += 32) cp_async16(to + c * 16, static_cast<const uint4 *>(from) + c);
        });
        cp_async_commit();
        if (!DOWN && gb == g_first) {  // vectors first: they need not wait for the weights behind them
            begin();
            wait_but(works ? stages - 1 : 0);
        } else {
            cp_async_wait<0>();
        }
        __syncwarp();
        vectors([&](int buf, int k, int group, int, uint32_t to) {
            const int e = DOWN ? scale_hidden(to, columns_of(group)) : scale_x(to, p.H);
            if (lane == 0) s_ex[buf][k] = e;
        });
        __syncthreads();

        for (; now.task < mine && now.group < gb + bufs; next(now)) {
            const int entry = DOWN ? now.group / nseg : now.group;
            const int base = r.base[entry], n = r.base[entry + 1] - base, buf = now.group - gb;
            const int cols = columns_of(now.group), c0 = chunk0(cols), c1 = chunk1(cols);
            uint32_t x = xs + buf * x_bytes + g * pitch + (t * 16 + c0 * (kChunk * 2)) * (DOWN ? 2 : 1);
            float acc[kNT][4];
#pragma unroll
            for (int i = 0; i < kNT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            for (int c = c0; c < c1; ++c) {
                wait_but(stages - 2);
                __syncwarp();
                load();  // into the stage that the step before this one read
                Scales s0, s1;
                s0.get(at + kTile + g * kScalePitch, odd);
                s1.get(at + kTile + (g + 8) * kScalePitch, odd);
                const int nb = min(kBlocks, (cols >> 5) - c * kBlocks);
                if (n <= 8)
                    nb == kBlocks ? stage_product<DOWN, 1, true>(at, code_at, s0, s1, nb, x, tok8, acc)
                                  : stage_product<DOWN, 1, false>(at, code_at, s0, s1, nb, x, tok8, acc);
                else  // one form: a second would cost the others more, in instructions to fetch, than it gives
                    stage_product<DOWN, kNT, false>(at, code_at, s0, s1, nb, x, tok8, acc);
                x += kChunk * (DOWN ? 4 : 2);
                at = at + kStage == ring_end ? ring : at + kStage;
            }
            if (share > 1) {  // add the shares up, in the order of the columns
                float *const to = s_join + (warp * 32 + lane) * 4 * kNT;
                auto meet = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * share) : "memory"); };
                if (part > 0) {
#pragma unroll
                    for (int i = 0; i < kNT; ++i) *reinterpret_cast<float4 *>(to + 4 * i) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                }
                meet();
                if (part == 0) {
                    for (int w = 1; w < share; ++w)
#pragma unroll
                        for (int i = 0; i < kNT; ++i) {
                            const float4 v = *reinterpret_cast<const float4 *>(to + w * 32 * 4 * kNT + 4 * i);
                            acc[i][0] += v.x, acc[i][1] += v.y, acc[i][2] += v.z, acc[i][3] += v.w;
                        }
                }
                meet();
                if (part > 0) continue;
            }
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = i * 8 + 2 * t + j;
                    if (k < n) {
                        const float down = scale_down(s_ex[buf][k]);
                        const float v0 = acc[i][j] * down, v1 = acc[i][2 + j] * down;
                        if constexpr (DOWN) {
                            float *const to = p.z + (static_cast<int64_t>(now.group % nseg) * (p.T * p.top_k) + base + k) * p.H +
                                              now.tile * 16 + g;
                            to[0] = v0;
                            to[8] = v1;
                        } else {
                            p.hidden[static_cast<int64_t>(base + k) * p.F + now.tile * 8 + g] = v0 / (1.0f + expf(-v0)) * v1;
                        }
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    return true;
}

// ---- all CTAs of the launch (a cooperative one: they all run) --------------------------------------
__device__ __forceinline__ void arrive(uint32_t *counter) {
    __syncthreads();
    if (threadIdx.x == 0) asm volatile("red.add.release.gpu.global.u32 [%0], 1;" ::"l"(counter) : "memory");
}
__device__ __forceinline__ bool wait_all(const uint32_t *counter, uint32_t *status, int &s_ok) {
    if (threadIdx.x == 0) {
        const uint64_t begun = globaltimer_ns();
        uint32_t n;
        bool late = false;
        while (true) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(counter) : "memory");
            if (n >= gridDim.x) break;
            if (globaltimer_ns() - begun > kWaitLimitNs) {
                late = true;
                break;
            }
        }
        if (late && status) atomicOr(status, Q8_DEV_TIMEOUT);
        s_ok = late ? 0 : 1;
    }
    __syncthreads();
    return s_ok != 0;
}

__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Routing r;
    __shared__ int s_ex[2][kGroup];  // the exponents that the vectors in shared memory were scaled by
    __shared__ int s_ok[2];
    const int tid = threadIdx.x;
    // counters[0] is zero here; counters[1] is what the call before left, and nobody counts with it
    // until this CTA has arrived at counters[0]
    if (blockIdx.x == 0 && tid == 0) p.counters[1] = 0;
    Making &mk = *reinterpret_cast<Making *>(smem);
    route(p, r, mk, blockIdx.x == 0);
    if (blockIdx.x == 0) {
        for (int i = tid; i < p.T * p.top_k; i += kThreads) {
            if (p.ids) p.ids[i] = mk.id[i];
            if (p.weights) p.weights[i] = r.w[i];
        }
        __syncthreads();
    }
    phase<false>(p, r, s_ex, smem, [] { return true; });
    arrive(&p.counters[0]);
    // the down weights come while the last hidden units are made
    if (!phase<true>(p, r, s_ex, smem, [&] { return wait_all(&p.counters[0], p.status, s_ok[0]); })) return;
    arrive(&p.counters[1]);
    const int nseg = (p.F + segment_of(r.most, p.F) - 1) / segment_of(r.most, p.F);
    if (!wait_all(&p.counters[1], p.status, s_ok[1])) return;
    if (blockIdx.x == 0 && tid == 0) p.counters[0] = 0;

    // ---- y_t = the sum over the token's experts and segments, in that order; four columns of one
    // token a thread ----------------------------------------------------------------------------------
    constexpr int kAt = 8;  // summands at once: their loads are under way together
    const int pairs = p.T * p.top_k, quarter = p.H / 4;
    for (int i = blockIdx.x * kThreads + tid; i < p.T * quarter; i += gridDim.x * kThreads) {
        const int t = i / quarter, c = (i - t * quarter) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int choice = 0, seg = 0; choice < p.top_k;) {
            float4 v[kAt];
            float w[kAt];
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int at = choice < p.top_k ? r.pair[t * p.top_k + choice] : -1;
                w[j] = at >= 0 ? r.w[t * p.top_k + choice] : 0.f;
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at >= 0) v[j] = __ldcg(reinterpret_cast<const float4 *>(p.z + (static_cast<int64_t>(seg) * pairs + at) * p.H + c));
                if (++seg == nseg) seg = 0, ++choice;
            }
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (w[j] == 0.f) continue;  // not chosen: its place holds nothing
                sum.x = fmaf(w[j], v[j].x, sum.x), sum.y = fmaf(w[j], v[j].y, sum.y);
                sum.z = fmaf(w[j], v[j].z, sum.z), sum.w = fmaf(w[j], v[j].w, sum.w);
            }
        }
        float *const y = p.y + t * p.ldy + c;
        y[0] = sum.x, y[1] = sum.y, y[2] = sum.z, y[3] = sum.w;  // rows of y are 4-byte aligned
    }
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeLayout {
    size_t hidden, z, total;  // after the counters
};
MoeLayout layout_of(int T, int H, int F, int top_k) {
    const size_t pairs = static_cast<size_t>(T) * top_k, segments = (F + 511) / 512;
    MoeLayout m;
    m.hidden = Q8_MOE_ZEROED_BYTES;  // after the counters
    m.z = m.hidden + up256(pairs * F * 4);
    m.total = m.z + up256(segments * pairs * H * 4);
    return m;
}

static_assert(sizeof(Routing) <= 6 * 1024, "kSmem leaves room for the routing");
static_assert(sizeof(Making) <= kSmem, "the routing is made in the ring's memory");
static_assert(8 * (2 * Q8_MOE_MAX_HIDDEN + 64) <= kMostX, "eight tokens' vectors fit beside two stages of every warp");
static_assert(kGroup * (4 * 512 + 16) <= kMostX && 8 * (4 * 1536 + 16) <= kMostX, "and so does a segment's");

}  // namespace

size_t moe_workspace(int T, int H, int F, int top_k) { return layout_of(T, H, F, top_k).total; }

q8_status launch_moe(const MoeArgs &a, void *ws, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (di->device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(moe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return Q8_ERR_CUDA;
        ready.fetch_or(bit);
    }
    const MoeLayout m = layout_of(a.T, a.H, a.F, a.top_k);
    // counters[0] is zero before and after; counters[1] is left as it is, like data
    const WsRange counters = {0, sizeof(uint32_t)}, data = {sizeof(uint32_t), m.total - sizeof(uint32_t)};
    const q8_status st = claim_workspace(ws, &counters, 1, &data, 1, stream);
    if (st != Q8_OK) return st;
    uint8_t *w = static_cast<uint8_t *>(ws);
    MoeParams p = {};
    p.x = a.x, p.logits = a.logits, p.q13 = a.q13, p.s13 = a.s13, p.q2 = a.q2, p.s2 = a.s2;
    p.y = a.y, p.ids = a.ids, p.weights = a.weights;
    p.counters = reinterpret_cast<uint32_t *>(w);
    p.hidden = reinterpret_cast<float *>(w + m.hidden), p.z = reinterpret_cast<float *>(w + m.z);
    p.status = dev_status;
    p.ldx = a.ldx, p.ldl = a.ldl, p.ldy = a.ldy;
    p.T = a.T, p.E = a.E, p.H = a.H, p.F = a.F, p.top_k = a.top_k, p.renorm = a.renorm;
    // entries of up to 16 tokens where the experts have more than 8 each on the average; else of 8, so
    // that a much liked expert is two entries' work for two CTAs and not a slow one for one (32
    // tokens, 8 of 128 experts: 151 us, 183 with entries of 16; 2 of 8 experts of 1536 x 4096: 59.6 and 60.9)
    p.cap = a.T * a.top_k > 8 * a.E && kGroup * (2 * a.H + 64) <= kMostX ? kGroup : 8;
    const int64_t pairs = static_cast<int64_t>(a.T) * a.top_k, entries = pairs < a.E ? pairs : a.E + pairs / p.cap;
    const int64_t tasks = entries * std::max<int64_t>(a.F / 8, static_cast<int64_t>(a.H / 16) * ((a.F + 511) / 512));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tasks < di->sm_count ? tasks : di->sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // its CTAs wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel, p) == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
