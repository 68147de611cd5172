// q8_moe.cu -- a mixture-of-experts layer for a few tokens (T <= 32) in two
// kernels: routing, gate and up products and SwiGLU in the first; down
// products and the weighted sum over experts in the second.
//
// Mathematics.  Token t takes the top_k experts of largest logit (ties: the
// lower index), w_j = exp(l_j - l_max) / z with z summed over the chosen (or
// all) experts; y_t = sum_j w_j W2_e(silu(W1_e x_t) * (W3_e x_t)).
//
// Bound: the chosen experts' weights, 1.0625 bytes each, read once for all
// tokens that chose them.  Both kernels are streams of 16-row x 256-column
// weight tiles through shared memory (16-byte asynchronous copies, a ring of
// stages per CTA) and m16n8k16 warp MMAs: 16 weight rows by 8 tokens, one
// block of 32 at a time, whose fp32 result is multiplied by the block's scale
// as in the matmuls.  The host does not know which experts are chosen: every
// CTA works the routing out for itself from the logits (a few hundred cycles
// a token) and cuts the same list of work into equal runs.
//
// gate/up kernel: a task is 32 hidden units of one expert, 8 per warp: MMA
// rows 0..7 are gate rows and 8..15 the same units' up rows, so a thread holds
// both factors of its unit and SwiGLU needs no exchange.  x is bf16 as given
// (products exact).
// Between the kernels a hidden unit must not lose what fp32 outputs keep, so
// it is stored as the sum of two binary16 values (22 bits), scaled by a power
// of two per token and block of 32 units.
// down kernel: a unit of work is 64 output rows x 256 hidden units of one
// expert; CTA c takes units [c * per, (c + 1) * per) of the list ordered by
// output rows, then expert, so a CTA's sums stay with it; output rows shared
// by CTAs are left in the workspace and joined in CTA order by the last.
#include <cuda_fp16.h>

#include <atomic>

#include "q8_async.cuh"
#include "q8_dev.cuh"
#include "q8_internal.h"

namespace q8 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxT = 32;
constexpr int kMaxE = 512;
constexpr int kMaxPairs = kMaxT * 16;  // tokens x chosen experts
constexpr int kChunk = 256;            // columns of a stage
constexpr int kTile = 16 * kChunk;     // bytes of a warp's codes in a stage
constexpr int kScaleTile = 16 * 32;    // bytes of its scales: rows of up to 20, 32 apart
constexpr int kWeights = kWarps * (kTile + kScaleTile);
constexpr int kMaxGrid = 1024;
constexpr int kDownRows = kWarps * 16;

struct MoeParams {
    const uint16_t *x;      // bf16 [T][ldx]
    const float *logits;    // [T][ldl]
    const int8_t *q13, *q2;
    const uint16_t *s13, *s2;
    float *y;               // [T][ldy]
    int32_t *ids;           // [T][top_k] or null
    float *weights;         // [T][top_k] or null
    uint16_t *hi, *lo;      // binary16 [pairs][F]: the hidden units' two parts
    float *fac;             // [pairs][F / 32]: the factor that undoes a block's scaling
    uint32_t *tickets;      // [kMaxGrid]
    float *parts;           // [2 * kMaxGrid][T * kDownRows]
    uint32_t *status;
    int64_t ldx, ldl, ldy;
    int32_t T, E, H, F, top_k, renorm;
    int32_t stages, tok_rows;  // ring; token rows of a stage (T rounded up to 8)
};

// The routing as every CTA holds it.
struct Routing {
    uint32_t mask[kMaxE];       // tokens that chose the expert
    uint16_t expert[kMaxE];     // the chosen experts, in order
    uint16_t base[kMaxE + 1];   // first pair of each
    uint8_t token[kMaxPairs];   // the pairs' tokens, by expert, then token
    float weight[kMaxPairs];    // and weights
    int16_t id[kMaxPairs];      // [T][top_k]
    float w[kMaxPairs];         // [T][top_k]
    int32_t used;               // chosen experts
};

// A total order of floats as unsigned integers; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

__device__ void route(const MoeParams &p, Routing &r, bool report) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < p.E; e += kThreads) r.mask[e] = 0;
    __syncthreads();
    for (int t = warp; t < p.T; t += kWarps) {
        const float *row = p.logits + t * p.ldl;
        uint32_t key[kMaxE / 32];
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = lane + 32 * i;
            key[i] = 0;
            if (e < p.E) {
                const float v = row[e];
                key[i] = order_key(v);
                nan = nan || v != v;
            }
        }
        if (report && __any_sync(0xffffffffu, nan) && lane == 0 && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
        float top = 0.f, z = 0.f, mine = 0.f;
        int mine_id = -1;
        for (int j = 0; j < p.top_k; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i) m = max(m, key[i]);
            const uint32_t best = __reduce_max_sync(0xffffffffu, m);
            if (best <= kKeyNegInf) break;  // nothing left to choose
            int at = kMaxE;
#pragma unroll
            for (int i = kMaxE / 32 - 1; i >= 0; --i)
                if (key[i] == best) at = lane + 32 * i;
            const int e = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (lane + 32 * i == e) key[i] = 0;
            const float v = __uint_as_float((best & 0x80000000u) ? best ^ 0x80000000u : ~best);
            if (j == 0) top = v;
            const float ex = v == top ? 1.f : expf(v - top);
            if (p.renorm) z += ex;
            if (lane == j) mine = ex, mine_id = e;
            if (lane == 0) atomicOr(&r.mask[e], 1u << t);
        }
        if (!p.renorm) {
            for (int e = lane; e < p.E; e += 32) {
                const float v = row[e];
                if (v == v) z += v == top ? 1.f : expf(v - top);
            }
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if (lane < p.top_k) {
            r.id[t * p.top_k + lane] = static_cast<int16_t>(mine_id);
            r.w[t * p.top_k + lane] = mine_id < 0 ? 0.f : __fdiv_rn(mine, z);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int used = 0, pairs = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t m = e < p.E ? r.mask[e] : 0u;
            const uint32_t some = __ballot_sync(0xffffffffu, m != 0);
            int n = __popc(m), run = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            if (m) {
                const int i = used + __popc(some & ((1u << lane) - 1));
                r.expert[i] = static_cast<uint16_t>(e);
                r.base[i] = static_cast<uint16_t>(pairs + run - n);
            }
            used += __popc(some);
            pairs += __shfl_sync(0xffffffffu, run, 31);
        }
        if (lane == 0) {
            r.base[used] = static_cast<uint16_t>(pairs);
            r.used = used;
        }
    }
    __syncthreads();
    for (int i = warp; i < r.used; i += kWarps) {
        const int e = r.expert[i];
        const uint32_t m = r.mask[e];
        if ((m >> lane) & 1) {
            const int at = r.base[i] + __popc(m & ((1u << lane) - 1));
            r.token[at] = static_cast<uint8_t>(lane);
            for (int j = 0; j < p.top_k; ++j)
                if (r.id[lane * p.top_k + j] == e) r.weight[at] = r.w[lane * p.top_k + j];
        }
    }
    __syncthreads();
}

// 16-byte chunk c of a weight tile's row r, and of a token row n: placed so
// that the MMA operand reads hit every bank once.
__device__ __forceinline__ uint32_t weight_at(int r, int c) {
    const uint32_t m = r * (kChunk / 16) + c;
    return (m ^ ((m >> 3) & 7)) * 16;
}
__device__ __forceinline__ uint32_t token_at(int n, int c) { return (n * 32 + (c ^ ((n & 1) << 2))) * 16; }

// One warp's weight tile: 16 rows (8 from row0, 8 from row8) x 256 columns
// from col, of a [rows][K] matrix.
__device__ __forceinline__ void load_tile(uint32_t codes, uint32_t scales, const int8_t *q, const uint16_t *s, int64_t row0,
                                          int64_t row8, int K, int col, int lane) {
    const int c = lane & 15;
    if (col + c * 16 < K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 2 * i + (lane >> 4);
            const int64_t row = r < 8 ? row0 + r : row8 + (r - 8);
            cp_async16(codes + weight_at(r, c), q + row * K + col + c * 16);
        }
    }
    const int nb = K >> 5;
    if ((K & 255) == 0) {
        if (lane < 16) {
            const int64_t row = lane < 8 ? row0 + lane : row8 + (lane - 8);
            cp_async16(scales + lane * 32, s + row * nb + (col >> 5));
        }
    } else {
        // rows of scales start at any 2-byte offset: take the aligned words
        // that hold this chunk's (the array ends on a word: rows % 32 == 0)
        const int words = min(5, (min(8, nb - (col >> 5)) + 2) >> 1);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int j = i * 32 + lane;
            const int r = j / 5, wd = j - r * 5;
            if (r < 16 && wd < words) {
                const int64_t row = r < 8 ? row0 + r : row8 + (r - 8);
                const int64_t at = (row * nb + (col >> 5)) & ~int64_t(1);
                if (at + wd * 2 < (row + 1) * nb) cp_async4(scales + r * 32 + wd * 4, s + at + wd * 2);
            }
        }
    }
}

// The 8 scales of a row's chunk, as four pairs.
__device__ __forceinline__ void row_scales(uint32_t scales, int r, bool odd, uint32_t *w) {
    const uint4 a = lds128(scales + r * 32);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if (odd) {
        const uint32_t last = lds32(scales + r * 32 + 16);
        w[0] = __funnelshift_r(a.x, a.y, 16);
        w[1] = __funnelshift_r(a.y, a.z, 16);
        w[2] = __funnelshift_r(a.z, a.w, 16);
        w[3] = __funnelshift_r(a.w, last, 16);
    }
}
__device__ __forceinline__ float pick_scale(const uint32_t *w, int b) {
    return f16_bits_to_f32((b & 1) ? w[b >> 1] >> 16 : w[b >> 1] & 0xFFFFu);
}

__device__ __forceinline__ void wait_stage(int stages) {
    // groups still under way: all but the oldest of stages - 1
    switch (stages) {
        case 2: cp_async_wait<0>(); break;
        case 3: cp_async_wait<1>(); break;
        case 4: cp_async_wait<2>(); break;
        case 5: cp_async_wait<3>(); break;
        default: cp_async_wait<4>(); break;
    }
}

__global__ void __launch_bounds__(kThreads) moe_gate_up_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Routing r;
    __shared__ float s_max[kWarps][kMaxT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    route(p, r, blockIdx.x == 0);
    if (blockIdx.x == 0) {
        for (int i = tid; i < p.T * p.top_k; i += kThreads) {
            if (p.ids) p.ids[i] = r.id[i];
            if (p.weights) p.weights[i] = r.w[i];
        }
    }
    const int blocks = p.F >> 5, chunks = (p.H + kChunk - 1) / kChunk;
    const int64_t tasks = static_cast<int64_t>(r.used) * blocks;
    const int64_t t0 = tasks * blockIdx.x / gridDim.x, t1 = tasks * (blockIdx.x + 1) / gridDim.x;
    if (t0 >= t1) return;

    const int stage_bytes = kWeights + p.tok_rows * 512;
    const uint32_t ring = smem_addr(smem);
    const int64_t total = (t1 - t0) * chunks;
    int64_t loaded = 0;
    int ld_i = static_cast<int>(t0 / blocks), ld_b = static_cast<int>(t0 % blocks), ld_c = 0, ld_slot = 0;
    auto load = [&]() {
        if (loaded < total) {
            const uint32_t st = ring + ld_slot * stage_bytes;
            const int64_t rows = static_cast<int64_t>(r.expert[ld_i]) * 2 * p.F;
            const int unit = ld_b * 32 + warp * 8, col = ld_c * kChunk;
            load_tile(st + warp * kTile, st + kWarps * kTile + warp * kScaleTile, p.q13, p.s13, rows + unit, rows + p.F + unit,
                      p.H, col, lane);
            const int base = r.base[ld_i], n = r.base[ld_i + 1] - base;
            if (col + lane * 8 < p.H)
                for (int i = warp; i < n; i += kWarps)
                    cp_async16(st + kWeights + token_at(i, lane), p.x + r.token[base + i] * p.ldx + col + lane * 8);
            ++loaded;
            if (++ld_c == chunks) {
                ld_c = 0;
                if (++ld_b == blocks) ld_b = 0, ++ld_i;
            }
        }
        ld_slot = ld_slot + 1 == p.stages ? 0 : ld_slot + 1;
        cp_async_commit();
    };
    for (int i = 0; i < p.stages - 1; ++i) load();

    int slot = 0, ei = static_cast<int>(t0 / blocks), blk = static_cast<int>(t0 % blocks);
    const bool odd0 = ((p.H >> 5) & 1) != 0;
    for (int64_t task = t0; task < t1; ++task) {
        const int base = r.base[ei], n = r.base[ei + 1] - base, nt = (n + 7) >> 3;
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        const int64_t rows = static_cast<int64_t>(r.expert[ei]) * 2 * p.F;
        const bool oddg = odd0 && ((rows + blk * 32 + warp * 8 + g) & 1), oddu = odd0 && ((rows + p.F + blk * 32 + warp * 8 + g) & 1);
        for (int c = 0; c < chunks; ++c) {
            wait_stage(p.stages);
            __syncthreads();
            load();
            const uint32_t st = ring + slot * stage_bytes, codes = st + warp * kTile;
            const uint32_t sc = st + kWarps * kTile + warp * kScaleTile, xs = st + kWeights;
            uint32_t sg[4], su[4];
            row_scales(sc, g, oddg, sg);
            row_scales(sc, g + 8, oddu, su);
            const int nb = min(8, (p.H >> 5) - c * 8);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (b < nb) {
                    const uint2 w0 = lds64(codes + weight_at(g, 2 * b + (t >> 1)) + (t & 1) * 8);
                    const uint2 w1 = lds64(codes + weight_at(g + 8, 2 * b + (t >> 1)) + (t & 1) * 8);
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    codes4_to_bf16x2(w0.x, a0, a2);
                    codes4_to_bf16x2(w1.x, a1, a3);
                    codes4_to_bf16x2(w0.y, b0, b2);
                    codes4_to_bf16x2(w1.y, b1, b3);
                    const float f0 = pick_scale(sg, b), f1 = pick_scale(su, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < nt) {
                            const uint4 xv = lds128(xs + token_at(i * 8 + g, 4 * b + t));
                            float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
                            mma_bf16_16816(d0, d1, d2, d3, a0, a1, a2, a3, xv.x, xv.y);
                            mma_bf16_16816(d0, d1, d2, d3, b0, b1, b2, b3, xv.z, xv.w);
                            acc[i][0] = fmaf(f0, d0, acc[i][0]);
                            acc[i][1] = fmaf(f0, d1, acc[i][1]);
                            acc[i][2] = fmaf(f1, d2, acc[i][2]);
                            acc[i][3] = fmaf(f1, d3, acc[i][3]);
                        }
                    }
                }
            }
            slot = slot + 1 == p.stages ? 0 : slot + 1;
        }
        // SwiGLU; the largest hidden unit of each token's block of 32 (four warps)
        float act[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = acc[i][j];
                act[i][j] = a / (1.0f + expf(-a)) * acc[i][2 + j];
                if (i < nt) {
                    float m = fabsf(act[i][j]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (g == 0) s_max[warp][i * 8 + 2 * t + j] = m;
                }
            }
        }
        __syncthreads();
        const int unit = blk * 32 + warp * 8 + g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = i * 8 + 2 * t + j;
                if (tok < n) {
                    const float m = fmaxf(fmaxf(s_max[0][tok], s_max[1][tok]), fmaxf(s_max[2][tok], s_max[3][tok]));
                    // the largest to [2^14, 2^15); a block of zeros or of non-finite units keeps a factor in range
                    const int ex = min(max(static_cast<int>(__float_as_uint(m) >> 23), 30), 240);
                    const float v = act[i][j] * __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
                    const __half h = __float2half_rn(v);
                    const __half l = __float2half_rn(v - __half2float(h));
                    const int64_t at = static_cast<int64_t>(base + tok) * p.F + unit;
                    p.hi[at] = __half_as_ushort(h);
                    p.lo[at] = __half_as_ushort(l);
                    if (warp == 0 && g == 0)
                        p.fac[static_cast<int64_t>(base + tok) * blocks + blk] = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
                }
            }
        }
        if (++blk == blocks) blk = 0, ++ei;
    }
    cp_async_wait<0>();
}

__global__ void __launch_bounds__(kThreads) moe_down_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Routing r;
    __shared__ uint32_t s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    route(p, r, false);
    const int chunks = (p.F + kChunk - 1) / kChunk, tiles = (p.H + kDownRows - 1) / kDownRows, blocks = p.F >> 5;
    const int64_t item = static_cast<int64_t>(r.used) * chunks;  // units of one tile of output rows
    const int64_t total = item * tiles;
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(1));
    const int64_t u0 = per * blockIdx.x, u1 = min(u0 + per, total);
    const int stage_bytes = kWeights + p.tok_rows * (1024 + 32);
    const uint32_t ring = smem_addr(smem);
    float *const s_y = reinterpret_cast<float *>(smem + p.stages * stage_bytes);  // [T][kDownRows]

    int64_t loaded = u0;
    int ld_rt = 0, ld_i = 0, ld_c = 0, ld_slot = 0;
    if (u0 < u1) {
        ld_rt = static_cast<int>(u0 / item);
        const int64_t in = u0 - ld_rt * item;
        ld_i = static_cast<int>(in / chunks);
        ld_c = static_cast<int>(in - static_cast<int64_t>(ld_i) * chunks);
    }
    int rt = ld_rt, ei = ld_i, ch = ld_c;
    // weights do not depend on the first kernel, hidden units do
    auto load_weights = [&](uint32_t st, int a_rt, int a_i, int a_c) {
        const int row = a_rt * kDownRows + warp * 16;
        if (row < p.H) {
            const int64_t rows = static_cast<int64_t>(r.expert[a_i]) * p.H + row;
            load_tile(st + warp * kTile, st + kWarps * kTile + warp * kScaleTile, p.q2, p.s2, rows, rows + 8, p.F, a_c * kChunk, lane);
        }
    };
    auto load_hidden = [&](uint32_t st, int a_i, int a_c) {
        const int base = r.base[a_i], n = r.base[a_i + 1] - base, col = a_c * kChunk;
        const uint32_t hs = st + kWeights;
        if (col + lane * 8 < p.F)
            for (int i = warp; i < n; i += kWarps) {
                const int64_t at = static_cast<int64_t>(base + i) * p.F + col + lane * 8;
                cp_async16(hs + token_at(i, lane), p.hi + at);
                cp_async16(hs + p.tok_rows * 512 + token_at(i, lane), p.lo + at);
            }
        const int nb = min(8, blocks - a_c * 8);
        for (int j = tid; j < n * 8; j += kThreads)
            if ((j & 7) < nb)
                cp_async4(hs + p.tok_rows * 1024 + (j & 7) * (p.tok_rows * 4) + (j >> 3) * 4,
                          p.fac + static_cast<int64_t>(base + (j >> 3)) * blocks + a_c * 8 + (j & 7));
    };
    auto step = [&](int &a_rt, int &a_i, int &a_c) {
        if (++a_c == chunks) {
            a_c = 0;
            if (++a_i == r.used) a_i = 0, ++a_rt;
        }
    };
    auto load = [&]() {
        if (loaded < u1) {
            const uint32_t st = ring + ld_slot * stage_bytes;
            load_weights(st, ld_rt, ld_i, ld_c);
            load_hidden(st, ld_i, ld_c);
            ++loaded;
            step(ld_rt, ld_i, ld_c);
        }
        ld_slot = ld_slot + 1 == p.stages ? 0 : ld_slot + 1;
        cp_async_commit();
    };
    pdl_wait_prior();
    if (r.used == 0) {
        for (int64_t i = blockIdx.x * kThreads + tid; i < static_cast<int64_t>(p.T) * p.H; i += gridDim.x * kThreads)
            p.y[i / p.H * p.ldy + i % p.H] = 0.f;
        return;
    }
    if (u0 >= u1) return;
    for (int i = 0; i < p.stages - 1; ++i) load();

    const bool odd = ((p.F >> 5) & 1) != 0;
    int slot = 0;
    int64_t u = u0;
    while (u < u1) {
        const int64_t seg0 = u, tile0 = rt * item, tile1 = tile0 + item, end = min(u1, tile1);
        const int this_rt = rt;
        for (int i = lane; i < p.T * 16; i += 32) s_y[(i >> 4) * kDownRows + warp * 16 + (i & 15)] = 0.f;
        __syncwarp();
        while (u < end) {
            const int base = r.base[ei], n = r.base[ei + 1] - base, nt = (n + 7) >> 3;
            const int64_t row0 = static_cast<int64_t>(r.expert[ei]) * p.H + rt * kDownRows + warp * 16;
            const bool odd0 = odd && ((row0 + g) & 1);
            const int this_e = ei;
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            do {
                wait_stage(p.stages);
                __syncthreads();
                load();
                const uint32_t st = ring + slot * stage_bytes, codes = st + warp * kTile;
                const uint32_t sc = st + kWarps * kTile + warp * kScaleTile, hs = st + kWeights;
                const uint32_t fs = hs + p.tok_rows * 1024 + 8 * t;
                uint32_t s0[4], s1[4];
                row_scales(sc, g, odd0, s0);
                row_scales(sc, g + 8, odd0, s1);
                const int nb = min(8, blocks - ch * 8);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (b < nb) {
                        const uint2 w0 = lds64(codes + weight_at(g, 2 * b + (t >> 1)) + (t & 1) * 8);
                        const uint2 w1 = lds64(codes + weight_at(g + 8, 2 * b + (t >> 1)) + (t & 1) * 8);
                        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                        codes4_to_f16x2(w0.x, a0, a2);
                        codes4_to_f16x2(w1.x, a1, a3);
                        codes4_to_f16x2(w0.y, b0, b2);
                        codes4_to_f16x2(w1.y, b1, b3);
                        const float f0 = pick_scale(s0, b), f1 = pick_scale(s1, b);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i < nt) {
                                const uint32_t at = hs + token_at(i * 8 + g, 4 * b + t);
                                const uint4 hv = lds128(at), lv = lds128(at + p.tok_rows * 512);
                                const uint2 fv = lds64(fs + b * (p.tok_rows * 4) + i * 32);
                                float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
                                mma_f16_16816(d0, d1, d2, d3, a0, a1, a2, a3, lv.x, lv.y);
                                mma_f16_16816(d0, d1, d2, d3, b0, b1, b2, b3, lv.z, lv.w);
                                mma_f16_16816(d0, d1, d2, d3, a0, a1, a2, a3, hv.x, hv.y);
                                mma_f16_16816(d0, d1, d2, d3, b0, b1, b2, b3, hv.z, hv.w);
                                const float c0 = __uint_as_float(fv.x), c1 = __uint_as_float(fv.y);
                                acc[i][0] = fmaf(f0 * c0, d0, acc[i][0]);
                                acc[i][1] = fmaf(f0 * c1, d1, acc[i][1]);
                                acc[i][2] = fmaf(f1 * c0, d2, acc[i][2]);
                                acc[i][3] = fmaf(f1 * c1, d3, acc[i][3]);
                            }
                        }
                    }
                }
                slot = slot + 1 == p.stages ? 0 : slot + 1;
                ++u;
                step(rt, ei, ch);
            } while (u < end && ei == this_e && ch != 0);
            // this expert's share of the rows, weighted
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = i * 8 + 2 * t + j;
                    if (k < n) {
                        float *at = s_y + r.token[base + k] * kDownRows + warp * 16 + g;
                        const float w = r.weight[base + k];
                        at[0] = fmaf(w, acc[i][j], at[0]);
                        at[8] = fmaf(w, acc[i][2 + j], at[8]);
                    }
                }
            __syncwarp();
        }
        const int row = this_rt * kDownRows;
        const int rows = min(kDownRows, p.H - row);
        __syncthreads();
        if (seg0 == tile0 && end == tile1) {
            for (int i = tid; i < p.T * kDownRows; i += kThreads) {
                const int tok = i / kDownRows, k = i - tok * kDownRows;
                if (k < rows) p.y[tok * p.ldy + row + k] = s_y[i];
            }
        } else {
            const int c0 = static_cast<int>(tile0 / per), c1 = static_cast<int>((tile1 - 1) / per);
            const int64_t size = static_cast<int64_t>(p.T) * kDownRows;
            float *const mine = p.parts + (2 * blockIdx.x + (seg0 == tile0 ? 1 : 0)) * size;
            for (int i = tid; i < size; i += kThreads) mine[i] = s_y[i];
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t k = atomicAdd(p.tickets + c0, 1u);
                s_last = k == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
                if (s_last) p.tickets[c0] = 0u;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int i = tid; i < size; i += kThreads) {
                    const int tok = i / kDownRows, k = i - tok * kDownRows;
                    float sum = 0.f;
#pragma unroll 8
                    for (int c = c0; c <= c1; ++c) sum += __ldcg(p.parts + (2 * c + (c == c0 ? 1 : 0)) * size + i);
                    if (k < rows) p.y[tok * p.ldy + row + k] = sum;
                }
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeLayout {
    size_t hi, lo, fac, parts, total;
};
MoeLayout layout_of(int T, int F, int top_k) {
    const size_t pairs = static_cast<size_t>(T) * top_k;
    MoeLayout m;
    m.hi = kMaxGrid * 4;
    m.lo = m.hi + up256(pairs * F * 2);
    m.fac = m.lo + up256(pairs * F * 2);
    m.parts = m.fac + up256(pairs * (F / 32) * 4);
    m.total = m.parts + static_cast<size_t>(2) * kMaxGrid * T * kDownRows * 4;
    return m;
}

constexpr int kSmemPerSm = 227 * 1024, kStaticSmem = 12 * 1024;

// Stages and CTAs per SM: as many CTAs as leave each a ring of three stages,
// at most 3; then as many stages as fit, at most 6.
struct Shape {
    int ctas, stages;
    size_t smem;
};
Shape shape_of(int stage, int extra) {
    for (int ctas = 3; ctas >= 1; --ctas) {
        const int room = kSmemPerSm / ctas - kStaticSmem - extra;
        const int stages = room / stage;
        if (stages >= 3 || ctas == 1) {
            const int n = stages > 6 ? 6 : stages;
            return {ctas, n, static_cast<size_t>(n) * stage + extra};
        }
    }
    return {0, 0, 0};
}

}  // namespace

size_t moe_workspace(int T, int F, int top_k) { return layout_of(T, F, top_k).total; }

q8_status launch_moe(const MoeArgs &a, void *ws, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (di->device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const int most = kSmemPerSm - kStaticSmem;
        if (cudaFuncSetAttribute(moe_gate_up_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaFuncSetAttribute(moe_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return Q8_ERR_CUDA;
        ready.fetch_or(bit);
    }
    const MoeLayout m = layout_of(a.T, a.F, a.top_k);
    uint8_t *w = static_cast<uint8_t *>(ws);
    MoeParams p = {};
    p.x = a.x, p.logits = a.logits, p.q13 = a.q13, p.s13 = a.s13, p.q2 = a.q2, p.s2 = a.s2;
    p.y = a.y, p.ids = a.ids, p.weights = a.weights;
    p.tickets = reinterpret_cast<uint32_t *>(w);
    p.hi = reinterpret_cast<uint16_t *>(w + m.hi), p.lo = reinterpret_cast<uint16_t *>(w + m.lo);
    p.fac = reinterpret_cast<float *>(w + m.fac), p.parts = reinterpret_cast<float *>(w + m.parts);
    p.status = dev_status;
    p.ldx = a.ldx, p.ldl = a.ldl, p.ldy = a.ldy;
    p.T = a.T, p.E = a.E, p.H = a.H, p.F = a.F, p.top_k = a.top_k, p.renorm = a.renorm;
    p.tok_rows = (a.T + 7) & ~7;
    const int64_t used = static_cast<int64_t>(a.T) * a.top_k < a.E ? static_cast<int64_t>(a.T) * a.top_k : a.E;

    const Shape up = shape_of(kWeights + p.tok_rows * 512, 0);
    p.stages = up.stages;
    int64_t grid = static_cast<int64_t>(up.ctas) * di->sm_count, need = used * (a.F / 32);
    if (grid > kMaxGrid) grid = kMaxGrid;
    if (grid > need) grid = need;
    if (launch_kernel(moe_gate_up_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), up.smem, stream, false, p) != cudaSuccess)
        return Q8_ERR_CUDA;

    const Shape down = shape_of(kWeights + p.tok_rows * (1024 + 32), a.T * kDownRows * 4);
    p.stages = down.stages;
    grid = static_cast<int64_t>(down.ctas) * di->sm_count;
    need = used * ((a.F + kChunk - 1) / kChunk) * ((a.H + kDownRows - 1) / kDownRows);
    if (grid > kMaxGrid) grid = kMaxGrid;
    if (grid > need) grid = need;
    if (launch_kernel(moe_down_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), down.smem, stream, true, p) != cudaSuccess)
        return Q8_ERR_CUDA;
    return Q8_OK;
}

}  // namespace q8
