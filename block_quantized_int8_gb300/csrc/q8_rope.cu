// q8_rope.cu -- rotary positions of query and key heads, by themselves and with the write of
// keys and values into the paged Q8_0 cache.
//
// Pair i of a head at position t turns by the angle t f_i (f_i radians a token):
//   (y1, y2) = factor * (x1 cos - x2 sin, x2 cos + x1 sin)
// with x1, x2 at dimensions i and i + rot / 2 (half layout) or 2 i and 2 i + 1 (interleaved); the
// dimensions from `rot` on pass.
//
// Angles: the table holds F_i = f_i / (2 pi) as a 64-bit fraction of a turn, so that t F_i modulo
// 2^64 is the angle within its turn, exactly for the F_i given, at any distance: off by |t| times
// the three units of 2^-64 turns that F_i may be off, below 2^-31 turns.  Its upper 32 bits go to fp32
// as half turns in [-1, 1) (2^-25 half turns of rounding at most), whose sine and cosine are taken.  A
// product t f_i in fp32 would be off by 0.008 at t = 200,000, two bf16 steps of the result.
//
// Bound by bytes: each row in once, rotated rows (bf16) or codes and scales out once.  A CTA has
// one token: its threads make the token's cosines and sines once, in shared memory, for all heads.
// Measured on the device (events around one call, L2 flushed before it; one after the other, as a part of the rows stays
// in L2, 29.4): 8192 tokens of 40 heads of 128 in bf16 32 us (5.2 TB/s; 256 threads 31 to 35, 512 35).  With the
// write to the cache, 4096 tokens of 32 / 8 heads 27.7 us (3.35 TB/s; 29, 35 and 46 with 256, 384 and 512 threads, 27 with
// 64), of which the angles' latency before the first store is most.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "q8_dev.cuh"
#include "q8_internal.h"
#include "q8_quant.cuh"
#include "q8_rows.cuh"

namespace q8 {

namespace {

constexpr int kRopeThreads = 128, kAppendThreads = 128;
constexpr int kCtas = 10;  // an SM's that registers must allow (8192 tokens 32.0 us, appending 4096 27.7; unasked 33.4 and 29.3, 16: 49.5 and 40.1)
constexpr int kMaxPairs = 128;  // head_dim 256

struct RopeParams {
    const void *x;       // q8_rope: all heads; q8_rope_append: query heads
    const void *k, *v;
    void *y;             // bf16
    int8_t *codes[2];
    uint16_t *scales[2];
    const uint64_t *turns;
    const int32_t *positions;
    const int64_t *slots;
    uint32_t *status;
    int64_t ldx, ldk, ldv, ldy, capacity;
    int32_t heads, kv_heads, d_shift, page_shift, rot;
    float factor;
};

// y1 and y2 of a pair; the products' roundings are written out, so that they are the same wherever a pair is turned.
__device__ __forceinline__ float turn1(float x1, float x2, float c, float s) { return fmaf(x1, c, -__fmul_rn(x2, s)); }
__device__ __forceinline__ float turn2(float x1, float x2, float c, float s) { return fmaf(x2, c, __fmul_rn(x1, s)); }

// The token's cosines and sines, times factor.
template <int kThreads>
__device__ __forceinline__ void make_angles(const RopeParams &p, int64_t token, float *s_cos, float *s_sin) {
    const int64_t pos = p.positions[token];
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
        const uint64_t turn = static_cast<uint64_t>(pos) * p.turns[i];
        // half turns: the upper 32 bits as a signed fraction
        const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        float s, c;
        sincospif(half_turns, &s, &c);
        s_cos[i] = c * p.factor;
        s_sin[i] = s * p.factor;
    }
}

__device__ __forceinline__ void lds8(const float *s, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(s)[0], b = reinterpret_cast<const float4 *>(s)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Sixteen values of a head (item i of D / 16), turned, to bf16: dimensions 8 i and rot / 2 + 8 i on of
// the half layout, 16 i on of the interleaved and of what passes.
template <typename T, bool kInter>
struct Item {
    Raw8<T> ra, rb;
    __device__ __forceinline__ void load(const RopeParams &p, const T *x, int i) {
        const bool half = !kInter && 16 * i < p.rot;
        ra.load(x + (half ? 8 * i : 16 * i));
        rb.load(x + (half ? p.rot / 2 + 8 * i : 16 * i + 8));
    }
    __device__ __forceinline__ void finish(const RopeParams &p, __nv_bfloat16 *y, int i, const float *s_cos, const float *s_sin) const {
        float a[8], b[8], c[8], s[8];
        ra.widen(a), rb.widen(b);
        const bool turns = 16 * i < p.rot;
        if (turns) {
            lds8(s_cos + 8 * i, c), lds8(s_sin + 8 * i, s);
            if constexpr (kInter) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x1 = a[2 * j], x2 = a[2 * j + 1], z1 = b[2 * j], z2 = b[2 * j + 1];
                    a[2 * j] = turn1(x1, x2, c[j], s[j]), a[2 * j + 1] = turn2(x1, x2, c[j], s[j]);
                    b[2 * j] = turn1(z1, z2, c[4 + j], s[4 + j]), b[2 * j + 1] = turn2(z1, z2, c[4 + j], s[4 + j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x1 = a[j], x2 = b[j];
                    a[j] = turn1(x1, x2, c[j], s[j]), b[j] = turn2(x1, x2, c[j], s[j]);
                }
            }
        }
        const bool half = !kInter && turns;
        store8(y + (half ? 8 * i : 16 * i), a), store8(y + (half ? p.rot / 2 + 8 * i : 16 * i + 8), b);
    }
};

// All heads of a row, each thread's next item on its way while it turns one; the first (begin()) while the
// angles are made.
template <typename T, bool kInter, int kThreads>
struct Heads {
    Item<T, kInter> item;
    int u, n, shift;
    const T *x;
    __device__ __forceinline__ int64_t head_of(const RopeParams &p, int v) const { return static_cast<int64_t>(v >> shift) << p.d_shift; }
    __device__ __forceinline__ void begin(const RopeParams &p, const T *row) {
        x = row, shift = p.d_shift - 4, n = p.heads << shift, u = threadIdx.x;
        if (u < n) item.load(p, x + head_of(p, u), u & ((1 << shift) - 1));
    }
    __device__ __forceinline__ void run(const RopeParams &p, __nv_bfloat16 *y, const float *s_cos, const float *s_sin) {
        while (u < n) {
            const Item<T, kInter> now = item;
            const int v = u;
            u += kThreads;
            // (y may be x: another item's values are read before this one's are written, and no two share any)
            if (u < n) item.load(p, x + head_of(p, u), u & ((1 << shift) - 1));
            now.finish(p, y + head_of(p, v), v & ((1 << shift) - 1), s_cos, s_sin);
        }
    }
};

template <typename T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kCtas) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
    const int64_t token = blockIdx.x;
    Heads<T, kInter, kRopeThreads> heads;
    heads.begin(p, static_cast<const T *>(p.x) + token * p.ldx);
    make_angles<kRopeThreads>(p, token, s_cos, s_sin);
    __syncthreads();
    heads.run(p, static_cast<__nv_bfloat16 *>(p.y) + token * p.ldy, s_cos, s_sin);
}

// Eight neighbouring dimensions d .. d + 7 of a key or value head.  A key's turn; in the half layout
// the other halves of their pairs are loaded too (from L1 for one of the two lanes that want them).
template <typename T, bool kInter>
struct Unit8 {
    Raw8<T> own, other;
    __device__ __forceinline__ void load(const RopeParams &p, const T *x, int d, bool turns) {
        own.load(x + d);
        if (!kInter && turns && d < p.rot) other.load(x + (d >= p.rot / 2 ? d - p.rot / 2 : d + p.rot / 2));
    }
    __device__ __forceinline__ void values(const RopeParams &p, int d, bool turns, float (&v)[8], const float *s_cos, const float *s_sin) const {
        own.widen(v);
        if (!turns || d >= p.rot) return;
        float c[8], s[8];
        if constexpr (kInter) {
            const float4 c4 = *reinterpret_cast<const float4 *>(s_cos + d / 2), s4 = *reinterpret_cast<const float4 *>(s_sin + d / 2);
            c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
            s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x1 = v[2 * j], x2 = v[2 * j + 1];
                v[2 * j] = turn1(x1, x2, c[j], s[j]), v[2 * j + 1] = turn2(x1, x2, c[j], s[j]);
            }
        } else {
            const bool second = d >= p.rot / 2;
            const int i = second ? d - p.rot / 2 : d;
            float o[8];
            other.widen(o);
            lds8(s_cos + i, c), lds8(s_sin + i, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = second ? turn2(o[j], v[j], c[j], s[j]) : turn1(v[j], o[j], c[j], s[j]);
        }
    }
};

template <typename T, bool kInter>
__global__ void __launch_bounds__(kAppendThreads, kCtas) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
    const int64_t token = blockIdx.x;
    const int64_t slot = p.slots[token];
    Heads<T, kInter, kAppendThreads> heads;
    heads.begin(p, static_cast<const T *>(p.x) + token * p.ldx);
    // keys, then values, eight to a lane; four lanes own a block (a head has a multiple of four).  A thread's next
    // unit is on its way while it works on one
    const int units = p.kv_heads << (p.d_shift - 3);
    const T *k = static_cast<const T *>(p.k) + token * p.ldk, *v = static_cast<const T *>(p.v) + token * p.ldv;
    Unit8<T, kInter> unit;
    auto fetch = [&](int u) {
        if (u >= 2 * units) return;
        const bool is_v = u >= units;
        const int at = (is_v ? u - units : u) * 8, d = at & ((1 << p.d_shift) - 1);
        unit.load(p, (is_v ? v : k) + (at - d), d, !is_v);
    };
    const bool held = slot >= 0 && slot < p.capacity;
    if (held) fetch(threadIdx.x);
    make_angles<kAppendThreads>(p, token, s_cos, s_sin);
    __syncthreads();
    // (y may be q, so the keys' and values' rows, which may lie behind it, are never written)
    heads.run(p, static_cast<__nv_bfloat16 *>(p.y) + token * p.ldy, s_cos, s_sin);
    if (!held) {
        if (slot >= 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, Q8_DEV_BAD_INDEX);
        return;
    }
    const int64_t page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    for (int u0 = 0; u0 < 2 * units; u0 += kAppendThreads) {
        const int u = u0 + threadIdx.x;
        const bool live = u < 2 * units, is_v = u >= units;
        const int at = (live ? (is_v ? u - units : u) : 0) * 8;
        const int h = at >> p.d_shift, d = at & ((1 << p.d_shift) - 1);
        float x[8];
        if (live) {
            unit.values(p, d, !is_v, x, s_cos, s_sin);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.f;
        }
        fetch(u + kAppendThreads);
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        __half hs;
        float sf;
        const uint32_t flags = block_scale(top, hs, sf);
        uint32_t packed[2] = {0u, 0u};
        if (!flags && sf != 0.f) codes_of<float, 8>(x, sf, packed);
        if (live) {
            const int64_t code = ((((page * p.kv_heads + h) << p.page_shift) + off) << p.d_shift) + d;
            *reinterpret_cast<uint2 *>(p.codes[is_v] + code) = make_uint2(packed[0], packed[1]);
            if ((threadIdx.x & 3) == 0) {
                p.scales[is_v][code >> 5] = flags ? 0 : __half_as_ushort(hs);
                if (flags && p.status) atomicOr(p.status, flags);
            }
        }
    }
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

template <typename T>
void launch(const RopeParams &p, int64_t T_, bool inter, bool append, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(T_);
    if (append)
        (inter ? rope_append_kernel<T, true> : rope_append_kernel<T, false>)<<<grid, kAppendThreads, 0, stream>>>(p);
    else
        (inter ? rope_kernel<T, true> : rope_kernel<T, false>)<<<grid, kRopeThreads, 0, stream>>>(p);
}

}  // namespace

q8_status launch_rope(const RopeArgs &a, const q8_kv_cache *c, uint32_t *dev_status, cudaStream_t stream) {
    RopeParams p = {};
    p.x = a.x, p.k = a.k, p.v = a.v, p.y = a.y;
    p.turns = a.turns, p.positions = a.positions, p.slots = a.slots, p.status = dev_status;
    p.ldx = a.ldx, p.ldk = a.ldk, p.ldv = a.ldv, p.ldy = a.ldy;
    p.heads = a.heads, p.d_shift = ilog2(a.head_dim), p.rot = a.rot, p.factor = a.factor;
    if (c) {
        p.codes[0] = c->kq, p.codes[1] = c->vq, p.scales[0] = c->ks, p.scales[1] = c->vs;
        p.kv_heads = c->kv_heads, p.page_shift = ilog2(c->page_size);
        p.capacity = static_cast<int64_t>(c->pages) * c->page_size;
    }
    if (a.dtype == Q8_DTYPE_F32)
        launch<float>(p, a.T, a.layout == Q8_ROPE_INTERLEAVED, c != nullptr, stream);
    else
        launch<__nv_bfloat16>(p, a.T, a.layout == Q8_ROPE_INTERLEAVED, c != nullptr, stream);
    return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

// f / (2 pi) as a 64-bit fraction of a turn.  1 / (2 pi) is taken as three doubles (Dekker's
// splitting of the constant 0.159154943091895335768883763372514362...), f's product with each
// as a rounded product and its exact remainder (fma), and the whole turns are dropped from each
// term (exact) before they are added, so that the fraction is good to its last bits for f up
// to thousands of radians.
void rope_turns(const double *inv_freq, int32_t n, uint64_t *turns) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kMid = -0x1.6b01ec5417056p-57, kLo = -0x1.6447e493ad4cep-111;
    for (int32_t i = 0; i < n; ++i) {
        const double f = inv_freq[i];
        const double terms[] = {f * kHi, std::fma(f, kHi, -(f * kHi)), f * kMid, std::fma(f, kMid, -(f * kMid)), f * kLo};
        uint64_t sum = 0;
        for (double t : terms) {
            const double x = std::fabs(t) - std::floor(std::fabs(t));
            const double hi = std::floor(x * 0x1p32);
            const double rest = (x * 0x1p32 - hi) * 0x1p32;
            const uint64_t part = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::floor(rest + 0.5));
            sum = t < 0.0 ? sum - part : sum + part;
        }
        turns[i] = sum;
    }
}

}  // namespace q8
