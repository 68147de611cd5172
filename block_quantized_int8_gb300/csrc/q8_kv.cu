// q8_kv.cu -- the paged key-value cache in Q8_0 blocks: writing new tokens'
// keys and values (quantized on the way in) and reading tokens back.
//
// A token's keys of one head are D values, cut into D / 32 blocks of the
// weights' format: s = binary16(amax / 127), code = |x| / s rounded half away
// from zero (q8_quant.cuh).  Codes lie at [page][kv_head][page_size][D],
// scales at [page][kv_head][page_size][D / 32], so 16 consecutive tokens of a
// head are one contiguous run of each -- what the attention streams.
//
// Bound by memory for many tokens and by the launch for few: per value 4 (or
// 2) bytes in and 1.0625 out for the write, the reverse for the read.  A lane
// holds 16 bytes of a row (4 fp32 or 8 bf16 values), so a warp's accesses to
// the rows are 512 contiguous bytes; 8 or 4 lanes own a block.  Each thread takes the same
// place of the keys and of the values (the write once it knows its slot) and is done (a grid of resident CTAs that loop was slower at
// every size).  Where there are more such units than run at once, a thread reads two (8192 tokens x 1024
// values in fp32: 16.7 us, 5.1 TB/s, with one 18.7; 1024 tokens 3.3 and 3.1; one token 1.9 and 1.7).  Writing
// two was slower at every size (8192 tokens 13.1 us and 13.0, 3.9 TB/s, from bf16; one token 2.7 and 2.1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q8_dev.cuh"
#include "q8_internal.h"
#include "q8_quant.cuh"

namespace q8 {

namespace {

constexpr int kThreads = 128;
constexpr uint32_t kMany = 1 << 19;  // units from which on a thread reads two

struct KvParams {
    int8_t *codes[2];      // keys, values
    uint16_t *scales[2];
    const void *in[2];     // append: [T][ld] values
    void *out[2];          // read:   [T][ld] values
    int64_t ld[2];         // elements from one token to the next
    const int64_t *slots;  // [T]
    uint32_t *status;
    int64_t capacity;      // pages * page_size
    uint32_t units;        // T * per_token
    uint32_t per_token;    // kv_heads * D / values of a unit
    uint32_t magic, shift; // u / per_token = (u * magic >> 32) >> shift for u < 2^31
    int32_t page_shift, d_shift, kv_heads;
};

// Unit u is W values of one token: where they are in the input or output row
// and in the cache.  false if the token has no slot (padding, or a slot that
// does not exist, which is flagged).
struct Place {
    uint32_t token, at;  // `at`: value offset within the token's row
    int64_t code;        // element offset into the codes
};
template <int W>
__device__ __forceinline__ bool place(const KvParams &p, uint32_t u, Place &o) {
    o.token = __umulhi(u, p.magic) >> p.shift;
    o.at = (u - o.token * p.per_token) * W;
    o.code = 0;
    const int64_t slot = p.slots[o.token];
    if (slot < 0 || slot >= p.capacity) {
        if (slot >= 0 && o.at == 0 && p.status) atomicOr(p.status, Q8_DEV_BAD_INDEX);
        return false;
    }
    const int64_t page = slot >> p.page_shift;
    const int64_t off = slot & ((1 << p.page_shift) - 1);
    const uint32_t h = o.at >> p.d_shift, d = o.at & ((1u << p.d_shift) - 1);
    o.code = ((((page * p.kv_heads + h) << p.page_shift) + off) << p.d_shift) + d;
    return true;
}

// The values in 16 bytes of a row, and back.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
    static constexpr int W = 4;
    static __device__ __forceinline__ void widen(const uint4 &r, float (&v)[W]) {
        v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint32_t largest(const uint4 &r) {
        return max(max(r.x & 0x7FFFFFFFu, r.y & 0x7FFFFFFFu), max(r.z & 0x7FFFFFFFu, r.w & 0x7FFFFFFFu));
    }
    static __device__ __forceinline__ uint4 narrow(const float (&v)[W]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Unit<__nv_bfloat16> {
    static constexpr int W = 8;
    static __device__ __forceinline__ void widen(const uint4 &r, float (&v)[W]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo_f32(w[i]), v[2 * i + 1] = bf16hi_f32(w[i]);
    }
    static __device__ __forceinline__ uint32_t largest(const uint4 &r) {
        const uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
        return max(m << 16, m & 0xFFFF0000u);
    }
    // s * q rounded once to bf16 (the product is exact in binary32)
    static __device__ __forceinline__ uint4 narrow(const float (&v)[W]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvParams p) {
    constexpr int W = Unit<T>::W, kLanes = 32 / W;  // lanes of a block
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    Place o;
    const bool live = u < p.units && place<W>(p, u, o);
    uint4 raw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.in[i]) + o.token * p.ld[i] + o.at));
    }
    // the lanes of a block are together in a warp and of one token (per_token is a multiple of kLanes)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x[W];
        Unit<T>::widen(raw[i], x);
        // the largest magnitude as bits: infinities and NaN are above every number
        uint32_t top = Unit<T>::largest(raw[i]);
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        __half h;
        float sf;
        const uint32_t flags = block_scale(top, h, sf);
        uint32_t packed[W / 4] = {};
        if (!flags && sf != 0.0f) codes_of<T, W>(x, sf, packed);
        if (live) {
            if constexpr (W == 4)
                *reinterpret_cast<uint32_t *>(p.codes[i] + o.code) = packed[0];
            else
                *reinterpret_cast<uint2 *>(p.codes[i] + o.code) = make_uint2(packed[0], packed[1]);
            if (threadIdx.x % kLanes == 0) {
                p.scales[i][o.code >> 5] = flags ? 0 : __half_as_ushort(h);
                if (flags && p.status) atomicOr(p.status, flags);
            }
        }
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvParams p) {
    constexpr int W = Unit<T>::W;
    const uint32_t u = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) * N + (threadIdx.x & 31);  // and u + 32, ...
    Place o[N];
    bool live[N];
    uint2 c[N][2];
    float s[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) live[n] = u + 32 * n < p.units && place<W>(p, u + 32 * n, o[n]);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[n][i] = make_uint2(0u, 0u);
            s[n][i] = 0.f;
            if (live[n]) {
                if constexpr (W == 4)
                    c[n][i].x = *reinterpret_cast<const uint32_t *>(p.codes[i] + o[n].code);
                else
                    c[n][i] = *reinterpret_cast<const uint2 *>(p.codes[i] + o[n].code);
                s[n][i] = f16_bits_to_f32(p.scales[i][o[n].code >> 5]);
            }
        }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (u + 32 * n >= p.units) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[W];
            codes4_to_f32(c[n][i].x, x[0], x[1], x[2], x[3]);
            if constexpr (W == 8) codes4_to_f32(c[n][i].y, x[4], x[5], x[6], x[7]);
#pragma unroll
            for (int j = 0; j < W; ++j) x[j] *= s[n][i];
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.out[i]) + o[n].token * p.ld[i] + o[n].at) = Unit<T>::narrow(x);
        }
    }
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

q8_status launch_kv(const q8_kv_cache &c, bool append, const void *k, const void *v, int64_t ldk, int64_t ldv,
                    int32_t dtype, const int64_t *slots, int64_t T, uint32_t *dev_status, cudaStream_t stream) {
    KvParams p = {};
    p.codes[0] = c.kq, p.codes[1] = c.vq;
    p.scales[0] = c.ks, p.scales[1] = c.vs;
    p.ld[0] = ldk, p.ld[1] = ldv;
    p.status = dev_status;
    p.capacity = static_cast<int64_t>(c.pages) * c.page_size;
    const uint32_t width = dtype == Q8_DTYPE_F32 ? Unit<float>::W : Unit<__nv_bfloat16>::W;
    p.per_token = static_cast<uint32_t>(c.kv_heads) * static_cast<uint32_t>(c.head_dim) / width;
    // with 2^(s - 1) < per_token <= 2^s: floor(2^(31 + s) / per_token) + 1 exceeds the true factor by at
    // most 2^-(31 + s) of it times per_token, less than one part in u
    const int bits = ilog2(p.per_token);
    p.magic = static_cast<uint32_t>((uint64_t(1) << (31 + bits)) / p.per_token + 1);
    p.shift = static_cast<uint32_t>(bits - 1);
    p.page_shift = ilog2(c.page_size), p.d_shift = ilog2(c.head_dim), p.kv_heads = c.kv_heads;
    const size_t esize = dtype == Q8_DTYPE_F32 ? 4 : 2;
    // 32-bit unit indexes: runs of tokens of fewer than 2^30 units each
    const int64_t most = (int64_t(1) << 30) / p.per_token;
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        const int64_t n = T - t0 < most ? T - t0 : most;
        p.units = static_cast<uint32_t>(n * p.per_token);
        p.slots = slots + t0;
        const size_t offk = static_cast<size_t>(t0) * ldk * esize, offv = static_cast<size_t>(t0) * ldv * esize;
        p.in[0] = static_cast<const uint8_t *>(k) + offk, p.in[1] = static_cast<const uint8_t *>(v) + offv;
        p.out[0] = const_cast<void *>(p.in[0]), p.out[1] = const_cast<void *>(p.in[1]);
        const unsigned grid = (p.units + kThreads - 1) / kThreads;
        const bool f32 = dtype == Q8_DTYPE_F32;
        if (append)
            (f32 ? kv_append_kernel<float> : kv_append_kernel<__nv_bfloat16>)<<<grid, kThreads, 0, stream>>>(p);
        else if (p.units < kMany)
            (f32 ? kv_read_kernel<float, 1> : kv_read_kernel<__nv_bfloat16, 1>)<<<grid, kThreads, 0, stream>>>(p);
        else
            (f32 ? kv_read_kernel<float, 2> : kv_read_kernel<__nv_bfloat16, 2>)<<<(grid + 1) / 2, kThreads, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return Q8_ERR_CUDA;
    }
    return Q8_OK;
}

}  // namespace

q8_status launch_kv_append(const q8_kv_cache &c, const void *k, const void *v, int64_t ldk, int64_t ldv, int32_t dtype,
                           const int64_t *slots, int64_t T, uint32_t *dev_status, cudaStream_t stream) {
    return launch_kv(c, true, k, v, ldk, ldv, dtype, slots, T, dev_status, stream);
}

q8_status launch_kv_read(const q8_kv_cache &c, const int64_t *slots, int64_t T, void *k, void *v, int64_t ldk,
                         int64_t ldv, int32_t dtype, uint32_t *dev_status, cudaStream_t stream) {
    return launch_kv(c, false, k, v, ldk, ldv, dtype, slots, T, dev_status, stream);
}

}  // namespace q8
