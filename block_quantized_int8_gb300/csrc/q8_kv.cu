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
// 2) bytes in and 1.0625 out for the write, the reverse for the read.  Four
// lanes own one block, 8 values each: a lane's loads are 16 bytes, its code
// store 8, and a warp's stores cover whole 32-byte sectors.  Each thread
// takes the same position of the keys and of the values, so two independent
// loads are in flight per thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q8_dev.cuh"
#include "q8_internal.h"
#include "q8_quant.cuh"

namespace q8 {

namespace {

constexpr int kThreads = 256;

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
    uint32_t per_token;    // kv_heads * D / 8
    int32_t page_shift, d_shift, kv_heads;
};

// Unit u is 8 values of one token: where they are in the input or output row
// and in the cache.  false if the token has no slot (padding, or a slot that
// does not exist, which is flagged).
struct Place {
    uint32_t token, at;  // `at`: value offset within the token's row
    int64_t code;        // element offset into the codes
};
__device__ __forceinline__ bool place(const KvParams &p, uint32_t u, Place &o) {
    o.token = u / p.per_token;
    o.at = (u - o.token * p.per_token) * 8;
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

template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <>
struct Eight<__nv_bfloat16> {
    float v[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo_f32(w[i]), v[2 * i + 1] = bf16hi_f32(w[i]);
    }
    // s * q rounded once to bf16 (the product is exact in binary32)
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvParams p) {
    const uint32_t stride = gridDim.x * kThreads;
    // whole warps stay in the loop: the four lanes of a block are always
    // together (per_token is a multiple of 8), tails are masked
    const uint32_t end = (p.units + 31u) & ~31u;
    for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < end; u += stride) {
        Place o;
        const bool live = u < p.units && place(p, u, o);
        Eight<T> x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i].v[j] = 0.f;
            if (live) x[i].load(static_cast<const T *>(p.in[i]) + o.token * p.ld[i] + o.at);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float amax = 0.f;
            uint32_t bad = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                amax = fmaxf(amax, fabsf(x[i].v[j]));
                bad |= isfinite(x[i].v[j]) ? 0u : 1u;
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                bad |= __shfl_xor_sync(0xffffffffu, bad, off);
            }
            const __half h = __float2half_rn(__fdiv_rn(amax, 127.0f));
            const float sf = __half2float(h);
            const uint32_t flags = bad ? Q8_DEV_NONFINITE : (isinf(sf) ? Q8_DEV_SCALE_OVF : 0u);
            uint2 packed = make_uint2(0u, 0u);
            uint16_t sbits = flags ? 0 : __half_as_ushort(h);
            if (!flags && sf != 0.0f) {
                const float rcp = __frcp_rn(sf);
                uint32_t c[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = static_cast<uint32_t>(code_of(x[i].v[j], sf, rcp)) & 0xFFu;
                packed.x = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
                packed.y = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
            }
            if (live) {
                *reinterpret_cast<uint2 *>(p.codes[i] + o.code) = packed;
                if ((u & 3) == 0) {
                    p.scales[i][o.code >> 5] = sbits;
                    if (flags && p.status) atomicOr(p.status, flags);
                }
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvParams p) {
    const uint32_t stride = gridDim.x * kThreads;
    for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < p.units; u += stride) {
        Place o;
        const bool live = place(p, u, o);
        uint2 c[2];
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = live ? *reinterpret_cast<const uint2 *>(p.codes[i] + o.code) : make_uint2(0u, 0u);
            s[i] = live ? f16_bits_to_f32(p.scales[i][o.code >> 5]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            Eight<T> x;
            codes4_to_f32(c[i].x, x.v[0], x.v[1], x.v[2], x.v[3]);
            codes4_to_f32(c[i].y, x.v[4], x.v[5], x.v[6], x.v[7]);
#pragma unroll
            for (int j = 0; j < 8; ++j) x.v[j] *= s[i];
            x.store(static_cast<T *>(p.out[i]) + o.token * p.ld[i] + o.at);
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
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    KvParams p = {};
    p.codes[0] = c.kq, p.codes[1] = c.vq;
    p.scales[0] = c.ks, p.scales[1] = c.vs;
    p.ld[0] = ldk, p.ld[1] = ldv;
    p.status = dev_status;
    p.capacity = static_cast<int64_t>(c.pages) * c.page_size;
    p.per_token = static_cast<uint32_t>(c.kv_heads) * static_cast<uint32_t>(c.head_dim) / 8;
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
        const int64_t want = (static_cast<int64_t>(p.units) + kThreads - 1) / kThreads;
        const int64_t cap = static_cast<int64_t>(di->sm_count) * 8;
        const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
        if (append) {
            if (dtype == Q8_DTYPE_F32)
                kv_append_kernel<float><<<grid, kThreads, 0, stream>>>(p);
            else
                kv_append_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
        } else {
            if (dtype == Q8_DTYPE_F32)
                kv_read_kernel<float><<<grid, kThreads, 0, stream>>>(p);
            else
                kv_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
        }
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
