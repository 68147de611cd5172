// q8_norm.cu -- root-mean-square norm of rows, with the residual's addition before it and
// bf16 or Q8_0 rows (or both) after it, in one pass over the data.
//
//   h = x + residual;   y = h / sqrt(mean of h^2 + eps) * (weight + offset)
//
// A CTA has one row: a thread holds up to NU units of 8 neighbouring values in registers from
// the load to the store, so that each input is read once and each output written once; four
// neighbouring lanes hold a block of 32, whose largest magnitude they find by two shuffles.
// All sums are fp32, in an order that the width alone sets.
//
// Bound by bytes for many wide rows, by the launch for few, and for many narrow ones by the CTAs: a row of 64
// values keeps 8 lanes busy.  Measured on the device (events around one call, L2 flushed before it): 4099 rows of
// 4096 in bf16 onto a bf16 residual 27.3 to 28.3 us (4.7 TB/s), with Q8_0 rows besides 33.4 to 35.5 (4.3); in bf16 alone
// 81,920 rows of 512 48 us (3.5 TB/s), 163,840 of 256 89 (1.9), 655,360 of 64 336 (0.5, two CTAs a nanosecond).
// One unit a thread up to 256 units, then two and, past 1024, four: fewer and wider would leave
// narrow rows a few warps, more would give the widest rows more than 1024 threads.
//
// Squares overflow binary32 from |h| of 2^64 on and vanish below 2^-75, where the row's norm does
// neither: rows whose sum of squares is not within [2^-80, 2^126] (below it, only where eps does
// not cover it) are summed again, scaled by the power of two of their largest value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q8_dev.cuh"
#include "q8_internal.h"
#include "q8_quant.cuh"
#include "q8_rows.cuh"

namespace q8 {

namespace {

struct NormParams {
    const void *x, *res;
    void *res_out;
    const float *weight;
    uint16_t *y;
    int8_t *q;
    uint16_t *s;
    uint32_t *status;
    int64_t ldx, ldr, ldo, ldy;
    int32_t units, width;  // of 8 values; values
    float offset, eps;
};

// Sum (or largest) over the CTA, the same in every thread.
template <bool kMax>
__device__ __forceinline__ float block_all(float v, float *s_part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    if (warps == 1) return v;
    __syncthreads();  // an earlier sum's parts have been read
    if (lane == 0) s_part[warp] = v;
    __syncthreads();
    v = lane < warps ? s_part[lane] : 0.f;
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    return v;
}

template <typename TX, typename TR, int NU>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float s_part[32];
    const int64_t row = blockIdx.x;
    const TX *x = static_cast<const TX *>(p.x) + row * p.ldx;
    const TR *r = p.res ? static_cast<const TR *>(p.res) + row * p.ldr : nullptr;
    float h[NU][8];
    {
        Raw8<TX> rx[NU];
        Raw8<TR> rr[NU];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = threadIdx.x + n * blockDim.x;
            if (u < p.units) {
                rx[n].load(x + 8 * u);
                if (r) rr[n].load(r + 8 * u);
            }
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = threadIdx.x + n * blockDim.x;
            if (u < p.units) {
                rx[n].widen(h[n]);
                if (r) {
                    float b[8];
                    rr[n].widen(b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[n][i] += b[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[n][i] = 0.f;
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[n][i], h[n][i], ss);
    ss = block_all<false>(ss, s_part);
    const float inv_w = 1.0f / static_cast<float>(p.width);
    float scale = rsqrtf(ss * inv_w + p.eps), before = 1.f;  // y = (h before) scale (weight + offset)
    if (!(ss <= 0x1p126f) || (ss < 0x1p-80f && p.eps < 0x1p-80f)) {
        float top = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(h[n][i]));  // passes NaN over: ss has it
        top = block_all<true>(top, s_part);
        // 2^-e with top 2^-e in [1, 2), within the normal powers
        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
        const float f = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        float s2 = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) s2 = fmaf(h[n][i] * f, h[n][i] * f, s2);
        s2 = block_all<false>(s2, s_part);
        if (isinf(top)) {
            scale = ss != ss ? ss : 0.f;  // an infinity over infinity is NaN, a number over it 0
        } else if (top == 0.f && ss == 0.f) {
            scale = p.eps > 0.f ? scale : 0.f;
        } else if (p.eps * f * f > 0x1p100f) {
            scale = rsqrtf(p.eps);  // the row's values are below 2^-50 of eps's root
        } else {
            before = f;
            scale = rsqrtf(s2 * inv_w + p.eps * f * f);
        }
    }

#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = threadIdx.x + n * blockDim.x;
        const bool live = u < p.units;
        if (live && p.res_out) store8(static_cast<TR *>(p.res_out) + row * p.ldo + 8 * u, h[n]);
        float y[8];
        if (live && p.weight) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * u);
            const float4 b = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * u + 1);
            const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[n][i] * before * scale * (w[i] + p.offset);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[n][i] * before * scale;
        }
        if (live && p.y) store8(reinterpret_cast<__nv_bfloat16 *>(p.y) + row * p.ldy + 8 * u, y);
        if (p.q) {
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            __half hs;
            float sf;
            const uint32_t flags = block_scale(top, hs, sf);
            uint32_t packed[2] = {0u, 0u};
            if (!flags && sf != 0.f) codes_of<float, 8>(y, sf, packed);
            if (live) {
                *reinterpret_cast<uint2 *>(p.q + row * p.width + 8 * u) = make_uint2(packed[0], packed[1]);
                if ((threadIdx.x & 3) == 0) {
                    p.s[(row * p.width + 8 * u) >> 5] = flags ? 0 : __half_as_ushort(hs);
                    if (flags && p.status) atomicOr(p.status, flags);
                }
            }
        }
    }
}

template <typename TX, typename TR>
void launch(const NormParams &p, int64_t rows, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(rows);
    const auto threads = [&](int nu) { return static_cast<unsigned>(((p.units + nu - 1) / nu + 31) / 32 * 32); };
    if (p.units <= 256)
        norm_kernel<TX, TR, 1><<<grid, threads(1), 0, stream>>>(p);
    else if (p.units <= 1024)
        norm_kernel<TX, TR, 2><<<grid, threads(2), 0, stream>>>(p);
    else
        norm_kernel<TX, TR, 4><<<grid, threads(4), 0, stream>>>(p);
}

}  // namespace

q8_status launch_norm(const NormArgs &a, uint32_t *dev_status, cudaStream_t stream) {
    NormParams p = {a.x, a.residual, a.residual_out, a.weight, a.y, a.q, a.s, dev_status, a.ldx, a.ldr, a.ldo, a.ldy,
                    a.width / 8, a.width, a.offset, a.eps};
    const bool xf = a.x_dtype == Q8_DTYPE_F32, rf = a.r_dtype == Q8_DTYPE_F32;
    if (xf)
        rf ? launch<float, float>(p, a.rows, stream) : launch<float, __nv_bfloat16>(p, a.rows, stream);
    else
        rf ? launch<__nv_bfloat16, float>(p, a.rows, stream) : launch<__nv_bfloat16, __nv_bfloat16>(p, a.rows, stream);
    return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
