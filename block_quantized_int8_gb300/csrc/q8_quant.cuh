// q8_quant.cuh -- the Q8_0 code of one value, shared by the weight quantizer, the key-value
// cache writes and the norm, and the codes and scale of a block that lanes share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q8.h"

namespace q8 {

// The code of v against the stored scale sf (rcp = 1 / sf rounded): the k with
// (k - 1/2) sf <= |v| < (k + 1/2) sf.  The estimate |v| * rcp is off by at
// most one; (k +- 1/2) * sf is exact in binary32, so one compare in each
// direction fixes it.
__device__ __forceinline__ int32_t code_of(float v, float sf, float rcp) {
    const float a = fabsf(v);
    float k = fminf(floorf(__fadd_rn(__fmul_rn(a, rcp), 0.5f)), 128.0f);
    if (__fmul_rn(__fadd_rn(k, 0.5f), sf) <= a) {
        k = __fadd_rn(k, 1.0f);
    } else if (k > 0.0f && __fmul_rn(__fsub_rn(k, 0.5f), sf) > a) {
        k = __fsub_rn(k, 1.0f);
    }
    const int32_t ki = static_cast<int32_t>(fminf(k, 127.0f));
    return v < 0.0f ? -ki : ki;
}

// The codes of W values by the scale sf, four to a word: |x| / sf rounded half away from zero.
// t = x * (1 / sf) is within 2^-16 of the quotient (at most 127.5), and adding 1.5 2^23 leaves its
// nearest integer in the low byte.
// bf16: x has 8 significant bits and sf 11, so a quotient that is no tie is at least 2^-12 from one
// (both are multiples of a power of two that small against sf); 2^-14 away from zero puts ties on the
// far side and nothing else across.  fp32: where t is within 2^-12 of a tie, the exact rule decides
// (one value in 2048).
template <typename T, int W>
__device__ __forceinline__ void codes_of(const float (&x)[W], float sf, uint32_t (&packed)[W / 4]) {
    constexpr float kMagic = 12582912.0f;
    const float rcp = __frcp_rn(sf);
    uint32_t c[W];
    bool close = false;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if constexpr (sizeof(T) == 2) {
            const float away = __uint_as_float(0x38800000u | (__float_as_uint(x[j]) & 0x80000000u));  // +- 2^-14
            c[j] = __float_as_uint(fminf(fmaxf(fmaf(x[j], rcp, away), -127.0f), 127.0f) + kMagic);
        } else {
            const float t = fminf(fmaxf(x[j] * rcp, -127.0f), 127.0f), z = t + kMagic;
            c[j] = __float_as_uint(z);
            close = close || fabsf(t - (z - kMagic)) > 0.5f - 0x1p-12f;
        }
    }
    if (sizeof(T) == 4 && close) {
#pragma unroll
        for (int j = 0; j < W; ++j) c[j] = static_cast<uint32_t>(code_of(x[j], sf, rcp));
    }
#pragma unroll
    for (int j = 0; j < W; j += 4)
        packed[j / 4] = __byte_perm(__byte_perm(c[j], c[j + 1], 0x0040), __byte_perm(c[j + 2], c[j + 3], 0x0040), 0x5410);
}

// A block whose largest magnitude has the bits `top` (infinities and NaN are above every
// number): its scale, and the flags of one that is stored as zeros.
__device__ __forceinline__ uint32_t block_scale(uint32_t top, __half &h, float &sf) {
    h = __float2half_rn(__fdiv_rn(__uint_as_float(top), 127.0f));
    sf = __half2float(h);
    return top >= 0x7F800000u ? Q8_DEV_NONFINITE : (isinf(sf) ? Q8_DEV_SCALE_OVF : 0u);
}

}  // namespace q8
