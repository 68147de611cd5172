// q8_quant.cuh -- the Q8_0 code of one value, shared by the weight quantizer
// and the key-value cache write.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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

}  // namespace q8
