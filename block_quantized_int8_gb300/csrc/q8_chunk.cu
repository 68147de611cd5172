// q8_chunk.cu -- attention of each sequence's newest tokens over a paged Q8_0 key-value cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q8_dev.cuh"
#include "q8_internal.h"

namespace q8 {

namespace {

struct ChunkParams {
    q8_kv_cache c;
    ChunkArgs a;
    uint32_t *status;
    int32_t page_shift;
};

// A block's scale, 0 (and flagged) where it is not finite.
__device__ __forceinline__ float scale_of(uint16_t bits, uint32_t *status) {
    if ((bits & 0x7C00u) != 0x7C00u) return f16_bits_to_f32(bits);
    if (status) atomicOr(status, Q8_DEV_NONFINITE);
    return 0.f;
}

// One warp per query head of (row, key head): scores of 32 tokens at a time, one a lane.
template <int D>
__global__ void __launch_bounds__(128) chunk_simple_kernel(const __grid_constant__ ChunkParams p) {
    const int row = blockIdx.x, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ChunkArgs &a = p.a;
    int b = -1, t0 = 0, n = 0;
    if (row == 0 && kvh == 0 && threadIdx.x == 0 && p.status) {
        for (int i = 0; i < a.batch; ++i) {
            const int s0 = a.starts[i], s1 = a.starts[i + 1], l = a.lens[i];
            if (s0 < 0 || s1 < s0 || s1 > a.T || l < 0 || l > a.table_width << p.page_shift || l < s1 - s0)
                atomicOr(p.status, Q8_DEV_BAD_INDEX);
        }
    }
    for (int i = 0; i < a.batch; ++i) {
        const int s0 = min(max(a.starts[i], 0), static_cast<int>(a.T)), s1 = min(max(a.starts[i + 1], s0), static_cast<int>(a.T));
        if (row >= s0 && row < s1) b = i, t0 = s0, n = s1 - s0;
    }
    if (b < 0) return;
    const int len = min(max(a.lens[b], 0), a.table_width << p.page_shift);
    const int pos = len - n + (row - t0);
    const int first = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const int group = a.q_heads / p.c.kv_heads;
    for (int g = warp; g < group; g += 4) {
        const int head = kvh * group + g;
        const uint16_t *q = a.q + row * a.ldq + static_cast<int64_t>(head) * D;
        float m = -INFINITY, l = 0.f, o[D / 32] = {};
        for (int t = first; t <= pos; t += 32) {
            const int tok = t + lane;
            float s = -INFINITY;
            int64_t base = -1;
            if (tok <= pos) {
                const int pg = a.table[static_cast<int64_t>(b) * a.table_width + (tok >> p.page_shift)];
                if (static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.c.pages)) {
                    base = ((static_cast<int64_t>(pg) * p.c.kv_heads + kvh) << p.page_shift) + (tok & ((1 << p.page_shift) - 1));
                    s = 0.f;
                    for (int d = 0; d < D; ++d)
                        s += __uint_as_float(static_cast<uint32_t>(q[d]) << 16) *
                             (p.c.kq[base * D + d] * scale_of(p.c.ks[(base * D + d) >> 5], p.status));
                    s *= a.scale;
                    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
                } else if (p.status) {
                    atomicOr(p.status, Q8_DEV_BAD_INDEX);
                }
            }
            if (__any_sync(0xffffffffu, s != s)) {  // a query of NaN or infinity: so is the row
                l = NAN, m = 0.f;
                continue;
            }
            float top = s;
            for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            top = fmaxf(top, m);
            if (top == -INFINITY) continue;
            const float f = expf(m - top), w = expf(s - top);
            m = top;
            l = l * f + w;
            for (int i = 0; i < D / 32; ++i) o[i] *= f;
            for (int j = 0; j < 32; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                const int64_t bj = __shfl_sync(0xffffffffu, base, j);
                if (bj < 0) continue;
                for (int i = 0; i < D / 32; ++i)
                    o[i] += wj * (p.c.vq[bj * D + 32 * i + lane] * scale_of(p.c.vs[bj * (D / 32) + i], p.status));
            }
        }
        for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
        const int64_t at = static_cast<int64_t>(row) * a.q_heads + head;
        for (int i = 0; i < D / 32; ++i)
            reinterpret_cast<__nv_bfloat16 *>(a.out)[at * D + 32 * i + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
        if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : m + logf(l);
    }
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

}  // namespace

size_t chunk_workspace(int, int, int) { return Q8_CHUNK_ZEROED_BYTES; }

q8_status launch_chunk(const q8_kv_cache &c, const ChunkArgs &a, void *, uint32_t *dev_status, cudaStream_t stream) {
    const ChunkParams p = {c, a, dev_status, ilog2(c.page_size)};
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(c.kv_heads));
    if (c.head_dim == 64) chunk_simple_kernel<64><<<grid, 128, 0, stream>>>(p);
    else if (c.head_dim == 128) chunk_simple_kernel<128><<<grid, 128, 0, stream>>>(p);
    else chunk_simple_kernel<256><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace q8
