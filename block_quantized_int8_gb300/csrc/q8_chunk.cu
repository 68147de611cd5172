// q8_chunk.cu -- attention of each sequence's newest tokens over a paged Q8_0 key-value cache, on
// the 5th generation tensor cores (tcgen05, tensor-memory accumulators).
//
// Mathematics.  As in q8_attn.cu: with s_t = scale * q . k_t in units of log 2 and any reference m,
// out = (sum_t 2^(s_t - m) v_t) / (sum_t 2^(s_t - m)).  A row walks tiles of BN tokens keeping
// (m, l, O); the reference is set 11 below the largest score, so that weights use binary16's range
// downwards, and moved only when a score passes it by 15; then O is multiplied in tensor memory.
// Two such triples join into (max m, ...), which is how CTAs that share a row's tokens are put
// together, in CTA order.
//
// An item is (sequence, run of 128 MT rows, key head), a row being (new token, query head of the
// key head's group): all heads of a group share the dequantised keys and values.  Per tile
//   S = Q K^T   (M = 128 rows, N = BN tokens, both operands from shared memory)
//   P = 2^(S - m), binary16, back into S's columns of tensor memory
//   O += P V    (A from tensor memory, B = V as it lies: [token][dimension])
// for each of MT tiles of 128 rows, whose softmaxes take turns with each other's products.
//
// Operands are binary16: a query row is scaled by a power of two (its bf16 values are then exact
// down to 2^-31 of its largest), keys and values are s * code rounded once (by 2^-11 of themselves;
// exact where the scale is subnormal, as all are whole multiples of 2^-24).  Tiles with a scale of
// 512 or more, whose products could overflow, are taken times 2^-9: the scores get the factor
// back, the weights are raised by 2^9 instead (their reference moves up for it).
//
// Roles (one CTA per SM):
//   softmax     4 warps per row tile, a thread per row: scores from tensor memory in two passes (the
//               largest, then the weights); the query rows into shared memory before an item, the answer after it
//   MMA         one warp, one thread of it issuing
//   loader      one warp: bulk copies of codes and scales, 16 tokens (a page's smallest part) each,
//               into a ring of raw tiles
//   converters  CW warps: codes times scales into a ring of binary16 tiles, in the 128-byte
//               swizzle that the tensor cores read: K-major for the keys, and the same bytes as
//               MN-major for the values, so nothing is transposed
//
// Split: units of one tile are counted out evenly over the CTAs from the device's lengths, as in
// q8_attn.cu; an item that crosses CTAs is joined by the last of them to arrive.
//
// All mbarrier waits are bounded; on expiry the CTA reports Q8_DEV_TIMEOUT, every wait gives up at
// once, and each role walks on to its end without work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>

#include "q8_async.cuh"
#include "q8_dev.cuh"
#include "q8_internal.h"
#include "q8_rows.cuh"

namespace q8 {

namespace {

constexpr int kMaxGrid = 160;   // CTAs a launch may have (sizes the workspace)
constexpr int kEndUnits = 3;    // what beginning and ending an item takes, in units' time
constexpr int kMinUnits = 2;    // units a CTA takes at least
constexpr int kScan = 512;      // sequences looked at together
constexpr float kLift = 11.0f;  // log2 of the largest weight when the reference is set
constexpr float kTop = 15.0f;   // and of the largest that leaves it
constexpr float kLiftEnd = 0x1p23f;  // magnitude of a score from which on there is neither
constexpr float kPlain = 0x1p20f;    // below it a score's rounding moves a weight by less than a factor 1.1
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSmemMax = 232448;

struct ChunkParams {
    const int8_t *kq, *vq;
    const uint16_t *ks, *vs;
    const uint16_t *q;
    const int32_t *table, *lens, *starts;
    uint16_t *out;
    float *lse;
    uint32_t *tickets;  // [2 * kMaxGrid][2]
    float *parts;       // [2 * kMaxGrid][MT][(D + 2) * 128]
    uint32_t *status;
    int64_t ldq;
    int32_t T, batch, q_heads, kv_heads, group;
    int32_t table_width, pages, page_shift, window;
    float scale, softcap;
};

// ---- tcgen05 --------------------------------------------------------------------
// Shared-memory matrix descriptor, 128-byte swizzle, 8-row groups 1024 bytes apart; `lead`: bytes
// between runs of 64 elements (MN-major operands of more than 64).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// Instruction descriptor, kind::f16: D f32, A and B f16, M = 128; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
           "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
           "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- small things -----------------------------------------------------------------
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
    return static_cast<unsigned long long>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t *p, uint32_t v) {
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void named_bar(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ bool named_bar_or(int id, int threads, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "barrier.cta.red.or.aligned.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"(v ? 1u : 0u), "r"(id), "r"(threads) : "memory");
    return r != 0;
}

// ---- shapes -------------------------------------------------------------------------
template <int D_, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr int BN = D == 256 ? 64 : 128;          // tokens of a tile
    static constexpr int RT = 128 * MT;                     // rows of an item
    static constexpr int CW = MT == 2 ? 6 : 8;              // converter warps (16 warps at most: 128 registers a thread)
    static constexpr int kSoftmax = 4 * MT;                 // softmax warps
    static constexpr int kWarps = kSoftmax + 2 + CW;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kQ = 256 * D;                      // bytes of a query tile
    static constexpr int kTile = BN * D * 2;                // bytes of a binary16 tile
    static constexpr int kChunk = BN * 128;                 // bytes of its first 64 dimensions
    static constexpr int kCodes = BN * D, kScales = BN * D / 16;
    static constexpr int kRaw = kCodes + kScales;
    static constexpr int NR = 3;                            // binary16 tiles
    static constexpr int kFixed = MT * kQ + NR * kTile;
    static constexpr int kRoom = (kSmemMax - 1024 - 1024 - kFixed) / kRaw;
    static constexpr int NW = kRoom < 6 ? kRoom : 6;        // raw tiles
    static constexpr int kRawAt = kFixed;
    static constexpr int kSmem = 1024 + kFixed + NW * kRaw;
    static constexpr int kPart = (D + 2) * 128;             // floats of a row tile's part
    static constexpr int kColO = 2 * BN;                    // first tensor-memory column of O
    static_assert(NW >= 2 && 2 * BN + MT * D <= 512, "shared and tensor memory");
};

struct Control {
    uint64_t raw_full[8], raw_empty[8];
    uint64_t t_full[4], t_empty[4];
    uint64_t s_full[2], p_full[2], q_full[2], pv_done[2];
    uint32_t runs[8];       // of a raw tile: which runs of 16 tokens were loaded
    uint32_t info[4];       // of the last tiles: bits 0-7 runs that must not be seen, 8 keys times 2^-9, 9 values
    uint32_t tmem, last[2];
    int32_t abort_flag;
    int32_t start;          // the sequence that this CTA begins in, and what the list holds before it
    long long before;
    long long sums[kScan / 32 + 1];
};

// ---- the list of items ------------------------------------------------------------------
struct Seq {
    int t0, n, len, pos0;  // first row of q, rows, tokens, position of the first row
};
__device__ __forceinline__ Seq seq_of(const ChunkParams &p, int b, uint32_t *status) {
    Seq s;
    const int a = p.starts[b], e = p.starts[b + 1], l = p.lens[b];
    s.t0 = min(max(a, 0), p.T);
    s.n = min(max(e, s.t0), p.T) - s.t0;
    s.len = min(max(l, 0), p.table_width << p.page_shift);
    s.pos0 = s.len - s.n;
    if (status && (a != s.t0 || e != s.t0 + s.n || l != s.len || s.pos0 < 0)) atomicOr(status, Q8_DEV_BAD_INDEX);
    return s;
}
// The tokens that rows [qt RT, (qt + 1) RT) of a sequence see: base (a multiple of 16), end, tiles.
template <class C>
__device__ __forceinline__ int tile_units(const ChunkParams &p, const Seq &s, int qt, int &base, int &end) {
    const int r0 = qt * C::RT, r1 = min(r0 + C::RT, s.n * p.group);
    end = s.pos0 + (r1 - 1) / p.group + 1;
    base = 0;
    if (end <= 0) return 0;
    if (p.window > 0) {
        const int64_t first = static_cast<int64_t>(s.pos0) + r0 / p.group + 1 - p.window;
        base = first > 0 ? static_cast<int>(first) & ~15 : 0;
    }
    return (end - base + C::BN - 1) / C::BN;
}
template <class C>
__device__ __forceinline__ int seq_tiles(const ChunkParams &p, const Seq &s) { return (s.n * p.group + C::RT - 1) / C::RT; }

template <class C>
struct Walk {
    int b, qt, kvh, unit;
    int units, base, end, nq;
    Seq s;
    __device__ __forceinline__ void enter(const ChunkParams &p) {
        s = seq_of(p, b, nullptr);
        nq = seq_tiles<C>(p, s);
        units = tile_units<C>(p, s, qt, base, end);
    }
    // the next item (the caller knows that there is one)
    __device__ __forceinline__ void next(const ChunkParams &p) {
        unit = 0;
        if (++kvh < p.kv_heads) return;
        kvh = 0;
        while (true) {
            if (++qt >= nq) {
                if (b + 1 >= p.batch) return;
                qt = 0;
                ++b;
                s = seq_of(p, b, nullptr);
                nq = seq_tiles<C>(p, s);
                if (nq == 0) continue;
            }
            units = tile_units<C>(p, s, qt, base, end);
            if (units > 0) return;
        }
    }
};

template <class C>
__device__ __forceinline__ bool wait_for(Control &sm, const ChunkParams &p, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int32_t *>(&sm.abort_flag)) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicExch(&sm.abort_flag, 1);
            if (p.status) atomicOr(p.status, Q8_DEV_TIMEOUT);
            return false;
        }
    }
}

template <int D_, int MT_>
__global__ void __launch_bounds__(Cfg<D_, MT_>::kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<D_, MT_>;
    constexpr int D = C::D, MT = C::MT, BN = C::BN, NR = C::NR, NW = C::NW;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control sm;
    static_assert(sizeof(Control) <= 1024, "static shared memory");
    uint8_t *const base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the list is looked at in the room of the binary16 tiles
    long long *const s_cost = reinterpret_cast<long long *>(base + MT * C::kQ);
    int32_t (*const s_seq)[kScan] = reinterpret_cast<int32_t (*)[kScan]>(s_cost + kScan);
    static_assert(24 * kScan <= NR * C::kTile, "room for the list");

    if (tid == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&sm.raw_full[i], 1), mbar_init(&sm.raw_empty[i], C::CW);
        for (int i = 0; i < 4; ++i) mbar_init(&sm.t_full[i], C::CW), mbar_init(&sm.t_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1), mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.q_full[i], 4), mbar_init(&sm.pv_done[i], 1);
        }
        sm.abort_flag = 0;
        sm.start = 0;
        fence_mbar_init();
    }

    // ---- how long the list is, and where this CTA begins --------------------------------------
    // cost of a sequence: for each of its row tiles that see something, kv_heads items of (units + kEndUnits)
    auto scan = [&](int b0, bool flag) -> long long {  // s_cost[i]: sum up to and with sequence b0 + i; returns the sum of all
        __syncthreads();
        const int held = min(kScan, p.batch - b0);
        for (int i = tid; i < held; i += C::kThreads) {
            const Seq s = seq_of(p, b0 + i, flag ? p.status : nullptr);
            s_seq[0][i] = s.t0, s_seq[1][i] = s.n, s_seq[2][i] = s.len, s_seq[3][i] = s.pos0;
        }
        __syncthreads();
        for (int i = warp; i < held; i += C::kWarps) {
            const Seq s = {s_seq[0][i], s_seq[1][i], s_seq[2][i], s_seq[3][i]};
            const int nq = seq_tiles<C>(p, s);
            long long sum = 0;
            for (int qt = lane; qt < nq; qt += 32) {
                int x, y;
                const int u = tile_units<C>(p, s, qt, x, y);
                sum += u > 0 ? u + kEndUnits : 0;
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) s_cost[i] = sum * p.kv_heads;
        }
        __syncthreads();
        // running sums within 32 sequences, and of all before them
        for (int w = warp; w < kScan / 32; w += C::kWarps) {
            const int i = 32 * w + lane;
            long long run = i < held ? s_cost[i] : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            s_cost[i] = run;
        }
        __syncthreads();
        if (warp == 0) {
            const long long own = lane < kScan / 32 ? s_cost[32 * lane + 31] : 0;
            long long run = own;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            if (lane <= kScan / 32) sm.sums[lane] = run - own;
        }
        __syncthreads();
        return sm.sums[kScan / 32];
    };
    static_assert(kScan / 32 < 32, "one warp sums the sums");
    long long total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kScan) total += scan(b0, blockIdx.x == 0);
    const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinUnits));
    const long long u0 = per * blockIdx.x, u1 = min(u0 + per, total);

    // rows whose tile sees nothing (more rows than tokens): their answer
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        const Seq s = seq_of(p, b, nullptr);
        if (s.pos0 >= 0 || s.n == 0) continue;
        const int rows = s.n * p.group, blind = -s.pos0 >= s.n ? rows : -s.pos0 * p.group / C::RT * C::RT;
        for (int kvh = 0; kvh < p.kv_heads; ++kvh)
            for (int r = warp; r < blind; r += C::kWarps) {
                const int64_t at = static_cast<int64_t>(s.t0 + r / p.group) * p.q_heads + kvh * p.group + r % p.group;
                for (int i = lane; i < D / 8; i += 32) reinterpret_cast<uint4 *>(p.out + at * D)[i] = make_uint4(0, 0, 0, 0);
                if (p.lse && lane == 0) p.lse[at] = -INFINITY;
            }
    }
    if (u0 >= u1) return;

    long long begin = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kScan) {
        const long long all = p.batch > kScan ? scan(b0, false) : total;
        if (begin + all > u0) {
            const int held = min(kScan, p.batch - b0);
            for (int i = tid; i < held; i += C::kThreads) {
                const long long up = begin + sm.sums[i >> 5] + s_cost[i];
                const long long down = i == 0 ? begin : begin + sm.sums[(i - 1) >> 5] + s_cost[i - 1];
                if (down <= u0 && u0 < up) sm.start = b0 + i, sm.before = down;
            }
            break;
        }
        begin += all;
    }
    __syncthreads();
    Walk<C> wk;
    long long left = u1 - u0, item0;
    wk.b = sm.start;
    wk.qt = wk.kvh = wk.unit = 0;
    wk.enter(p);
    {
        // every warp finds the row tile for itself, 32 at a time
        long long before = sm.before;
        int qt = 0, u = 0;
        for (int q0 = 0; q0 < wk.nq; q0 += 32) {
            int x, y;
            u = q0 + lane < wk.nq ? tile_units<C>(p, wk.s, q0 + lane, x, y) : 0;
            const long long c = u > 0 ? static_cast<long long>(u + kEndUnits) * p.kv_heads : 0;
            long long run = c;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, before + run > u0);
            if (hit) {
                const int src = __ffs(hit) - 1;
                qt = q0 + src;
                before += __shfl_sync(0xffffffffu, run - c, src);
                break;
            }
            before += __shfl_sync(0xffffffffu, run, 31);
        }
        wk.qt = qt;
        wk.enter(p);
        const int cost = wk.units + kEndUnits;
        const long long in = u0 - before;
        wk.kvh = static_cast<int>(in / cost);
        wk.unit = static_cast<int>(in - static_cast<long long>(wk.kvh) * cost);
        item0 = u0 - wk.unit;
        if (wk.unit >= wk.units) {  // at the end of an item that others work on: begin with the next
            left -= cost - wk.unit;
            item0 += cost;
            if (left > 0) wk.next(p);
        }
    }
    if (left <= 0) return;

    if (warp == C::kSoftmax) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const uint32_t q_at = smem_addr(base), tile_at = q_at + MT * C::kQ, raw_at = q_at + C::kRawAt;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, wait_for<C>(sm, p, bar, parity & 1u));
    };

    if (warp == C::kSoftmax) {
        // ------------------------------------------------------------------ MMA
        uint32_t c = 0, items = 0;  // tiles, items so far
        const auto bar_of = [&](uint32_t pos) { return pos % NR; };
        while (left > 0) {
            const int seg = static_cast<int>(min(left, static_cast<long long>(wk.units - wk.unit)));
            auto qk = [&](int m, uint32_t tile) {  // scores of row tile m, tile `tile`
                const uint32_t pos = 2 * tile, slot = bar_of(pos);
                const uint32_t buf = MT == 2 ? m : (tile & 1);
                if (ok && lane == 0) {
                    const uint64_t a = sw128_desc(q_at + m * C::kQ, 16), b = sw128_desc(tile_at + slot * C::kTile, 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_ss(tmem + buf * BN, a + ((k / 4) * 16384 + (k % 4) * 32) / 16, b + ((k / 4) * C::kChunk + (k % 4) * 32) / 16,
                                idesc(BN, false), k > 0);
                    umma_commit(&sm.s_full[buf]);
                    if (m == MT - 1) umma_commit(&sm.t_empty[slot]);
                }
                __syncwarp();
            };
            for (int m = 0; m < MT; ++m) wait(&sm.q_full[m], items);
            wait(&sm.t_full[bar_of(2 * c)], 2 * c / NR);
            tc_fence_after();
            for (int m = 0; m < MT; ++m) qk(m, c);
            for (int j = 0; j < seg; ++j, ++c) {
                const bool more = j + 1 < seg;
                const uint32_t vpos = 2 * c + 1, vslot = bar_of(vpos);
                if (MT == 1 && more) {
                    wait(&sm.t_full[bar_of(2 * c + 2)], (2 * c + 2) / NR);
                    tc_fence_after();
                    qk(0, c + 1);
                }
                wait(&sm.t_full[vslot], vpos / NR);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint32_t buf = MT == 2 ? m : (c & 1);
                    wait(&sm.p_full[buf], MT == 2 ? c : c >> 1);
                    tc_fence_after();
                    if (ok && lane == 0) {
                        const uint64_t b = sw128_desc(tile_at + vslot * C::kTile, C::kChunk);
#pragma unroll
                        for (int k = 0; k < BN / 16; ++k)
                            umma_ts(tmem + C::kColO + m * D, tmem + buf * BN + 8 * k, b + 2048 * k / 16, idesc(D, true), j > 0 || k > 0);
                        umma_commit(&sm.pv_done[m]);
                        if (m == MT - 1) umma_commit(&sm.t_empty[vslot]);
                    }
                    __syncwarp();
                    if (MT == 2 && more) {
                        if (m == 0) {
                            wait(&sm.t_full[bar_of(2 * c + 2)], (2 * c + 2) / NR);
                            tc_fence_after();
                        }
                        qk(m, c + 1);
                    }
                }
            }
            ++items;
            left -= seg + kEndUnits;
            if (left > 0) wk.next(p);
        }
    } else if (warp == C::kSoftmax + 1) {
        // --------------------------------------------------------------- loader
        uint32_t pos = 0;
        const int page_mask = (1 << p.page_shift) - 1;
        while (left > 0) {
            const int seg = static_cast<int>(min(left, static_cast<long long>(wk.units - wk.unit)));
            const int32_t *row = p.table + static_cast<int64_t>(wk.b) * p.table_width;
            auto page_of = [&](int j) {
                const int tok = wk.base + (wk.unit + j) * BN + 16 * lane;
                return j < seg && lane < BN / 16 && tok < wk.end ? row[tok >> p.page_shift] : -1;
            };
            int page = page_of(0);
            for (int j = 0; j < seg; ++j) {
                const int tok = wk.base + (wk.unit + j) * BN + 16 * lane;
                const bool in = lane < BN / 16 && tok < wk.end;
                const bool good = in && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages);
                const uint32_t runs = __ballot_sync(0xffffffffu, good);
                if (in && !good && p.status) atomicOr(p.status, Q8_DEV_BAD_INDEX);
                const int64_t at = ((static_cast<int64_t>(good ? page : 0) * p.kv_heads + wk.kvh) << p.page_shift) + (tok & page_mask);
                page = page_of(j + 1);
#pragma unroll
                for (int v = 0; v < 2; ++v, ++pos) {
                    const uint32_t slot = pos % NW;
                    if (pos >= NW) wait(&sm.raw_empty[slot], pos / NW - 1);
                    if (!ok) continue;
                    if (lane == 0) {
                        sm.runs[slot] = runs;
                        mbar_arrive_expect_tx(&sm.raw_full[slot], __popc(runs) * 17 * D);
                    }
                    __syncwarp();
                    if (good) {
                        uint8_t *to = base + C::kRawAt + slot * C::kRaw;
                        bulk_g2s(to + lane * 16 * D, (v ? p.vq : p.kq) + at * D, 16 * D, &sm.raw_full[slot]);
                        bulk_g2s(to + C::kCodes + lane * D, (v ? p.vs : p.ks) + at * (D / 32), D, &sm.raw_full[slot]);
                    }
                }
            }
            left -= seg + kEndUnits;
            if (left > 0) wk.next(p);
        }
    } else if (warp > C::kSoftmax) {
        // ----------------------------------------------------------- converters
        constexpr int kCT = C::CW * 32;
        const int ct = tid - (C::kSoftmax + 2) * 32;
        uint32_t pos = 0;
        while (left > 0) {
            const int seg = static_cast<int>(min(left, static_cast<long long>(wk.units - wk.unit)));
            for (int jj = 0; jj < 2 * seg; ++jj, ++pos) {
                const int j = jj >> 1;
                const bool is_v = jj & 1;
                const int tok0 = wk.base + (wk.unit + j) * BN;
                const uint32_t slot = pos % NW, to = pos % NR;
                const uint32_t raw = raw_at + slot * C::kRaw, scales = raw + C::kCodes;
                wait(&sm.raw_full[slot], pos / NW);
                // scales: of tokens that are not there 0, of what is not finite 0; are there any of 512 and more?
                const uint32_t runs = ok ? sm.runs[slot] : 0u;
                const int here = min(BN, wk.end - tok0);  // tokens of this tile
                const bool whole = runs == (1u << (BN / 16)) - 1u && here == BN;
                constexpr int kWords = BN * D / 64;       // pairs of scales
                uint32_t odd = 0u;
                for (int i = ct; i < kWords; i += kCT) odd |= __vcmpgeu2(lds32(scales + 4 * i) & 0x7FFF7FFFu, 0x60006000u);
                bool big = named_bar_or(1, kCT, odd != 0u);
                if (big || !whole) {
                    bool over = false;
                    for (int i = ct; i < kWords; i += kCT) {
                        uint32_t w = lds32(scales + 4 * i);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int t = (2 * i + h) / (D / 32);
                            const uint32_t mag = (w >> (16 * h)) & 0x7FFFu;
                            const bool there = t < here && ((runs >> (t >> 4)) & 1u);
                            if (there && mag >= 0x7C00u && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
                            if (!there || mag >= 0x7C00u) w &= h ? 0x0000FFFFu : 0xFFFF0000u;
                            else over = over || mag >= 0x6000u;
                        }
                        asm volatile("st.shared.u32 [%0], %1;" :: "r"(scales + 4 * i), "r"(w) : "memory");
                    }
                    big = named_bar_or(1, kCT, over);
                }
                if (pos >= NR) wait(&sm.t_empty[to], pos / NR - 1);
                if (ct == 0) {
                    uint32_t &info = sm.info[(pos >> 1) & 3];
                    if (is_v) info |= big ? 0x200u : 0u;
                    else info = (~runs & ((1u << (BN / 16)) - 1u)) | (big ? 0x100u : 0u);
                }
                if (ok) {
                    const uint32_t down = big ? 0x18001800u : 0x3C003C00u;  // 2^-9, or 1
                    const uint32_t tile = tile_at + to * C::kTile;
                    constexpr int kPer = D / 16;  // units of 16 codes a token
#pragma unroll
                    for (int n = 0; n < (BN * kPer + kCT - 1) / kCT; ++n) {
                        const int u = ct + n * kCT, t = u / kPer, x = u % kPer;
                        if (BN * kPer % kCT != 0 && u >= BN * kPer) break;
                        // which half of the 16 codes first: both the loads and the stores of a warp then hit all banks once
                        const int h = D == 64 ? (t >> 1) & 1 : (D == 128 ? ((x >> 2) ^ t) & 1 : ((x >> 2) ^ (x >> 3)) & 1);
                        const uint32_t from = raw + t * D + x * 16;
                        const uint2 c0 = lds64(from + 8 * h), c1 = lds64(from + 8 * (h ^ 1));
                        uint32_t s2 = lds16(scales + (t * (D / 32) + (x >> 1)) * 2);
                        s2 = hmul2(s2 | s2 << 16, down);
                        const uint32_t row = tile + (x >> 2) * C::kChunk + t * 128;
                        uint32_t a, b, c, d;
                        codes4_to_f16x2(c0.x, a, b);
                        codes4_to_f16x2(c0.y, c, d);
                        sts128(row + (((2 * (x & 3) + h) ^ (t & 7)) << 4), make_uint4(hmul2(a, s2), hmul2(b, s2), hmul2(c, s2), hmul2(d, s2)));
                        codes4_to_f16x2(c1.x, a, b);
                        codes4_to_f16x2(c1.y, c, d);
                        sts128(row + (((2 * (x & 3) + (h ^ 1)) ^ (t & 7)) << 4), make_uint4(hmul2(a, s2), hmul2(b, s2), hmul2(c, s2), hmul2(d, s2)));
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.t_full[to]);
                    mbar_arrive(&sm.raw_empty[slot]);
                }
            }
            left -= seg + kEndUnits;
            if (left > 0) wk.next(p);
        }
    } else {
        // -------------------------------------------------------------- softmax
        const int m = warp >> 2, r = tid & 127;  // row tile, row
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t o_at = tmem + lanes + C::kColO + m * D;
        uint32_t c = 0;
        while (left > 0) {
            const int seg = static_cast<int>(min(left, static_cast<long long>(wk.units - wk.unit)));
            const int rr = wk.qt * C::RT + m * 128 + r;  // row of the sequence
            const bool live = rr < wk.s.n * p.group;
            const int tok = live ? rr / p.group : 0, head = wk.kvh * p.group + (live ? rr - tok * p.group : 0);
            const int64_t qrow = static_cast<int64_t>(wk.s.t0 + tok);
            // the tokens [lo, hi) that the row sees (a row that is not there: all, so that nothing is masked for it)
            const int p1 = wk.s.pos0 + tok + 1;
            const int64_t from = static_cast<int64_t>(p1) - p.window;
            const int hi = live ? p1 : INT32_MAX, lo = live && p.window > 0 && from > 0 ? static_cast<int>(from) : 0;

            // ---- the query row: scaled to a largest magnitude in [2^14, 2^15), binary16, into the tile
            float fac;
            {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + qrow * p.ldq + static_cast<int64_t>(head) * D);
                uint32_t top = 0u;  // of bf16 magnitudes, in either half
                if (live) {
#pragma unroll 8
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 v = __ldg(src + i);
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                    }
                }
                const int ex = min(max(static_cast<int>(max(top >> 16, top & 0xFFFFu) >> 7), 30), 254);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23) * (p.scale < 0.f ? -1.f : 1.f);
                fac = fabsf(p.scale) * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
                fac = p.softcap > 0.f ? fac / p.softcap : fac * kLog2e;
                fac = fminf(fac, FLT_MAX);  // a score of zero stays one
                const uint32_t to = q_at + m * C::kQ + r * 128;
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = f32x2_to_f16x2(bf16lo_f32(w[k]) * up, bf16hi_f32(w[k]) * up);
                    sts128(to + (i >> 3) * 16384 + (((i & 7) ^ (r & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_full[m]);
            }

            float mm = -INFINITY, ref = 0.f, top = -INFINITY, l = 0.f;
            for (int j = 0; j < seg; ++j, ++c) {
                const int tok0 = wk.base + (wk.unit + j) * BN;
                const uint32_t buf = MT == 2 ? m : (c & 1);
                const uint32_t s_at = tmem + lanes + buf * BN;
                const uint32_t vpos = 2 * c + 1;
                wait(&sm.s_full[buf], MT == 2 ? c : c >> 1);
                wait(&sm.t_full[vpos % NR], vpos / NR);
                tc_fence_after();
                if (ok) {
                    const uint32_t info = *reinterpret_cast<volatile uint32_t *>(&sm.info[c & 3]);
                    const float f = info & 0x100u ? fminf(fac * 512.f, FLT_MAX) : fac;
                    const float lift = info & 0x200u ? 9.f : 0.f;
                    // bits of the tokens of 32 that the row sees
                    auto seen = [&](int c0) -> uint32_t {
                        const int a = lo - tok0 - c0, b = hi - tok0 - c0;  // [a, b)
                        uint32_t bits = b >= 32 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << b) - 1u);
                        if (a > 0) bits &= a >= 32 ? 0u : ~((1u << a) - 1u);
                        if ((info >> (c0 >> 4)) & 1u) bits &= 0xFFFF0000u;
                        if ((info >> ((c0 >> 4) + 1)) & 1u) bits &= 0x0000FFFFu;
                        return bits;
                    };
                    const bool masked = __any_sync(0xffffffffu, lo > tok0 || hi < tok0 + BN) || (info & 0xFFu);
                    float y = -INFINITY;
#pragma unroll 1
                    for (int c0 = 0; c0 < BN; c0 += 32) {
                        uint32_t v[32];
                        tmem_ld32(s_at + c0, v);
                        tmem_ld_wait();
                        if (masked) {
                            const uint32_t bits = seen(c0);
#pragma unroll
                            for (int i = 0; i < 32; ++i) y = fmaxf(y, (bits >> i) & 1u ? __uint_as_float(v[i]) : -INFINITY);
                        } else {
                            float y1 = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) y = fmaxf(y, __uint_as_float(v[i])), y1 = fmaxf(y1, __uint_as_float(v[i + 1]));
                            y = fmaxf(y, y1);
                        }
                    }
                    // (fac >= 0: the sign of scale is in the query)
                    y = y == -INFINITY ? y : y * f;
                    if (p.softcap > 0.f && y != -INFINITY) y = p.softcap * kLog2e * tanhf(y);
                    const float z = y + lift;
                    const bool grows = z > top;
                    if (__any_sync(0xffffffffu, grows)) {
                        float g = 1.f;
                        if (grows) {
                            const float to = fmaxf(z - (fabsf(y) < kLiftEnd ? kLift : 0.f), mm);
                            g = mm == -INFINITY ? 0.f : ex2(mm - to);
                            mm = to;
                            ref = to == -INFINITY ? 0.f : to;
                            top = to + (fabsf(y) < kLiftEnd ? kTop : 0.f);
                            l *= g;
                        }
                        if (j > 0) {
                            wait(&sm.pv_done[m], c - 1);
                            tc_fence_after();
                            if (ok) {
#pragma unroll 1
                                for (int d = 0; d < D; d += 32) {
                                    uint32_t v[32];
                                    tmem_ld32(o_at + d, v);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * g);
                                    tmem_st32(o_at + d, v);
                                }
                            }
                        }
                    }
                    const float shift = ref - lift;  // weights are 2^(s - shift)
                    const bool slow = masked || p.softcap > 0.f || __any_sync(0xffffffffu, !(fabsf(y) < kPlain));
                    unsigned long long sum = 0ull;
#pragma unroll 1
                    for (int c0 = 0; c0 < BN; c0 += 32) {
                        uint32_t v[32], h[16];
                        tmem_ld32(s_at + c0, v);
                        tmem_ld_wait();
                        if (slow) {
                            const uint32_t bits = masked ? seen(c0) : 0xFFFFFFFFu;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                float x[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    x[k] = __fmul_rn(__uint_as_float(v[i + k]), f);
                                    if (p.softcap > 0.f) x[k] = p.softcap * kLog2e * tanhf(x[k]);
                                    x[k] = (bits >> (i + k)) & 1u ? ex2(__fadd_rn(x[k], -shift)) : 0.f;
                                }
                                h[i / 2] = f32x2_to_f16x2(x[0], x[1]);
                                sum = add2(sum, pack2(x[0], x[1]));
                            }
                        } else {
                            const unsigned long long f2 = pack2(f, f), n2 = pack2(-shift, -shift);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const unsigned long long x = fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f2, n2);
                                const float x0 = ex2(lo2(x)), x1 = ex2(hi2(x));
                                h[i / 2] = f32x2_to_f16x2(x0, x1);
                                sum = add2(sum, pack2(x0, x1));
                            }
                        }
                        tmem_st16(s_at + c0 / 2, h);
                    }
                    const float part = lo2(sum) + hi2(sum);
                    l += lift > 0.f ? part * 0x1p-9f : part;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[buf]);
            }
            wait(&sm.pv_done[m], c - 1);
            tc_fence_after();

            // ---- the answer, or a part of it
            const int64_t at = qrow * p.q_heads + head;
            auto store = [&](int d, const float (&v)[8]) { store8(reinterpret_cast<__nv_bfloat16 *>(p.out) + at * D + d, v); };
            auto give_lse = [&](float mx, float ls) {
                if (p.lse) p.lse[at] = ls == 0.f ? -INFINITY : fmaf(mx + kLift, 0.69314718055994531f, logf(ls * 0x1p-11f));
            };
            if (seg == wk.units) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int d = 0; d < D && ok; d += 32) {
                    uint32_t v[32];
                    tmem_ld32(o_at + d, v);
                    tmem_ld_wait();
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = l == 0.f ? 0.f : __uint_as_float(v[i + k]) * inv;
                            store(d + i, x);
                        }
                    }
                }
                if (live && ok) give_lse(mm, l);
            } else {
                const int c0 = static_cast<int>(item0 / per), c1 = static_cast<int>((item0 + wk.units - 1) / per);
                auto slot_of = [&](int k) { return 2 * k + (k == c0 ? 1 : 0); };
                auto part = [&](int k) { return p.parts + (static_cast<int64_t>(slot_of(k)) * MT + m) * C::kPart; };
                float *mine = part(blockIdx.x);
#pragma unroll 1
                for (int d = 0; d < D && ok; d += 32) {
                    uint32_t v[32];
                    tmem_ld32(o_at + d, v);
                    tmem_ld_wait();
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            __stcg(reinterpret_cast<uint4 *>(mine) + (d + i) / 4 * 128 + r, make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]));
                    }
                }
                if (live) __stcg(reinterpret_cast<float2 *>(mine + D * 128) + r, make_float2(mm, l));
                named_bar(2 + m, 128);
                if (r == 0) {
                    uint32_t *ticket = p.tickets + slot_of(c0) * 2 + m;
                    sm.last[m] = ok && atomic_add_acq_rel(ticket, 1u) == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
                    if (sm.last[m]) *ticket = 0u;
                }
                named_bar(2 + m, 128);
                if (sm.last[m] && live) {
                    float mx = -INFINITY, ls = 0.f;
                    auto ml = [&](int k) { return __ldcg(reinterpret_cast<const float2 *>(part(k) + D * 128) + r); };
                    for (int k = c0; k <= c1; ++k) mx = fmaxf(mx, ml(k).x);
                    auto weight = [&](float m1) { return m1 == -INFINITY ? (mx == -INFINITY ? 1.f : 0.f) : ex2(m1 - mx); };
                    for (int k = c0; k <= c1; ++k) {
                        const float2 v = ml(k);
                        ls = fmaf(v.y, weight(v.x), ls);
                    }
                    const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0.f;
#pragma unroll 1
                        for (int k = c0; k <= c1; ++k) {
                            const float w = weight(ml(k).x);
                            const float4 *src = reinterpret_cast<const float4 *>(part(k)) + d / 4 * 128 + r;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 v = __ldcg(src + i * 128);
                                x[4 * i] = fmaf(v.x, w, x[4 * i]), x[4 * i + 1] = fmaf(v.y, w, x[4 * i + 1]);
                                x[4 * i + 2] = fmaf(v.z, w, x[4 * i + 2]), x[4 * i + 3] = fmaf(v.w, w, x[4 * i + 3]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float o[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = ls == 0.f ? 0.f : x[i + k] * inv;
                            store(d + i, o);
                        }
                    }
                    give_lse(mx, ls);
                }
                named_bar(2 + m, 128);  // the flag has been read
            }
            left -= seg + kEndUnits;
            item0 += wk.units + kEndUnits;
            if (left > 0) wk.next(p);
        }
    }

    // ------------------------------------------------------------------ teardown
    __syncwarp();
    if (tid == 0 && *reinterpret_cast<volatile int32_t *>(&sm.abort_flag)) drain_after_timeout();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kSoftmax) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
}

int ilog2(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

template <int D, int MT>
q8_status launch(const ChunkParams &p, const DeviceInfo *di, cudaStream_t stream) {
    using C = Cfg<D, MT>;
    static std::atomic<bool> set[64];
    if (di->device >= 64 || !set[di->device].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(chunk_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return Q8_ERR_CUDA;
        if (di->device < 64) set[di->device].store(true, std::memory_order_relaxed);
    }
    const unsigned grid = static_cast<unsigned>(di->sm_count < kMaxGrid ? di->sm_count : kMaxGrid);
    chunk_kernel<D, MT><<<grid, C::kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

}  // namespace

// Counters, then two parts per CTA.
size_t chunk_workspace(int, int, int head_dim) {
    const int rows = head_dim == 256 ? 128 : 256;
    return Q8_CHUNK_ZEROED_BYTES + static_cast<size_t>(2) * kMaxGrid * rows * (head_dim + 2) * 4;
}
static_assert(2 * kMaxGrid * 2 * 4 <= Q8_CHUNK_ZEROED_BYTES, "the tickets");

q8_status launch_chunk(const q8_kv_cache &c, const ChunkArgs &a, void *ws, uint32_t *dev_status, cudaStream_t stream) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    const WsRange counters = {0, Q8_CHUNK_ZEROED_BYTES};
    const WsRange data = {Q8_CHUNK_ZEROED_BYTES, chunk_workspace(a.q_heads, c.kv_heads, c.head_dim) - Q8_CHUNK_ZEROED_BYTES};
    const q8_status st = claim_workspace(ws, &counters, 1, &data, 1, stream);
    if (st != Q8_OK) return st;
    ChunkParams p = {};
    p.kq = c.kq, p.vq = c.vq, p.ks = c.ks, p.vs = c.vs;
    p.q = a.q, p.table = a.table, p.lens = a.lens, p.starts = a.starts, p.out = a.out, p.lse = a.lse;
    p.tickets = static_cast<uint32_t *>(ws);
    p.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + Q8_CHUNK_ZEROED_BYTES);
    p.status = dev_status;
    p.ldq = a.ldq, p.T = static_cast<int32_t>(a.T), p.batch = a.batch, p.q_heads = a.q_heads, p.kv_heads = c.kv_heads;
    p.group = a.q_heads / c.kv_heads;
    p.table_width = a.table_width, p.pages = c.pages, p.page_shift = ilog2(c.page_size);
    // a cap from 2^40 on is none (see q8_attn.cu)
    p.window = a.window, p.scale = a.scale, p.softcap = a.softcap < 0x1p40f ? a.softcap : 0.f;
    // two row tiles share a tile of keys and values where sequences have the rows for them
    const bool two = a.T * p.group > int64_t{128} * a.batch;
    if (c.head_dim == 64) return two ? launch<64, 2>(p, di, stream) : launch<64, 1>(p, di, stream);
    if (c.head_dim == 128) return two ? launch<128, 2>(p, di, stream) : launch<128, 1>(p, di, stream);
    return launch<256, 1>(p, di, stream);
}

}  // namespace q8
