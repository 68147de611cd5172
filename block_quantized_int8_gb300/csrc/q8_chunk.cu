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
// exact where the scale is subnormal, as all are whole multiples of 2^-24).  Tokens with a scale of
// 512 or more, whose products could overflow, are taken times 2^-9 (what their small blocks hold to
// 2^-16): the scores get the factor back, or the weights are raised by 2^9 (their reference moves up for
// it, and stays, so that the row's other weights are good down to 2^-16 of the largest from then on).
//
// A row's arithmetic does not depend on what other rows hold, whichever branch its warp takes.
//
// Roles (one CTA per SM):
//   softmax     4 warps per row tile, a thread per row, its scores of a tile in registers; the query rows
//               into shared memory before an item, the answer after it
//   MMA         one warp, an elected thread of it issuing
//   loader      one warp: bulk copies of codes and scales, 16 tokens (a page's smallest part) each,
//               into a ring of raw tiles
//   converters  CW warps: codes times scales into a ring of binary16 tiles, in the 128-byte
//               swizzle that the tensor cores read: K-major for the keys, and the same bytes as
//               MN-major for the values, so nothing is transposed
//
// Bound: a tile of 128 tokens and 256 rows needs 2048 clocks of the tensor cores, 1024 of exponentials and
// about 2600 of shared memory (operands, raw tiles in and out); it takes 4100, the turn of a row tile: scores out of tensor
// memory, weights, product, next scores.  With 128 rows it is as much, converters and softmax about
// 3000 each.  Measured on the device (events around one call, L2 flushed before it): 1024 new tokens over 65,536 (32 / 8
// heads of 128) 916 us, 1.19 PFLOP/s; 4096 tokens alone 176 to 187 us, 0.75; 16 sequences of 1 to 5 new tokens
// over up to 6000 60 us; 32 new tokens over 262,144 229 us, 2.49 TB/s; 1024 over 65,536 with 12 / 4 heads of 256
// 1103 us, 0.74 PFLOP/s.  (Calls one after the other hold the clock lower: the first takes 990 us then.)  Tiles of 80
// tokens with a place of their own for the weights, so that the next scores need not wait for the product: 1225 us where
// this form took 1004.
//
// Two row tiles where sequences have more than 128 rows on average (a tile takes 2.1 us with 128 rows and with 256, so
// that below it half of the work would be nobody's); at 256 dimensions tensor memory has room for one.
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

namespace q8 {

namespace {

constexpr int kMaxGrid = 160;   // CTAs a launch may have (sizes the workspace)
constexpr int kEndUnits = 3;    // what beginning and ending an item takes, in units' time
constexpr int kMinUnits = 2;    // units a CTA takes at least
constexpr int kWhole = 4;       // items of up to so many are not divided (a join takes longer than three tiles)
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
// These are executed by a whole warp, one of whose threads is elected for the instruction: the operands are
// then made in the warp's uniform registers.  (Behind a branch on the lane an MMA took 97 clocks to issue,
// for 40 of the tensor cores'.)
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync r|q, 0xFFFFFFFF;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync r|q, 0xFFFFFFFF;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("{\n\t.reg .pred q;\n\t.reg .b32 r;\n\telect.sync r|q, 0xFFFFFFFF;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// n columns of the warp's lanes; the wait stands in the same statement, so that nothing can use (or
// spill) the registers before it
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(t), "r"(t + 32) : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(t), "r"(t + 32), "r"(t + 64), "r"(t + 96) : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
        : "memory");
}
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t *p, uint32_t v) {
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void named_bar(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }

// ---- shapes -------------------------------------------------------------------------
template <int D_, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr int BN = D == 256 ? 64 : 128;          // tokens of a tile
    static constexpr int RT = 128 * MT;                     // rows of an item
    static constexpr int kSoftmax = 4 * MT;                 // softmax warps
    static constexpr int CW = 14 - kSoftmax;                // converter warps: what is left of 16
    // A softmax thread has a row's scores in registers: the other roles leave it what they do without of the
    // 128 that each thread begins with (8 x 184 + 8 x 72, or 4 x 200 + 12 x 104)
    static constexpr int kRegs = MT == 2 ? 184 : 200, kRegsLess = MT == 2 ? 72 : 104;
    static constexpr int kWarps = kSoftmax + 2 + CW;
    static_assert(kWarps == 16 && kSoftmax * kRegs + (16 - kSoftmax) * kRegsLess <= 16 * 128, "registers");
    static_assert(kSoftmax % 4 == 0, "registers are moved between whole warpgroups");
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
    uint32_t meta[8];       // of a raw tile: bits 0-7 the runs of 16 tokens that were loaded, 8-15 tokens
    uint32_t unseen[8];     // of the last tiles: runs that were not loaded
    uint4 big[2][8];        // and tokens whose keys (values) are times 2^-9, a bit each
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
    // the units of this item that a CTA takes with `left` of its stretch of the list left: short items are not
    // divided, but belong to the CTA that they begin in
    __device__ __forceinline__ int stretch(long long left) const {
        return units <= kWhole ? units : static_cast<int>(min(left, static_cast<long long>(units - unit)));
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

// c tanh(x / cap) in units of log 2 (c = cap log2(e)), y being x / cap times 2 log2(e): c - 2 c / (1 + 2^y) is
// off by 2^-22 c, which is 2^-13 at most for caps up to kCapEnd.  Above, where |x / cap| < 1/4, the series
// of tanh to its ninth power (2^-26 of it off), and elsewhere the same form, 2^-20 of the score off.
constexpr float kCapEnd = 256.f;
__device__ __forceinline__ float capped(const ChunkParams &p, float y) {
    const float c = p.softcap * kLog2e;
    const float far = fmaf(-2.f * c, rcp(1.f + ex2(y)), c);
    if (p.softcap <= kCapEnd) return far;
    const float x = y * (0.5f / kLog2e), z = x * x;
    const float series = fmaf(z, fmaf(z, fmaf(z, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
    return fabsf(x) < 0.25f ? c * fmaf(x * z, series, x) : far;
}

// One try that sleeps in the barrier for up to 20 us (a loop of short tries took half of all issue slots).
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_more(Control &sm, uint32_t *status, uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (try_wait_long(bar, parity)) return true;
        if (*reinterpret_cast<volatile int32_t *>(&sm.abort_flag)) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicExch(&sm.abort_flag, 1);
            if (status) atomicOr(status, Q8_DEV_TIMEOUT);
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
    const int tid = threadIdx.x, lane = tid & 31;
    // From lane 0, so that branches on it are the warp's: the MMA warp's operands are then made in uniform registers
    // (1024 over 65,536 takes 998 us, 1293 without)
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

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
        for (int i = 0; i < 8; ++i) sm.big[0][i] = sm.big[1][i] = make_uint4(0, 0, 0, 0);
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
        if (wk.unit >= wk.units || (wk.unit > 0 && wk.units <= kWhole)) {  // in an item that others end: begin with the next
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
        if (ok && __any_sync(0xffffffffu, !try_wait_long(bar, parity & 1u)))
            ok = __all_sync(0xffffffffu, wait_more(sm, p.status, bar, parity & 1u));
    };

    // One setmaxnreg for all warps of a warpgroup: PTX asks that they execute the same one.  (The softmax first: with the other
    // roles before it more instruction fetches missed, 1.28 in place of 0.8 stalls an instruction, 1105 us in place of 915)
    if (warp < C::kSoftmax) {
        // -------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::kRegs));
        constexpr int kLanes = D / 8;            // lanes of a query or answer row, 16 bytes each
        const int m = warp >> 2, r = tid & 127;  // row tile, row
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t o_at = tmem + lanes + C::kColO + m * D;
        uint32_t c = 0;
        while (left > 0) {
            const int seg = wk.stretch(left);
            const int rr = wk.qt * C::RT + m * 128 + r;  // row of the sequence
            const bool live = rr < wk.s.n * p.group;
            const int tok = live ? rr / p.group : 0, head = wk.kvh * p.group + (live ? rr - tok * p.group : 0);
            const int64_t qrow = static_cast<int64_t>(wk.s.t0 + tok);
            // the tokens [lo, hi) that the row sees (a row that is not there: all, so that nothing is masked for it)
            const int p1 = wk.s.pos0 + tok + 1;
            const int64_t from = static_cast<int64_t>(p1) - p.window;
            const int hi = live ? p1 : INT32_MAX, lo = live && p.window > 0 && from > 0 ? static_cast<int>(from) : 0;

            // ---- the query row: scaled to a largest magnitude in [2^14, 2^15), binary16, into the tile
            // (kLanes lanes have a row: a warp loads whole rows, and each thread learns its own row's exponent)
            float fac;
            {
                const uint64_t src = reinterpret_cast<uint64_t>(p.q + qrow * p.ldq + static_cast<int64_t>(head) * D);
                int ex = 30;
                uint4 raw[8];  // eight loads under way at a time
#pragma unroll 1
                for (int i0 = 0; i0 < kLanes; i0 += 8) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const int x = (i0 + b) * (32 / kLanes) + lane / kLanes;  // row of the warp
                    const uint64_t from = __shfl_sync(0xffffffffu, src, x);
                    const bool there = __shfl_sync(0xffffffffu, live, x);
                    // (out may be q: not by the loads that ask for memory that the kernel leaves alone)
                    raw[b] = there ? __ldcg(reinterpret_cast<const uint4 *>(from) + lane % kLanes) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const int i = i0 + b, x = i * (32 / kLanes) + lane / kLanes;
                    const uint4 v = raw[b];
                    uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int e = min(max(static_cast<int>(max(top >> 16, top & 0xFFFFu) >> 7), 30), 254);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - e) << 23) * (p.scale < 0.f ? -1.f : 1.f);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = f32x2_to_f16x2(bf16lo_f32(w[k]) * up, bf16hi_f32(w[k]) * up);
                    const int c8 = lane % kLanes, row = 32 * (warp & 3) + x;
                    sts128(q_at + m * C::kQ + (c8 >> 3) * 16384 + row * 128 + (((c8 & 7) ^ (row & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                    const int of_mine = __shfl_sync(0xffffffffu, e, lane % (32 / kLanes) * kLanes);
                    if (i == lane / (32 / kLanes)) ex = of_mine;
                }
                }
                fac = fabsf(p.scale) * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
                fac = p.softcap > 0.f ? fac / p.softcap * (2.f * kLog2e) : fac * kLog2e;
                fac = fminf(fac, FLT_MAX);  // a score of zero stays one
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
                tc_fence_after();
                if (ok) {
                    const uint32_t unseen = *reinterpret_cast<volatile uint32_t *>(&sm.unseen[c & 7]);
                    const uint4 bk = *const_cast<const uint4 *>(&sm.big[0][c & 7]);
                    const float f = fac;
                    const bool cap = p.softcap > 0.f;
                    // bits of the tokens of 32 that the row sees
                    auto seen = [&](int c0) -> uint32_t {
                        const int a = lo - tok0 - c0, b = hi - tok0 - c0;  // [a, b)
                        uint32_t bits = b >= 32 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << b) - 1u);
                        if (a > 0) bits &= a >= 32 ? 0u : ~((1u << a) - 1u);
                        if ((unseen >> (c0 >> 4)) & 1u) bits &= 0xFFFF0000u;
                        if ((unseen >> ((c0 >> 4) + 1)) & 1u) bits &= 0x0000FFFFu;
                        return bits;
                    };
                    const bool masked = __any_sync(0xffffffffu, lo > tok0 || hi < tok0 + BN) || unseen;
                    uint32_t v[BN];  // the row's scores
                    tmem_ld(s_at, v);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < BN; k += 32) {
                            const uint32_t bits = seen(k);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[k + i] = (bits >> i) & 1u ? v[k + i] : 0xFF800000u;
                        }
                    }
                    const bool shrunk = __any_sync(0xffffffffu, (bk.x | bk.y | bk.z | bk.w) != 0u);
                    if (shrunk) {  // keys that are times 2^-9
                        const uint32_t w[4] = {bk.x, bk.y, bk.z, bk.w};
#pragma unroll
                        for (int i = 0; i < BN; ++i)
                            if ((w[i >> 5] >> (i & 31)) & 1u) v[i] = __float_as_uint(__uint_as_float(v[i]) * 512.f);
                    }
                    float y4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < BN; i += 8)
#pragma unroll
                        for (int n = 0; n < 4; ++n) y4[n] = max3(y4[n], __uint_as_float(v[i + n]), __uint_as_float(v[i + 4 + n]));
                    float y = fmaxf(max3(y4[0], y4[1], y4[2]), y4[3]);
                    // (f >= 0: the sign of scale is in the query)
                    y = y == -INFINITY ? y : y * f;
                    if (cap && y != -INFINITY) y = capped(p, y);
                    wait(&sm.t_full[vpos % NR], vpos / NR);
                    const uint4 bv = *const_cast<const uint4 *>(&sm.big[1][c & 7]);
                    // values that are times 2^-9: their weights are raised by 2^9
                    const bool raised = __any_sync(0xffffffffu, (bv.x | bv.y | bv.z | bv.w) != 0u);
                    const float lift = raised ? 9.f : 0.f;
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
                                for (int d = 0; d < D; d += 16) {
                                    uint32_t o[16];
                                    tmem_ld(o_at + d, o);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * g);
                                    tmem_st(o_at + d, o);
                                }
                            }
                        }
                    }
                    const float shift = ref;  // weights are 2^(s - shift)
                    unsigned long long sum[2] = {0ull, 0ull};
                    // large scores, whose product's rounding would show in the weight: product and difference one after the other
                    const bool apart = !(f > 0.f) || (y > -INFINITY && !(fabsf(y) < kPlain));
                    if (raised || p.softcap > kCapEnd || __any_sync(0xffffffffu, apart)) {
                        // raised weights, wide caps, and warps with a row of large scores: few at a time, read again, from the last
                        // to the first, as the weights go where scores lay that have been read.  The other rows of such a warp get
                        // what the other branch would give them, bit for bit: their sums are taken in its order, in a pass before
                        const bool late = raised || p.softcap > kCapEnd || apart;  // the row's sum is taken in the last pass
                        const float c1 = p.softcap * kLog2e, c2 = -2.f * c1, c3 = c1 - shift;
                        const uint32_t wk4[4] = {bk.x, bk.y, bk.z, bk.w}, wv4[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll 1
                        for (int pass = __all_sync(0xffffffffu, late) ? 1 : 0; pass < 2; ++pass) {
#pragma unroll 1
                            for (int b = 0; b < BN; b += 16) {
                                const int k = pass ? BN - 16 - b : b;
                                uint32_t x[16], h[8];
                                tmem_ld(s_at + k, x);
                                const uint32_t bits = masked ? seen(k & ~31) >> (k & 16) : 0xFFFFu;
                                uint32_t bigk = 0u, bigv = 0u;
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    if ((k >> 5) == n) bigk = wk4[n] >> (k & 16), bigv = wv4[n] >> (k & 16);
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    float w[2], u[2];
#pragma unroll
                                    for (int n = 0; n < 2; ++n) {
                                        w[n] = __uint_as_float(x[i + n]);
                                        if ((bigk >> (i + n)) & 1u) w[n] *= 512.f;
                                        const float s = __fmul_rn(w[n], f);
                                        float e = apart ? __fadd_rn(s, -shift) : fmaf(w[n], f, -shift);
                                        if (cap) e = p.softcap > kCapEnd ? __fadd_rn(capped(p, s), -shift) : fmaf(c2, rcp(1.f + ex2(s)), c3);
                                        w[n] = (bits >> (i + n)) & 1u ? ex2(e) : 0.f;
                                        u[n] = (bigv >> (i + n)) & 1u ? w[n] * 512.f : w[n];
                                    }
                                    h[i / 2] = f32x2_to_f16x2(u[0], u[1]);
                                    if ((pass != 0) == late) sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(w[0], w[1]));
                                }
                                if (pass) tmem_st(s_at + BN / 2 + k / 2, h);
                            }
                        }
                    } else {
                        if (cap) {
                            const float c1 = p.softcap * kLog2e, c2 = -2.f * c1, c3 = c1 - shift;
#pragma unroll
                            for (int i = 0; i < BN; ++i) {
                                const float e = fmaf(c2, rcp(1.f + ex2(__uint_as_float(v[i]) * f)), c3);
                                v[i] = masked && v[i] == 0xFF800000u ? v[i] : __float_as_uint(e);
                            }
                        } else {
                            const unsigned long long f2 = pack2(f, f), n2 = pack2(-shift, -shift);
#pragma unroll
                            for (int i = 0; i < BN; i += 2) {
                                const unsigned long long e = fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f2, n2);
                                v[i] = static_cast<uint32_t>(e), v[i + 1] = static_cast<uint32_t>(e >> 32);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < BN; k += 32) {
                            uint32_t h[16];
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float w0 = ex2(__uint_as_float(v[k + i])), w1 = ex2(__uint_as_float(v[k + i + 1]));
                                h[i / 2] = f32x2_to_f16x2(w0, w1);
                                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(w0, w1));
                            }
                            tmem_st(s_at + BN / 2 + k / 2, h);
                        }
                    }
                    const float part = (lo2(sum[0]) + hi2(sum[0])) + (lo2(sum[1]) + hi2(sum[1]));
                    l += part;
                    tmem_st_wait();
                }
                // Every phase of pv_done is waited for in its turn: a wait on a later one alone could take the phase before
                // it, unfinished, for its own.  (Where two row tiles take turns, these scores came after that product.)
                if (MT == 1 && j > 0) wait(&sm.pv_done[m], c - 1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[buf]);
            }
            wait(&sm.pv_done[m], c - 1);
            tc_fence_after();

            // ---- the answer, or a part of it
            const int64_t at = qrow * p.q_heads + head;
            // An answer row lies in the query tile's place (same size, same swizzle) before it goes out, whole rows at a time
            auto stage = [&](int d, const float (&x)[8]) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    h[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
                sts128(q_at + m * C::kQ + (d >> 6) * 16384 + r * 128 + ((((d >> 3) & 7) ^ (r & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
            };
            auto send = [&]() {
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < kLanes; ++i) {
                    const int x = i * (32 / kLanes) + lane / kLanes, row = 32 * (warp & 3) + x, c8 = lane % kLanes;
                    const int64_t to = __shfl_sync(0xffffffffu, at, x);
                    const bool there = __shfl_sync(0xffffffffu, live, x);
                    const uint4 v = lds128(q_at + m * C::kQ + (c8 >> 3) * 16384 + row * 128 + (((c8 & 7) ^ (row & 7)) << 4));
                    if (there) *reinterpret_cast<uint4 *>(p.out + to * D + 8 * c8) = v;
                }
                __syncwarp();
            };
            auto give_lse = [&](float mx, float ls) {
                if (p.lse) p.lse[at] = ls == 0.f ? -INFINITY : fmaf(mx + kLift, 0.69314718055994531f, logf(ls * 0x1p-11f));
            };
            if (seg == wk.units) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int d = 0; d < D && ok; d += 32) {
                    uint32_t v[32];
                    tmem_ld(o_at + d, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = l == 0.f ? 0.f : __uint_as_float(v[i + k]) * inv;
                        stage(d + i, x);
                    }
                }
                if (ok) send();
                if (live && ok) give_lse(mm, l);
            } else {
                const int c0 = static_cast<int>(item0 / per), c1 = static_cast<int>((item0 + wk.units - 1) / per);
                auto slot_of = [&](int k) { return 2 * k + (k == c0 ? 1 : 0); };
                auto part = [&](int k) { return p.parts + (static_cast<int64_t>(slot_of(k)) * MT + m) * C::kPart; };
                float *mine = part(blockIdx.x);
#pragma unroll 1
                for (int d = 0; d < D && ok; d += 32) {
                    uint32_t v[32];
                    tmem_ld(o_at + d, v);
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
                if (sm.last[m]) {
                    float mx = -INFINITY, ls = 0.f;
                    auto ml = [&](int k) { return live ? __ldcg(reinterpret_cast<const float2 *>(part(k) + D * 128) + r) : make_float2(0.f, 1.f); };
                    for (int k = c0; k <= c1; ++k) mx = fmaxf(mx, ml(k).x);
                    auto weight = [&](float m1) { return m1 == -INFINITY ? (mx == -INFINITY ? 1.f : 0.f) : ex2(m1 - mx); };
                    for (int k = c0; k <= c1; ++k) {
                        const float2 v = ml(k);
                        ls = fmaf(v.y, weight(v.x), ls);
                    }
                    const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll 1
                    for (int d = 0; d < D; d += 64) {
                        float x[64];
#pragma unroll
                        for (int i = 0; i < 64; ++i) x[i] = 0.f;
#pragma unroll 1
                        for (int k = c0; k <= c1; ++k) {
                            const float4 *src = reinterpret_cast<const float4 *>(part(k)) + d / 4 * 128 + r;
                            float4 v[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = live ? __ldcg(src + i * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
                            const float w = weight(ml(k).x);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                x[4 * i] = fmaf(v[i].x, w, x[4 * i]), x[4 * i + 1] = fmaf(v[i].y, w, x[4 * i + 1]);
                                x[4 * i + 2] = fmaf(v[i].z, w, x[4 * i + 2]), x[4 * i + 3] = fmaf(v[i].w, w, x[4 * i + 3]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 64; i += 8) {
                            float o[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = ls == 0.f ? 0.f : x[i + k] * inv;
                            stage(d + i, o);
                        }
                    }
                    send();
                    if (live) give_lse(mx, ls);
                }
                named_bar(2 + m, 128);  // the flag has been read
            }
            left -= seg + kEndUnits;
            item0 += wk.units + kEndUnits;
            if (left > 0) wk.next(p);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::kRegsLess));
        if (warp == C::kSoftmax) {
            // ------------------------------------------------------------------ MMA
            uint32_t c = 0, items = 0;  // tiles, items so far
            const auto bar_of = [&](uint32_t pos) { return pos % NR; };
            while (left > 0) {
                const int seg = wk.stretch(left);
                auto qk = [&](int m, uint32_t tile) {  // scores of row tile m, tile `tile`
                    const uint32_t pos = 2 * tile, slot = bar_of(pos);
                    const uint32_t buf = MT == 2 ? m : (tile & 1);
                    if (ok) {
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
                        if (ok) {
                            const uint64_t b = sw128_desc(tile_at + vslot * C::kTile, C::kChunk);
#pragma unroll
                            for (int k = 0; k < BN / 16; ++k)
                                umma_ts(tmem + C::kColO + m * D, tmem + buf * BN + BN / 2 + 8 * k, b + 2048 * k / 16, idesc(D, true), j > 0 || k > 0);
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
                const int seg = wk.stretch(left);
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
                            sm.meta[slot] = runs | static_cast<uint32_t>(min(BN, wk.end - (wk.base + (wk.unit + j) * BN))) << 8;
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
        } else {
            // ----------------------------------------------------------- converters
            constexpr int kCT = C::CW * 32, kPer = D / 16, kUnits = BN * kPer;  // units of 16 codes, of a token and a tile
            constexpr int kMine = (kUnits + kCT - 1) / kCT;
            const int ct = tid - (C::kSoftmax + 2) * 32;
            // This thread's units are ct, ct + kCT, ...: unit x0 of tokens t0, t0 + kStep, ..., in the order of the raw tile.
            // Which half of a unit's 16 codes comes first is chosen so that a warp's loads and its stores each hit all
            // banks once
            constexpr int kStep = kCT / kPer;
            static_assert(kStep % 4 == 0, "the same place in the swizzle");
            const int t0 = ct / kPer, x0 = ct % kPer;
            const int half = D == 64 ? (t0 >> 1) & 1 : (D == 128 ? ((x0 >> 2) ^ t0) & 1 : ((x0 >> 2) ^ (x0 >> 3)) & 1);
            const uint32_t from = ct * 16 + 8 * half, scale_at = (t0 * (D / 32) + (x0 >> 1)) * 2;
            const uint32_t place = (x0 >> 2) * C::kChunk + t0 * 128;
            const uint32_t piece0 = place + (((2 * (x0 & 3) + half) ^ (t0 & 7)) << 4), piece1 = place + (((2 * (x0 & 3) + (half ^ 1)) ^ (t0 & 7)) << 4);
            uint32_t pos = 0;
            while (left > 0) {
                const int n = wk.stretch(left);
                for (int jj = 0; jj < 2 * n; ++jj, ++pos) {
                    const uint32_t slot = pos % NW, to = pos % NR;
                    const uint32_t raw = raw_at + slot * C::kRaw;
                    wait(&sm.raw_full[slot], pos / NW);
                    if (pos >= NR) wait(&sm.t_empty[to], pos / NR - 1);
                    if (ok) {
                        const uint32_t meta = sm.meta[slot];
                        const bool is_v = pos & 1u;
                        const int here = (meta >> 8) & 0xFF, ring = (pos >> 1) & 7;
                        if (ct == 0 && !is_v) {
                            sm.unseen[ring] = ~meta & ((1u << (BN / 16)) - 1u);
                            // for a tile to come (the last that had the place is long done)
                            sm.big[0][ring ^ 4] = sm.big[1][ring ^ 4] = make_uint4(0, 0, 0, 0);
                        }
                        uint2 w0[kMine], w1[kMine];
                        uint32_t sc[kMine];
#pragma unroll
                        for (int i = 0; i < kMine; ++i) {
                            if (kUnits % kCT != 0 && ct + i * kCT >= kUnits) break;
                            w0[i] = lds64(raw + from + i * (kCT * 16));
                            w1[i] = lds64(raw + (from ^ 8) + i * (kCT * 16));
                            sc[i] = lds16(raw + C::kCodes + scale_at + i * (kStep * (D / 32) * 2));
                        }
                        // tokens that are not there and scales that are not finite count as 0, tokens with a scale of 512 or
                        // more are taken times 2^-9 (a token's units are neighbouring lanes): such a scale before the product,
                        // which would overflow; the token's others after it, as a small scale would lose its digits
                        uint32_t top = 0u, after = 0u;  // bit i: unit i's products are still to be taken times 2^-9
#pragma unroll
                        for (int i = 0; i < kMine; ++i) {
                            if (kUnits % kCT != 0 && ct + i * kCT >= kUnits) break;
                            top = max(top, sc[i] & 0x7FFFu);
                        }
                        if (__any_sync(0xffffffffu, top >= 0x6000u) || here < BN || (meta & 0xFFu) != (1u << (BN / 16)) - 1u) {
#pragma unroll
                            for (int i = 0; i < kMine; ++i) {
                                if (kUnits % kCT != 0 && ct + i * kCT >= kUnits) break;  // (whole warps)
                                const int t = t0 + i * kStep;
                                const bool there = t < here && ((meta >> (t >> 4)) & 1u), finite = (sc[i] & 0x7C00u) != 0x7C00u;
                                if (there && !finite && p.status) atomicOr(p.status, Q8_DEV_NONFINITE);
                                if (!there || !finite) sc[i] = 0u;
                                const uint32_t mine = __ballot_sync(0xffffffffu, (sc[i] & 0x7FFFu) >= 0x6000u);
                                if ((mine >> (lane & ~(kPer - 1))) & ((1u << kPer) - 1u)) {
                                    if ((sc[i] & 0x7FFFu) >= 0x6000u) sc[i] = hmul2(sc[i], 0x1800u);
                                    else after |= 1u << i;
                                    if ((lane & (kPer - 1)) == 0) atomicOr(reinterpret_cast<uint32_t *>(&sm.big[is_v][ring]) + (t >> 5), 1u << (t & 31));
                                }
                            }
                        }
                        const uint32_t row = tile_at + to * C::kTile;
#pragma unroll
                        for (int i = 0; i < kMine; ++i) {
                            if (kUnits % kCT != 0 && ct + i * kCT >= kUnits) break;
                            const uint32_t s2 = sc[i] | sc[i] << 16;
                            // (kStep tokens on, where that is an odd multiple of four as for 256 dimensions, the swizzle's
                            // third bit is the other one)
                            const uint32_t flip = kStep % 8 == 0 ? 0u : (i & 1) * 64u, on = i * (kStep * 128);
                            uint32_t a, b, c, d;
                            codes4_to_f16x2(w0[i].x, a, b);
                            codes4_to_f16x2(w0[i].y, c, d);
                            sts128(row + (piece0 ^ flip) + on, make_uint4(hmul2(a, s2), hmul2(b, s2), hmul2(c, s2), hmul2(d, s2)));
                            codes4_to_f16x2(w1[i].x, a, b);
                            codes4_to_f16x2(w1[i].y, c, d);
                            sts128(row + (piece1 ^ flip) + on, make_uint4(hmul2(a, s2), hmul2(b, s2), hmul2(c, s2), hmul2(d, s2)));
                        }
#pragma unroll 1
                        for (; after; after &= after - 1u) {
                            const int i = __ffs(after) - 1;
                            const uint32_t flip = kStep % 8 == 0 ? 0u : (i & 1) * 64u, on = i * (kStep * 128);
                            for (const uint32_t at : {row + (piece0 ^ flip) + on, row + (piece1 ^ flip) + on}) {
                                const uint4 v = lds128(at);
                                sts128(at, make_uint4(hmul2(v.x, 0x18001800u), hmul2(v.y, 0x18001800u), hmul2(v.z, 0x18001800u), hmul2(v.w, 0x18001800u)));
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.t_full[to]);
                        mbar_arrive(&sm.raw_empty[slot]);
                    }
                }
                left -= n + kEndUnits;
                if (left > 0) wk.next(p);
            }
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
