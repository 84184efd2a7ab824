// Tensor-core (tcgen05) partial kernel for attention units of many query rows.
//
// A shared-prefix segment read by R query rows per KV head is a dense
// contraction of R rows against the segment's keys and values: R flops per
// byte of K + V.  Beyond about 64 rows the mma.sync kernel (16-row tiles,
// accumulators in registers) is bound by its tensor and softmax issue rate,
// not by HBM.  This kernel takes those units (up to 256 rows: two row tiles
// of 128) and runs both products on the fifth-generation tensor cores with
// the accumulators in tensor memory (TMEM):
//
//   S_r = Q_r K^T   M = 128 rows, N = 16..64 tokens, K = head_dim 128
//   O_r += P_r V    M = 128 rows, N = head_dim 128,  K = 16..64 tokens
//
// P_r is never staged in shared memory: the softmax writes it (bf16, two per
// 32-bit column) over the S buffer it was computed from, and the P V
// product reads its A operand from tensor memory.  Each row tile has two S/P
// buffers, so the softmax of stage k + 1 writes its P while P V of stage k
// still runs; an S buffer is reused for stage k + 2 once P V of stage k,
// which read P from it, has completed.
//
// Warp roles (448 threads, one CTA per SM):
//   warps 0, 11 TMA producers: stream 64-token stages (4 blocks of 16 tokens)
//               of K and of V into two 4-stage rings, block ids fetched 32
//               tiles at a time.
//   warps 1, 12 TMEM owner (warp 1); one lane issues the S MMAs of row tile
//               0 (warp 1) or 1 (warp 12) and their commits.
//   warps 10, 13 one lane issues the P V MMAs of row tile 0 or 1.
//   warps 2-9   softmax, one query row per thread (warps 2-5 row tile 0,
//               warps 6-9 row tile 1): read the row of S from TMEM, mask,
//               exponentiate (base 2), write P (bf16) back into the first 32
//               columns of the same S buffer, keep (m, l).
// TMEM (512 columns): row tile r holds O_r in columns [256 r, 256 r + 128)
// and two S/P buffers of 64 columns after it, so the MMA of S for the next
// stage overlaps the softmax of this one and P V of the previous one.
//
// Online softmax with a lazy reference: each row keeps a reference max m and
// rescales O (a TMEM read-modify-write) only when a stage's max exceeds m by
// more than 8 (base-2 units), so P <= 2^8 and the fp32 accumulators stay far
// from overflow; (m, l, O) is a valid partial for any reference m, so the
// log-sum-exp merge is unchanged.  P is rounded to bf16 before the MMA and
// the row sum l is taken over the rounded values, as in the mma.sync kernel.
//
// Work split: the plan's tensor-core class has its own tile list and CTA
// partition; a CTA walks its tile range unit by unit and writes one partial
// (m, l, acc) per row of every unit chunk it processed.
//
// Every mbarrier wait is bounded (about 2 s of %globaltimer).  On expiry the
// CTA records DENDRITE_ETIMEOUT, every role stops issuing work, the MMA warp
// waits (bounded) for its issued MMAs and the producer for its copies in
// flight, and the TMEM is freed before the CTA exits.
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "rows.h"

using namespace dendrite;

namespace {

constexpr int TC_TOK = 64;                                   // tokens per stage (4 blocks)
constexpr int TC_HALF = TC_TOK * 128;                        // 64 tokens x 64 columns bf16 = 8 KiB
constexpr int TC_RING_STAGE = 2 * TC_HALF;                   // K (or V) of a stage: half 0, half 1
constexpr int TC_QTILE = 128 * D * 2;                        // 128 rows x 128 columns bf16 = 32 KiB
constexpr int TC_ROWTILES = 2;
constexpr int TC_SOFTMAX_WARP0 = 2;
constexpr int TC_PV_WARP = TC_SOFTMAX_WARP0 + 4 * TC_ROWTILES;   // 10
constexpr int TC_V_WARP = TC_PV_WARP + 1;                          // 11
constexpr int TC_S1_WARP = TC_V_WARP + 1;                          // 12
// Shared memory and roles of a bf16 pool's kernel, and of an 8-bit pool's (F8).
// The K ring of that one is two stages (a slot is free again once S is issued;
// V's is held until P V is done) to make room for the tiles as they are stored:
// F8_RAW slots of a stage's four tiles (K and V each).  Its 21 warps, of 80
// registers a thread: 0-7 softmax, 8-11 the issuers (S and PV of row tile 0, then
// of 1), 12 copies the stored tiles, 13-20 convert one half tile (K or V) each.
//
// What bounds it are the chains of the roles side by side: 4,096 scores and
// 16,384 codes a stage of 64 rows take some 2,000 cycles, in which every role works
// most of the time, the SM issues in 56 of 100 cycles and shared memory moves about
// half of what it can (fewer instructions alone do not help: with fp16 operands a
// pair of codes takes two instructions less, and the first case 150 us).  The attention of
// 32 draft trees of 16 nodes (64 rows a kv head) over 7,000 tokens each, 360 MB of
// codes, takes 143 us (2.5 TB/s); of 12 trees of 32 nodes (256 rows) over 16,000
// tokens 128 us, of 61 nodes (488 rows) 230.  On the way there, in these cases:
//   - one branch-selected issuer thread a row tile, one unit on one row tile: 191 / 148 / 277 us
//   - an elected lane of a converged warp as issuer, units of up to 128 rows
//     split along their tokens (below): 154 / 134 / 244
//   - packed fp32 arithmetic, scores not held over a stage, an issuer each
//     for S and PV of both row tiles, K ring of 2 and V ring of 4 stages: 142 / 124 / 243
//   - scores read once, maximum and weights half a stage at a time: 143 / 128 / 230
// Waits and the rescaling of O are out of line and the issuers share their code:
// with everything in line a tenth of the instruction fetches missed the SM's cache.
constexpr int F8_RAW = 3;
constexpr int F8_RAW_TILE = 2 * kFp8TileBytes;
constexpr int F8_RAW_SLOT = 4 * F8_RAW_TILE;
constexpr int F8_ISSUE_WARP = 8, F8_COPY_WARP = 12, F8_CONV_WARP = 13;
template <bool F8>
struct TcLayout {
    static constexpr int NK = F8 ? 2 : 4, NV = 4;   // stages of the K and V rings
    static constexpr int S0_WARP = F8 ? F8_ISSUE_WARP : 1;   // owns the TMEM too
    static constexpr int PV1_WARP = TC_S1_WARP + 1;
    static constexpr int SOFTMAX_WARP0 = F8 ? 0 : TC_SOFTMAX_WARP0;
    static constexpr int THREADS = F8 ? 672 : (PV1_WARP + 1) * 32;
    // K ring, then V ring, in stages of 64 tokens
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = NK * TC_RING_STAGE;
    static constexpr int OFF_Q = (NK + NV) * TC_RING_STAGE;
    static constexpr int OFF_RAW = OFF_Q + TC_ROWTILES * TC_QTILE;
    // draft trees: the mask of each row, written and read by the row's thread
    static constexpr int OFF_MASK = OFF_RAW + (F8 ? F8_RAW * F8_RAW_SLOT : 0);
    static constexpr int OFF_BAR = OFF_MASK + TC_ROWTILES * 128 * 8;
    // mbarriers; S/P buffers are indexed 2 r + b (row tile r, buffer b):
    // S_FULL when S is in the buffer, P_FULL when P overwrote it, PV_DONE when
    // the P V product that read that P has completed (the buffer is free again)
    static constexpr int B_K_FULL = 0;
    static constexpr int B_K_EMPTY = B_K_FULL + NK;
    static constexpr int B_V_FULL = B_K_EMPTY + NK;
    static constexpr int B_V_EMPTY = B_V_FULL + NV;
    static constexpr int B_S_FULL = B_V_EMPTY + NV;
    static constexpr int B_P_FULL = B_S_FULL + 4;
    static constexpr int B_PV_DONE = B_P_FULL + 4;
    static constexpr int B_Q_FULL = B_PV_DONE + 4;
    static constexpr int B_FINAL = B_Q_FULL + 2;   // one per issuer: S0, PV0, S1, PV1
    static constexpr int B_RAW_FULL = B_FINAL + 4;      // F8: the copied tiles
    static constexpr int B_RAW_EMPTY = B_RAW_FULL + (F8 ? F8_RAW : 0);
    // F8, split units: (m, l) of both groups written; both accumulators read
    static constexpr int B_ML_FULL = B_RAW_EMPTY + (F8 ? F8_RAW : 0);
    static constexpr int B_ML_DONE = B_ML_FULL + (F8 ? 1 : 0);
    static constexpr int B_COUNT = B_ML_DONE + (F8 ? 1 : 0);
    // a packed unit's extra tiles (logical block, member mask), per row tile
    static constexpr int OFF_XINFO = OFF_BAR + B_COUNT * 8 + 16;
    // and how many of their tokens a branch of the mask holds
    static constexpr int OFF_XHELD = OFF_XINFO + TC_ROWTILES * kMaxTcExtraTiles * 8;
    // F8: (m, l) of the rows of a split unit, per group
    static constexpr int OFF_ML = OFF_XHELD + TC_ROWTILES * kMaxTcExtraTiles;
    // WHOLE, bf16: 32 rows of 64 bytes of each softmax warp, on their way out (row stride 80 bytes)
    static constexpr int OFF_OUT = (OFF_ML + (F8 ? TC_ROWTILES * 128 * 8 : 0) + 15) & ~15;
    static constexpr int OUT_WARP = 32 * 80;
    static constexpr int SMEM = 1024 + OFF_ML + (F8 ? TC_ROWTILES * 128 * 8 : 0);
    static constexpr int SMEM_WHOLE = F8 ? SMEM : 1024 + OFF_OUT + 8 * OUT_WARP;
};
static_assert(TcLayout<false>::SMEM_WHOLE <= 227 * 1024 - 64 && TcLayout<true>::SMEM <= 227 * 1024 - 64,
              "shared memory budget");
constexpr uint32_t TMEM_COLS = 512;
constexpr float RESCALE_THRESHOLD = 8.f;

// ------------------------------------------------------------- tcgen05 helpers
// Shared-memory matrix descriptor, 128-byte swizzle: start >> 4 in bits
// [0, 14), leading byte offset >> 4 in [16, 30), stride byte offset >> 4 in
// [32, 46), descriptor version 1 at bit 46, swizzle mode 2 (128 B) at [61, 64).
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// A descriptor `bytes` further (the start address does not leave its field:
// shared memory ends below 2^18).
__device__ __forceinline__ uint64_t sdesc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
// Instruction descriptor of kind::f16: fp32 accumulator, bf16 A and B,
// A/B major-ness (0 = K-major, 1 = MN-major), N >> 3, M >> 4.
__device__ __forceinline__ uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// The same with A (M x K, two bf16 per 32-bit column, row i in lane i) read
// from tensor memory at a_tmem.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
// 2^x by the SFU (PTX ex2.approx.ftz.f32: relative error about 2^-22,
// results below 2^-126 flushed to zero; 2^-inf = +0).
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 in one register pair and their packed arithmetic (each rounded as
// the scalar instruction rounds).
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float low(f32x2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high(f32x2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Adds a pair's two bf16 to two fp32 sums.
__device__ __forceinline__ void add_bf16(float& a, float& b, uint32_t x) {
    uint16_t lo, hi;
    asm("mov.b32 {%0, %1}, %2;" : "=h"(lo), "=h"(hi) : "r"(x));
    asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(a) : "h"(lo));
    asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(b) : "h"(hi));
}
// The largest of three (a NaN counts for nothing, as in fmaxf).
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define TC_R8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), \
                 "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define TC_W8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), \
                 "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 consecutive fp32 columns of this thread's TMEM lane (32x32b shape).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : TC_R8(0), TC_R8(8), TC_R8(16), TC_R8(24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        TC_W8(0), TC_W8(8), TC_W8(16), TC_W8(24)
        : "memory");
}
// 16 columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        TC_W8(0), TC_W8(8)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : TC_R8(0), TC_R8(8)
        : "r"(taddr));
}
#define TC_RW8(i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), \
                  "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
// Wait for this thread's tcgen05.ld results.  The registers pass through the
// statement so that no use of them is scheduled before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : TC_RW8(0), TC_RW8(8), TC_RW8(16), TC_RW8(24)::"memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : TC_RW8(0), TC_RW8(8)::"memory");
}
// Half a stage's scores: what the row does not see becomes -inf.
__device__ __forceinline__ void mask_half(uint32_t (&v)[32], uint32_t see) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = (see >> i) & 1u ? v[i] : 0xff800000u;
}
// Orders later uses of v after the preceding statement (a wait issued for
// several loads at once).
__device__ __forceinline__ void reg_tie(uint32_t (&v)[32]) {
    asm volatile("" : TC_RW8(0), TC_RW8(8), TC_RW8(16), TC_RW8(24));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Non-blocking test of an mbarrier phase.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Bounded wait by one thread; on failure marks the CTA aborted and records
// DENDRITE_ETIMEOUT (a no-op when another error is already recorded).
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, volatile int* abortp, DevMeta* meta) {
    if (mbar_test(bar, parity)) return true;   // usually complete already
    if (*abortp) return false;
    if (mbar_wait(bar, parity, abortp)) return true;
    *abortp = 1;
    atomicCAS(&meta->status, 0, DENDRITE_ETIMEOUT);
    return false;
}
// Bounded wait by a whole warp; the result is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abortp, DevMeta* meta) {
    bool ok = !*abortp && mbar_wait(bar, parity, abortp);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && (threadIdx.x & 31) == 0 && !*abortp) {
        *abortp = 1;
        atomicCAS(&meta->status, 0, DENDRITE_ETIMEOUT);
    }
    return ok;
}
// The same, looking for a while before it reads the clock and the abort flag: every look that they delay
// lengthens the chain of a stage (S, its softmax, P V, S again), which is what bounds direct plans.
__device__ __forceinline__ bool eager_wait(uint32_t bar, uint32_t parity, volatile int* abortp, DevMeta* meta) {
    bool ok = false;
    for (int i = 0; i < 128 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    return warp_wait(bar, parity, abortp, meta);
}
// The same by a call where the first look does not settle it, for the 8-bit
// pools' kernel, whose roles have to share the instruction cache.
__device__ __noinline__ bool long_wait(uint32_t bar, uint32_t parity, volatile int* abortp, DevMeta* meta) {
    return thread_wait(bar, parity, abortp, meta);
}
template <bool F8, bool WHOLE = false>
__device__ __forceinline__ bool warp_wait_(uint32_t bar, uint32_t parity, volatile int* abortp, DevMeta* meta) {
    if constexpr (!F8 && WHOLE) return eager_wait(bar, parity, abortp, meta);
    if constexpr (!F8) return warp_wait(bar, parity, abortp, meta);
    return __all_sync(0xffffffffu, mbar_test(bar, parity) || long_wait(bar, parity, abortp, meta));
}
// Wait without an abort exit, used only to drain work already issued.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < WAIT_LIMIT_NS) {
    }
}

// ------------------------------------------------ 8-bit pools: converting warps
// Two warps bring tile w of each stage, one K and one V, to the bf16 stages the
// products read.  A tile's values are code * 2^e, bf16 numbers exactly, so from here on
// the kernel is the bf16 one.
//   - By fp32 products, two codes at a time: a path of bf16 products beside it for
//     small exponents made the roles' loops outgrow the instruction cache (1,450
//     cycles a tile in place of 450).
//   - A lane converts 16 codes at a time: one 16-byte load, two 16-byte stores
//     into the two 16-byte chunks they fill in the 128-byte-swizzled stage.
//     Eight neighbouring lanes take four chunks of one 64-column half of two
//     tokens t and t ^ 5: their loads then differ in bit 2 of the swizzle and
//     their stores in bit 0, and no two meet in a bank.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Two codes (the low 16 bits of c) times f as a pair of bf16.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t c, float f) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const f32x2 y = mul2(pair(x.x, x.y), pair(f, f));
    return pack_bf16(low(y), high(y));
}
// The stages of a CTA's tile range, in order.
struct StageWalk {
    int32_t t, u, cend = 0;    // next stage's first tile; its unit; the end of the unit's tiles here
    int32_t unit_end = 0;      // the end of the unit's tiles
    int64_t row = 0;           // table offset of tile 0 of the unit
    int32_t head = 0;
    __device__ __forceinline__ StageWalk(int32_t t0, int32_t u0) : t(t0), u(u0 - 1) {}
    // Moves on to the unit of the next stage; false past the range's end.
    __device__ __forceinline__ bool more(const AttnPlanDev& pl, int32_t t_end, int32_t bpb) {
        if (t >= t_end) return false;
        while (t >= cend) {
            const AttnUnit& U = pl.units[++u];
            unit_end = U.tile_off + U.n_blk;
            cend = min(t_end, unit_end);
            row = (int64_t)U.table_row * bpb + U.blk_start - U.tile_off;
            head = U.kv_head;
        }
        return true;
    }
    __device__ __forceinline__ int tiles() const { return min(4, cend - t); }
    __device__ __forceinline__ void step() { t = min(t + 4, cend); }
};

// Tokens of the last of the unit's n_tiles own tiles that one of its branches holds.
__device__ __noinline__ int32_t held_tokens(const AttnPlanDev& pl, const AttnUnit& U, int32_t n_tiles) {
    const int32_t rm = pl.q_len * pl.group;
    int32_t len = 0;
    for (int32_t i = U.row_lo / rm + (threadIdx.x & 31); i <= (U.row_lo + U.n_rows - 1) / rm; i += 32)
        len = max(len, pl.members[U.mem_off + i].len);
    len = __reduce_max_sync(0xffffffffu, len);
    return min(kBlockSize, len - (U.blk_start + n_tiles - 1) * kBlockSize);
}
// Makes the rows of V behind the first `held` of a tile's 16 zero (tile: its 64-
// column half 0 in the V ring; a warp's work): left there by a roll-back or the
// block's last owner they may be NaN, and would spread through their weight of zero.
__device__ __forceinline__ void clear_unheld(unsigned char* tile, int32_t held) {
    for (int i = held * 16 + (threadIdx.x & 31); i < kBlockSize * 16; i += 32)
        *reinterpret_cast<uint4*>(tile + ((i >> 3) & 1) * TC_HALF + (i >> 4) * 128 + (i & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
}

// bf16 pools, a softmax warp: of a stage's tiles those that may end behind their
// branches (the last of the unit's own range, extra ones), once V has landed.  All
// warps of a unit make the same zeros, each before it passes on the P that is
// multiplied with them.  first: the stage's first tile in the unit; limit: of the
// lane's row; g: stage of the CTA; xheld: held tokens of the extra tiles.
__device__ __noinline__ bool clear_tails(const AttnArgs& a, unsigned char* sm, uint32_t bars, volatile int* abortp,
                                         const AttnUnit& U, int32_t first, int ntiles, int32_t limit, int32_t g,
                                         const unsigned char* xheld) {
    using Y = TcLayout<false>;
    const int slot = g % Y::NV;
    bool landed = false;
    for (int j = max(0, U.n_shared - 1 - first); j < ntiles; ++j) {
        const int32_t x = first + j - U.n_shared;   // of the extra tiles
        // a row that sees the tile to its end spares the look at the branches
        if (x < 0 && __any_sync(0xffffffffu, limit >= (U.blk_start + U.n_shared) * kBlockSize)) continue;
        const int32_t held =
            x < 0 ? held_tokens(a.plan, U, U.n_shared) : (int32_t)xheld[min(x, kMaxTcExtraTiles - 1)];
        if (held >= kBlockSize) continue;
        if (!landed && !warp_wait(bars + 8 * (Y::B_V_FULL + slot), (uint32_t)(g / Y::NV) & 1u, abortp, a.meta))
            return false;
        landed = true;
        clear_unheld(sm + Y::OFF_V + slot * TC_RING_STAGE + j * 16 * 128, held);
    }
    if (landed) fence_async_smem();
    return true;
}

// Copies the stages' tiles as they are stored, F8_RAW stages ahead; lane i < 4
// copies tile i, whose block id it loaded a stage before.
template <typename Y>
__device__ __forceinline__ void copy_tiles(const AttnArgs& a, uint32_t base, uint32_t bars, volatile int* abortp,
                                           int32_t t_begin, int32_t t_end, int32_t u0) {
    const AttnPlanDev& pl = a.plan;
    const int lane = threadIdx.x & 31;
    auto bar = [bars](int i) { return bars + 8u * (uint32_t)i; };
    const char* kp = reinterpret_cast<const char*>(a.pool_k);
    const char* vp = reinterpret_cast<const char*>(a.pool_v);
    StageWalk at(t_begin, u0);
    int slot = 0, rounds = 0;          // rounds: stages copied so far
    bool left = at.more(pl, t_end, a.bpb);
    int n = left ? at.tiles() : 0;
    int32_t blk = lane < n ? a.table[at.row + at.t + lane] : 0, head = at.head;
    while (left) {
        // the next stage's block ids while this one waits for its slot
        at.step();
        left = at.more(pl, t_end, a.bpb);
        const int n_next = left ? at.tiles() : 0;
        const int32_t blk_next = lane < n_next ? a.table[at.row + at.t + lane] : 0, head_next = at.head;
        const uint32_t ph = (uint32_t)(rounds / F8_RAW) & 1u;
        if (!warp_wait_<true>(bar(Y::B_RAW_EMPTY + slot), ph ^ 1u, abortp, a.meta)) break;
        const uint32_t rb = bar(Y::B_RAW_FULL + slot);
        if (lane == 0) mbar_expect_tx(rb, (uint32_t)(n * F8_RAW_TILE));
        __syncwarp();
        if (lane < n) {
            if ((uint32_t)blk >= (uint32_t)a.n_blocks) {   // broken table: poison, read a valid block
                atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                blk = 0;
            }
            const int64_t off = ((int64_t)blk * a.n_kv + head) * kFp8TileBytes;
            const uint32_t dst = base + Y::OFF_RAW + slot * F8_RAW_SLOT + lane * F8_RAW_TILE;
            bulk_load(dst, kp + off, kFp8TileBytes, rb);
            bulk_load(dst + kFp8TileBytes, vp + off, kFp8TileBytes, rb);
        }
        ++rounds;
        slot = slot == F8_RAW - 1 ? 0 : slot + 1;
        n = n_next;
        blk = blk_next;
        head = head_next;
    }
    __syncwarp();
    if (lane == 0 && *abortp) {   // copies still in flight land before the CTA exits
        for (int i = max(0, rounds - F8_RAW); i < rounds; ++i)
            drain_wait(bar(Y::B_RAW_FULL + i % F8_RAW), (uint32_t)(i / F8_RAW) & 1u);
    }
}

template <typename Y>
__device__ __forceinline__ void convert_tiles(const AttnArgs& a, unsigned char* sm, uint32_t bars, volatile int* abortp,
                                              int32_t t_begin, int32_t t_end, int32_t u0, int w, int kv) {
    const AttnPlanDev& pl = a.plan;
    const int lane = threadIdx.x & 31;
    auto bar = [bars](int i) { return bars + 8u * (uint32_t)i; };
    const int b_full = kv ? Y::B_V_FULL : Y::B_K_FULL, b_empty = kv ? Y::B_V_EMPTY : Y::B_K_EMPTY;
    // this lane's share: chunk c (16 codes) of four tokens; the two chunks
    // 2 c, 2 c + 1 of the stage row they fill
    const int c = 4 * ((lane >> 3) & 1) + (lane & 3), up = c >> 2, k = (2 * c) & 7;
    const int flip = (lane & 4) ? 5 : 0;
    unsigned char* ring = sm + (kv ? Y::OFF_V : Y::OFF_K) + up * TC_HALF + w * 16 * 128;
    const unsigned char* raws = sm + Y::OFF_RAW + w * F8_RAW_TILE + kv * kFp8TileBytes;
    StageWalk now(t_begin, u0);
    int slot = 0, stage = 0;
    uint32_t raw_ph = 0, empty_ph = 1;
    for (; now.more(pl, t_end, a.bpb); now.step()) {
        if (!warp_wait_<true>(bar(Y::B_RAW_FULL + slot), raw_ph, abortp, a.meta)) break;
        if (!warp_wait_<true>(bar(b_empty + stage), empty_ph, abortp, a.meta)) break;
        if (w < now.tiles()) {
            const unsigned char* src = raws + slot * F8_RAW_SLOT;
            unsigned char* dst = ring + stage * TC_RING_STAGE;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = (((2 * i + (lane >> 4)) & 3) ^ flip) + 8 * (i >> 1), sw = tok & 7;
                const uint4 x = *reinterpret_cast<const uint4*>(src + tok * kFp8Dim + ((c ^ sw) << 4));
                const float f = __uint_as_float((uint32_t)src[kBlockSize * kFp8Dim + tok] << 23);   // 2^e
                *reinterpret_cast<uint4*>(dst + tok * 128 + ((k ^ sw) << 4)) =
                    make_uint4(codes_bf16(x.x, f), codes_bf16(x.x >> 16, f), codes_bf16(x.y, f),
                               codes_bf16(x.y >> 16, f));
                *reinterpret_cast<uint4*>(dst + tok * 128 + (((k + 1) ^ sw) << 4)) =
                    make_uint4(codes_bf16(x.z, f), codes_bf16(x.z >> 16, f), codes_bf16(x.w, f),
                               codes_bf16(x.w >> 16, f));
            }
        }
        if (kv && w < now.tiles() && now.t + w == now.unit_end - 1) {
            __syncwarp();
            const AttnUnit& U = pl.units[now.u];
            clear_unheld(sm + Y::OFF_V + stage * TC_RING_STAGE + w * 16 * 128, held_tokens(pl, U, U.n_blk));
        }
        fence_async_smem();   // the stores, before the products read them
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar(b_full + stage));
            mbar_arrive(bar(Y::B_RAW_EMPTY + slot));
        }
        if (++slot == F8_RAW) { slot = 0; raw_ph ^= 1u; }
        if (++stage == (kv ? Y::NV : Y::NK)) { stage = 0; empty_ph ^= 1u; }
    }
}

// Eight values times inv as 16 bytes of bf16.
__device__ __forceinline__ uint4 out_words(const uint32_t* v, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The row tiles of a unit's chunk of nst stages, 8-bit pools.  A unit of up to
// 128 rows is split along its tokens instead: both groups of softmax warps hold
// its rows, group r takes the stages k with k % 2 = r, and the two (m, l, O) are
// joined when the chunk ends.
struct RowTiles {
    bool split;
    int n;
    __device__ __forceinline__ RowTiles(const AttnUnit& U, int32_t nst)
        : split(U.rt == 1), n(split ? min(nst, 2) : U.rt) {}
    __device__ __forceinline__ bool mine(int r, int32_t k) const { return r < n && (!split || (k & 1) == r); }
};

// One issuer of row tile r, stage by stage: of S_r(k) = Q_r K^T once stage k's K
// landed and the P V that read its buffer completed, or of O_r += P_r V once
// stage k's V landed and P_r(k) is in tensor memory.  Where the row tile does not
// take part it simply gives the ring slot back.
//   - All lanes run the loop and one is elected for the products: their operands
//     then are the warp's, not one thread's (from a branch on the lane a stage's
//     products took about 2,000 cycles to issue, 250 this way).
//   - Both kinds share the code, which has to stay in the instruction cache.
template <typename Y>
__device__ __forceinline__ void issue_products(const AttnArgs& a, uint32_t base, uint32_t bars, uint32_t tmem,
                                               volatile int* abortp, int32_t t_begin, int32_t t_end, int32_t u0,
                                               bool scores, int r) {
    const AttnPlanDev& pl = a.plan;
    const uint64_t dq = sdesc(base + Y::OFF_Q + r * TC_QTILE, 16, 1024), dk = sdesc(base + Y::OFF_K, 16, 1024),
                   dv = sdesc(base + Y::OFF_V, TC_HALF, 1024);
    const uint32_t ring_full = bars + 8 * (scores ? Y::B_K_FULL : Y::B_V_FULL);
    const uint32_t ring_empty = bars + 8 * (scores ? Y::B_K_EMPTY : Y::B_V_EMPTY);
    const uint32_t ready = bars + 8 * ((scores ? Y::B_PV_DONE : Y::B_P_FULL) + 2 * r);   // + 8 b
    const uint32_t done = bars + 8 * ((scores ? Y::B_S_FULL : Y::B_PV_DONE) + 2 * r);
    const uint32_t q_full = bars + 8 * (Y::B_Q_FULL + r), fin = bars + 8 * (Y::B_FINAL + 2 * r + (scores ? 0 : 1));
    int32_t t = t_begin, u = u0, js = 0;   // js: stages of this row tile
    int stage = 0;
    uint32_t ph = 0, qph = 0;
    bool ok = true;
    while (ok && t < t_end) {
        const AttnUnit& U = pl.units[u];
        const int32_t uend = U.tile_off + U.n_blk;
        if (t >= uend) { ++u; continue; }
        const int32_t cend = min(t_end, uend);
        const RowTiles tiles(U, (cend - t + 3) >> 2);
        const int32_t first = tiles.split ? r : 0;
        if (scores && r < tiles.n) {
            ok = warp_wait_<true>(q_full, qph, abortp, a.meta);
            qph ^= 1u;
        }
#pragma unroll 1
        for (int32_t k = 0; ok && t < cend; ++k, t += 4) {
            const int ntiles = min(4, cend - t);
            ok = warp_wait_<true>(ring_full + 8 * stage, ph, abortp, a.meta);
            if (!ok) break;
            if (tiles.mine(r, k)) {
                const int b = js & 1;
                ok = warp_wait_<true>(ready + 8 * b, ((uint32_t)(js >> 1) & 1u) ^ (scores ? 1u : 0u), abortp, a.meta);
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tmem + r * 256 + 128 + b * 64;   // S, then P: 16 tokens per 8 columns
                if (elect_one()) {
                    if (scores) {
                        const uint64_t dK = sdesc_at(dk, stage * TC_RING_STAGE);
                        const uint32_t id = idesc_bf16(128, 16 * ntiles, 0, 0);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16(tS, sdesc_at(dq, (kk >> 2) * 16384 + (kk & 3) * 32),
                                      sdesc_at(dK, (kk >> 2) * TC_HALF + (kk & 3) * 32), id, kk > 0);
                    } else {
                        const uint64_t dV = sdesc_at(dv, stage * TC_RING_STAGE);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (kk < ntiles)
                                umma_bf16_ta(tmem + r * 256, tS + kk * 8, sdesc_at(dV, kk * 2048),
                                             idesc_bf16(128, 128, 0, 1), kk > 0 || k > first);
                    }
                    umma_commit(done + 8 * b);
                    umma_commit(ring_empty + 8 * stage);
                }
                ++js;
            } else if (elect_one()) {
                mbar_arrive(ring_empty + 8 * stage);
            }
            __syncwarp();
            if (++stage == (scores ? Y::NK : Y::NV)) { stage = 0; ph ^= 1u; }
        }
        t = cend;
        ++u;
    }
    if (js && elect_one()) {   // every MMA issued here has finished before the TMEM is freed
        umma_commit(fin);
        drain_wait(fin, 0);
    }
    __syncwarp();
}

// 8-bit pools: brings what a row has so far to a reference 2^-d higher, where
// need: O, once the PV before this stage (bar_pv, phase) has completed (with_o),
// and the stage's first 32 weights (with_p).  d is whole, so the weights stay
// the rounded ones they were.
__device__ __noinline__ bool rescale_rows(bool need, float d, uint32_t tl, uint32_t tP, bool with_o, bool with_p,
                                          uint32_t bar_pv, uint32_t phase, volatile int* abortp, DevMeta* meta) {
    const float alpha = need ? ex2_approx(d) : 1.f;
    if (with_p) {
        uint32_t v[16];
        tmem_wait_st();
        tmem_ld16(tP, v);
        tmem_wait_ld16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = pack_bf16(__uint_as_float(v[i] << 16) * alpha, __uint_as_float(v[i] & 0xffff0000u) * alpha);
        tmem_st16(tP, v);
    }
    if (with_o) {
        if (!warp_wait_<true>(bar_pv, phase, abortp, meta)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tl + c0, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st32(tl + c0, v);
        }
    }
    tmem_wait_st();
    return true;
}

// DRAFT: the rows are nodes of draft trees (masked by their ancestors too).
// F8: an 8-bit pool's blocks (tmK and tmV unused).
// CUT: bf16, some branch was rolled back into a block, where V rows may stand behind
// its end (8-bit pools' V is cleared there as it is converted, in every call).
// WHOLE: direct plans (cross attention), whose units that one CTA runs whole are written out here.
// Nothing there waits for HBM (256 rows a unit, several units a KV head through L2), so the roles' chains
// and instructions are what a stage takes, 1,700 cycles of which the products need 1,280 (S with N = 64
// reads its operands from shared memory for longer than it multiplies).  4 prompts of 515 tokens, 32
// heads, over 6,404 states (215 GFLOP): 178 us, 1.2 PFLOP/s, tensor pipe 57 % (whole calls 180 to 188 us on
// different GPUs of this kind); 16 prompts of 448, 16
// heads, over 1,500 (86 GFLOP, a unit starts every 24 stages): 102 us.  On the way there, as whole calls:
//   - partial rows for every unit and the general merge: 248 / 229 us
//   - rows of whole units written here, split units merged by unit: 238 / 138
//   - elected issuers, packed fp32 arithmetic: 216 / 130
//   - tiles and starts weighed by what they take here: 205 / 124
//   - Q in and rows out in whole lines, Q on its way to L2 a unit ahead, descriptors by additions: 193 / 120
//   - K slots given back by the softmax, row sums by mixed additions: 188 / 115
//   - the next unit's Q copied while rows go out: 183 / 106
//   - units of two chunks joined where the second ends, no merge behind: 180 / 104
// Tried there and left: S in one buffer and P in two of its own, so that S is issued a stage ahead (196 /
// 120: the softmax warps then all compute at once, and have more waits), a quarter of the exponentials as
// polynomials (209 / 122: instructions are short, not the SFU).
template <bool DRAFT, bool F8, bool CUT, bool WHOLE>
__global__ void __launch_bounds__(TcLayout<F8>::THREADS, 1)
k_attn_partial_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const AttnArgs a) {
    using Y = TcLayout<F8>;
    constexpr int TC_NSTAGE = Y::NV, OFF_K = Y::OFF_K, OFF_V = Y::OFF_V, OFF_Q = Y::OFF_Q, OFF_BAR = Y::OFF_BAR,
                  OFF_XINFO = Y::OFF_XINFO, B_K_FULL = Y::B_K_FULL, B_K_EMPTY = Y::B_K_EMPTY, B_V_FULL = Y::B_V_FULL,
                  B_V_EMPTY = Y::B_V_EMPTY, B_S_FULL = Y::B_S_FULL, B_P_FULL = Y::B_P_FULL, B_PV_DONE = Y::B_PV_DONE,
                  B_Q_FULL = Y::B_Q_FULL, B_FINAL = Y::B_FINAL, B_COUNT = Y::B_COUNT, TC_PV1_WARP = Y::PV1_WARP,
                  TC_S0_WARP = Y::S0_WARP;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int abort_flag, unclean_flag;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* sm = smem_raw + (base - raw);
    const uint32_t bars = base + OFF_BAR;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_BAR + B_COUNT * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [bars](int i) { return bars + 8u * (uint32_t)i; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < Y::NK; ++s) {
            mbar_init(bar(B_K_FULL + s), F8 ? 4 : 1);   // F8: every converting warp
            mbar_init(bar(B_K_EMPTY + s), 2);    // both S issuers (row tiles 0 and 1)
        }
        for (int s = 0; s < Y::NV; ++s) {
            mbar_init(bar(B_V_FULL + s), F8 ? 4 : 1);
            mbar_init(bar(B_V_EMPTY + s), 2);    // both PV issuers
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(B_S_FULL + i), 1);
            mbar_init(bar(B_P_FULL + i), 4);     // the row tile's four softmax warps
            mbar_init(bar(B_PV_DONE + i), 1);
        }
        for (int r = 0; r < TC_ROWTILES; ++r) mbar_init(bar(B_Q_FULL + r), 4);
        for (int i = 0; i < 4; ++i) mbar_init(bar(B_FINAL + i), 1);
        for (int i = Y::B_RAW_FULL; i < B_COUNT; ++i) mbar_init(bar(i), i < Y::B_RAW_EMPTY ? 1 : 8);   // 8 warps
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    pdl_trigger();
    if (a.plan.counts && (int32_t)blockIdx.x >= a.plan.counts[1]) return;   // past the device-expanded split
    if (threadIdx.x == 0) {
        abort_flag = a.meta->status != 0;
        if (CUT) unclean_flag = a.meta->unclean;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (abort_flag) return;
    if (warp == TC_S0_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const AttnPlanDev& pl = a.plan;
    const int c = blockIdx.x;
    const int32_t t_begin = pl.tc_cta_begin[c], t_end = pl.tc_cta_begin[c + 1];
    const int32_t u0 = pl.tc_cta_unit[c];
    volatile int* abortp = &abort_flag;

    if (F8 && warp >= 8) {
        if (warp < F8_COPY_WARP)
            issue_products<Y>(a, base, bars, tmem, abortp, t_begin, t_end, u0, !(warp & 1),
                              (warp - F8_ISSUE_WARP) >> 1);
        else if (warp == F8_COPY_WARP) copy_tiles<Y>(a, base, bars, abortp, t_begin, t_end, u0);
        else
            convert_tiles<Y>(a, sm, bars, abortp, t_begin, t_end, u0, (warp - F8_CONV_WARP) >> 1,
                             (warp - F8_CONV_WARP) & 1);
    } else if (!F8 && (warp == 0 || warp == TC_V_WARP)) {
        // ------------------------------------------------------ producers
        // Warp 0 streams K into the K ring, warp 11 V into the V ring, so a
        // K slot is refilled as soon as its S is done and a V slot as soon as
        // its P V is done.  Lane i < ntiles issues tile i of the stage: two
        // 64-column halves at token offset 16 i of the stage's two 8 KiB halves.
        const bool k_role = warp == 0;
        const CUtensorMap* tmap = k_role ? &tmK : &tmV;
        const uint32_t ring = base + (k_role ? OFF_K : OFF_V);
        const int b_full = k_role ? B_K_FULL : B_V_FULL, b_empty = k_role ? B_K_EMPTY : B_V_EMPTY;
        uint32_t issued = 0, parity_bits = 0;
        int32_t g = 0;
        int32_t t = t_begin, u = u0;
        while (t < t_end && !*abortp) {
            const AttnUnit U = pl.units[u];
            const int32_t uend = U.tile_off + U.n_blk;
            if (t >= uend) { ++u; continue; }
            const int32_t cend = min(t_end, uend);
            const int32_t* trow = a.table + (int64_t)U.table_row * a.bpb + U.blk_start - U.tile_off;
            // block id of tile t: from the unit's table row, or for a packed
            // unit's extra tile through its entry in the plan
            auto blk_at = [&](int32_t tt) -> int32_t {
                const int32_t ti = tt - U.tile_off;
                if (ti < U.n_shared) return trow[tt];
                const AttnXTile e = pl.xtiles[U.x_off + ti - U.n_shared];
                return a.table[(int64_t)e.table_row * a.bpb + e.blk];
            };
            // block ids, 32 tiles per batch, the next batch loaded one batch ahead
            int32_t cur_base = t, nxt_base = t + 32;
            int32_t cur = t + lane < cend ? blk_at(t + lane) : 0;
            int32_t nxt = nxt_base + lane < cend ? blk_at(nxt_base + lane) : 0;
            for (int32_t st = t; st < cend; st += 4, ++g) {
                if (st >= cur_base + 32) {
                    cur = nxt;
                    cur_base = nxt_base;
                    nxt_base += 32;
                    nxt = nxt_base + lane < cend ? blk_at(nxt_base + lane) : 0;
                }
                int32_t blk = __shfl_sync(0xffffffffu, cur, (st - cur_base) + (lane & 3));
                const int slot = g % TC_NSTAGE;
                const uint32_t ph = (uint32_t)(g / TC_NSTAGE) & 1u;
                const int ntiles = min(4, cend - st);
                int ok = 1;
                if (lane == 0) ok = thread_wait(bar(b_empty + slot), ph ^ 1u, abortp, a.meta);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(bar(b_full + slot), (uint32_t)(ntiles * 2 * HALF_BYTES));
                __syncwarp();
                if (lane < ntiles) {
                    if ((uint32_t)blk >= (uint32_t)a.n_blocks) {   // broken table: poison, read zeros
                        atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                        blk = -1;
                    }
                    const int32_t row0 = (blk * a.n_kv + U.kv_head) * BS;
                    const uint32_t dst = ring + slot * TC_RING_STAGE + lane * HALF_BYTES;
                    const uint32_t fb = bar(b_full + slot);
                    tma_load_3d(dst, tmap, 0, 0, row0, fb);
                    tma_load_3d(dst + TC_HALF, tmap, 0, 1, row0, fb);
                }
                issued |= 1u << slot;
                parity_bits = (parity_bits & ~(1u << slot)) | (ph << slot);
            }
            t = cend;
            ++u;
        }
        if (lane == 0 && *abortp) {   // copies still in flight land before the CTA exits
            for (int s = 0; s < TC_NSTAGE; ++s)
                if (issued >> s & 1u) drain_wait(bar(b_full + s), parity_bits >> s & 1u);
        }
    } else if (!F8 && (warp == 1 || warp == TC_PV_WARP || warp == TC_S1_WARP || warp == TC_PV1_WARP)) {
        // ------------------------------------------------------ MMA issuers
        // Four single-thread issuers, one chain of waits each: for row tile
        // r, an S issuer (warp 1 for r = 0, warp 12 for r = 1) issues
        // S_r(k) = Q_r K^T as soon as stage k's K landed and the P V of
        // stage k - 2, which read the buffer S_r(k) overwrites, completed;
        // a PV issuer (warp 10, warp 13) issues O_r += P_r V as soon as stage
        // k's V landed and P_r(k) is in tensor memory.  A ring
        // slot goes back to its producer once both issuers of its kind have
        // committed it; the issuer of a row tile a unit does not have simply
        // arrives.
        const bool s_role = warp == 1 || warp == TC_S1_WARP;
        const int my_r = (warp == 1 || warp == TC_PV_WARP) ? 0 : 1;
        // Draft trees: all lanes run the loop and one is elected for the
        // products, as in the 8-bit pools' issuers (96 rows, 8,192 tokens:
        // 173 -> 166 us).  Without them it is one lane's loop: electing gained
        // 0.5 % of a verification call and lost 1.2 % of the stress step, where
        // memory is the bound.
        auto one = [] {
            if constexpr (DRAFT || WHOLE) return elect_one();
            return true;
        };
        auto wait = [&](uint32_t wb, uint32_t parity) {
            if constexpr (WHOLE) return eager_wait(wb, parity, abortp, a.meta);
            if constexpr (DRAFT) return warp_wait(wb, parity, abortp, a.meta);
            return thread_wait(wb, parity, abortp, a.meta);
        };
        if (DRAFT || WHOLE || lane == 0) {
            const uint32_t sQ = base + OFF_Q + my_r * TC_QTILE;
            const uint64_t dq = sdesc(sQ, 16, 1024), dk = sdesc(base + OFF_K, 16, 1024), dv = sdesc(base + OFF_V, TC_HALF, 1024);
            int32_t g = 0, js = 0, qc = 0;
            bool ok = true, any = false;
            int32_t t = t_begin, u = u0;
            while (ok && t < t_end) {
                const AttnUnit U = pl.units[u];
                const int32_t uend = U.tile_off + U.n_blk;
                if (t >= uend) { ++u; continue; }
                const int32_t cend = min(t_end, uend);
                const bool active = my_r < U.rt;
                const int32_t nst = (cend - t + 3) >> 2;
                if (s_role && active) ok = wait(bar(B_Q_FULL + my_r), (uint32_t)qc++ & 1u);
                for (int32_t k = 0; k < nst && ok; ++k) {
                    const int32_t gg = g + k;
                    const int slot = gg % TC_NSTAGE;
                    const uint32_t ph = (uint32_t)(gg / TC_NSTAGE) & 1u;
                    const int ntiles = min(4, cend - (t + 4 * k));
                    if (s_role) {
                        ok = wait(bar(B_K_FULL + slot), ph);
                        if (ok && active) {
                            const int b = js & 1;
                            ok = wait(bar(B_PV_DONE + 2 * my_r + b), ((uint32_t)(js >> 1) & 1u) ^ 1u);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t stage = base + OFF_K + slot * TC_RING_STAGE;
                            const uint32_t id = idesc_bf16(128, 16 * ntiles, 0, 0);
                            const uint32_t dS = tmem + my_r * 256 + 128 + b * 64;
                            if constexpr (WHOLE) {   // descriptors by one addition each
                                if (one()) {
                                    const uint64_t dK = sdesc_at(dk, slot * TC_RING_STAGE);
#pragma unroll
                                    for (int kk = 0; kk < 8; ++kk)
                                        umma_bf16(dS, sdesc_at(dq, (kk >> 2) * 16384 + (kk & 3) * 32),
                                                  sdesc_at(dK, (kk >> 2) * TC_HALF + (kk & 3) * 32), id, kk > 0);
                                    umma_commit(bar(B_S_FULL + 2 * my_r + b));   // (the softmax gives the K slot back)
                                }
                            } else if (one()) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk) {
                                    const uint32_t qoff = (kk >> 2) * 16384 + (kk & 3) * 32;
                                    const uint32_t koff = (kk >> 2) * TC_HALF + (kk & 3) * 32;
                                    umma_bf16(dS, sdesc(sQ + qoff, 16, 1024), sdesc(stage + koff, 16, 1024), id, kk > 0);
                                }
                                umma_commit(bar(B_S_FULL + 2 * my_r + b));
                                umma_commit(bar(B_K_EMPTY + slot));
                            }
                            ++js;
                            any = true;
                        } else if (ok && one()) {
                            mbar_arrive(bar(B_K_EMPTY + slot));
                        }
                    } else {
                        ok = wait(bar(B_V_FULL + slot), ph);
                        if (ok && active) {
                            const int b = js & 1;
                            ok = wait(bar(B_P_FULL + 2 * my_r + b), (uint32_t)(js >> 1) & 1u);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t vst = base + OFF_V + slot * TC_RING_STAGE;
                            const uint32_t id = idesc_bf16(128, 128, 0, 1);
                            const uint32_t tP = tmem + my_r * 256 + 128 + b * 64;   // 16 tokens per 8 columns
                            if constexpr (WHOLE) {
                                if (one()) {
                                    const uint64_t dV = sdesc_at(dv, slot * TC_RING_STAGE);
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        if (kk < ntiles)
                                            umma_bf16_ta(tmem + my_r * 256, tP + kk * 8, sdesc_at(dV, kk * 2048), id, kk > 0 || k > 0);
                                    umma_commit(bar(B_PV_DONE + 2 * my_r + b));
                                    umma_commit(bar(B_V_EMPTY + slot));
                                }
                            } else if (one()) {
                                for (int kk = 0; kk < ntiles; ++kk)
                                    umma_bf16_ta(tmem + my_r * 256, tP + kk * 8, sdesc(vst + kk * 2048, TC_HALF, 1024),
                                                 id, kk > 0 || k > 0);
                                umma_commit(bar(B_PV_DONE + 2 * my_r + b));
                                umma_commit(bar(B_V_EMPTY + slot));
                            }
                            ++js;
                            any = true;
                        } else if (ok && one()) {
                            mbar_arrive(bar(B_V_EMPTY + slot));
                        }
                    }
                    if constexpr (DRAFT || WHOLE) __syncwarp();
                }
                g += nst;
                t = cend;
                ++u;
            }
            if (any && one()) {   // every MMA issued here has finished before the TMEM is freed
                const uint32_t fb = bar(B_FINAL + (s_role ? 0 : 1) + 2 * my_r);
                umma_commit(fb);
                drain_wait(fb, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax
        const int r = (warp - Y::SOFTMAX_WARP0) >> 2;
        const int sub = warp & 3;                 // TMEM lanes 32 sub .. 32 sub + 31
        const int trow = sub * 32 + lane;         // row within the row tile
        const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16) + r * 256;
        unsigned char* sQ = sm + OFF_Q + r * TC_QTILE;
        const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
        // row of the unit (F8: both groups hold the rows of a split unit)
        auto row_of = [&](const AttnUnit& V) { return F8 && V.rt == 1 ? trow : r * 128 + trow; };
        int2* xinfo = reinterpret_cast<int2*>(sm + OFF_XINFO) + r * kMaxTcExtraTiles;
        unsigned char* xheld = sm + Y::OFF_XHELD + r * kMaxTcExtraTiles;
        // draft trees: the row's mask, in shared memory: in registers, or made
        // again from the unit where it is needed, it cost spills in the loop
        // (a third of its time)
        uint64_t* mask_slot = reinterpret_cast<uint64_t*>(sm + Y::OFF_MASK) + r * 128 + trow;
        // This thread's row of a unit's Q into the K-major swizzled tile, and
        // the row's record.  A unit's Q is staged as soon as the previous
        // chunk's last S was read (no S MMA of it is pending then), before
        // that chunk's epilogue, so the next chunk's S overlaps the epilogue.
        auto stage_q = [&](const AttnUnit& V) -> AttnRow {
            const int row = row_of(V);
            const bool v_ok = row < V.n_rows;
            const AttnRow RR = v_ok ? unit_row(pl, V, row) : AttnRow{0, 0};
            if constexpr (WHOLE && !F8) {
                // two rows an instruction (sixteen lanes each), so that a request covers whole lines: a row
                // a lane, 16 bytes at a time, took 4,000 cycles for the 256 rows.  On their way while the
                // previous unit's rows go out (q_there)
                const int32_t from = v_ok ? RR.q_row : -1;
                const int ch = lane & 15;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int32_t q_row = __shfl_sync(0xffffffffu, from, 2 * i + (lane >> 4));
                    const int tr = sub * 32 + 2 * i + (lane >> 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     smem_u32(sQ + (ch >> 3) * 16384 + tr * 128 + (((ch & 7) ^ (tr & 7)) << 4))),
                                 "l"(reinterpret_cast<const uint4*>(Q + (int64_t)max(q_row, 0) * D) + ch), "r"(q_row >= 0 ? 16 : 0)
                                 : "memory");
                }
                return RR;
            }
            const uint4* q = reinterpret_cast<const uint4*>(Q + (int64_t)RR.q_row * D);
#pragma unroll
            for (int ch = 0; ch < 16; ++ch) {
                const uint4 v = v_ok ? __ldg(q + ch) : make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(sQ + (ch >> 3) * 16384 + trow * 128 + (((ch & 7) ^ (trow & 7)) << 4)) = v;
            }
            if constexpr (DRAFT) *mask_slot = v_ok ? draft_mask(pl, V, row) : 0;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_Q_FULL + r));
            return RR;
        };
        int32_t js = 0;
        bool ok = true;
        int32_t t = t_begin, u = u0;
        // WHOLE: the tile's Q is there, and S may be issued
        auto q_there = [&] {
            if constexpr (WHOLE && !F8) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q_FULL + r));
            }
        };
        int32_t staged_u = -1;      // unit whose Q is already in the tile
        AttnRow staged_R{0, 0};
        uint32_t joined = 0;        // phase of the joins of split units
        int32_t g = 0;              // CUT: stages before this chunk
        const bool unclean = CUT && unclean_flag;   // V may hold rows that are not finite
        while (ok && t < t_end) {
            const AttnUnit U = pl.units[u];
            const int32_t uend = U.tile_off + U.n_blk;
            if (t >= uend) { ++u; continue; }
            const int32_t cend = min(t_end, uend);
            const int32_t nst = (cend - t + 3) >> 2;
            const RowTiles tiles(U, nst);
            if (r >= (F8 ? tiles.n : U.rt)) {
                g += nst;
                t = cend;
                ++u;
                continue;
            }
            const int row = row_of(U);
            const bool valid = row < U.n_rows;
            const bool staged = staged_u == u;
            const AttnRow R = staged ? staged_R : stage_q(U);
            if (!staged) q_there();
            if (!F8 && !WHOLE && U.n_blk > U.n_shared) {   // (no unit of a direct plan is packed)
                // a packed unit: its extra tiles' logical blocks, member masks
                // and held tokens into shared memory, once every warp of the row tile
                // is done with the previous unit's (the plan keeps them to
                // kMaxTcExtraTiles; a unit past that reads none and is flagged)
                const int32_t nx = U.n_blk - U.n_shared;
                if (nx > kMaxTcExtraTiles && trow == 0) atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                asm volatile("bar.sync %0, 128;" ::"r"(1 + r) : "memory");
                for (int32_t i = trow; i < min(nx, kMaxTcExtraTiles); i += 128) {
                    const int2 e = *reinterpret_cast<const int2*>(pl.xtiles + U.x_off + i);
                    xinfo[i] = e;
                    if constexpr (CUT) {
                        int32_t len = 0;
                        for (uint32_t mm = (uint32_t)e.y; mm; mm &= mm - 1u)
                            len = max(len, pl.members[U.mem_off + __ffs(mm) - 1].len);
                        xheld[i] = (unsigned char)min(BS, len - e.x * BS);
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + r) : "memory");
            }
            if constexpr (WHOLE && !F8) {   // the next chunk's Q, on its way to L2 meanwhile
                if (u + 1 < pl.n_units && cend < t_end) {
                    const AttnUnit& V = pl.units[u + 1];
                    if (row_of(V) < V.n_rows) {
                        const char* q = reinterpret_cast<const char*>(Q + (int64_t)unit_row(pl, V, row_of(V)).q_row * D);
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 128));
                    }
                }
            }
            const int32_t k0 = F8 && tiles.split ? r : 0, k_step = F8 && tiles.split ? 2 : 1;
            float m_ref = -INFINITY, l = 0.f;
            for (int32_t k = k0; k < nst && ok; k += k_step, ++js) {
                const int32_t st = t + 4 * k;
                const int ntiles = min(4, cend - st);
                const int b = js & 1;
                ok = warp_wait_<F8, WHOLE>(bar(B_S_FULL + 2 * r + b), (uint32_t)(js >> 1) & 1u, abortp, a.meta);
                if (!ok) break;
                tc_fence_after();
                // (a commit takes its issuer some 150 cycles, an arrival next to nothing)
                if (WHOLE && !F8 && sub == 0 && lane == 0) mbar_arrive(bar(B_K_EMPTY + (g + k) % TC_NSTAGE));
                if ((DRAFT || F8) && row - lane >= U.n_rows) {
                    // a warp without a row of the unit: its rows of Q are zero,
                    // hence of S, which is zero as P too; it only passes the buffer on
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P_FULL + 2 * r + b));
                    continue;
                }
                if constexpr (F8) {
                    // half a stage at a time: 32 scores fit the 80 registers a thread
                    // has, and a reference that the second half outgrows is raised
                    // for the first half's weights too
                    const int32_t off = R.limit - (U.blk_start + st - U.tile_off) * BS;
                    const bool plain = __all_sync(0xffffffffu, off >= TC_TOK) && ntiles == 4;
                    const uint32_t tS = tl + 128 + b * 64;
                    uint64_t see = ~0ull;
                    if (!plain) {
                        see = DRAFT       ? draft_visible(*mask_slot, off)
                              : off >= 64 ? ~0ull
                              : off > 0   ? (1ull << off) - 1ull
                                          : 0ull;
                        if (ntiles < 4) see &= (1ull << (ntiles * BS)) - 1ull;
                    }
                    f32x2 l2[2] = {0, 0};
                    const f32x2 scale2 = pair(a.scale_log2, a.scale_log2);
#pragma unroll 1
                    for (int half = 0; half < 2;) {
                        uint32_t v[32];
                        tmem_ld32(tS + 32 * half, v);
                        tmem_wait_ld(v);
                        if (!plain) mask_half(v, (uint32_t)(see >> (32 * half)));
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; i += 2) m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], v[i], v[i + 1]);
                        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
                        // whole references: what is rescaled keeps its bits
                        if (k == k0 && half == 0) {
                            m_ref = ceilf(mx);
                        } else {
                            const bool need = mx > m_ref + RESCALE_THRESHOLD;
                            if (__any_sync(0xffffffffu, need)) {
                                const float m_new = ceilf(mx);
                                ok = rescale_rows(need, m_ref - m_new, tl, tS, k != k0, half != 0,
                                                  bar(B_PV_DONE + 2 * r + ((js - 1) & 1)), (uint32_t)((js - 1) >> 1) & 1u,
                                                  abortp, a.meta);
                                if (!ok) break;
                                if (need) {
                                    const float alpha = ex2_approx(m_ref - m_new);
                                    l *= alpha;
                                    l2[0] = mul2(l2[0], pair(alpha, alpha));
                                    l2[1] = mul2(l2[1], pair(alpha, alpha));
                                    m_ref = m_new;
                                }
                                continue;   // this half again: its scores need not outlive the call
                            }
                        }
                        const float nref = m_ref == -INFINITY ? 0.f : -m_ref;
                        const f32x2 nref2 = pair(nref, nref);
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const f32x2 x = fma2(pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale2,
                                                 nref2);
                            pk[i] = pack_bf16(ex2_approx(low(x)), ex2_approx(high(x)));
                            l2[i & 1] = add2(l2[i & 1], pair(__uint_as_float(pk[i] << 16),
                                                             __uint_as_float(pk[i] & 0xffff0000u)));
                        }
                        tmem_st16(tS + 16 * half, pk);   // over columns already read
                        ++half;
                    }
                    if (!ok) break;
                    const f32x2 ls = add2(l2[0], l2[1]);
                    l += low(ls) + high(ls);
                } else {
                float s[64];
                {
                    uint32_t v0[32], v1[32];
                    tmem_ld32(tl + 128 + b * 64, v0);
                    tmem_ld32(tl + 128 + b * 64 + 32, v1);
                    tmem_wait_ld(v0);
                    reg_tie(v1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        s[i] = __uint_as_float(v0[i]);
                        s[32 + i] = __uint_as_float(v1[i]);
                    }
                }
                // mask stage columns past the chunk and positions the row does
                // not see (only stages some row of the warp does not fully see)
                const int32_t ti0 = st - U.tile_off;
                if (WHOLE || ti0 + ntiles <= U.n_shared) {
                    const int32_t vis = min(ntiles * BS, R.limit - (U.blk_start + ti0) * BS);
                    if (!__all_sync(0xffffffffu, vis >= TC_TOK)) {
                        if constexpr (DRAFT) {
                            // draft trees: the stage's seen positions as bits
                            uint64_t see = draft_visible(*mask_slot, R.limit - (U.blk_start + ti0) * BS);
                            if (ntiles < 4) see &= (1ull << (ntiles * BS)) - 1ull;
#pragma unroll
                            for (int i = 0; i < 64; ++i) s[i] = (see >> i) & 1ull ? s[i] : -INFINITY;
                        } else {
#pragma unroll
                            for (int i = 0; i < 64; ++i) s[i] = i < vis ? s[i] : -INFINITY;
                        }
                    }
                } else {
                    // a stage with a packed unit's extra tiles: each tile counts
                    // only for the rows of the members in its mask
                    const int32_t mi = div_rcp(U.row_lo + row, pl.q_len * pl.group, pl.rcp_rows_per_member);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int32_t tj = ti0 + j;
                        int32_t lb = U.blk_start + tj;
                        bool seen = j < ntiles;
                        if (seen && tj >= U.n_shared) {
                            const int2 e = xinfo[min(tj - U.n_shared, kMaxTcExtraTiles - 1)];
                            lb = e.x;
                            seen = ((uint32_t)e.y >> (mi & 31)) & 1u;
                        }
                        const int32_t v = seen ? min(BS, R.limit - lb * BS) : 0;
                        if constexpr (DRAFT) {
                            const uint32_t see =
                                seen ? (uint32_t)draft_visible(*mask_slot, R.limit - lb * BS) : 0u;
#pragma unroll
                            for (int c = 0; c < BS; ++c) s[BS * j + c] = (see >> c) & 1u ? s[BS * j + c] : -INFINITY;
                        } else {
#pragma unroll
                            for (int c = 0; c < BS; ++c) s[BS * j + c] = c < v ? s[BS * j + c] : -INFINITY;
                        }
                    }
                }
                // row max of the raw scores (eight independent chains), then
                // in base-2 units (the scale is positive)
                float mx;
                if constexpr (WHOLE) {
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 64; i += 2)
                        m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __float_as_uint(s[i]), __float_as_uint(s[i + 1]));
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
                } else {
                    float m8[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) m8[j] = s[j];
#pragma unroll
                    for (int i = 8; i < 64; ++i) m8[i & 7] = fmaxf(m8[i & 7], s[i]);
                    mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                               fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                    mx *= a.scale_log2;
                }
                if (k == 0) {
                    m_ref = mx;   // this stage's PV overwrites O
                } else {
                    const bool need = mx > m_ref + RESCALE_THRESHOLD;
                    if (__any_sync(0xffffffffu, need)) {
                        // O holds the PV of the previous stage once it completes
                        ok = warp_wait(bar(B_PV_DONE + 2 * r + ((js - 1) & 1)), (uint32_t)((js - 1) >> 1) & 1u,
                                       abortp, a.meta);
                        if (!ok) break;
                        tc_fence_after();
                        const float alpha = need ? ex2_approx(m_ref - mx) : 1.f;
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t v[32];
                            tmem_ld32(tl + c0, v);
                            tmem_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                            tmem_st32(tl + c0, v);
                        }
                        tmem_wait_st();
                        if (need) {
                            l *= alpha;
                            m_ref = mx;
                        }
                    }
                }
                const float nref = m_ref == -INFINITY ? 0.f : -m_ref;
                // P = 2^(s * scale - m_ref) in bf16; the row sum is taken over
                // the rounded values (eight independent chains)
                uint32_t pk[32];
                if constexpr (WHOLE) {   // the same sums, two to an instruction
                    const f32x2 scale2 = pair(a.scale_log2, a.scale_log2), nref2 = pair(nref, nref);
                    float l8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const f32x2 x = fma2(pair(s[2 * i], s[2 * i + 1]), scale2, nref2);
                        pk[i] = pack_bf16(ex2_approx(low(x)), ex2_approx(high(x)));
                        add_bf16(l8[(2 * i) & 7], l8[(2 * i + 1) & 7], pk[i]);
                    }
                    l += ((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7]));
                } else {
                    float l8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        pk[i] = pack_bf16(ex2_approx(fmaf(s[2 * i], a.scale_log2, nref)),
                                          ex2_approx(fmaf(s[2 * i + 1], a.scale_log2, nref)));
                        l8[(2 * i) & 7] += __uint_as_float(pk[i] << 16);
                        l8[(2 * i + 1) & 7] += __uint_as_float(pk[i] & 0xffff0000u);
                    }
                    l += ((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7]));
                }
                // P over the S it came from (token 2 i in the low half of
                // column i); unused columns past the chunk hold P = 0
                tmem_st32(tl + 128 + b * 64, pk);
                if (CUT && unclean && ti0 + ntiles >= U.n_shared) {
                    ok = clear_tails(a, sm, bars, abortp, pl.units[u], ti0, ntiles, R.limit, g + k, xheld);
                    if (!ok) break;
                }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_FULL + 2 * r + b));
            }
            if (!ok) break;
            // the next chunk this row tile works on: stage its Q now
            bool coming;
            {
                int32_t t2 = cend, u2 = u + 1;
                while (t2 < t_end) {
                    const AttnUnit& V = pl.units[u2];
                    const int32_t e2 = V.tile_off + V.n_blk;
                    if (t2 >= e2) { ++u2; continue; }
                    if (r < (F8 ? RowTiles(V, (min(t_end, e2) - t2 + 3) >> 2).n : V.rt)) break;
                    t2 = min(t_end, e2);
                    ++u2;
                }
                if (t2 < t_end) {
                    staged_R = stage_q(pl.units[u2]);
                    staged_u = u2;
                }
                coming = t2 < t_end;
            }
            g += nst;
            // chunk done: O after the last PV -> partial row
            ok = warp_wait_<F8, WHOLE>(bar(B_PV_DONE + 2 * r + ((js - 1) & 1)), (uint32_t)((js - 1) >> 1) & 1u, abortp, a.meta);
            if (!ok) break;
            tc_fence_after();
            const int32_t prow = U.prow_base + (c - U.cfirst) * U.n_rows + row;
            float* dst = a.part_acc + (int64_t)(valid ? prow : 0) * D;
            if (F8 && tiles.split && tiles.n == 2) {
                // join: each group stores half of the columns of both
                float2* ml = reinterpret_cast<float2*>(sm + Y::OFF_ML);
                ml[r * 128 + trow] = make_float2(m_ref, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Y::B_ML_FULL));
                ok = warp_wait_<F8>(bar(Y::B_ML_FULL), joined, abortp, a.meta);
                if (!ok) break;
                tc_fence_after();
                const float2 o = ml[(r ^ 1) * 128 + trow];
                const float m = fmaxf(m_ref, o.x);
                const float mine = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
                const float other = o.x == -INFINITY ? 0.f : ex2_approx(o.x - m);
                const uint32_t tl_o = tmem + ((uint32_t)(sub * 32) << 16) + (r ^ 1) * 256;
                const bool whole = WHOLE && U.nchunks == 1;
                const float sum = l * mine + o.y * other, inv = 1.f / sum;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
                if (whole && valid) out += (int64_t)unit_row(pl, U, row).q_row * D;
#pragma unroll 1
                for (int c0 = r * (D / 2); c0 < (r + 1) * (D / 2); c0 += 32) {
                    uint32_t v[32], w[32];
                    tmem_ld32(tl + c0, v);
                    tmem_ld32(tl_o + c0, w);
                    tmem_wait_ld(v);
                    reg_tie(w);
                    if (valid && whole) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint(__uint_as_float(v[i]) * mine + __uint_as_float(w[i]) * other);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(out + c0 + i) = out_words(v + i, inv);
                    } else if (valid) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float4 x;
                            x.x = __uint_as_float(v[i]) * mine + __uint_as_float(w[i]) * other;
                            x.y = __uint_as_float(v[i + 1]) * mine + __uint_as_float(w[i + 1]) * other;
                            x.z = __uint_as_float(v[i + 2]) * mine + __uint_as_float(w[i + 2]) * other;
                            x.w = __uint_as_float(v[i + 3]) * mine + __uint_as_float(w[i + 3]) * other;
                            *reinterpret_cast<float4*>(dst + c0 + i) = x;
                        }
                    }
                }
                if (valid && !whole && r == 0) a.part_ml[prow] = make_float2(m, sum);
                // neither accumulator is written again, nor its (m, l), before both groups are done
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Y::B_ML_DONE));
                ok = warp_wait_<F8>(bar(Y::B_ML_DONE), joined, abortp, a.meta);
                if (!ok) break;
                tc_fence_after();
                joined ^= 1u;
                t = cend;
                ++u;
                continue;
            }
            const bool whole = WHOLE && U.nchunks == 1;   // no other partial: O / l is the output row
            const float inv = 1.f / l;
            if constexpr (WHOLE && !F8) {
                // 64 bytes of each of the warp's rows at a time through shared memory, so that a store
                // covers whole sectors of eight rows
                unsigned char* box = sm + Y::OFF_OUT + (warp - Y::SOFTMAX_WARP0) * Y::OUT_WARP;
                int32_t to = !valid ? -1 : whole ? unit_row(pl, U, row).q_row : prow;
                char* base_out = whole ? static_cast<char*>(a.out) : reinterpret_cast<char*>(a.part_acc);
                int32_t row_bytes = whole ? D * 2 : D * 4;
                auto send = [&](const uint4 (&x)[4], int32_t at) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(box + lane * 80 + i * 16) = x[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = 8 * i + (lane >> 2);
                        const int32_t out_row = __shfl_sync(0xffffffffu, to, rr);
                        const uint4 y = *reinterpret_cast<const uint4*>(box + rr * 80 + (lane & 3) * 16);
                        if (out_row >= 0)
                            *reinterpret_cast<uint4*>(base_out + (int64_t)out_row * row_bytes + at + (lane & 3) * 16) = y;
                    }
                    __syncwarp();
                };
                // a unit of two chunks: each warp's rows are joined by the CTA that ends second, which has its
                // own in TMEM yet; none waits for the other.  (The one with the second chunk does it first of
                // all, the other last.)  Sums are in the chunks' order, whoever makes them
                const bool two = U.nchunks == 2, later = c != U.cfirst;
                int32_t* met = a.joins + U.cfirst * 8 + (warp - Y::SOFTMAX_WARP0);
                int32_t other = 0;   // the other's partial rows are there
                if (two) other = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(met, 0) : 0, 0);
#pragma unroll 1
                for (int c0 = 0; c0 < (other ? 0 : D); c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(tl + c0, v);
                    tmem_wait_ld(v);
                    if (c0 == D / 2 && coming) {
                        q_there();
                        coming = false;
                    }
                    if (whole) {
                        send({out_words(v, inv), out_words(v + 8, inv), out_words(v + 16, inv), out_words(v + 24, inv)}, c0 * 2);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 16)
                            send({make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]), make_uint4(v[i + 4], v[i + 5], v[i + 6], v[i + 7]),
                                  make_uint4(v[i + 8], v[i + 9], v[i + 10], v[i + 11]), make_uint4(v[i + 12], v[i + 13], v[i + 14], v[i + 15])},
                                 (c0 + i) * 4);
                    }
                }
                if (valid && !whole && !other) a.part_ml[prow] = make_float2(m_ref, l);
                if (two && !other) {
                    __threadfence();
                    __syncwarp();
                    other = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(met, 1) : 0, 0);
                }
                if (two && other) {
                    __threadfence();
                    const int64_t there = (int64_t)U.prow_base + (later ? 0 : U.n_rows) + row;
                    const float2 o = valid ? __ldcg(a.part_ml + there) : make_float2(-INFINITY, 0.f);
                    const float m = fmaxf(m_ref, o.x), ref = m == -INFINITY ? 0.f : m;
                    const float w = exp2f(m_ref - ref), w_o = exp2f(o.x - ref);
                    const float w0 = later ? w_o : w, w1 = later ? w : w_o;
                    const float inv2 = 1.f / (later ? fmaf(w1, l, w0 * o.y) : fmaf(w1, o.y, w0 * l));
                    to = valid ? unit_row(pl, U, row).q_row : -1;
                    base_out = static_cast<char*>(a.out);
                    row_bytes = D * 2;
                    // the other's rows 64 bytes at a time, eight rows a load (a row a lane: 16 us more), through the
                    // same box; the next 128 are on their way meanwhile
                    const int32_t from = valid ? (int32_t)there : -1;
                    float4 next[2][4];
                    auto load = [&](int32_t c0, float4 (&to)[4]) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int32_t at = __shfl_sync(0xffffffffu, from, 8 * i + (lane >> 2));
                            to[i] = at >= 0 ? __ldcg(reinterpret_cast<const float4*>(a.part_acc + (int64_t)at * D + c0) + (lane & 3))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    };
                    load(0, next[0]);
                    load(16, next[1]);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t v[32];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<float4*>(box + (8 * i + (lane >> 2)) * 80 + (lane & 3) * 16) = next[half][i];
                            __syncwarp();
                            if (c0 + 32 < D) load(c0 + 32 + 16 * half, next[half]);
                            float x[16];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 y = *reinterpret_cast<const float4*>(box + lane * 80 + i * 16);
                                x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
                            }
                            __syncwarp();
                            if (half == 0) {
                                tmem_ld32(tl + c0, v);
                                tmem_wait_ld(v);
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float own = __uint_as_float(v[16 * half + i]);
                                v[16 * half + i] = __float_as_uint(later ? fmaf(w1, own, w0 * x[i]) : fmaf(w1, x[i], w0 * own));
                            }
                        }
                        if (c0 == D / 2 && coming) {
                            q_there();
                            coming = false;
                        }
                        send({out_words(v, inv2), out_words(v + 8, inv2), out_words(v + 16, inv2), out_words(v + 24, inv2)}, c0 * 2);
                    }
                    if (lane == 0) atomicExch(met, 0);   // as the next call expects it
                }
                tc_fence_before();
                t = cend;
                ++u;
                continue;
            }
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
            if (whole && valid) out += (int64_t)unit_row(pl, U, row).q_row * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tl + c0, v);
                tmem_wait_ld(v);
                if (valid && whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4*>(out + c0 + i) = out_words(v + i, inv);
                } else if (valid) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(dst + c0 + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (valid && !whole) a.part_ml[prow] = make_float2(m_ref, l);
            tc_fence_before();
            t = cend;
            ++u;
        }
        if (WHOLE && !F8) asm volatile("cp.async.wait_all;" ::: "memory");   // (an aborted unit's)
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == TC_S0_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

}  // namespace

namespace dendrite {

template <bool DRAFT, bool F8, bool CUT, bool WHOLE = false>
static int setup_one() {
    constexpr auto fn = k_attn_partial_tc<DRAFT, F8, CUT, WHOLE>;
    constexpr int smem = WHOLE ? TcLayout<F8>::SMEM_WHOLE : TcLayout<F8>::SMEM;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return DENDRITE_ECUDA;
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, TcLayout<F8>::THREADS, smem) !=
            cudaSuccess ||
        occ != 1)
        return DENDRITE_ECUDA;   // the kernel's 512 TMEM columns need exactly one CTA per SM
    return DENDRITE_OK;
}

int attn_tc_setup(bool f8) {
    if (f8) {
        DENDRITE_TRY((setup_one<false, true, false>()));
        DENDRITE_TRY((setup_one<false, true, false, true>()));
        return setup_one<true, true, false>();
    }
    DENDRITE_TRY((setup_one<false, false, false, true>()));
    DENDRITE_TRY((setup_one<false, false, true, true>()));
    DENDRITE_TRY((setup_one<false, false, false>()));
    DENDRITE_TRY((setup_one<true, false, false>()));
    DENDRITE_TRY((setup_one<false, false, true>()));
    return setup_one<true, false, true>();
}

template <bool F8, bool CUT>
static void launch_one(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, int n_ctas, cudaStream_t s) {
    using Y = TcLayout<F8>;
    if (a.plan.masks) k_attn_partial_tc<true, F8, CUT, false><<<n_ctas, Y::THREADS, Y::SMEM, s>>>(mk, mv, a);
    else if (a.plan.direct) k_attn_partial_tc<false, F8, CUT, true><<<n_ctas, Y::THREADS, Y::SMEM_WHOLE, s>>>(mk, mv, a);
    else k_attn_partial_tc<false, F8, CUT, false><<<n_ctas, Y::THREADS, Y::SMEM, s>>>(mk, mv, a);
}

int launch_attn_tc(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, int n_ctas, bool f8, cudaStream_t s) {
    if (f8) launch_one<true, false>(mk, mv, a, n_ctas, s);
    else if (a.cut) launch_one<false, true>(mk, mv, a, n_ctas, s);
    else launch_one<false, false>(mk, mv, a, n_ctas, s);
    return cudaGetLastError() == cudaSuccess ? DENDRITE_OK : DENDRITE_ECUDA;
}

}  // namespace dendrite
