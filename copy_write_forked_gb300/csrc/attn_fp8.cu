// Partial attention kernel over 8-bit blocks (DENDRITE_FP8 pools).
//
// The plan, its units and the partial rows are those of the bf16 kernels; a
// unit is up to 64 query rows over tiles of 16 tokens.  A tile is 2,064 bytes
// of K and 2,064 of V (e4m3 codes, one power-of-two scale per token): at the
// HBM rate an SM is handed about 23 bytes per cycle, so what bounds the kernel
// is how few instructions turn a code into a tensor core operand.
//
//   Operands are fp16: one cvt.f16x2.e4m3x2 per two codes, exact, and no
//   scaling per element.  The scales go where there is one per token:
//     S[r][t] = (q_r . c_t) 2^e_t     on the score, with the softmax's scale;
//     O[r]    = sum_t (p_rt 2^f_t) v_t   on the weight.
//   A row of Q is brought to (-4, 4) by a power of two (returned with the
//   score), which loses nothing that fp16 keeps of a bf16 row: elements under
//   2^-14 of the row's largest lose bits below 2^-25 of it.
//   The weights w_rt = p_rt 2^f_t get a running reference W of their own, as
//   log2 w is score + f_t: w is stored as 2^(score + f_t - W) in fp16, whatever the
//   spread of the tokens' scales, while the row sum l takes p = 2^(score - m) in
//   fp32.  W is whole and 15 below the largest (weights reach 2^15: fp16 keeps 11
//   bits of those down to 2^-29 of the largest, where a reference at the largest
//   would end at 2^-14, and the many small weights beside one large would be off by
//   the same side of a step).  acc is in units of 2^W and is brought to 2^m when the
//   chunk's partial row is written.
//
//   K needs no ldmatrix: the mma's k order is free as long as Q and K agree,
//   so a lane takes 32 consecutive codes of its token (two 16-byte loads).
//   V goes through ldmatrix.trans on pairs of codes; one byte permutation
//   parts the even dimensions from the odd ones, and each of the two is an
//   operand (their accumulators interleave to four consecutive columns).
//
// Four warps share a unit: each row tile of 16 rows belongs to 4, 2 or 1 of
// them, which take the unit's tiles two at a time in turn and combine their
// states at the chunk's end.  Every warp copies its own tiles (cp.async.bulk
// into a ring of two slots of two tiles): the next copy into a slot is issued
// when the warp is done with it, no warp waits for another, and the registers
// of a copying warp go to a third CTA on the SM.  What bounds the kernel is
// the latency of a step's chain (products, maximum over four lanes,
// exponentials, products), so warps side by side and two tiles per step pay:
// with a producer warp, two CTAs and one tile per step, eight warps kept up
// with 70 % of the HBM rate.  A row tile's warps beyond one copy of the tiles
// read them from L2 (units of more than 16 rows).
//
// 8 contexts of 32,768 tokens, 4 rows a kv head: 96 us for 549 MB (5.7 TB/s; at
// 18 % of the warps and 50 % of the issue slots it is the chain's latency that
// keeps it from 6.8); 8 prefixes of 4,096 tokens read by 16 rows each, with 256
// tokens behind them for each of 4 branches: 31.6 us a call for 85 MB, where a call
// on one short context takes 12 to 17 (the host's pace).
//
// Every mbarrier wait is bounded, as in the bf16 kernel.
#include <cuda_fp16.h>

#include <climits>

#include "attn_common.cuh"
#include "attn_fp8.h"
#include "rows.h"

using namespace dendrite;

namespace {

constexpr int F8_TILE = 2 * kFp8TileBytes;               // K then V of one tile
constexpr int F8_SLOT = 2 * F8_TILE;                     // two tiles
constexpr int F8_SLOTS = 2;                              // per warp
constexpr int F8_WARPS = 4;
constexpr int F8_THREADS = F8_WARPS * 32;
constexpr int F8_ML = F8_WARPS * F8_SLOTS * F8_SLOT;     // per warp and row (m, l)
constexpr int F8_BAR = F8_ML + F8_WARPS * 16 * 8;
constexpr size_t F8_SMEM = F8_BAR + F8_WARPS * F8_SLOTS * 8;
// at a chunk's end a warp leaves its 16 rows of fp32 sums in the slot it read last
static_assert(F8_SLOT >= 16 * D * 4 && F8_SLOT % 16 == 0 && F8_BAR % 8 == 0, "layout");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Four e4m3 codes to fp16, exactly.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// (not volatile: the compiler may interleave the chains of several accumulators)
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The least reference under which weights of up to 2^x stay in fp16: whole, so that
// sums rescaled from one to another keep their bits.  (From 2^23 on x is whole itself,
// and x - 15 might round to a reference more than 15 below: there it is x.)
constexpr float kWeightTop = 15.f;
__device__ __forceinline__ float weight_ref(float x) { return ceilf(x) - (fabsf(x) < 0x1p23f ? kWeightTop : 0.f); }

// A row's 32 elements 32 q .. 32 q + 31 (q = lane % 4) as fp16 pairs w[0..15],
// scaled by a power of two common to the row; returns that power's inverse
// times the softmax scale.
__device__ __forceinline__ float load_q(const __nv_bfloat16* row, bool valid, int q, float scale, uint32_t (&w)[16]) {
    uint32_t raw[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint4 v = valid ? __ldg(reinterpret_cast<const uint4*>(row + 32 * q) + k) : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * k] = v.x;
        raw[4 * k + 1] = v.y;
        raw[4 * k + 2] = v.z;
        raw[4 * k + 3] = v.w;
    }
    uint32_t top = 0;   // magnitudes of bf16 order as integers
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, max(raw[k] & 0x7fffu, (raw[k] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = min(max((int)(top >> 7), 1), 253);          // biased exponent of the largest
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e)
#pragma unroll
    for (int k = 0; k < 16; ++k)
        w[k] = pack_f16(__uint_as_float(raw[k] << 16) * inv, __uint_as_float(raw[k] & 0xffff0000u) * inv);
    return scale * __uint_as_float((uint32_t)e << 23);
}

// The pairs of tiles a warp reads, in order: of every chunk of the CTA's range
// those of its turn.
struct PairWalk {
    int32_t t, u, cend = 0;              // next pair's first tile; its unit; the chunk's end
    int64_t row = 0;                     // table offset of the unit's tile 0
    int32_t head = 0, step = 1;
    int32_t t_next;                      // where the next chunk begins
    __device__ __forceinline__ PairWalk(int32_t t0, int32_t u0) : t(0), u(u0 - 1), t_next(t0) {}
    // Moves on to the chunk of the next pair; false past the range's end.
    __device__ __forceinline__ bool more(const AttnPlanDev& pl, int32_t t_end, int32_t bpb, int warp) {
        while (t >= cend) {
            if (t_next >= t_end) return false;
            const AttnUnit& U = pl.units[++u];
            if (t_next >= U.tile_off + U.n_blk) continue;
            cend = min(t_end, U.tile_off + U.n_blk);
            const int P = F8_WARPS / U.rt;
            // a row tile past the unit's rows has no warps
            t = (warp / P) * 16 >= U.n_rows ? cend : t_next + 2 * (warp % P);
            t_next = cend;
            step = 2 * P;
            row = (int64_t)U.table_row * bpb + U.blk_start - U.tile_off;
            head = U.kv_head;
        }
        return true;
    }
};

template <bool DRAFT>
__global__ void __launch_bounds__(F8_THREADS, 3) k_attn_partial_fp8(const AttnArgs a) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ int abort_flag;
    __shared__ int last_slot[F8_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bars = smem_u32(sm) + F8_BAR + warp * F8_SLOTS * 8;
    if (lane < F8_SLOTS) mbar_init(bars + 8 * lane, 1);
    // The kernels after this one are let in at each CTA's end only: let in at
    // the start, the merge and, behind it, the next call's partial kernel take
    // SM slots as the first CTAs here end, and that call's CTAs crowd on few
    // SMs (8 contexts of 32,768 tokens, calls back to back: 142 us, and 98 so).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnPlanDev& pl = a.plan;
    const int c = blockIdx.x;
    const int32_t t_begin = pl.cta_begin[c], t_end = pl.cta_begin[c + 1];
    const int32_t u0 = pl.cta_unit[c];
    if (threadIdx.x == 0) abort_flag = a.meta->status != 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    if (abort_flag) return;
    volatile int* abortp = &abort_flag;
    const float NEG_INF = -INFINITY;
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
    float2* ml = reinterpret_cast<float2*>(sm + F8_ML);
    unsigned char* slots = sm + warp * F8_SLOTS * F8_SLOT;
    const int q = lane & 3, g = lane >> 2;

    // ---- copies: lane i < 2 copies tile i of a pair, its block id loaded a
    // pair before
    PairWalk ahead(t_begin, u0);
    int32_t blk = 0, n_ahead = 0, head_ahead = 0, issued = 0;
    auto look = [&]() {
        n_ahead = ahead.more(pl, t_end, a.bpb, warp) ? min(2, ahead.cend - ahead.t) : 0;
        if (lane < n_ahead) blk = a.table[ahead.row + ahead.t + lane];
        head_ahead = ahead.head;
    };
    auto issue = [&]() {
        if (!n_ahead) return;
        const int slot = issued & 1;
        if (lane == 0) mbar_expect_tx(bars + 8 * slot, (uint32_t)(n_ahead * F8_TILE));
        __syncwarp();
        if (lane < n_ahead) {
            if ((uint32_t)blk >= (uint32_t)a.n_blocks) {   // broken table: poison, read a valid block
                atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                blk = 0;
            }
            const int64_t off = ((int64_t)blk * a.n_kv + head_ahead) * kFp8TileBytes;
            const uint32_t dst = smem_u32(slots) + slot * F8_SLOT + lane * F8_TILE;
            bulk_load(dst, reinterpret_cast<const char*>(a.pool_k) + off, kFp8TileBytes, bars + 8 * slot);
            bulk_load(dst + kFp8TileBytes, reinterpret_cast<const char*>(a.pool_v) + off, kFp8TileBytes, bars + 8 * slot);
        }
        ++issued;
        ahead.t += ahead.step;
        look();
    };
    static_assert(F8_SLOTS == 2, "slots alternate");
    look();
    for (int i = 0; i < F8_SLOTS; ++i) issue();

    int32_t done = 0;           // pairs this warp has read
    bool ok = true;
    int32_t t = t_begin, u = u0;
    while (t < t_end) {
        const AttnUnit& U = pl.units[u];            // read again at the chunk's end: not held over the loop
        const int32_t uend = U.tile_off + U.n_blk;
        if (t >= uend) { ++u; continue; }
        const int32_t cend = min(t_end, uend);
        const int32_t pos_of = (U.blk_start - U.tile_off) * BS;   // position of tile st: pos_of + 16 st
        const int P = F8_WARPS / U.rt;              // warps per row tile
        const int r = warp / P, part = warp % P;
        const int row0 = r * 16 + g, row1 = row0 + 8;
        const bool idle = r * 16 >= U.n_rows;       // a row tile past the unit's rows
        uint32_t qa[8][4];
        int32_t lim0 = 0, lim1 = 0;
        uint64_t mask0 = 0, mask1 = 0;
        float f0, f1;
        {
            const bool v0 = row0 < U.n_rows, v1 = row1 < U.n_rows;
            const AttnRow R0 = v0 ? unit_row(pl, U, row0) : AttnRow{0, 0};
            const AttnRow R1 = v1 ? unit_row(pl, U, row1) : AttnRow{0, 0};
            // rows past the unit's (queries of zero, results unused) mask nothing
            lim0 = v0 ? R0.limit : INT_MAX;
            lim1 = v1 ? R1.limit : INT_MAX;
            if (DRAFT) {
                mask0 = v0 ? draft_mask(pl, U, row0) : 0;
                mask1 = v1 ? draft_mask(pl, U, row1) : 0;
            }
            uint32_t w[16];
            f0 = load_q(Q + (int64_t)R0.q_row * D, v0, q, a.scale_log2, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                qa[k][0] = w[2 * k];
                qa[k][2] = w[2 * k + 1];
            }
            f1 = load_q(Q + (int64_t)R1.q_row * D, v1, q, a.scale_log2, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                qa[k][1] = w[2 * k];
                qa[k][3] = w[2 * k + 1];
            }
        }
        float o[16][4];   // chunk c of 16 columns: o[2 c] the even ones, o[2 c + 1] the odd ones
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m0 = NEG_INF, m1 = NEG_INF, w0 = NEG_INF, w1 = NEG_INF, l0 = 0.f, l1 = 0.f;
        int slot = 0;     // of the chunk's last pair, once the loop is through

        for (int32_t st = idle ? cend : t + 2 * part; st < cend; st += 2 * P) {
            slot = done & 1;
            if (ok) ok = mbar_wait(bars + 8 * slot, (uint32_t)(done >> 1) & 1u, abortp);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0 && !*abortp) {
                    *abortp = 1;
                    atomicCAS(&a.meta->status, 0, DENDRITE_ETIMEOUT);
                }
                break;
            }
            ++done;
            {
                const unsigned char* kt = slots + slot * F8_SLOT;
                const bool two = st + 1 < cend;   // else the second tile is not there
                // S = Q C^T: token group h (8 tokens) of the pair, lane's token 8 h + g
                float s[4][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
                // the four groups' chains step by step beside one another: a
                // product waits 24 cycles for the one before it in its chain
                auto scores = [&](int h0) {
                    uint4 v[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const unsigned char* row = kt + (h0 >> 1) * F8_TILE + (8 * h + g) * kFp8Dim;
                        v[h][0] = *reinterpret_cast<const uint4*>(row + (((2 * q) ^ g) << 4));
                        v[h][1] = *reinterpret_cast<const uint4*>(row + (((2 * q + 1) ^ g) << 4));
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4& x = v[h][k >> 2];
                            const uint32_t w = (k & 3) == 0 ? x.x : (k & 3) == 1 ? x.y : (k & 3) == 2 ? x.z : x.w;
                            uint32_t b0, b1;
                            unpack4(w, b0, b1);
                            mma_f16(s[h0 + h], qa[k], b0, b1);
                        }
                    }
                };
                scores(0);
                if (two) scores(2);
                // scale by the tokens' and rows' powers of two; the weights'
                // logarithms are the scores plus the tokens' exponents vl
                uint32_t vb[4] = {0u, 0u, 0u, 0u};   // exponent bytes of the lane's tokens of group h, as they are
                auto vl = [&](int h, int e) {   // byte - 127, by way of 2^23 + byte
                    return __uint_as_float(0x4b000000u | ((vb[h] >> (8 * e)) & 255u)) - 8388735.f;
                };
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const unsigned char* ex = kt + (h >> 1 && two ? F8_TILE : 0) + BS * kFp8Dim + 8 * (h & 1) + 2 * q;
                    const uint32_t ke = *reinterpret_cast<const uint16_t*>(ex);
                    vb[h] = *reinterpret_cast<const uint16_t*>(ex + kFp8TileBytes);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float kf = __uint_as_float(((ke >> (8 * e)) & 255u) << 23);
                        // (one after the other: the two together may pass fp32's range
                        // where the score, of rows that hardly meet, does not)
                        s[h][e] = s[h][e] * kf * f0;
                        s[h][2 + e] = s[h][2 + e] * kf * f1;
                    }
                }
                // mask: only where some row does not see the whole pair
                const int32_t pos0 = pos_of + st * BS;
                if (!two || __any_sync(0xffffffffu, pos0 + 2 * BS > min(lim0, lim1))) {
                    const uint32_t have = two ? 0xffffffffu : 0xffffu;
                    uint32_t see0, see1;
                    if (DRAFT) {
                        see0 = (uint32_t)draft_visible(mask0, lim0 - pos0) & have;
                        see1 = (uint32_t)draft_visible(mask1, lim1 - pos0) & have;
                    } else {
                        see0 = lim0 - pos0 >= 32 ? have : lim0 > pos0 ? have & ((1u << (lim0 - pos0)) - 1u) : 0u;
                        see1 = lim1 - pos0 >= 32 ? have : lim1 > pos0 ? have & ((1u << (lim1 - pos0)) - 1u) : 0u;
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int bit = 8 * h + 2 * q + e;
                            s[h][e] = (see0 >> bit) & 1u ? s[h][e] : NEG_INF;
                            s[h][2 + e] = (see1 >> bit) & 1u ? s[h][2 + e] : NEG_INF;
                        }
                    }
                    // A V row of NaN that no row sees (left behind a branch's
                    // end by a roll-back, or by the block's last owner) would
                    // spread through its weight of zero: it becomes zero here.
                    bool nan_row = false;
#pragma unroll
                    for (int h = 0; h < 4; ++h) nan_row |= (vb[h] & 255u) == 255u || vb[h] >> 8 == 255u;
                    if (__any_sync(0xffffffffu, nan_row)) {
                        const uint32_t seen = __reduce_or_sync(0xffffffffu, (row0 < U.n_rows ? see0 : 0u) |
                                                                                (row1 < U.n_rows ? see1 : 0u));
                        for (int tk = 0; tk < (two ? 32 : 16); ++tk) {
                            if ((seen >> tk) & 1u) continue;
                            unsigned char* row = slots + slot * F8_SLOT + (tk >> 4) * F8_TILE + kFp8TileBytes +
                                                 (tk & 15) * kFp8Dim;
                            reinterpret_cast<uint32_t*>(row)[lane] = 0u;
                        }
                        fence_async_smem();   // before the slot's next copy
                        __syncwarp();
                    }
                }
                float mx0 = NEG_INF, mx1 = NEG_INF, wx0 = NEG_INF, wx1 = NEG_INF;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx0 = fmaxf(mx0, s[h][e]);
                        mx1 = fmaxf(mx1, s[h][2 + e]);
                        wx0 = fmaxf(wx0, s[h][e] + vl(h, e));
                        wx1 = fmaxf(wx1, s[h][2 + e] + vl(h, e));
                    }
                }
#pragma unroll
                for (int x = 1; x <= 2; x <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
                    wx0 = fmaxf(wx0, __shfl_xor_sync(0xffffffffu, wx0, x));
                    wx1 = fmaxf(wx1, __shfl_xor_sync(0xffffffffu, wx1, x));
                }
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                const float x0 = fmaxf(w0, weight_ref(wx0)), x1 = fmaxf(w1, weight_ref(wx1));
                const float nu0 = n0 == NEG_INF ? 0.f : n0, nu1 = n1 == NEG_INF ? 0.f : n1;
                const float xu0 = x0 == NEG_INF ? 0.f : x0, xu1 = x1 == NEG_INF ? 0.f : x1;
                l0 *= ex2(m0 - nu0);
                l1 *= ex2(m1 - nu1);
                const float al0 = ex2(w0 - xu0), al1 = ex2(w1 - xu1);
                m0 = n0;
                m1 = n1;
                w0 = x0;
                w1 = x1;
                uint32_t pa[2][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    l0 += ex2(s[h][0] - nu0) + ex2(s[h][1] - nu0);
                    l1 += ex2(s[h][2] - nu1) + ex2(s[h][3] - nu1);
                    // weights in fp16: rounded by 2^-11, or 2^-40 of the row's largest weight
                    pa[h >> 1][2 * (h & 1)] = pack_f16(ex2(s[h][0] + vl(h, 0) - xu0), ex2(s[h][1] + vl(h, 1) - xu0));
                    pa[h >> 1][2 * (h & 1) + 1] = pack_f16(ex2(s[h][2] + vl(h, 0) - xu1), ex2(s[h][3] + vl(h, 1) - xu1));
                }
                if (!__all_sync(0xffffffffu, al0 == 1.f && al1 == 1.f)) {
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        o[n][0] *= al0;
                        o[n][1] *= al0;
                        o[n][2] *= al1;
                        o[n][3] *= al1;
                    }
                }
                // O += W V
                const int mi = lane >> 3, tok = (mi & 1) * 8 + (lane & 7);
                const uint32_t va = smem_u32(kt + kFp8TileBytes) + tok * kFp8Dim;
                // (a loop over the two tiles: unrolled, the step outgrows the instruction cache)
#pragma unroll 1
                for (int half = 0; half <= (two ? 1 : 0); ++half) {
                    const uint32_t tile = va + half * F8_TILE;
                    const uint32_t p[4] = {half ? pa[1][0] : pa[0][0], half ? pa[1][1] : pa[0][1], half ? pa[1][2] : pa[0][2],
                                           half ? pa[1][3] : pa[0][3]};
#pragma unroll
                    for (int cc = 0; cc < 8; cc += 2) {
                        uint32_t v[4];
                        ldsm_x4_t(tile + (((cc + (mi >> 1)) ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {   // chunk cc + k: tokens 0-7 in v[2 k], 8-15 in v[2 k + 1]
                            uint32_t e0, d0, e1, d1;
                            unpack4(__byte_perm(v[2 * k], 0u, 0x3120), e0, d0);
                            unpack4(__byte_perm(v[2 * k + 1], 0u, 0x3120), e1, d1);
                            mma_f16(o[2 * (cc + k)], p, e0, e1);
                            mma_f16(o[2 * (cc + k) + 1], p, d0, d1);
                        }
                    }
                }
            }
            __syncwarp();
            if (st + 2 * P < cend) issue();   // (the chunk's last slot is still needed)
        }

        {
            // ---------------------------------------- end of this unit's chunk
            if (cend == t_end) pdl_trigger();   // the CTA's last
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            // acc from units of 2^w to units of 2^m (in two steps: w - m may be 15 below
            // the least exponent, with values of that size)
            const float back0 = w0 == NEG_INF ? 0.f : ex2(w0 - m0 + kWeightTop);
            const float back1 = w1 == NEG_INF ? 0.f : ex2(w1 - m1 + kWeightTop);
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                o[n][0] *= 0x1p-15f;
                o[n][1] *= 0x1p-15f;
                o[n][2] *= 0x1p-15f;
                o[n][3] *= 0x1p-15f;
            }
            const int32_t prow0 = U.prow_base + (c - U.cfirst) * U.n_rows;
            if (P == 1) {
                if (ok && !idle) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int row = hh ? row1 : row0;
                        const float back = hh ? back1 : back0;
                        if (row < U.n_rows) {
                            float* dst = a.part_acc + (int64_t)(prow0 + row) * D + 4 * q;
#pragma unroll
                            for (int n = 0; n < 8; ++n)
                                *reinterpret_cast<float4*>(dst + 16 * n) =
                                    make_float4(o[2 * n][2 * hh] * back, o[2 * n + 1][2 * hh] * back,
                                                o[2 * n][2 * hh + 1] * back, o[2 * n + 1][2 * hh + 1] * back);
                            if (q == 0) a.part_ml[prow0 + row] = hh ? make_float2(m1, l1) : make_float2(m0, l0);
                        }
                    }
                }
            } else {
                // the P warps of each row tile combine through the slots they
                // read last (16-byte words XOR-ed with the row, so that a
                // quarter warp's stores fall in distinct banks); a warp that
                // had no pair of this chunk takes no part, its slots hold
                // copies for later ones
                const bool took = t + 2 * part < cend;
                if (took) {
                    float* ob = reinterpret_cast<float*>(slots + slot * F8_SLOT);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int row = g + 8 * hh;
                        const float back = hh ? back1 : back0;
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            *reinterpret_cast<float4*>(ob + row * D + (((4 * n + q) ^ (row & 7)) << 2)) =
                                make_float4(o[2 * n][2 * hh] * back, o[2 * n + 1][2 * hh] * back,
                                            o[2 * n][2 * hh + 1] * back, o[2 * n + 1][2 * hh + 1] * back);
                    }
                }
                if (q == 0) {
                    ml[warp * 16 + g] = make_float2(m0, l0);
                    ml[warp * 16 + g + 8] = make_float2(m1, l1);
                }
                if (lane == 0) last_slot[warp] = slot;
                __syncthreads();
                if (!*abortp) {
                    const int took_of = (cend - t + 1) >> 1;   // warps of a row tile that had a pair: at most P
                    for (int idx = threadIdx.x; idx < U.n_rows * (D / 4); idx += F8_THREADS) {
                        const int grow = idx / (D / 4), d4 = idx % (D / 4);
                        const int row = grow & 15, wf = (grow >> 4) * P, np = min(P, took_of);
                        float M = NEG_INF;
                        for (int p2 = 0; p2 < np; ++p2) M = fmaxf(M, ml[(wf + p2) * 16 + row].x);
                        const float Mu = M == NEG_INF ? 0.f : M;
                        float L = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int p2 = 0; p2 < np; ++p2) {
                            const float2 s2 = ml[(wf + p2) * 16 + row];
                            const float wgt = exp2f(s2.x - Mu);
                            L += s2.y * wgt;
                            const float* ob = reinterpret_cast<const float*>(
                                sm + ((wf + p2) * F8_SLOTS + last_slot[wf + p2]) * F8_SLOT);
                            const float4 v = *reinterpret_cast<const float4*>(ob + row * D + ((d4 ^ (row & 7)) << 2));
                            acc.x += v.x * wgt;
                            acc.y += v.y * wgt;
                            acc.z += v.z * wgt;
                            acc.w += v.w * wgt;
                        }
                        *reinterpret_cast<float4*>(a.part_acc + (int64_t)(prow0 + grow) * D + 4 * d4) = acc;
                        if (d4 == 0) a.part_ml[prow0 + grow] = make_float2(M, L);
                    }
                }
                fence_async_smem();
                __syncthreads();   // the slots are free again before the next copy lands in them
            }
            if (ok && !idle && t + 2 * part < cend) issue();   // the chunk's last slot
        }
        t = cend;
        ++u;
    }
    // after a timeout, wait (bounded) for this warp's copies still in flight
    if (lane == 0 && *abortp) {
        for (int i = max(0, issued - F8_SLOTS); i < issued; ++i) {
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(bars + 8 * (i & 1), (uint32_t)(i >> 1) & 1u) && globaltimer() - t0 < WAIT_LIMIT_NS) {
            }
        }
    }
}

}  // namespace

namespace dendrite {

int attn_fp8_setup(int* ctas_per_sm) {
    if (cudaFuncSetAttribute(k_attn_partial_fp8<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F8_SMEM) !=
            cudaSuccess ||
        cudaFuncSetAttribute(k_attn_partial_fp8<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F8_SMEM) !=
            cudaSuccess)
        return cuda_err(cudaGetLastError());
    int occ = 0, occ_draft = 0;
    DENDRITE_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k_attn_partial_fp8<false>, F8_THREADS, F8_SMEM));
    DENDRITE_CUDA(
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ_draft, k_attn_partial_fp8<true>, F8_THREADS, F8_SMEM));
    *ctas_per_sm = occ < occ_draft ? occ : occ_draft;
    if (*ctas_per_sm < 1) *ctas_per_sm = 1;
    return DENDRITE_OK;
}

int launch_attn_fp8(const AttnArgs& a, bool after_event, cudaStream_t s) {
    if (a.plan.n_ctas <= 0) return DENDRITE_OK;
    if (after_event) {
        if (a.plan.masks) k_attn_partial_fp8<true><<<a.plan.n_ctas, F8_THREADS, F8_SMEM, s>>>(a);
        else k_attn_partial_fp8<false><<<a.plan.n_ctas, F8_THREADS, F8_SMEM, s>>>(a);
        DENDRITE_CUDA(cudaGetLastError());
    } else if (a.plan.masks)
        DENDRITE_CUDA(launch_pdl(k_attn_partial_fp8<true>, dim3(a.plan.n_ctas), dim3(F8_THREADS), F8_SMEM, s, a));
    else
        DENDRITE_CUDA(launch_pdl(k_attn_partial_fp8<false>, dim3(a.plan.n_ctas), dim3(F8_THREADS), F8_SMEM, s, a));
    return DENDRITE_OK;
}

}  // namespace dendrite
