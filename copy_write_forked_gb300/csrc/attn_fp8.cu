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
//   The weights w_rt = p_rt 2^f_t get a running reference of their own, as
//   log2 w is score + f_t: w is stored as 2^(score + f_t - m2) in [0, 1] in
//   fp16, whatever the spread of the tokens' scales, while the row sum l takes
//   p = 2^(score - m) in fp32.  acc is in units of 2^m2 and is brought to
//   2^m when the chunk's partial row is written.
//
//   K needs no ldmatrix: the mma's k order is free as long as Q and K agree,
//   so a lane takes 32 consecutive codes of its token (two 16-byte loads).
//   V goes through ldmatrix.trans on pairs of codes; one byte permutation
//   parts the even dimensions from the odd ones, and each of the two is an
//   operand (their accumulators interleave to four consecutive columns).
//
// One producer warp streams tiles with cp.async.bulk into an mbarrier ring
// (4 tiles a stage); four consumer warps share a unit: each row tile of 16
// rows belongs to 4, 2 or 1 warps, which then take the stage's tiles in turn
// and combine their states at the chunk's end.
//
// Every mbarrier wait is bounded, as in the bf16 kernel.
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "attn_fp8.h"
#include "rows.h"

using namespace dendrite;

namespace {

constexpr int F8_STAGES = 4;
constexpr int F8_TILES = 4;                              // tiles per stage
constexpr int F8_SLOT = 2 * kFp8TileBytes;               // K then V of one tile
constexpr int F8_STAGE = F8_TILES * F8_SLOT;
constexpr int F8_WARPS = 4;
constexpr int F8_THREADS = (F8_WARPS + 1) * 32;
constexpr int F8_COMB = F8_STAGES * F8_STAGE;            // combine buffer: 4 warps x 16 rows x 128 fp32
constexpr int F8_ML = F8_COMB + F8_WARPS * 16 * D * 4;   // per warp and row (m, l)
constexpr int F8_BAR = F8_ML + F8_WARPS * 16 * 8;
constexpr size_t F8_SMEM = F8_BAR + 2 * F8_STAGES * 8;
static_assert(F8_STAGE % 16 == 0 && F8_BAR % 8 == 0, "alignment");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Two e4m3 codes to fp16, exactly.
__device__ __forceinline__ uint32_t unpack2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = unpack2((uint16_t)w);
    hi = unpack2((uint16_t)(w >> 16));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^(byte - 127); byte 0 is the denormal 2^-127.
__device__ __forceinline__ float exp_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x400000u); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

template <bool DRAFT>
__global__ void __launch_bounds__(F8_THREADS, 2) k_attn_partial_fp8(const AttnArgs a) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ int abort_flag;
    const uint32_t base = smem_u32(sm);
    const uint32_t bar_full = base + F8_BAR, bar_empty = bar_full + F8_STAGES * 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < F8_STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, F8_WARPS);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    pdl_trigger();
    const AttnPlanDev& pl = a.plan;
    const int c = blockIdx.x;
    const int32_t t_begin = pl.cta_begin[c], t_end = pl.cta_begin[c + 1];
    const int32_t u0 = pl.cta_unit[c];
    if (threadIdx.x == 0) {
        abort_flag = a.meta->status != 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (abort_flag) return;
    volatile int* abortp = &abort_flag;

    if (warp == F8_WARPS) {
        // ------------------------------------------------------ producer
        const char* kp = reinterpret_cast<const char*>(a.pool_k);
        const char* vp = reinterpret_cast<const char*>(a.pool_v);
        uint32_t issued = 0, parity_bits = 0;
        int32_t stage = 0, t = t_begin, u = u0;
        while (t < t_end) {
            const AttnUnit U = pl.units[u];
            const int32_t uend = U.tile_off + U.n_blk;
            if (t >= uend) { ++u; continue; }
            const int32_t cend = min(t_end, uend);
            const int32_t* trow = a.table + (int64_t)U.table_row * a.bpb + U.blk_start - U.tile_off;
            int32_t next = lane < F8_TILES && t + lane < cend ? trow[t + lane] : 0;
            for (int32_t st = t; st < cend; st += F8_TILES, ++stage) {
                const int slot = stage % F8_STAGES;
                const uint32_t ph = (uint32_t)(stage / F8_STAGES) & 1u;
                const int ntiles = min(F8_TILES, cend - st);
                int32_t blk = next;
                if (lane < F8_TILES && st + F8_TILES + lane < cend) next = trow[st + F8_TILES + lane];
                bool ok = true;
                if (lane == 0 && !*abortp) {
                    ok = mbar_wait(bar_empty + 8 * slot, ph ^ 1u, abortp);
                    if (!ok) {
                        *abortp = 1;
                        atomicCAS(&a.meta->status, 0, DENDRITE_ETIMEOUT);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) && !*abortp;
                if (!__all_sync(0xffffffffu, ok)) continue;
                if (lane == 0) mbar_expect_tx(bar_full + 8 * slot, (uint32_t)(ntiles * F8_SLOT));
                __syncwarp();
                if (lane < ntiles) {
                    if ((uint32_t)blk >= (uint32_t)a.n_blocks) {   // broken table: poison, read a valid block
                        atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                        blk = 0;
                    }
                    const int64_t off = ((int64_t)blk * a.n_kv + U.kv_head) * kFp8TileBytes;
                    const uint32_t dst = base + slot * F8_STAGE + lane * F8_SLOT;
                    bulk_load(dst, kp + off, kFp8TileBytes, bar_full + 8 * slot);
                    bulk_load(dst + kFp8TileBytes, vp + off, kFp8TileBytes, bar_full + 8 * slot);
                }
                issued |= 1u << slot;
                parity_bits = (parity_bits & ~(1u << slot)) | (ph << slot);
            }
            t = cend;
            ++u;
        }
        if (lane == 0 && *abortp) {   // copies still in flight land before the CTA exits
            for (int s = 0; s < F8_STAGES; ++s) {
                if (!(issued >> s & 1u)) continue;
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(bar_full + 8 * s, parity_bits >> s & 1u) && globaltimer() - t0 < WAIT_LIMIT_NS) {
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------- consumers
    const float NEG_INF = -INFINITY;
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
    float2* ml = reinterpret_cast<float2*>(sm + F8_ML);
    const int q = lane & 3, g = lane >> 2;
    int32_t stage = 0, t = t_begin, u = u0;
    while (t < t_end) {
        const AttnUnit U = pl.units[u];
        const int32_t uend = U.tile_off + U.n_blk;
        if (t >= uend) { ++u; continue; }
        const int32_t cend = min(t_end, uend);
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
            lim0 = R0.limit;
            lim1 = R1.limit;
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

        for (int32_t st = t; st < cend; st += F8_TILES, ++stage) {
            const int slot = stage % F8_STAGES;
            const uint32_t ph = (uint32_t)(stage / F8_STAGES) & 1u;
            const int ntiles = min(F8_TILES, cend - st);
            const bool last = st + F8_TILES >= cend;
            bool ok = !*abortp;
            if (ok) {
                ok = mbar_wait(bar_full + 8 * slot, ph, abortp);
                if (!ok) {
                    *abortp = 1;
                    atomicCAS(&a.meta->status, 0, DENDRITE_ETIMEOUT);
                }
            }
            ok = __all_sync(0xffffffffu, ok) && !*abortp;
            ok = __all_sync(0xffffffffu, ok);
            for (int ti = part; ok && !idle && ti < ntiles; ti += P) {
                const unsigned char* kt = sm + slot * F8_STAGE + ti * F8_SLOT;
                const unsigned char* vt = kt + kFp8TileBytes;
                // S = Q C^T: token group h (8 tokens), lane's token 8 h + g
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned char* row = kt + (8 * h + g) * kFp8Dim;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 v = *reinterpret_cast<const uint4*>(row + (((2 * q + k) ^ g) << 4));
                        uint32_t b0, b1;
                        unpack4(v.x, b0, b1);
                        mma_f16(s[h], qa[4 * k], b0, b1);
                        unpack4(v.y, b0, b1);
                        mma_f16(s[h], qa[4 * k + 1], b0, b1);
                        unpack4(v.z, b0, b1);
                        mma_f16(s[h], qa[4 * k + 2], b0, b1);
                        unpack4(v.w, b0, b1);
                        mma_f16(s[h], qa[4 * k + 3], b0, b1);
                    }
                }
                // scale by the tokens' and rows' powers of two, mask; the
                // weights' logarithms beside the scores
                const int32_t tile_pos = (U.blk_start + (st - U.tile_off) + ti) * BS;
                uint32_t see0 = 0, see1 = 0;
                if (DRAFT) {
                    see0 = (uint32_t)draft_visible(mask0, lim0 - tile_pos);
                    see1 = (uint32_t)draft_visible(mask1, lim1 - tile_pos);
                }
                float wl[2][4];
                float mx0 = NEG_INF, mx1 = NEG_INF, wx0 = NEG_INF, wx1 = NEG_INF;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t ke = *reinterpret_cast<const uint16_t*>(kt + BS * kFp8Dim + 8 * h + 2 * q);
                    const uint32_t ve = *reinterpret_cast<const uint16_t*>(vt + BS * kFp8Dim + 8 * h + 2 * q);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float kf = exp_of((ke >> (8 * e)) & 255u);
                        const float vl = (float)((ve >> (8 * e)) & 255u) - 127.f;
                        const int bit = 8 * h + 2 * q + e;
                        const bool on0 = DRAFT ? (see0 >> bit) & 1u : tile_pos + bit < lim0;
                        const bool on1 = DRAFT ? (see1 >> bit) & 1u : tile_pos + bit < lim1;
                        // factors past fp32 are cut, so that a zero product stays zero
                        s[h][e] = on0 ? s[h][e] * fminf(kf * f0, 3.4e38f) : NEG_INF;
                        s[h][2 + e] = on1 ? s[h][2 + e] * fminf(kf * f1, 3.4e38f) : NEG_INF;
                        wl[h][e] = s[h][e] + vl;
                        wl[h][2 + e] = s[h][2 + e] + vl;
                        mx0 = fmaxf(mx0, s[h][e]);
                        mx1 = fmaxf(mx1, s[h][2 + e]);
                        wx0 = fmaxf(wx0, wl[h][e]);
                        wx1 = fmaxf(wx1, wl[h][2 + e]);
                    }
                }
#pragma unroll
                for (int x = 1; x <= 2; x <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
                    wx0 = fmaxf(wx0, __shfl_xor_sync(0xffffffffu, wx0, x));
                    wx1 = fmaxf(wx1, __shfl_xor_sync(0xffffffffu, wx1, x));
                }
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1), x0 = fmaxf(w0, wx0), x1 = fmaxf(w1, wx1);
                const float nu0 = n0 == NEG_INF ? 0.f : n0, nu1 = n1 == NEG_INF ? 0.f : n1;
                const float xu0 = x0 == NEG_INF ? 0.f : x0, xu1 = x1 == NEG_INF ? 0.f : x1;
                l0 *= ex2(m0 - nu0);
                l1 *= ex2(m1 - nu1);
                const float al0 = ex2(w0 - xu0), al1 = ex2(w1 - xu1);
                m0 = n0;
                m1 = n1;
                w0 = x0;
                w1 = x1;
                uint32_t pa[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    l0 += ex2(s[h][0] - nu0) + ex2(s[h][1] - nu0);
                    l1 += ex2(s[h][2] - nu1) + ex2(s[h][3] - nu1);
                    // weights in fp16: rounded by 2^-12, or 2^-25 of the row's largest weight
                    pa[2 * h] = pack_f16(ex2(wl[h][0] - xu0), ex2(wl[h][1] - xu0));
                    pa[2 * h + 1] = pack_f16(ex2(wl[h][2] - xu1), ex2(wl[h][3] - xu1));
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
                const uint32_t va = smem_u32(vt);
                const int mi = lane >> 3, tok = (mi & 1) * 8 + (lane & 7);
#pragma unroll
                for (int cc = 0; cc < 8; cc += 2) {
                    uint32_t v[4];
                    ldsm_x4_t(va + tok * kFp8Dim + (((cc + (mi >> 1)) ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {   // chunk cc + k: tokens 0-7 in v[2 k], 8-15 in v[2 k + 1]
                        uint32_t e0, d0, e1, d1;
                        unpack4(__byte_perm(v[2 * k], 0u, 0x3120), e0, d0);
                        unpack4(__byte_perm(v[2 * k + 1], 0u, 0x3120), e1, d1);
                        mma_f16(o[2 * (cc + k)], pa, e0, e1);
                        mma_f16(o[2 * (cc + k) + 1], pa, d0, d1);
                    }
                }
            }
            // the stage's tiles are read: back to the producer
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * slot);
            if (!last) continue;

            // ---------------------------------------- end of this unit's chunk
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            // acc from units of 2^w to units of 2^m
            const float back0 = w0 == NEG_INF ? 0.f : ex2(w0 - m0), back1 = w1 == NEG_INF ? 0.f : ex2(w1 - m1);
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
                continue;
            }
            // the P warps of each row tile combine through shared memory
            // (16-byte words XOR-ed with the row, so that a quarter warp's
            // stores fall in distinct banks)
            {
                float* ob = reinterpret_cast<float*>(sm + F8_COMB) + warp * 16 * D;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int row = g + 8 * hh;
                    const float back = hh ? back1 : back0;
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        *reinterpret_cast<float4*>(ob + row * D + (((4 * n + q) ^ (row & 7)) << 2)) =
                            make_float4(o[2 * n][2 * hh] * back, o[2 * n + 1][2 * hh] * back,
                                        o[2 * n][2 * hh + 1] * back, o[2 * n + 1][2 * hh + 1] * back);
                    if (q == 0) ml[warp * 16 + row] = hh ? make_float2(m1, l1) : make_float2(m0, l0);
                }
            }
            consumer_sync();
            if (ok) {
                const float* obase = reinterpret_cast<const float*>(sm + F8_COMB);
                for (int idx = threadIdx.x; idx < U.n_rows * (D / 4); idx += F8_WARPS * 32) {
                    const int grow = idx / (D / 4), d4 = idx % (D / 4);
                    const int row = grow & 15, wf = (grow >> 4) * P;
                    float M = NEG_INF;
                    for (int p2 = 0; p2 < P; ++p2) M = fmaxf(M, ml[(wf + p2) * 16 + row].x);
                    const float Mu = M == NEG_INF ? 0.f : M;
                    float L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int p2 = 0; p2 < P; ++p2) {
                        const float2 s2 = ml[(wf + p2) * 16 + row];
                        const float wgt = exp2f(s2.x - Mu);
                        L += s2.y * wgt;
                        const float4 v = *reinterpret_cast<const float4*>(obase + ((wf + p2) * 16 + row) * D +
                                                                          ((d4 ^ (row & 7)) << 2));
                        acc.x += v.x * wgt;
                        acc.y += v.y * wgt;
                        acc.z += v.z * wgt;
                        acc.w += v.w * wgt;
                    }
                    *reinterpret_cast<float4*>(a.part_acc + (int64_t)(prow0 + grow) * D + 4 * d4) = acc;
                    if (d4 == 0) a.part_ml[prow0 + grow] = make_float2(M, L);
                }
            }
            consumer_sync();   // the buffer is free again
        }
        t = cend;
        ++u;
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

int launch_attn_fp8(const AttnArgs& a, cudaStream_t s) {
    if (a.plan.n_ctas <= 0) return DENDRITE_OK;
    if (a.plan.masks)
        DENDRITE_CUDA(launch_pdl(k_attn_partial_fp8<true>, dim3(a.plan.n_ctas), dim3(F8_THREADS), F8_SMEM, s, a));
    else
        DENDRITE_CUDA(launch_pdl(k_attn_partial_fp8<false>, dim3(a.plan.n_ctas), dim3(F8_THREADS), F8_SMEM, s, a));
    return DENDRITE_OK;
}

}  // namespace dendrite
