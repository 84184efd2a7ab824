// Cross attention over fp32 blocks, on the CUDA cores.
//
// The row-by-row kernel of fp32 pools reads a key for every row that meets it
// and adds its products up over a warp's lanes, which takes ten times as long as
// the products.  Here a CTA of 128 threads holds a unit's rows of Q and 32 tokens at
// a time in shared memory and multiplies in tiles of registers, with the online softmax
// between the two products (a row's tokens over 8 lanes).  Products and sums are fp32
// throughout (no TF32).  For 16 R rows, R = 2, 4, 8:
//   S = Q K^T    16 R x 32, a thread R rows x 4 tokens: R + 4 16-byte loads for 16 R products
//   O += P V     16 R x d,  a thread the same R rows x d/8 columns: R/4 + d/32 for R d/8
// and for 4 R rows, R = 1, 2, 4, the tokens shared out to the warps (k_attn_cross_f32_few).
//
// Thread (rg, tg) = (tid / 8, tid % 8) has rows rg + 16 i and tokens tg + 8 j.  The 16-byte
// words of a row of Q or K are permuted by the row's last three bits, and P's rows are
// 4 floats longer than they need be, so that no load or store meets a bank twice.  K of
// the next 32 tokens is copied while O is summed, V while S is; a second buffer would
// cost a resident CTA.  Units, CTA split and partial rows are the plan's, as for the
// other kernels; a unit that one CTA runs whole writes its rows out itself.
//
// Many rows are bound by instructions (products 58 % of the FMA pipe's rate, all of them 69 % of
// the issue slots, shared memory 46 %): 200 queries, 32 heads of 8 kv heads, over 4,000
// tokens 347 us, 38 TFLOP/s; the row-by-row kernel 3,513, 64 rows a unit 529, plain torch 620.
// 448 x 2 over 1,500 of 16 heads, d = 64: 171 (2,764; plain 428).  5 over 4,636 of 32 heads
// of 8, 3 sequences: 41 (325).  Two products an instruction (fma.rn.f32x2) gave 340 and, by
// registers, 182.
// Few rows are bound by HBM: one query of 8 heads, a kv head each, over 32 x 1,500 tokens 79 us for
// 393 MB (5.0 TB/s; 540 row by row, 202 with the tokens not shared out, 123 in units of 16 rows),
// over one sequence of 60,000 with 32 heads 103 (4.8 TB/s; 669, 282, 176).
#include "attn_f32.h"

using namespace dendrite;

namespace {

constexpr int TT = 32, NT = 128;   // tokens a step, threads

template <int DIM, int R>
struct F32Smem {
    static constexpr int TR = 16 * R, PS = TR + 4;   // rows; floats of a token's row of P
    static constexpr int Q = 0, K = Q + TR * DIM, V = K + TT * DIM, P = V + TT * DIM, LIM = P + TT * PS;
    static constexpr int BYTES = (LIM + TR) * 4;
    static constexpr int CTAS = BYTES <= 76 * 1024 ? 3 : BYTES <= 113 * 1024 ? 2 : 1;   // that fit an SM
};

__device__ __forceinline__ void copy16(float* to, const float* from, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 fma4(float w, float4 x, float4 a) {
    return make_float4(fmaf(w, x.x, a.x), fmaf(w, x.y, a.y), fmaf(w, x.z, a.z), fmaf(w, x.w, a.w));
}

// n <= 4: one load or store; 8: two
template <int N>
__device__ __forceinline__ void load_row(float (&to)[N], const float* from) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = lds4(from + i);
            to[i] = v.x; to[i + 1] = v.y; to[i + 2] = v.z; to[i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(from);
        to[0] = v.x; to[1] = v.y;
    } else {
        to[0] = *from;
    }
}

template <int N>
__device__ __forceinline__ void store_row(float* to, const float (&x)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(to) = make_float2(x[0], x[1]);
    } else {
        *to = x[0];
    }
}

template <int DIM, int R>
__global__ void __launch_bounds__(NT, F32Smem<DIM, R>::CTAS) k_attn_cross_f32(const AttnArgs a) {
    using S = F32Smem<DIM, R>;
    constexpr int TR = S::TR, C = DIM / 32;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, rg = tid >> 3, tg = tid & 7;
    int32_t* lims = reinterpret_cast<int32_t*>(sm + S::LIM);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    pdl_trigger();
    if (__syncthreads_or(tid == 0 && a.meta->status)) return;
    const AttnPlanDev& pl = a.plan;
    const int c = blockIdx.x;
    int32_t t = pl.cta_begin[c];
    const int32_t t_end = pl.cta_begin[c + 1];
    int32_t u = pl.cta_unit[c];
    const float* Q = static_cast<const float*>(a.Q);
    while (t < t_end) {
        const AttnUnit U = pl.units[u];
        const int32_t uend = U.tile_off + U.n_blk;
        if (t >= uend) { ++u; continue; }
        const int32_t cend = min(t_end, uend);
        const int32_t* trow = a.table + (int64_t)U.table_row * a.bpb + U.blk_start - U.tile_off;
        auto block_of = [&](int32_t tile) {
            int32_t blk = tile < cend ? __ldg(trow + tile) : 0;
            if ((uint32_t)blk >= (uint32_t)a.n_blocks) {
                atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                blk = 0;   // read a valid block; the pool is poisoned anyway
            }
            return ((int64_t)blk * a.n_kv + U.kv_head) * (BS * DIM);
        };
        // copies 32 tokens from tile tt on, swizzled for K; what lies past the chunk, or past every row's end,
        // becomes zero (a weight of zero times what stands there may be NaN)
        int32_t held = 0;   // positions that some row sees
        auto fetch = [&](const float* pool, float* to, int swizzle, int32_t tt, int64_t b0, int64_t b1) {
            const int32_t left = min(held - (U.blk_start + tt - U.tile_off) * BS, (cend - tt) * BS);
#pragma unroll
            for (int e0 = 0; e0 < TT * (DIM / 4); e0 += NT) {
                const int e = e0 + tid, tok = e / (DIM / 4), w = e % (DIM / 4);
                copy16(to + tok * DIM + 4 * (w ^ (tok & swizzle)), pool + (tok < BS ? b0 : b1) + (tok & 15) * DIM + 4 * w,
                       tok < left);
            }
            copies_commit();
        };
        __syncthreads();   // the last unit's shared memory is done with
        int32_t* qrows = reinterpret_cast<int32_t*>(sm + S::P);
        if (tid < TR) {
            const AttnRow row = unit_row(pl, U, min(tid, U.n_rows - 1));
            lims[tid] = tid < U.n_rows ? row.limit : 0;
            qrows[tid] = row.q_row;
        }
        int64_t b0 = block_of(t), b1 = block_of(t + 1);
        __syncthreads();
        int32_t seen_by_all = INT32_MAX;
        for (int r = 0; r < U.n_rows; ++r) {
            held = max(held, lims[r]);
            seen_by_all = min(seen_by_all, lims[r]);
        }
#pragma unroll 4
        for (int e = tid; e < TR * (DIM / 4); e += NT) {
            const int r = e / (DIM / 4), w = e % (DIM / 4);
            copy16(sm + S::Q + r * DIM + 4 * (w ^ (r & 7)), Q + (int64_t)qrows[r] * DIM + 4 * w, r < U.n_rows);
        }
        copies_commit();
        fetch(a.pool_k, sm + S::K, 7, t, b0, b1);
        fetch(a.pool_v, sm + S::V, 0, t, b0, b1);
        float m[R], l[R];
        float4 acc[R][C];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int k = 0; k < C; ++k) acc[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int32_t tt = t; tt < cend; tt += 2) {
            b0 = block_of(tt + 2);
            b1 = block_of(tt + 3);
            copies_wait<1>();
            __syncthreads();   // Q and K are there
            float s[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
            for (int k = 0; k < DIM / 4; ++k) {
                float4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = lds4(sm + S::K + (tg + 8 * j) * DIM + 4 * (k ^ tg));
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float4 q = lds4(sm + S::Q + (rg + 16 * i) * DIM + 4 * (k ^ (rg & 7)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(q.w, x[j].w, fmaf(q.z, x[j].z, fmaf(q.y, x[j].y, fmaf(q.x, x[j].x, s[i][j]))));
                }
            }
            const int32_t pos0 = (U.blk_start + tt - U.tile_off) * BS, n_tok = min(TT, (cend - tt) * BS);
            const bool plain = n_tok == TT && pos0 + TT <= seen_by_all;
            bool moved = false;
            float al[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = tg + 8 * j;
                    s[i][j] *= a.scale_log2;
                    if (!plain && (tok >= n_tok || pos0 + tok >= lims[rg + 16 * i])) s[i][j] = -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
                al[i] = exp2f(m[i] - ref);
                moved |= mn != m[i];
                m[i] = mn;
                l[i] *= al[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2f(s[i][j] - ref);
                    l[i] += s[i][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p[R];
#pragma unroll
                for (int i = 0; i < R; ++i) p[i] = s[i][j];
                store_row(sm + S::P + (tg + 8 * j) * S::PS + R * rg, p);
            }
            copies_wait<0>();
            __syncthreads();   // V and P are there, K is free
            if (tt + 2 < cend) fetch(a.pool_k, sm + S::K, 7, tt + 2, b0, b1);
            else copies_commit();
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int k = 0; k < C; ++k)
                        acc[i][k] = make_float4(acc[i][k].x * al[i], acc[i][k].y * al[i], acc[i][k].z * al[i], acc[i][k].w * al[i]);
            }
            if (plain) {
#pragma unroll 2
                for (int tok = 0; tok < TT; ++tok) {
                    float w[R];
                    load_row(w, sm + S::P + tok * S::PS + R * rg);
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const float4 v = lds4(sm + S::V + tok * DIM + 4 * tg + 32 * k);
#pragma unroll
                        for (int i = 0; i < R; ++i) acc[i][k] = fma4(w[i], v, acc[i][k]);
                    }
                }
            } else {   // a masked token's V may be infinite: it is left out, not weighed by zero
#pragma unroll 1
                for (int tok = 0; tok < n_tok; ++tok) {
                    float w[R];
                    load_row(w, sm + S::P + tok * S::PS + R * rg);
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const float4 v = lds4(sm + S::V + tok * DIM + 4 * tg + 32 * k);
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if (pos0 + tok < lims[rg + 16 * i]) acc[i][k] = fma4(w[i], v, acc[i][k]);
                    }
                }
            }
            __syncthreads();   // V and P are free
            if (tt + 2 < cend) fetch(a.pool_v, sm + S::V, 0, tt + 2, b0, b1);
            else copies_commit();
        }
        copies_wait<0>();
        const bool whole = pl.direct && U.nchunks == 1;
        const int32_t prow0 = U.prow_base + (c - U.cfirst) * U.n_rows;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = rg + 16 * i;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (r >= U.n_rows) continue;
            const float f = whole ? 1.f / l[i] : 1.f;
            float* to = whole ? static_cast<float*>(a.out) + (int64_t)unit_row(pl, U, r).q_row * DIM : a.part_acc + (int64_t)(prow0 + r) * DIM;
#pragma unroll
            for (int k = 0; k < C; ++k)
                *reinterpret_cast<float4*>(to + 4 * tg + 32 * k) =
                    make_float4(acc[i][k].x * f, acc[i][k].y * f, acc[i][k].z * f, acc[i][k].w * f);
            if (!whole && tg == 0) a.part_ml[prow0 + r] = make_float2(m[i], l[i]);
        }
        t = cend;
        ++u;
    }
}

// Units of up to 16 rows, where the tiles above would read each K and V word in every warp.  Here
// the warps share the tokens instead, eight of 32 each, and run on their own (their copies, running maximum
// and sums); a thread has the products of four rows and one token, then of its four rows and d/8 columns.
// The four (m, l, O) are joined at a unit's end in K's and V's place.
template <int DIM, int R>
struct FewSmem {
    static constexpr int TR = 4 * R, PS = R == 1 ? 4 : TR + 4;   // rows; floats of a token's row of P
    static constexpr int Q = 0, K = Q + TR * DIM, V = K + TT * DIM, P = V + TT * DIM, ML = P + TT * PS, LIM = ML + 2 * 64;
    static constexpr int BYTES = (LIM + 32) * 4;
    static constexpr int FIT = 228 * 1024 / (BYTES + 1024), MOST = R == 1 ? 6 : R == 2 ? 5 : DIM <= 64 ? 5 : DIM <= 128 ? 4 : 2;
    static constexpr int CTAS = FIT < MOST ? FIT : MOST;   // that an SM holds
};

template <int DIM, int R>
__global__ void __launch_bounds__(NT, FewSmem<DIM, R>::CTAS) k_attn_cross_f32_few(const AttnArgs a) {
    using S = FewSmem<DIM, R>;
    constexpr int TR = S::TR, C = DIM / 32, TW = TT / 4;   // TW: a warp's tokens
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = lane >> 3, tg = lane & 7;
    int32_t *lims = reinterpret_cast<int32_t*>(sm + S::LIM), *qrows = lims + 16;
    float* ml = sm + S::ML;   // [warp][row] m, then l
    asm volatile("griddepcontrol.wait;" ::: "memory");
    pdl_trigger();
    if (__syncthreads_or(tid == 0 && a.meta->status)) return;
    const AttnPlanDev& pl = a.plan;
    const int c = blockIdx.x;
    int32_t t = pl.cta_begin[c];
    const int32_t t_end = pl.cta_begin[c + 1];
    int32_t u = pl.cta_unit[c];
    const float* Q = static_cast<const float*>(a.Q);
    float *kw = sm + S::K + warp * TW * DIM, *vw = sm + S::V + warp * TW * DIM, *pw = sm + S::P + warp * TW * S::PS;
    while (t < t_end) {
        const AttnUnit U = pl.units[u];
        const int32_t uend = U.tile_off + U.n_blk;
        if (t >= uend) { ++u; continue; }
        const int32_t cend = min(t_end, uend);
        const int32_t* trow = a.table + (int64_t)U.table_row * a.bpb + U.blk_start - U.tile_off;
        const int32_t half = warp >> 1;   // of the two tiles of a step, this warp's
        auto block_of = [&](int32_t tile) {
            int32_t blk = tile < cend ? __ldg(trow + tile) : 0;
            if ((uint32_t)blk >= (uint32_t)a.n_blocks) {
                atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
                blk = 0;   // read a valid block; the pool is poisoned anyway
            }
            return ((int64_t)blk * a.n_kv + U.kv_head) * (BS * DIM) + (warp & 1) * TW * DIM;
        };
        int32_t held = 0;   // positions that some row sees: what lies behind becomes zero
        auto first_pos = [&](int32_t tt) { return (U.blk_start + tt + half - U.tile_off) * BS + (warp & 1) * TW; };
        auto fetch = [&](const float* pool, float* to, int swizzle, int32_t tt, int64_t from) {
            const int32_t left = tt + half < cend ? held - first_pos(tt) : 0;
#pragma unroll
            for (int e0 = 0; e0 < TW * (DIM / 4); e0 += 32) {
                const int e = e0 + lane, tok = e / (DIM / 4), w = e % (DIM / 4);
                copy16(to + tok * DIM + 4 * (w ^ (tok & swizzle)), pool + from + tok * DIM + 4 * w, tok < left);
            }
            copies_commit();
        };
        __syncthreads();   // the last unit's shared memory is done with
        if (tid < TR) {
            const AttnRow row = unit_row(pl, U, min(tid, U.n_rows - 1));
            lims[tid] = tid < U.n_rows ? row.limit : 0;
            qrows[tid] = row.q_row;
        }
        int64_t from = block_of(t + half);
        __syncthreads();
        int32_t seen_by_all = INT32_MAX;
        for (int r = 0; r < U.n_rows; ++r) {
            held = max(held, lims[r]);
            seen_by_all = min(seen_by_all, lims[r]);
        }
        for (int e = tid; e < TR * (DIM / 4); e += NT) {
            const int r = e / (DIM / 4), w = e % (DIM / 4);
            copy16(sm + S::Q + r * DIM + 4 * (w ^ (r & 7)), Q + (int64_t)qrows[r] * DIM + 4 * w, r < U.n_rows);
        }
        copies_commit();
        fetch(a.pool_k, kw, 7, t, from);
        fetch(a.pool_v, vw, 0, t, from);
        copies_wait<2>();
        __syncthreads();   // Q is there
        float m[R], l[R];
        float4 acc[R][C];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int k = 0; k < C; ++k) acc[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int32_t tt = t; tt < cend; tt += 2) {
            const bool more = tt + 2 < cend;
            from = block_of(tt + 2 + half);
            copies_wait<1>();
            __syncwarp();   // the warp's K is there
            float s[R] = {};
#pragma unroll 4
            for (int k = 0; k < DIM / 4; ++k) {
                const float4 x = lds4(kw + tg * DIM + 4 * (k ^ tg));
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float4 q = lds4(sm + S::Q + (rg + 4 * i) * DIM + 4 * (k ^ (rg + 4 * (i & 1))));
                    s[i] = fmaf(q.w, x.w, fmaf(q.z, x.z, fmaf(q.y, x.y, fmaf(q.x, x.x, s[i]))));
                }
            }
            __syncwarp();   // K is free
            if (more) fetch(a.pool_k, kw, 7, tt + 2, from);
            else copies_commit();
            const int32_t pos = first_pos(tt) + tg, n_tok = tt + half < cend ? TW : 0;
            const bool plain = n_tok && pos - tg + TW <= seen_by_all;   // (of a warp alike)
            bool moved = false;
            float al[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                s[i] *= a.scale_log2;
                if (!plain && (!n_tok || pos >= lims[rg + 4 * i])) s[i] = -INFINITY;
                float mx = s[i];
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
                al[i] = exp2f(m[i] - ref);
                moved |= mn != m[i];
                m[i] = mn;
                s[i] = exp2f(s[i] - ref);
                l[i] = fmaf(l[i], al[i], s[i]);
            }
            store_row(pw + tg * S::PS + R * rg, s);
            copies_wait<1>();
            __syncwarp();   // V and P are there
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int k = 0; k < C; ++k)
                        acc[i][k] = make_float4(acc[i][k].x * al[i], acc[i][k].y * al[i], acc[i][k].z * al[i], acc[i][k].w * al[i]);
            }
            if (plain) {
#pragma unroll 2
                for (int tok = 0; tok < TW; ++tok) {
                    float w[R];
                    load_row(w, pw + tok * S::PS + R * rg);
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const float4 v = lds4(vw + tok * DIM + 4 * tg + 32 * k);
#pragma unroll
                        for (int i = 0; i < R; ++i) acc[i][k] = fma4(w[i], v, acc[i][k]);
                    }
                }
            } else {   // a masked token's V may be infinite: it is left out, not weighed by zero
#pragma unroll 1
                for (int tok = 0; tok < n_tok; ++tok) {
                    float w[R];
                    load_row(w, pw + tok * S::PS + R * rg);
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const float4 v = lds4(vw + tok * DIM + 4 * tg + 32 * k);
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if (pos - tg + tok < lims[rg + 4 * i]) acc[i][k] = fma4(w[i], v, acc[i][k]);
                    }
                }
            }
            __syncwarp();   // V and P are free
            if (more) fetch(a.pool_v, vw, 0, tt + 2, from);
            else copies_commit();
        }
        copies_wait<0>();
        __syncthreads();   // K's and V's place is free
        float* join = sm + S::K;   // [warp][row][DIM]
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            const int r = TR * warp + rg + 4 * i;
            if (tg == 0) {
                ml[r] = m[i];
                ml[64 + r] = l[i];
            }
#pragma unroll
            for (int k = 0; k < C; ++k) *reinterpret_cast<float4*>(join + r * DIM + 4 * tg + 32 * k) = acc[i][k];
        }
        __syncthreads();
        const bool whole = pl.direct && U.nchunks == 1;
        const int32_t prow0 = U.prow_base + (c - U.cfirst) * U.n_rows;
        for (int e = tid; e < U.n_rows * (DIM / 4); e += NT) {
            const int r = e / (DIM / 4), w = e % (DIM / 4);
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[TR * k + r]);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = exp2f(ml[TR * k + r] - ref);
                L = fmaf(f, ml[64 + TR * k + r], L);
                o = fma4(f, lds4(join + (TR * k + r) * DIM + 4 * w), o);
            }
            if (whole) {
                const float f = 1.f / L;
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (int64_t)qrows[r] * DIM + 4 * w) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            } else {
                *reinterpret_cast<float4*>(a.part_acc + (int64_t)(prow0 + r) * DIM + 4 * w) = o;
                if (w == 0) a.part_ml[prow0 + r] = make_float2(M, L);
            }
        }
        t = cend;
        ++u;
    }
}

template <int DIM, typename F>
int by_rows(int rows, F f) {
    if constexpr (DIM <= 128)
        if (rows == 128) return f(k_attn_cross_f32<DIM, 8>, F32Smem<DIM, 8>::BYTES);
    switch (rows) {
        case 4: return f(k_attn_cross_f32_few<DIM, 1>, FewSmem<DIM, 1>::BYTES);
        case 8: return f(k_attn_cross_f32_few<DIM, 2>, FewSmem<DIM, 2>::BYTES);
        case 16: return f(k_attn_cross_f32_few<DIM, 4>, FewSmem<DIM, 4>::BYTES);
        case 32: return f(k_attn_cross_f32<DIM, 2>, F32Smem<DIM, 2>::BYTES);
        case 64: return f(k_attn_cross_f32<DIM, 4>, F32Smem<DIM, 4>::BYTES);
        default: return DENDRITE_EDTYPE;
    }
}

template <typename F>
int by_dim(int dim, int rows, F f) {
    switch (dim) {
        case 32: return by_rows<32>(rows, f);
        case 64: return by_rows<64>(rows, f);
        case 96: return by_rows<96>(rows, f);
        case 128: return by_rows<128>(rows, f);
        case 160: return by_rows<160>(rows, f);
        case 192: return by_rows<192>(rows, f);
        case 224: return by_rows<224>(rows, f);
        case 256: return by_rows<256>(rows, f);
        default: return DENDRITE_EDTYPE;
    }
}

}  // namespace

namespace dendrite {

int attn_f32_tiled_setup(int head_dim, int (&ctas_per_sm)[kF32TiledKernels]) {
    for (int i = 0, rows = kF32TiledMinRows; rows <= f32_tiled_max_rows(head_dim); ++i, rows *= 2) {
        DENDRITE_TRY(by_dim(head_dim, rows, [&](auto fn, int bytes) -> int {
            DENDRITE_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
            int occ = 0;
            DENDRITE_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, NT, bytes));
            ctas_per_sm[i] = occ > 1 ? occ : 1;
            return DENDRITE_OK;
        }));
    }
    return DENDRITE_OK;
}

int launch_attn_f32_tiled(const AttnArgs& a, cudaStream_t s) {
    if (a.plan.n_ctas <= 0) return DENDRITE_OK;
    return by_dim(a.head_dim, a.plan.tiled, [&](auto fn, int bytes) -> int {
        DENDRITE_CUDA(launch_pdl(fn, dim3((unsigned)a.plan.n_ctas), dim3(NT), (size_t)bytes, s, a));
        return DENDRITE_OK;
    });
}

}  // namespace dendrite
