// Rows into and out of the blocks.
//
// k_append_rows writes the new rows of an append and, on the way, applies
// rotary positions and the 8-bit quantisation, so that a row is read once and
// written once.
//
// Rotary positions.  Pair i of a head (elements (i, i + r/2), or (2 i, 2 i + 1)
// when interleaved; r = rot_dim) turns by a = position * inv_freq[i]:
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a).
// The angle is kept in turns, as a 64-bit fixed-point fraction: position *
// fraction wraps at whole turns, so the range reduction is one integer
// product and exact however far the position is (an fp32 angle at position
// 10^6 would be off by 2^-4 rad).  sine and cosine come from the fraction's
// distance to the nearest quarter turn, as a sum of two floats, by Taylor
// polynomials, and are rounded once (sincos_turns).
//
// 8-bit rows.  e is the least integer >= -126 with max|x| <= 448 * 2^e and
// element k is stored as the e4m3 number nearest to x_k * 2^-e, ties to even
// (with e = 120 at most 240, which is finite when read back); a row with a NaN
// or an infinity is stored as NaN throughout.  The scale
// is a power of two: x * 2^-e is exact in fp32, so a code depends on its
// row's bits alone, and code * 2^e is again a bf16 number, exactly.
//
// A thread owns 16 elements (two 8-element chunks that hold whole pairs) of
// the row of one token and walks the heads with them: the 8 angles are
// computed once per thread, not once per head.  All of a tile's tokens and
// heads are spread over 128 threads; tiles are (branch, block) pairs, and few
// tiles are split over their heads (grid.z) until the SMs are full.
// The kernel is bound by HBM at large sizes and by its chain of dependent
// reads (table, row) at small ones.  4 x 4,099 tokens of 8 + 8 + 32 heads,
// rotated: 67 us for 402 MB in and out (6.0 TB/s); 8 x 4,096 tokens of 8 + 8
// heads, quantised: 43 us for 202 MB (4.7 TB/s, 67 % of the issue slots: there
// the instructions of the quantisation count as much); the same read back: 35 us
// (5.8 TB/s).  One token of 16 branches is 4 us, all of it latency.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "rows.h"

using namespace dendrite;

namespace {

__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Per-call argument words: as kernel parameters up to CAP words, staged in
// device memory beyond.
template <int CAP>
struct ParamWords {
    int32_t v[CAP];
    __device__ __forceinline__ int32_t operator[](int64_t i) const { return v[i]; }
};
struct GlobalWords {
    const int32_t* p;
    __device__ __forceinline__ int32_t operator[](int64_t i) const { return __ldg(p + i); }
};
constexpr int kRowsSmall = 256, kRowsCap = 1536;   // small calls copy fewer parameter bytes per launch

template <typename A>
__device__ __forceinline__ int32_t byte_of(const A& args, int64_t word0, int64_t i) {
    return (int32_t)((uint32_t)args[word0 + (i >> 2)] >> (8 * (int)(i & 3))) & 255;
}

// Branch holding entry t of the concatenated per-branch ranges that start at
// args[off + i] (ascending), and its range's start: a division when every
// branch has `uniform` entries.
template <typename A>
__device__ __forceinline__ int32_t find_branch(const A& args, int64_t off, int32_t n, int32_t t, int32_t uniform,
                                               int32_t& first) {
    if (uniform > 0) {
        const int32_t i = t / uniform;
        first = i * uniform;
        return i;
    }
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (args[off + mid] <= t) lo = mid; else hi = mid - 1;
    }
    first = args[off + lo];
    return lo;
}

struct RowsArgs {
    int32_t n, n_new, bpb, n_kv, nq, dim, rot, interleaved, n_blocks, uniform, n_tiles, has_depth, one_tree;
    float m;
    const int32_t* table;
    const int32_t* call;    // the metadata kernel's scratch: copy-on-write sources at [n, 2 n)
    const void* K;
    const void* V;
    const void* Q;
    void* q_out;
    char* kp;
    char* vp;
    int64_t kv_layer, q_layer;   // elements
    int64_t pool_layer;          // bytes
    DevMeta* meta;
    uint64_t freq[128];          // turns per position, as a fraction of 2^64
};

// Eight consecutive elements as they are; input rows are read once, through L2
// and not the read-only path: the queries may be rotated in place.
template <typename T>
struct Chunk {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load(const T* p, Chunk<T>& x) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(T) / 2); ++k) x.w[k] = __ldcg(reinterpret_cast<const uint4*>(p) + k);
}
template <typename T>
__device__ __forceinline__ void store(T* p, const Chunk<T>& x) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(T) / 2); ++k) reinterpret_cast<uint4*>(p)[k] = x.w[k];
}
__device__ __forceinline__ void to_float(const Chunk<__nv_bfloat16>& c, float (&x)[8]) {
    const uint32_t w[4] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_float(const Chunk<float>& c, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[4 * k] = __uint_as_float(c.w[k].x);
        x[4 * k + 1] = __uint_as_float(c.w[k].y);
        x[4 * k + 2] = __uint_as_float(c.w[k].z);
        x[4 * k + 3] = __uint_as_float(c.w[k].w);
    }
}
__device__ __forceinline__ void from_float(const float (&x)[8], Chunk<__nv_bfloat16>& c) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    c.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void from_float(const float (&x)[8], Chunk<float>& c) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
        c.w[k] = make_uint4(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]), __float_as_uint(x[4 * k + 2]),
                            __float_as_uint(x[4 * k + 3]));
}
// The bits of max|x| as fp32: magnitudes order as integers, with what is not
// finite above all.
__device__ __forceinline__ uint32_t top_bits(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // of two 16-bit pairs
    uint32_t y;
    asm("max.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t top_bits(const Chunk<__nv_bfloat16>& c) {
    const uint32_t m = max2(max2(c.w[0].x & 0x7fff7fffu, c.w[0].y & 0x7fff7fffu),
                            max2(c.w[0].z & 0x7fff7fffu, c.w[0].w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}

// m cos and m sin of u / 2^64 turns, each rounded once (about half a step off;
// through one fp32 angle it would be two).  With q the nearest quarter turn,
// the rest x = 2 pi (u / 2^64 - q / 4), |x| <= pi/4, is p + e: p the rounded
// product of its top 22 bits with 2 pi, e what that leaves out.
//     sin x = p + (p^3 S(p^2) + e cos p),       S: Taylor to x^9
//     cos x = (1 - p^2/2) + (p^4 C(p^2) - e sin p), C: Taylor to x^10
// (first omitted terms 2^-29 and 2^-33 of the result), both sums with the
// rounding of their first term and of p^2 carried in the second.
__device__ __forceinline__ void sincos_turns(uint64_t u, float m, float& sn, float& cs) {
    const uint32_t q = (uint32_t)((u + (1ull << 61)) >> 62);
    const int64_t r = (int64_t)(u - ((uint64_t)q << 62));
    const float hi = (float)(int32_t)(r >> 40);                    // 2^-24 turns
    const float lo = (float)(uint32_t)((uint64_t)(r >> 16) & 0xffffffu);   // 2^-48 turns
    constexpr float kTwoPi = 6.28318530717958647692f;
    constexpr float kTwoPiRest = (float)(6.28318530717958647692 - (double)kTwoPi);
    const float p = hi * (kTwoPi * 0x1p-24f);
    float e = fmaf(hi, kTwoPi * 0x1p-24f, -p);
    e = fmaf(hi, kTwoPiRest * 0x1p-24f, e);
    e = fmaf(lo, kTwoPi * 0x1p-48f, e);
    const float z = p * p;
    const float zl = fmaf(p, p, -z);
    float t = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    t = fmaf(z, t, 1.f / 120.f);
    t = fmaf(z, t, -1.f / 6.f);
    const float st = fmaf(p * z, t, fmaf(-0.5f * z, e, e));
    const float w = fmaf(-0.5f, z, 1.f);
    float k = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    k = fmaf(z, k, -1.f / 720.f);
    k = fmaf(z, k, 1.f / 24.f);
    float ct = fmaf(-0.5f, z, 1.f - w);            // what rounding 1 - z/2 left out
    ct = fmaf(-0.5f, zl, ct);
    ct = fmaf(z * z, k, ct);
    ct = fmaf(-e, p + st, ct);
    const float s = fmaf(p, m, st * m), c = fmaf(w, m, ct * m);
    const float a = q & 1u ? c : s, b = q & 1u ? s : c;
    sn = q & 2u ? -a : a;
    cs = (q + 1u) & 2u ? -b : b;
}

// The exponent byte e + 127: e is the least >= -126 with top <= 448 * 2^e
// (top = (1 + f) 2^(E - 127), and 448 = 1.75 * 2^8); 255 for a row that is not
// finite.
__device__ __forceinline__ uint32_t fp8_exponent(uint32_t top) {
    if (top >= 0x7f800000u) return 255u;
    return (uint32_t)max(1, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
}
// Two codes of (x, y) * 2^-e (inv: that power of two, twice).
__device__ __forceinline__ uint32_t two_codes(float x, float y, uint64_t inv) {
    uint64_t v;
    float2 f;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(inv));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}
// Eight codes of x * 2^-e.  At e = 120 they end at 240 (256 * 2^120 would read
// back as an infinity); out of line, for it hardly ever happens.
__device__ __noinline__ uint2 fp8_codes_top(float4 x, float4 y, uint32_t byte) {
    if (byte == 255u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = __nv_cvt_float2_to_fp8x2(make_float2(fminf(fmaxf(f[2 * k] * 0x1p-120f, -240.f), 240.f),
                                                    fminf(fmaxf(f[2 * k + 1] * 0x1p-120f, -240.f), 240.f)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
__device__ __forceinline__ uint2 fp8_codes(const float (&x)[8], uint32_t byte) {
    if (byte >= 247u)
        return fp8_codes_top(make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]), byte);
    const uint32_t b = (254u - byte) << 23;   // e in [-126, 119]
    const uint64_t inv = (uint64_t)b << 32 | b;
    return make_uint2(two_codes(x[0], x[1], inv) | two_codes(x[2], x[3], inv) << 16,
                      two_codes(x[4], x[5], inv) | two_codes(x[6], x[7], inv) << 16);
}
// Byte offset of element d (a multiple of 8) of slot s in an 8-bit tile.
__device__ __forceinline__ int32_t fp8_at(int32_t s, int32_t d) {
    return s * kFp8Dim + (((d >> 4) ^ (s & 7)) << 4) + (d & 8);
}

// args: branch[n], length[n], prefix of touched blocks[n], then the draft
// tree depths as bytes.
// T: the rows' type; FP8: the blocks hold 8-bit rows (else rows of T); ROPE:
// keys and queries turn (else every row is stored as it is).
// Rows go through a thread U at a time, loads first.  Rotating rows of 16 bits:
// four, at four CTAs an SM (three or six at a time lost 1 to 5 %, two at six CTAs
// 17 %).  Rows that are only quantised: two, at eight CTAs (32,768 tokens of 8
// heads appended and read back 94.9 us, against 98.7 with four at five CTAs and
// 104 with one at twelve).
template <typename T, bool FP8, bool ROPE, typename A>
__global__ void __launch_bounds__(128, ROPE ? 4 : 8) k_append_rows(const __grid_constant__ A args, const __grid_constant__ RowsArgs a) {
    pdl_wait();
    constexpr int bs = kBlockSize;
    constexpr int U = ROPE && sizeof(T) == 2 ? 4 : 2;
    const int32_t n = a.n, dim = a.dim;
    const int32_t items = dim >> 4;                     // threads per row
    const int32_t lanes = 128 / items;                  // rows in flight, cut to a power of two
    const int32_t lp2 = 1 << (31 - __clz(lanes));
    const int32_t item = threadIdx.x % items, lane = threadIdx.x / items;
    // this thread's two chunks, whether they turn, and their first pair
    int32_t c0, c1;
    if (!ROPE || a.interleaved) {
        c0 = 8 * item;
        c1 = dim / 2 + 8 * item;
    } else if (16 * item < a.rot) {
        c0 = 8 * item;
        c1 = a.rot / 2 + 8 * item;
    } else {
        c0 = a.rot + 8 * (item - a.rot / 16);
        c1 = c0 + (dim - a.rot) / 2;
    }
    const bool turn0 = ROPE && c0 < a.rot, turn1 = ROPE && c1 < a.rot;
    const int32_t n_rows = 2 * a.n_kv + a.nq;           // rows per token: K heads, V heads, Q heads
    const int32_t status = a.meta->status, unclean = a.meta->unclean;
    const T* K = static_cast<const T*>(a.K) + blockIdx.y * a.kv_layer;
    const T* V = static_cast<const T*>(a.V) + blockIdx.y * a.kv_layer;
    const T* Q = static_cast<const T*>(a.Q) + blockIdx.y * a.q_layer;
    T* q_out = static_cast<T*>(a.q_out) + blockIdx.y * a.q_layer;
    char* kp = a.kp + blockIdx.y * a.pool_layer;
    char* vp = a.vp + blockIdx.y * a.pool_layer;
    const int64_t tile_bytes = FP8 ? kFp8TileBytes : (int64_t)bs * dim * (int)sizeof(T);
    if (__any_sync(0xffffffffu, status)) return;   // a whole warp leaves: shuffles below
    for (int32_t t = blockIdx.x; t < a.n_tiles; t += gridDim.x) {
        int32_t first;
        const int32_t i = find_branch(args, 2 * (int64_t)n, n, t, a.uniform, first);
        const int32_t L = args[n + i];
        const int32_t lblk = L / bs + (t - first);
        const int32_t s0 = lblk == L / bs ? L % bs : 0;
        const int32_t s1 = min(bs, L + a.n_new - lblk * bs);
        const int32_t dst = a.table[(int64_t)args[i] * a.bpb + lblk];
        const int32_t csrc = lblk == L / bs ? a.call[n + i] : -1;
        if ((uint32_t)dst >= (uint32_t)a.n_blocks || csrc >= a.n_blocks) {
            if (threadIdx.x == 0) atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
            return;
        }
        // tokens side by side over the lanes, as many as there are (to a power of two)
        const int32_t nt = s1 - s0;
        const int32_t tp = min(lp2, nt <= 1 ? 1 : 1 << (32 - __clz(nt - 1)));
        const int32_t r0 = lane / tp, rstep = lp2 / tp;
        for (int32_t k0 = 0; k0 < nt; k0 += tp) {
            const int32_t k = k0 + lane % tp;
            const bool live = lane < lp2 && k < nt;
            const int32_t slot = s0 + (live ? k : 0);
            const int32_t tok = lblk * bs + slot - L;       // 0 .. n_new - 1
            const int64_t in_row = (int64_t)i * a.n_new + tok;
            const int64_t kv_at = in_row * a.n_kv * dim, q_at = in_row * a.nq * dim;
            const int32_t n_iter = (n_rows + rstep * (int)gridDim.z - 1) / (rstep * (int)gridDim.z);
            float cs[8], sn[8];
            for (int32_t it0 = 0; it0 < n_iter; it0 += U) {
                Chunk<T> x[U], y[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t rr = ((it0 + u) * (int)gridDim.z + (int)blockIdx.z) * rstep + r0;
                    if (!live || rr >= n_rows) continue;
                    const T* src = rr < a.n_kv       ? K + kv_at + rr * dim
                                   : rr < 2 * a.n_kv ? V + kv_at + (rr - a.n_kv) * dim
                                                     : Q + q_at + (rr - 2 * a.n_kv) * dim;
                    load(src + c0, x[u]);
                    load(src + c1, y[u]);
                }
                if (ROPE && it0 == 0) {   // the angles, while the first rows are on their way
                    const int32_t pos = L + (a.has_depth ? byte_of(args, 3 * (int64_t)n, (int64_t)(a.one_tree ? 0 : i) * a.n_new + tok) : tok);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int32_t pair = a.interleaved ? (q < 4 ? c0 / 2 + q : c1 / 2 + q - 4) : c0 + q;
                        const bool on = a.interleaved ? (q < 4 ? turn0 : turn1) : turn0;
                        cs[q] = 1.f;
                        sn[q] = 0.f;
                        if (on) sincos_turns(a.freq[pair & 127] * (uint64_t)(uint32_t)pos, a.m, sn[q], cs[q]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t rr = ((it0 + u) * (int)gridDim.z + (int)blockIdx.z) * rstep + r0;
                    const bool act = live && rr < n_rows;
                    const int32_t kind = rr < a.n_kv ? 0 : rr < 2 * a.n_kv ? 1 : 2;   // K, V, Q
                    const int32_t h = rr - (kind == 0 ? 0 : kind == 1 ? a.n_kv : 2 * a.n_kv);
                    float f[8], g[8];
                    uint32_t top = 0;
                    const bool turns = ROPE && act && kind != 1;
                    if (turns) {
                        to_float(x[u], f);
                        to_float(y[u], g);
                        if (a.interleaved) {
                            if (turn0) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const float c = f[2 * q], d = f[2 * q + 1];
                                    f[2 * q] = c * cs[q] - d * sn[q];
                                    f[2 * q + 1] = d * cs[q] + c * sn[q];
                                }
                            }
                            if (turn1) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const float c = g[2 * q], d = g[2 * q + 1];
                                    g[2 * q] = c * cs[4 + q] - d * sn[4 + q];
                                    g[2 * q + 1] = d * cs[4 + q] + c * sn[4 + q];
                                }
                            }
                        } else if (turn0) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float c = f[q], d = g[q];
                                f[q] = c * cs[q] - d * sn[q];
                                g[q] = d * cs[q] + c * sn[q];
                            }
                        }
                        if (!FP8 || kind == 2) {
                            from_float(f, x[u]);
                            from_float(g, y[u]);
                        }
                    }
                    if constexpr (FP8) {
                        if (act && kind != 2) {
                            if (turns) top = max(top_bits(f), top_bits(g));
                            else top = max(top_bits(x[u]), top_bits(y[u]));
                        }
                        // the row's largest element: its eight threads are eight neighbouring lanes
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    }
                    if (!act) continue;
                    char* tile = (kind == 0 ? kp : vp) + ((int64_t)dst * a.n_kv + (kind == 2 ? 0 : h)) * tile_bytes;
                    if (kind == 2) {
                        T* out = q_out + q_at + h * dim;
                        store(out + c0, x[u]);
                        store(out + c1, y[u]);
                    } else if constexpr (FP8) {
                        if (!turns) {
                            to_float(x[u], f);
                            to_float(y[u], g);
                        }
                        const uint32_t e = fp8_exponent(top);
                        *reinterpret_cast<uint2*>(tile + fp8_at(slot, c0)) = fp8_codes(f, e);
                        *reinterpret_cast<uint2*>(tile + fp8_at(slot, c1)) = fp8_codes(g, e);
                        if (item == 0) tile[bs * kFp8Dim + slot] = (char)e;
                    } else {
                        T* out = reinterpret_cast<T*>(tile) + slot * dim;
                        store(out + c0, x[u]);
                        store(out + c1, y[u]);
                        if constexpr (sizeof(T) == 2)   // (fp32 attention reads no row that nothing sees)
                            if (kind == 1 && max(top_bits(x[u]), top_bits(y[u])) >= 0x7f800000u) a.meta->unclean = 1;
                    }
                }
            }
        }
        // bf16: V behind the branch's new end becomes finite
        if (!FP8 && sizeof(T) == 2 && unclean)
            for (int32_t h = blockIdx.z; h < a.n_kv; h += gridDim.z) {
                uint4* to = reinterpret_cast<uint4*>(vp + ((int64_t)dst * a.n_kv + h) * tile_bytes);
                for (int32_t w = s1 * (dim / 8) + threadIdx.x; w < bs * (dim / 8); w += 128) to[w] = make_uint4(0u, 0u, 0u, 0u);
            }
        // the valid slots of a copied-on-write tail, stored rows as they are
        if (csrc >= 0 && s0 > 0) {
            const int32_t words = FP8 ? kFp8Dim / 16 : dim * (int)sizeof(T) / 16;
            for (int32_t r = blockIdx.z; r < 2 * a.n_kv; r += gridDim.z) {
                char* pool = r < a.n_kv ? kp : vp;
                const int32_t h = r < a.n_kv ? r : r - a.n_kv;
                const char* from = pool + ((int64_t)csrc * a.n_kv + h) * tile_bytes;
                char* to = pool + ((int64_t)dst * a.n_kv + h) * tile_bytes;
                for (int32_t w = threadIdx.x; w < s0 * words; w += 128)
                    reinterpret_cast<uint4*>(to)[w] = reinterpret_cast<const uint4*>(from)[w];
                if (FP8 && (int32_t)threadIdx.x < s0) to[bs * kFp8Dim + threadIdx.x] = from[bs * kFp8Dim + threadIdx.x];
            }
        }
    }
}

// ------------------------------------------------------------------ gather
// args: branch[n], first position[n], output row[n], prefix of touched blocks[n],
// row count[n].  One CTA per (branch, block) and share of the heads.  A thread
// owns 8 elements of the row of one slot and walks the heads with them, U rows'
// loads in flight, so that nothing is divided in the loop (8-bit rows: eight
// rather than four, 92.4 against 94.9 us for the case above, sixteen 97.8); a warp's
// stores cover whole 128-byte lines.
struct ReadArgs {
    int32_t n, bpb, n_kv, dim, n_blocks, uniform, n_tiles;
    const int32_t* table;
    const char* kp;
    const char* vp;
    void* K;
    void* V;
    DevMeta* meta;
};

template <typename T, bool FP8, typename A>
__global__ void __launch_bounds__(256) k_read_rows(const __grid_constant__ A args, const __grid_constant__ ReadArgs a) {
    pdl_wait();
    constexpr int bs = kBlockSize;
    constexpr int U = FP8 ? 8 : 4;
    const int32_t n = a.n, dim = a.dim;
    const int32_t chunks = dim >> 3;                    // threads per row
    const int32_t lp2 = 1 << (31 - __clz(256 / chunks));
    const int32_t d = 8 * (threadIdx.x % chunks), lane = threadIdx.x / chunks;
    if (a.meta->status) return;
    const int64_t tile_bytes = FP8 ? kFp8TileBytes : (int64_t)bs * dim * (int)sizeof(T);
    for (int32_t t = blockIdx.x; t < a.n_tiles; t += gridDim.x) {
        int32_t first;
        const int32_t i = find_branch(args, 3 * (int64_t)n, n, t, a.uniform, first);
        const int32_t p0 = args[n + i], count = args[4 * (int64_t)n + i];
        const int32_t lblk = p0 / bs + (t - first);
        const int32_t s0 = max(0, p0 - lblk * bs), s1 = min(bs, p0 + count - lblk * bs);
        const int32_t src = a.table[(int64_t)args[i] * a.bpb + lblk];
        if ((uint32_t)src >= (uint32_t)a.n_blocks) {
            if (threadIdx.x == 0) atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
            return;
        }
        if (lane >= lp2) continue;
        const int64_t row0 = (int64_t)args[2 * (int64_t)n + i] + lblk * bs - p0;   // output row of slot 0
        const int32_t nt = s1 - s0;
        const int32_t tp = min(lp2, nt <= 1 ? 1 : 1 << (32 - __clz(nt - 1)));
        const int32_t rstep = lp2 / tp * (int)gridDim.z;
        for (int32_t slot = s0 + lane % tp; slot < s1; slot += tp) {
            for (int32_t r0 = (int)blockIdx.z * (lp2 / tp) + lane / tp; r0 < 2 * a.n_kv; r0 += U * rstep) {
                Chunk<T> x[U];
                uint2 w[U];
                uint32_t e[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t r = r0 + u * rstep;
                    if (r >= 2 * a.n_kv) continue;
                    const char* tile = (r < a.n_kv ? a.kp : a.vp) +
                                       ((int64_t)src * a.n_kv + (r < a.n_kv ? r : r - a.n_kv)) * tile_bytes;
                    if constexpr (FP8) {
                        w[u] = *reinterpret_cast<const uint2*>(tile + fp8_at(slot, d));
                        e[u] = (unsigned char)tile[bs * kFp8Dim + slot];
                    } else {
                        load(reinterpret_cast<const T*>(tile) + slot * dim + d, x[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t r = r0 + u * rstep;
                    if (r >= 2 * a.n_kv) continue;
                    T* out = static_cast<T*>(r < a.n_kv ? a.K : a.V) +
                             ((row0 + slot) * a.n_kv + (r < a.n_kv ? r : r - a.n_kv)) * dim + d;
                    if constexpr (FP8) {
                        const float s = __uint_as_float(e[u] << 23);   // 2^e
                        const uint32_t q[2] = {w[u].x, w[u].y};
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                                (__nv_fp8x2_storage_t)(q[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
                            const float2 v = __half22float2(__half2(hr));
                            f[2 * k] = v.x * s;
                            f[2 * k + 1] = v.y * s;
                        }
                        from_float(f, x[u]);
                    }
                    store(out, x[u]);
                }
            }
        }
    }
}

// ------------------------------------------------------------- kept drafts
// args: branch[n], base length[n], kept rows[n], prefix of kept nodes[n], then
// the kept nodes as bytes.  Row base + node[k] moves to base + k.  Nodes are
// ascending (node[k] >= k), so a write to row k never hits a row that a later
// k still reads, and every thread moves its own 16-byte column: the order of
// the loop is all the synchronisation it needs.  CTA (branch, kv head, layer).
struct KeepArgs {
    int32_t n, bpb, n_kv, n_blocks, words;   // words: 16-byte words of a stored row
    int64_t tile_bytes, pool_layer;
    int32_t fp8;
    const int32_t* table;
    char* kp;
    char* vp;
    DevMeta* meta;
};

template <typename A>
__global__ void __launch_bounds__(128) k_keep_rows(const __grid_constant__ A args, const __grid_constant__ KeepArgs a) {
    pdl_wait();
    constexpr int bs = kBlockSize;
    __shared__ int32_t blocks[kMaxDraft / bs + 1];
    __shared__ int32_t bad;
    const int32_t n = a.n, i = blockIdx.x, h = blockIdx.y;
    if (a.meta->status) return;
    const int32_t base = args[n + i], kept = args[2 * n + i], off = args[3 * n + i];
    if (kept == 0) return;
    const int32_t b0 = base / bs;
    const int32_t top = base + byte_of(args, 4 * (int64_t)n, off + kept - 1);   // the last row read
    const int32_t nb = top / bs - b0 + 1;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    if ((int32_t)threadIdx.x < nb) {
        const int32_t blk = a.table[(int64_t)args[i] * a.bpb + b0 + threadIdx.x];
        blocks[threadIdx.x] = blk;
        if ((uint32_t)blk >= (uint32_t)a.n_blocks) {
            bad = 1;
            atomicCAS(&a.meta->status, 0, DENDRITE_ECORRUPT);
        }
    }
    __syncthreads();
    if (bad) return;
    const int32_t cols = 2 * a.words + (a.fp8 ? 2 : 0);   // K words, V words, then the two exponent columns
    for (int32_t c = threadIdx.x; c < cols; c += blockDim.x) {
        const bool v = c < 2 * a.words ? c >= a.words : c - 2 * a.words == 1;
        char* pool = (v ? a.vp : a.kp) + blockIdx.z * a.pool_layer;
        if (c < 2 * a.words) {
            const int32_t w = v ? c - a.words : c;
            auto at = [&](int32_t pos) {
                const int32_t s = pos % bs;
                return reinterpret_cast<uint4*>(pool + ((int64_t)blocks[pos / bs - b0] * a.n_kv + h) * a.tile_bytes) +
                       s * a.words + (a.fp8 ? w ^ (s & 7) : w);
            };
            constexpr int U = 8;
            for (int32_t k0 = 0; k0 < kept; k0 += U) {
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k0 + u < kept) x[u] = *at(base + byte_of(args, 4 * (int64_t)n, off + k0 + u));
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k0 + u < kept) *at(base + k0 + u) = x[u];
            }
        } else {
            auto at = [&](int32_t pos) {
                return pool + ((int64_t)blocks[pos / bs - b0] * a.n_kv + h) * a.tile_bytes + bs * kFp8Dim + pos % bs;
            };
            for (int32_t k = 0; k < kept; ++k) *at(base + k) = *at(base + byte_of(args, 4 * (int64_t)n, off + k));
        }
    }
}

// Calls `go` with the argument words: as kernel parameters, or staged.
template <typename Fill, typename Go>
int with_words(dendrite_pool* p, size_t words, cudaStream_t s, Fill fill, Go go) {
    if (words <= (size_t)kRowsSmall) {
        ParamWords<kRowsSmall> a;
        fill(a.v);
        return go(a);
    }
    if (words <= (size_t)kRowsCap) {
        ParamWords<kRowsCap> a;
        fill(a.v);
        return go(a);
    }
    char *h, *d;
    DENDRITE_TRY(p->staging.reserve(words * 4, &h, &d));
    fill(reinterpret_cast<int32_t*>(h));
    DENDRITE_TRY(p->staging.upload(s, h, words * 4));
    DENDRITE_TRY(go(GlobalWords{reinterpret_cast<const int32_t*>(d)}));
    return p->staging.release(s);
}

// CTAs along the heads so that `tiles` tiles make about per_sm per SM, at most `most`.
unsigned head_splits(const dendrite_pool* p, int64_t tiles, int64_t most, int per_sm) {
    const int64_t want = (per_sm * (int64_t)p->sm_count + tiles - 1) / std::max<int64_t>(tiles, 1);
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, most), 64));
}

}  // namespace

namespace dendrite {

// Captured calls would be replayed with the lengths, tables and staged
// arguments of the capture: refused.
int check_not_capturing(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) {
        cudaGetLastError();
        return DENDRITE_EINVAL;
    }
    return st == cudaStreamCaptureStatusNone ? DENDRITE_OK : DENDRITE_EINVAL;
}

}  // namespace dendrite

namespace {

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

}  // namespace

namespace dendrite {

int check_trees(const int32_t* parents, int32_t n_trees, int32_t n, int32_t t) {
    if (!parents || (n_trees != 1 && n_trees != n)) return DENDRITE_EINVAL;
    if (t < 1 || t > kMaxDraft) return DENDRITE_EINVAL;
    for (int64_t i = 0; i < n_trees; ++i)
        for (int32_t j = 0; j < t; ++j) {
            const int32_t up = parents[i * t + j];
            if (up < -1 || up >= j) return DENDRITE_EINVAL;
        }
    return DENDRITE_OK;
}

void tree_depths(const int32_t* parents, int32_t n_trees, int32_t t, std::vector<uint8_t>& depth) {
    depth.resize((size_t)n_trees * t);
    for (int64_t i = 0; i < n_trees; ++i)
        for (int32_t j = 0; j < t; ++j) {
            const int32_t up = parents[i * t + j];
            depth[i * t + j] = up < 0 ? 0 : (uint8_t)(depth[i * t + up] + 1);
        }
}

// branch[n], length[n], prefix of touched blocks[n], then the draft tree depths as bytes.
static size_t rows_words(const RowsCall& c) {
    const size_t n_depth = c.depth ? (size_t)c.n_trees * c.n_new : 0;
    return 3 * (size_t)c.n + (n_depth + 3) / 4;
}

size_t staged_rows_words(const RowsCall& c) {
    const size_t words = rows_words(c);
    return words > (size_t)kRowsCap ? words : 0;
}

void fill_rows_words(const RowsCall& c, int32_t bs, int32_t* w) {
    const size_t n = c.n;
    int32_t acc = 0;
    for (size_t i = 0; i < n; ++i) {
        w[i] = c.branches[i];
        w[n + i] = c.lens[i];
        w[2 * n + i] = acc;
        acc += (c.lens[i] + c.n_new - 1) / bs - c.lens[i] / bs + 1;
    }
    if (c.depth) {
        w[rows_words(c) - 1] = 0;   // the bytes after the last depth
        std::memcpy(w + 3 * n, c.depth, (size_t)c.n_trees * c.n_new);
    }
}

int launch_append_rows(dendrite_pool* p, const RowsCall& c, const int32_t* staged, cudaStream_t s) {
    const int32_t bs = p->block_size, n = c.n, n_new = c.n_new;
    RowsArgs a{};
    a.n = n;
    a.n_new = n_new;
    a.bpb = p->bpb;
    a.n_kv = p->n_kv;
    a.nq = c.Q ? c.n_q_heads : 0;
    a.dim = p->head_dim;
    a.n_blocks = (int32_t)p->num_blocks;
    a.n_tiles = (int32_t)c.touched;
    a.table = p->d_table;
    a.call = p->d_call_i32;
    a.K = c.K;
    a.V = c.V;
    a.Q = c.Q;
    a.q_out = c.q_out;
    a.kp = static_cast<char*>(p->d_k) + (size_t)c.layer0 * p->layer_bytes;
    a.vp = static_cast<char*>(p->d_v) + (size_t)c.layer0 * p->layer_bytes_v;
    a.kv_layer = c.kv_layer;
    a.q_layer = c.q_layer;
    a.pool_layer = (int64_t)p->layer_bytes;
    a.meta = p->d_meta;
    a.m = 1.f;
    if (c.rope) {
        a.rot = c.rope->rot_dim;
        a.interleaved = c.rope->interleaved;
        a.m = (float)c.rope->scale;
        for (int k = 0; k < a.rot / 2; ++k) {
            // turns per position modulo one: whole turns change nothing at whole positions
            const double turns = c.rope->inv_freq[k] * 0.15915494309189533577;   // 1 / (2 pi)
            const double frac = turns - std::floor(turns);
            a.freq[k] = frac >= 1.0 ? 0 : (uint64_t)(frac * 18446744073709551616.0);
        }
        a.has_depth = c.depth != nullptr;
        a.one_tree = c.n_trees == 1;
    }
    int32_t uniform = -1;
    for (int32_t i = 0; i < n && uniform != 0; ++i) {
        const int32_t k = (c.lens[i] + n_new - 1) / bs - c.lens[i] / bs + 1;
        uniform = uniform < 0 ? k : (uniform == k ? k : 0);
    }
    a.uniform = std::max(uniform, 0);
    // rows side by side in a CTA: 128 / (dim / 16) threads over a tile's tokens, the rest over heads
    const int32_t n_rows = 2 * a.n_kv + a.nq;
    int32_t lanes = 128 / (a.dim / 16), tp = 1;
    while (lanes & (lanes - 1)) lanes &= lanes - 1;
    while (tp < lanes && tp < std::min(n_new, bs)) tp *= 2;
    // (rotating rows: as many as run at once, for each CTA makes the angles anew:
    // 32 x 16 tokens of 48 heads 8 us, and 10 with 8 an SM)
    const unsigned z = head_splits(p, c.touched * c.n_layers_in, (n_rows + lanes / tp - 1) / (lanes / tp), c.rope ? 4 : 8);
    const dim3 grid((unsigned)std::min<int64_t>(c.touched, (int64_t)p->sm_count * 64), (unsigned)c.n_layers_in, z);
    auto go = [&](auto args) -> int {
        using A = decltype(args);
        if (p->dtype == DENDRITE_FP8 && !c.rope)
            DENDRITE_CUDA(launch_pdl(k_append_rows<__nv_bfloat16, true, false, A>, grid, dim3(128), 0, s, args, a));
        else if (p->dtype == DENDRITE_FP8)
            DENDRITE_CUDA(launch_pdl(k_append_rows<__nv_bfloat16, true, true, A>, grid, dim3(128), 0, s, args, a));
        else if (p->dtype == DENDRITE_BF16)
            DENDRITE_CUDA(launch_pdl(k_append_rows<__nv_bfloat16, false, true, A>, grid, dim3(128), 0, s, args, a));
        else
            DENDRITE_CUDA(launch_pdl(k_append_rows<float, false, true, A>, grid, dim3(128), 0, s, args, a));
        return DENDRITE_OK;
    };
    if (staged) return go(GlobalWords{staged});
    if (rows_words(c) <= (size_t)kRowsSmall) {
        ParamWords<kRowsSmall> w;
        fill_rows_words(c, bs, w.v);
        return go(w);
    }
    ParamWords<kRowsCap> w;
    fill_rows_words(c, bs, w.v);
    return go(w);
}

}  // namespace dendrite

extern "C" {

int dendrite_rope_init(dendrite_rope* r, int32_t rot_dim, int32_t interleaved, double base, int32_t scaling,
                       double factor, double original_len, double turns_low, double turns_high) {
    if (!r || rot_dim < 16 || rot_dim > 256 || rot_dim % 16) return DENDRITE_EINVAL;
    if (interleaved != 0 && interleaved != 1) return DENDRITE_EINVAL;
    if (!(base > 1.0) || !std::isfinite(base)) return DENDRITE_EINVAL;
    if (scaling < DENDRITE_ROPE_PLAIN || scaling > DENDRITE_ROPE_BANDS) return DENDRITE_EINVAL;
    if (scaling != DENDRITE_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return DENDRITE_EINVAL;
    const bool banded = scaling == DENDRITE_ROPE_YARN || scaling == DENDRITE_ROPE_BANDS;
    if (banded && (!(original_len > 0.0) || !std::isfinite(original_len) || !(turns_low > 0.0) ||
                   !(turns_high > turns_low) || !std::isfinite(turns_high)))
        return DENDRITE_EINVAL;
    std::memset(r, 0, sizeof(*r));
    r->rot_dim = rot_dim;
    r->interleaved = interleaved;
    r->scale = scaling == DENDRITE_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    const double two_pi = 6.283185307179586476925;
    const double b = scaling == DENDRITE_ROPE_NTK ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
    // the pair that makes `turns` turns over the original length, as a real index
    auto pair_of = [&](double turns) { return rot_dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(base)); };
    double low = 0.0, high = 0.0;
    if (scaling == DENDRITE_ROPE_YARN) {
        low = std::max(std::floor(pair_of(turns_high)), 0.0);
        high = std::min(std::ceil(pair_of(turns_low)), rot_dim - 1.0);
    }
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(b, -2.0 * i / rot_dim);
        double stretched = 0.0;   // share of the pair that is slowed down by factor
        if (scaling == DENDRITE_ROPE_LINEAR) stretched = 1.0;
        if (scaling == DENDRITE_ROPE_YARN)
            stretched = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
        if (scaling == DENDRITE_ROPE_BANDS) {
            const double turns = original_len * f / two_pi;
            stretched = 1.0 - std::min(std::max((turns - turns_low) / (turns_high - turns_low), 0.0), 1.0);
        }
        r->inv_freq[i] = stretched > 0.0 ? stretched * f / factor + (1.0 - stretched) * f : f;
    }
    return DENDRITE_OK;
}

int dendrite_read_kv(dendrite_pool* p, int32_t layer, const int32_t* branches, const int32_t* starts,
                     const int32_t* counts, int32_t n, void* K, void* V, void* stream) {
    if (!p) return DENDRITE_EINVAL;
    if (p->poisoned) return p->poisoned;
    if (p->dtype == DENDRITE_TURBO) return DENDRITE_EDTYPE;
    if (layer < 0 || layer >= p->n_layers) return DENDRITE_EINVAL;
    if (p->pending.active && !p->pending.layer_done[layer]) return DENDRITE_EINVAL;
    if (n < 0 || (n > 0 && (!branches || !starts || !counts))) return DENDRITE_EINVAL;
    const int32_t bs = p->block_size;
    int64_t rows = 0, tiles = 0;
    int32_t uniform = -1;
    for (int32_t i = 0; i < n; ++i) {
        DENDRITE_TRY(check_live(p, branches[i]));
        if (starts[i] < 0 || counts[i] < 0 || (int64_t)starts[i] + counts[i] > p->br[branches[i]].len) return DENDRITE_EINVAL;
        const int32_t k = counts[i] ? (starts[i] + counts[i] - 1) / bs - starts[i] / bs + 1 : 0;
        rows += counts[i];
        tiles += k;
        uniform = uniform < 0 ? k : (uniform == k ? k : 0);
    }
    if (rows == 0) return DENDRITE_OK;
    if (rows > INT32_MAX / 2 || tiles > INT32_MAX / 2) return DENDRITE_ELIMIT;
    if (!K || !V || (((uintptr_t)K | (uintptr_t)V) & 15)) return DENDRITE_EINVAL;
    const size_t bytes = (size_t)rows * p->n_kv * p->head_dim * p->elt;
    if (overlap(K, bytes, V, bytes)) return DENDRITE_EINVAL;
    DENDRITE_CUDA(cudaSetDevice(p->device));
    cudaStream_t s = (cudaStream_t)stream;
    DENDRITE_TRY(check_not_capturing(s));
    ReadArgs a{};
    a.n = n;
    a.bpb = p->bpb;
    a.n_kv = p->n_kv;
    a.dim = p->head_dim;
    a.n_blocks = (int32_t)p->num_blocks;
    a.uniform = std::max(uniform, 0);
    a.n_tiles = (int32_t)tiles;
    a.table = p->d_table;
    a.kp = static_cast<const char*>(p->d_k) + (size_t)layer * p->layer_bytes;
    a.vp = static_cast<const char*>(p->d_v) + (size_t)layer * p->layer_bytes_v;
    a.K = K;
    a.V = V;
    a.meta = p->d_meta;
    auto fill = [&](int32_t* w) {
        int32_t row = 0, tile = 0;
        for (int32_t i = 0; i < n; ++i) {
            w[i] = branches[i];
            w[n + i] = starts[i];
            w[2 * (size_t)n + i] = row;
            w[3 * (size_t)n + i] = tile;
            w[4 * (size_t)n + i] = counts[i];
            row += counts[i];
            tile += counts[i] ? (starts[i] + counts[i] - 1) / bs - starts[i] / bs + 1 : 0;
        }
    };
    // rows side by side in a CTA, as in the append: over a tile's tokens first, the rest over heads
    int32_t lanes = 256 / (p->head_dim / 8), tp = 1, longest = 0;
    while (lanes & (lanes - 1)) lanes &= lanes - 1;
    for (int32_t i = 0; i < n; ++i) longest = std::max(longest, counts[i]);
    while (tp < lanes && tp < std::min(longest, bs)) tp *= 2;
    const dim3 grid((unsigned)std::min<int64_t>(tiles, (int64_t)p->sm_count * 64), 1,
                    head_splits(p, tiles, (2 * p->n_kv + lanes / tp - 1) / (lanes / tp), 8));
    return with_words(p, 5 * (size_t)n, s, fill, [&](auto args) -> int {
        using A = decltype(args);
        if (p->dtype == DENDRITE_FP8)
            DENDRITE_CUDA(launch_pdl(k_read_rows<__nv_bfloat16, true, A>, grid, dim3(256), 0, s, args, a));
        else if (p->dtype == DENDRITE_BF16)
            DENDRITE_CUDA(launch_pdl(k_read_rows<__nv_bfloat16, false, A>, grid, dim3(256), 0, s, args, a));
        else
            DENDRITE_CUDA(launch_pdl(k_read_rows<float, false, A>, grid, dim3(256), 0, s, args, a));
        return DENDRITE_OK;
    });
}

int dendrite_accept_draft(dendrite_pool* p, const int32_t* branches, int32_t n, int32_t n_draft,
                          const int32_t* n_keep, const int32_t* nodes, void* stream) {
    if (!p) return DENDRITE_EINVAL;
    if (p->poisoned) return p->poisoned;
    if (p->dtype == DENDRITE_TURBO) return DENDRITE_EDTYPE;
    if (p->pending.active) return DENDRITE_EINVAL;
    if (n < 0 || n_draft < 0 || n_draft > kMaxDraft || (n > 0 && (!branches || !n_keep))) return DENDRITE_EINVAL;
    if (n == 0) return DENDRITE_OK;
    int64_t total = 0;
    for (int32_t i = 0; i < n; ++i) {
        DENDRITE_TRY(check_live(p, branches[i]));
        const Branch& b = p->br[branches[i]];
        if (b.len < n_draft || n_keep[i] < 0 || n_keep[i] > n_draft) return DENDRITE_EINVAL;
        total += n_keep[i];
    }
    {
        std::vector<int32_t> o(branches, branches + n);
        std::sort(o.begin(), o.end());
        if (std::adjacent_find(o.begin(), o.end()) != o.end()) return DENDRITE_EINVAL;
    }
    if (total > 0 && !nodes) return DENDRITE_EINVAL;
    std::vector<int32_t> new_lens(n);
    bool moves = false;
    const int32_t* nd = nodes;
    for (int32_t i = 0; i < n; ++i) {
        const Branch& b = p->br[branches[i]];
        const int32_t base = b.len - n_draft;
        bool mine = false;
        for (int32_t k = 0; k < n_keep[i]; ++k) {
            if (nd[k] < 0 || nd[k] >= n_draft || (k && nd[k] <= nd[k - 1])) return DENDRITE_EINVAL;
            mine |= nd[k] != k;
        }
        if (mine) {
            // rows move in place: the drafted blocks must be this branch's
            // own, so no fork may stand behind the base (this branch forked
            // or rolled back there, or a child forked there)
            const Node& nde = p->nodes[b.node];
            if (nde.fork_len > base) return DENDRITE_EINVAL;
            for (int32_t c = nde.first_child; c >= 0; c = p->nodes[c].next_sib)
                if (p->nodes[c].fork_len > base) return DENDRITE_EINVAL;
        }
        moves |= mine;
        new_lens[i] = base + n_keep[i];
        nd += n_keep[i];
    }
    DENDRITE_CUDA(cudaSetDevice(p->device));
    cudaStream_t s = (cudaStream_t)stream;
    DENDRITE_TRY(check_not_capturing(s));
    if (moves) {
        KeepArgs a{};
        a.n = n;
        a.bpb = p->bpb;
        a.n_kv = p->n_kv;
        a.n_blocks = (int32_t)p->num_blocks;
        a.fp8 = p->dtype == DENDRITE_FP8;
        a.words = a.fp8 ? kFp8Dim / 16 : p->head_dim * p->elt / 16;
        a.tile_bytes = (int64_t)(p->layer_bytes / p->num_blocks / p->n_kv);
        a.pool_layer = (int64_t)p->layer_bytes;
        a.table = p->d_table;
        a.kp = static_cast<char*>(p->d_k);
        a.vp = static_cast<char*>(p->d_v);
        a.meta = p->d_meta;
        const size_t words = 4 * (size_t)n + (size_t)(total + 3) / 4;
        auto fill = [&](int32_t* w) {
            int32_t acc = 0;
            w[words - 1] = 0;
            uint8_t* bytes = reinterpret_cast<uint8_t*>(w + 4 * (size_t)n);
            for (int32_t i = 0; i < n; ++i) {
                w[i] = branches[i];
                w[n + i] = p->br[branches[i]].len - n_draft;
                w[2 * (size_t)n + i] = n_keep[i];
                w[3 * (size_t)n + i] = acc;
                for (int32_t k = 0; k < n_keep[i]; ++k) bytes[acc + k] = (uint8_t)nodes[acc + k];
                acc += n_keep[i];
            }
        };
        DENDRITE_TRY(with_words(p, words, s, fill, [&](auto args) -> int {
            DENDRITE_CUDA(launch_pdl(k_keep_rows<decltype(args)>, dim3((unsigned)n, (unsigned)p->n_kv, (unsigned)p->n_layers),
                                     dim3(128), 0, s, args, a));
            return DENDRITE_OK;
        }));
    }
    return dendrite_truncate(p, branches, new_lens.data(), n, stream);
}

}  // extern "C"
