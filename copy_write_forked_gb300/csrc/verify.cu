// Verification of drafted tokens against the target's probabilities.
//
// At a node with target row p and draft row q, the children x_1, x_2, ... (each
// drawn from q by itself) are tried in order: x_k is accepted with probability
// min(1, r(x_k) / q(x_k)), and a refusal makes r the normalised max(r - q, 0).
// With r = w / S unnormalised, w = max(p - c q, 0) and S = sum w, the residual
// of w / S is max(w - S q, 0) / S = max(p - (c + S) q, 0) / S: so c, a number,
// is all that a refusal changes, and any residual of a node is made from its
// two rows in one pass.  (Certain drafts: q is 1 at the child, so w is p
// without the refused tokens.)  The first child of a node needs p and q at its
// token alone, so a path of accepted nodes touches no row until its end, where
// the next token is drawn: the least token whose running sum of w passes u S.
//
// A cluster of CTAs takes one sequence.  Its first CTA gathers the numbers of
// all nodes (one round of loads, whatever the path turns out to be) and gives
// them to the others, so that every CTA walks the tree alike; where a row's sum
// is needed, each sums its share and adds all shares in the same order.  Ranges
// are contiguous per warp: the token is found by looking for u S among the CTAs'
// sums, the warps', and a warp's lanes'.
//
// Sums decide which token a number falls to, and a vocabulary of 2^17 tokens puts
// borders 2^-17 apart: fp32 sums would move some.  They are held as pairs of
// floats (48 bits) with the error of every addition and product carried along,
// fp64 adds being 1/64 of the fp32 rate here (with fp64 in the walk and in the
// joins of the sums a pass took 12 us where it takes 5).
//
// What bounds it is the chain of a sequence's passes: the gather (two dependent
// loads), one pass over the last node's rows, and one for every second and later
// refusal at a node.  A pass that finds its rows held takes some 8,000 cycles where
// all SMs work on two CTAs (4,000 sums, 2,000 exchange between the CTAs, 2,000
// walk), 2 us alone.  32 trees of 24 nodes, 128,256 tokens in fp32, six passes in
// the longest: 44 us (33 MB that have to be read: 5 us); 256 sequences of 7 certain
// drafts, 50,257 tokens in bf16: 30 us (26 MB); one of 5 in a row, 32,000 tokens: 14 us
// (16 CTAs).  On the way there, in these cases:
//   - rows read anew in every pass, an element a load, sums joined in fp64: 97 / 93 us
//   - 16-byte words, held between passes, 16 CTAs a sequence in two waves: 55 / 79
//   - as many CTAs a sequence as fit one wave, packed fp32 pairs without fp64: 49 / 40
//   - certain drafts' sums by subtraction, only warps that lost a token anew: 47 / 36
//   - short additions of a row's own weights, below the largest of them: 45 / 31
//   - residuals added by whole two_sums (beside a probability that the draft has too they would lose digits
//     that a pair of their own holds), the largest weight taken of what is left, two bf16 at a time: 44 / 30
// Half the threads a CTA and twice the CTAs: 45 / 33, and 28 us in place of 23 where
// every sequence takes one pass.
// Draft rows that lie otherwise in their 16 bytes than the target's (vocabularies of odd sizes) are loaded
// element by element: 32 sequences of 7 drafts, 50,257 tokens, fp32 33.7 us (50,256: 32.4), bf16 32.8 (31.3).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "rows.h"

using namespace dendrite;

namespace {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32, kVerifyCluster = 16, kHeld = 8;
constexpr int kDraftSmem = kHeld * kVerifyThreads * 16;
constexpr int kTreeWordsCap = 1536;   // tree bytes as kernel parameters, four to a word

struct VerifyArgs {
    int32_t n_draft, vocab, one_tree, cluster;
    const int32_t* tokens;
    const void* target;
    const void* draft;
    int64_t target_stride, draft_stride;
    const float* accept;
    const float* sample;
    int32_t* path;
    int32_t* n_keep;
    int32_t* next;
    const DevMeta* meta;
};

// A number as the sum of two floats, h + l, with l a rounding error of h (after norm) or a sum of such.
struct alignas(8) Pair {
    float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair norm(Pair a) { return two_sum(a.h, a.l); }
__device__ __forceinline__ Pair add(Pair a, Pair b) {   // (not normal: for sums of a few)
    const Pair s = two_sum(a.h, b.h);
    return {s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ Pair product(Pair a, float b) {
    const float h = __fmul_rn(a.h, b);
    return norm({h, __fmaf_rn(a.l, b, __fmaf_rn(a.h, b, -h))});
}
__device__ __forceinline__ Pair product(Pair a, Pair b) {
    const float h = __fmul_rn(a.h, b.h);
    return norm({h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -h)))});
}
// Of normal pairs.
__device__ __forceinline__ bool less(Pair a, Pair b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }
__device__ __forceinline__ Pair of_lane(Pair x, int lane) {
    return {__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}
// Sum over 2^STEPS lanes (in every one of them).
template <int STEPS>
__device__ __forceinline__ Pair lanes_sum(Pair x) {
#pragma unroll
    for (int o = 1 << (STEPS - 1); o > 0; o >>= 1)
        x = add(x, Pair{__shfl_xor_sync(0xffffffffu, x.h, o), __shfl_xor_sync(0xffffffffu, x.l, o)});
    return norm(x);
}
// Inclusive sums over 2^STEPS lanes.
template <int STEPS>
__device__ __forceinline__ Pair lanes_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 1 << STEPS; o <<= 1) {
        const Pair y = {__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
        if (lane >= o) x = add(y, x);
    }
    return norm(x);
}

// A probability: what is not positive and finite counts as zero.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

__device__ __forceinline__ float load_prob(const float* p) { return prob(__ldg(p)); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) { return prob(__bfloat162float(__ldg(p))); }

// Two fp32 in a register pair, and their packed arithmetic (each rounded as the scalar instruction rounds).
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pack(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack(f32x2 x) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
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
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, pack(-1.f, -1.f), a); }   // a - b, rounded once
// Two sums side by side: h + l each.
struct Pair2 {
    f32x2 h, l;
};
__device__ __forceinline__ Pair2 two_sum2(f32x2 a, f32x2 b) {
    const f32x2 s = add2(a, b), t = sub2(s, a);
    return {s, add2(sub2(a, sub2(s, t)), sub2(b, t))};
}
// Adds w, of any size.
__device__ __forceinline__ void accumulate(Pair2& sum, Pair2 w) {
    const Pair2 s = two_sum2(sum.h, w.h);
    sum = {s.h, add2(sum.l, add2(s.l, w.l))};
}
// Adds w, at most sum.h in size: the short form of two_sum.
__device__ __forceinline__ void accumulate_below(Pair2& sum, f32x2 w) {
    const f32x2 s = add2(sum.h, w);
    sum = {s, add2(sum.l, add2(sub2(sum.h, s), w))};
}

// max(p - c q, 0), p and c q to 48 bits: the product's error and the difference's are carried (the latter by the
// short form for |p| >= |c q|: where that does not hold the result is zero, or the difference is exact).  What is
// left may be below the last digit of either, so the sign is that of both parts' sum; the high part may be the
// smaller one, or negative.  ONE: c is 1, and the result exact and normal.
struct Factor {
    f32x2 h, l, minus;   // c, twice each; -c.h
    __device__ __forceinline__ explicit Factor(Pair c) : h(pack(c.h, c.h)), l(pack(c.l, c.l)), minus(pack(-c.h, -c.h)) {}
};
template <bool ONE>
__device__ __forceinline__ Pair2 residual(f32x2 p, f32x2 q, const Factor& c) {
    if constexpr (ONE) {   // p - min(p, q)
        const float2 x = unpack(p), y = unpack(q);
        const f32x2 m = pack(fminf(x.x, y.x), fminf(x.y, y.y)), s = sub2(p, m);
        return {s, sub2(sub2(p, s), m)};
    } else {
        const f32x2 nph = mul2(c.minus, q), s = add2(p, nph);
        const f32x2 e = sub2(add2(sub2(p, s), nph), fma2(c.l, q, fma2(c.h, q, nph)));
        const float2 h = unpack(s), l = unpack(e), x = unpack(add2(s, e));
        return {pack(x.x > 0.f ? h.x : 0.f, x.y > 0.f ? h.y : 0.f), pack(x.x > 0.f ? l.x : 0.f, x.y > 0.f ? l.y : 0.f)};
    }
}
__device__ __forceinline__ Pair residual(float p, float q, Pair c) {
    const Pair2 w = residual<false>(pack(p, 0.f), pack(q, 0.f), Factor(c));
    return norm({unpack(w.h).x, unpack(w.l).x});
}

// A row is read in words of 16 bytes that are aligned whatever its address: element e of a row
// stands at e + skew, with skew = the elements between the aligned address below the row and the row.
template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);   // elements of a word
template <typename T>
__device__ __forceinline__ uint32_t clean(uint32_t x) {
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(prob(__uint_as_float(x)));
    } else {
        __nv_bfloat162 v;
        memcpy(&v, &x, 4);
        return x & __hgt2_mask(v, __float2bfloat162_rn(0.f)) & __hlt2_mask(v, __float2bfloat162_rn(INFINITY));
    }
}
// A word at a row's end, or of a row whose words are not aligned: element by element.
template <typename T>
__device__ __noinline__ uint4 some(const T* base, int32_t skew, int32_t vocab, int32_t e) {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            x[j] = e + j >= skew && e + j < skew + vocab ? __ldg(reinterpret_cast<const uint32_t*>(base) + e + j) : 0u;
        } else {
            const uint16_t* b = reinterpret_cast<const uint16_t*>(base);
            const int32_t f = e + 2 * j;
            const uint32_t lo = f >= skew && f < skew + vocab ? __ldg(b + f) : 0u;
            const uint32_t hi = f + 1 >= skew && f + 1 < skew + vocab ? __ldg(b + f + 1) : 0u;
            x[j] = lo | hi << 16;
        }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}
// The word at e of a row with its elements at [skew, skew + vocab), as probabilities.
template <typename T>
__device__ __forceinline__ uint4 word(const T* base, bool aligned, int32_t skew, int32_t vocab, int32_t e) {
    constexpr int PER = kPer<T>;
    return aligned && e >= skew && e + PER <= skew + vocab ? __ldg(reinterpret_cast<const uint4*>(base + e)) : some(base, skew, vocab, e);
}
template <typename T>
__device__ __forceinline__ uint4 clean(uint4 w) {
    return make_uint4(clean<T>(w.x), clean<T>(w.y), clean<T>(w.z), clean<T>(w.w));
}
// Elements 2 j, 2 j + 1 of a word.
template <typename T>
__device__ __forceinline__ f32x2 two(const uint4& w, int j) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) return pack(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
    else return pack(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
}
// The largest element of words of probabilities.
template <typename T, int N>
__device__ __forceinline__ float largest(const uint4 (&w)[N]) {
    if constexpr (sizeof(T) == 4) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(w[k].x), __uint_as_float(w[k].y)), fmaxf(__uint_as_float(w[k].z), __uint_as_float(w[k].w))));
        return top;
    } else {   // (two at a time as they are: unpacked, they would stay in registers for the sum)
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            __nv_bfloat162 x[4];
            memcpy(x, &w[k], 16);
            top = __hmax2(top, __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3])));
        }
        return fmaxf(__low2float(top), __high2float(top));
    }
}
// Takes element r of a word away, where it has one.
template <typename T>
__device__ __forceinline__ void drop(uint4& w, int32_t r) {
    if (r < 0 || r >= kPer<T>) return;
    const uint32_t keep = sizeof(T) == 4 ? 0u : r & 1 ? 0x0000ffffu : 0xffff0000u;
    const int32_t j = sizeof(T) == 4 ? r : r >> 1;
    if (j == 0) w.x &= keep;
    if (j == 1) w.y &= keep;
    if (j == 2) w.z &= keep;
    if (j == 3) w.w &= keep;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
    uint32_t y;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return y;
}
__device__ __forceinline__ void store_peer(uint32_t at, Pair x) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(x.h), "f"(x.l) : "memory");
}
__device__ __forceinline__ uint32_t load_peer(uint32_t at) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The tree as bytes, parent + 1 of each node: kernel parameters, or staged.
template <int CAP>
struct ParamTree {
    uint32_t v[CAP];
    __device__ __forceinline__ int32_t operator()(int64_t i) const { return (int32_t)(v[i >> 2] >> (8 * (int)(i & 3))) & 255; }
};
struct GlobalTree {
    const uint8_t* p;
    __device__ __forceinline__ int32_t operator()(int64_t i) const { return __ldg(p + i); }
};

// What the first CTA of a cluster found about the nodes, the same in every CTA.
struct Nodes {
    int32_t token[kMaxDraft];   // -1: no such node
    float accept[kMaxDraft], p[kMaxDraft], q[kMaxDraft];
    uint32_t real[2], first[2];   // bits of the nodes that there are, and that are accepted if they are tried first
    int32_t status;
    float sample;
};

// Where the walk of the tree stands: the current node's row, and its residual.  Warp 0's, in
// shared memory between the passes (in registers it would cost every warp's share of the row some).
struct Walk {
    Pair c, S, S_pass;           // w = max(p - c q, 0); its sum; the sum that was last taken over the row
    uint64_t refused, left;      // certain drafts: refused nodes; children to try
    uint64_t first;              // nodes that are accepted if they are tried first
    int32_t cur, kept, lost;     // lost: tokens that S went without since S_pass
    bool fresh, stale, last;     // none refused yet; S is not the sum of w; nothing is left to try
};

// Each thread holds kHeld words of the target's row in registers and as many of the draft's in shared
// memory.  A share of the row that fits them is read once, however many children of the node are refused.
template <typename T, bool DRAFT, typename A>
__global__ void __launch_bounds__(kVerifyThreads, 2) k_verify_draft(const __grid_constant__ A tree, const __grid_constant__ VerifyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint4 held_q[];   // [kHeld][threads], each thread's own
    __shared__ Nodes nodes;
    __shared__ Pair cta_sum[2][kVerifyCluster];   // every CTA's, of two passes in turn
    __shared__ Pair warp_sums[kVerifyWarps];
    __shared__ Walk walk;
    __shared__ struct {
        int32_t done, cur, again;   // again: the row has to be summed
        Pair c;
        uint64_t refused;
    } order;
    __shared__ struct {
        int32_t here, none;   // whether the token is in this CTA's share; no weight at all
        Pair before, goal;
    } find;
    const int32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int32_t cs = a.cluster, nd = a.n_draft;
    const int32_t rank = cs > 1 ? (int32_t)cluster_rank() : 0;
    const int64_t i = blockIdx.x / cs;
    const T* P = static_cast<const T*>(a.target) + i * (1 + nd) * a.target_stride;
    const T* Q = static_cast<const T*>(a.draft) + i * nd * a.draft_stride;
    // the rows that node t, and (warp 0, which walks) node 32 + t hang on
    const int32_t up = t < nd ? tree((a.one_tree ? 0 : i * nd) + t) : -1;
    const int32_t up1 = warp == 0 && 32 + lane < nd ? tree((a.one_tree ? 0 : i * nd) + 32 + lane) : -1;
    // the nodes: gathered by the first CTA, fetched by the others
    if (rank == 0) {
        if (t < kMaxDraft) {
            const int32_t x = t < nd ? __ldg(a.tokens + i * nd + t) : -1;
            const bool real = x >= 0 && x < a.vocab;
            const float u = real ? __ldg(a.accept + i * nd + t) : 0.f;
            const float p = real ? load_prob(P + up * a.target_stride + x) : 0.f;
            const float q = !real ? 0.f : DRAFT ? load_prob(Q + up * a.draft_stride + x) : 1.f;
            nodes.token[t] = real ? x : -1;
            nodes.accept[t] = u;
            nodes.p[t] = p;
            nodes.q[t] = q;
            const uint32_t all = __ballot_sync(0xffffffffu, real);
            const uint32_t first = __ballot_sync(0xffffffffu, p > 0.f && less(product(Pair{u, 0.f}, q), Pair{p, 0.f}));
            if (lane == 0) {
                nodes.real[warp] = all;
                nodes.first[warp] = first;
            }
        } else if (t == kMaxDraft) {
            nodes.status = a.meta->status;
            const float u = __ldg(a.sample + i);
            nodes.sample = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
        }
    }
    if (cs > 1) {
        cluster_arrive();
        cluster_wait();
        constexpr int words = sizeof(Nodes) / 4;
        static_assert(words <= kVerifyThreads, "a word a thread");
        if (rank && t < words) reinterpret_cast<uint32_t*>(&nodes)[t] = load_peer(peer(reinterpret_cast<const uint32_t*>(&nodes) + t, 0));
    }
    __syncthreads();
    // (the first CTA is there until the others have fetched: each waits for all once more, or leaves here)
    if (nodes.status) {
        if (cs > 1) {
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    // (before the passes' exchanges: whoever finds a token writes it after this)
    if (rank == 0 && t == 0) a.next[i] = -1;

    constexpr int PER = kPer<T>;
    uint4 hp[kHeld];
    uint4* const hq = held_q + t;
    int32_t p_row = -1, q_row = -1;   // the rows that are held, where a share fits the registers

    // the real nodes that hang on a row (warp 0)
    auto kids = [&](int32_t row) {
        const uint32_t lo = __ballot_sync(0xffffffffu, up == row) & nodes.real[0], hi = __ballot_sync(0xffffffffu, up1 == row) & nodes.real[1];
        return (uint64_t)hi << 32 | lo;
    };
    if (warp == 0) {
        const uint64_t left = kids(0);
        if (lane == 0)
            walk = Walk{{0.f, 0.f}, {1.f, 0.f}, {0.f, 0.f}, 0, left, (uint64_t)nodes.first[1] << 32 | nodes.first[0], 0, 0, 0, true, false, false};
        __syncwarp();
    }
    bool fell_back = false;
    int32_t parity = 0;
    uint64_t counted = 0;   // refused nodes whose tokens the sums are without

    for (;;) {
        if (warp == 0) {
            Walk z = walk;
            __syncwarp();
            while (!z.last && z.left && !z.stale) {
                const int32_t j = __ffsll((long long)z.left) - 1;
                z.left &= z.left - 1;
                bool ok;
                Pair w = {nodes.p[j], 0.f};
                if (z.fresh) {
                    ok = z.first >> j & 1;
                } else {
                    if (DRAFT) w = residual(nodes.p[j], nodes.q[j], z.c);
                    else
                        for (uint64_t r = z.refused; r; r &= r - 1)
                            if (nodes.token[__ffsll((long long)r) - 1] == nodes.token[j]) w.h = 0.f;
                    ok = w.h > 0.f && less(product(product(Pair{nodes.accept[j], 0.f}, nodes.q[j]), z.S), w);
                }
                if (ok) {
                    if (rank == 0 && lane == 0) a.path[i * nd + z.kept] = j;
                    ++z.kept;
                    z.cur = j + 1;
                    z.left = kids(z.cur);
                    z.c = {0.f, 0.f};
                    z.S = {1.f, 0.f};
                    z.refused = 0;
                    z.fresh = true;
                } else if (DRAFT) {
                    z.c = norm(add(z.c, z.S));
                    z.fresh = false;
                    z.stale = true;
                } else {
                    // the sum without one more token: a new one only where subtractions would lose digits (each is off
                    // by 2^-49 of the last sum at most, so S by 2^-41 of itself)
                    z.S = norm(add(z.S, Pair{-w.h, 0.f}));
                    ++z.lost;
                    z.stale = z.fresh || z.S.h < z.S_pass.h * (0x1p-8f * (float)z.lost);
                    z.refused |= 1ull << j;
                    z.fresh = false;
                }
            }
            z.last = z.last || !z.left;   // (a sum that nothing asks for is the last pass's)
            if (lane == 0) {
                walk = z;
                order.done = z.last;
                order.again = DRAFT || z.fresh || z.stale;   // (else it was, and S went on by subtraction)
                order.cur = z.cur;
                order.c = z.c;
                order.refused = z.refused;
            }
        }
        __syncthreads();
        const bool fin = order.done != 0, again = order.again || fell_back;
        const int32_t row = order.cur;
        const Pair pc = fell_back ? Pair{0.f, 0.f} : order.c;
        const uint64_t gone = fell_back ? 0 : order.refused;
        const bool with_q = DRAFT && pc.h != 0.f;
        const T* rp = P + row * a.target_stride;
        const T* rq = Q + row * a.draft_stride;
        // this warp's range of the row, in its words' numbering
        const int32_t skew = (int32_t)((uintptr_t)rp & 15) / (int32_t)sizeof(T), words = (skew + a.vocab + PER - 1) / PER;
        const int32_t share = (words + cs * kVerifyWarps - 1) / (cs * kVerifyWarps) * PER;
        const int32_t lo = min(words * PER, (rank * kVerifyWarps + warp) * share), hi = min(words * PER, lo + share);
        const bool fits = share <= 32 * PER * kHeld;
        // certain drafts: where the row was summed before, the warps that have lost a token since do it again
        uint64_t here = 0;   // tokens of this warp's range that are gone
        for (uint64_t r = gone; r; r &= r - 1) {
            const int32_t at = nodes.token[__ffsll((long long)r) - 1] + skew;
            if (at >= lo && at < hi) here |= r & (0 - r);
        }
        const bool mine = again || (here & ~counted);
        counted = gone;
        Pair2 sum2 = {0, 0};
        const Factor fc(pc);
        for (int32_t base = mine ? lo : hi; base < hi; base += 32 * PER * kHeld) {
            const int32_t e0 = base + PER * lane;
            const bool new_q = with_q && (!fits || q_row != row);
            if (new_q) {
                const T* qb = rq - skew;
                const bool aligned = ((uintptr_t)qb & 15) == 0;
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int32_t e = e0 + 32 * PER * k;
                    if (e >= hi) continue;
                    if (aligned && e >= skew && e + PER <= skew + a.vocab) copy_async(hq + k * kVerifyThreads, qb + e);
                    else hq[k * kVerifyThreads] = some(qb, skew, a.vocab, e);
                }
            }
            if (!fits || p_row != row) {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int32_t e = e0 + 32 * PER * k;
                    hp[k] = e < hi ? word(rp - skew, true, skew, a.vocab, e) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < kHeld; ++k) hp[k] = clean<T>(hp[k]);
            }
            if (new_q) copies_done();
            auto drafted = [&](auto one) {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    if (e0 + 32 * PER * k >= hi) continue;
                    uint4 q = hq[k * kVerifyThreads];
                    if (new_q) hq[k * kVerifyThreads] = q = clean<T>(q);
#pragma unroll
                    for (int j = 0; j < PER / 2; ++j) accumulate(sum2, residual<decltype(one)::value>(two<T>(hp[k], j), two<T>(q, j), fc));
                }
            };
            if (DRAFT && with_q) {
                if (pc.h == 1.f && pc.l == 0.f) drafted(std::true_type());
                else drafted(std::false_type());
                sum2 = two_sum2(sum2.h, sum2.l);
            } else {
                for (uint64_t r = here; r; r &= r - 1) {
                    const int32_t at = nodes.token[__ffsll((long long)r) - 1] + skew - e0;
#pragma unroll
                    for (int k = 0; k < kHeld; ++k) drop<T>(hp[k], at - 32 * PER * k);
                }
                // The sum stands above the largest weight meanwhile, so that each addition is the short form.  Not the
                // largest probability: the sum's last digits are as far below what it stands on as a pair's are.
                const float top = largest<T>(hp);
                const Pair2 up2 = two_sum2(sum2.h, pack(top, top));
                sum2 = {up2.h, add2(sum2.l, up2.l)};
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    if (e0 + 32 * PER * k >= hi) continue;
#pragma unroll
                    for (int j = 0; j < PER / 2; ++j) accumulate_below(sum2, two<T>(hp[k], j));
                }
                const Pair2 down = two_sum2(sum2.h, pack(-top, -top));
                sum2 = two_sum2(down.h, add2(sum2.l, down.l));
            }
        }
        if (mine) p_row = row;   // (of one node more tokens may go, none come back)
        if (with_q) q_row = row;
        const float2 sh = unpack(sum2.h), sl = unpack(sum2.l);
        const Pair sum = lanes_sum<5>(add(Pair{sh.x, sl.x}, Pair{sh.y, sl.y}));
        if (mine && lane == 0) warp_sums[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const Pair x = lanes_sum<4>(warp_sums[lane & (kVerifyWarps - 1)]);
            if (lane < cs) store_peer(peer(&cta_sum[parity][rank], lane), x);
        }
        if (cs > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        // every CTA's sum, added in the same order in every CTA
        if (warp == 0) {
            const Pair own = lane < cs ? cta_sum[parity][lane] : Pair{0.f, 0.f}, incl = lanes_scan<4>(own, lane);
            const Pair S = of_lane(incl, 15);
            if (lane == 0) {
                walk.S = walk.S_pass = S;
                walk.stale = false;
                walk.lost = 0;
            }
            if (fin) {
                Pair goal = product(S, nodes.sample);
                // (of the least numbers a part rounds to the whole, which no token would pass; S.l is zero there)
                if (S.h > 0.f && !less(goal, S)) goal = {__uint_as_float(__float_as_uint(S.h) - 1), 0.f};
                // The CTA: of those with weight the first whose end passes the goal, or the last.  (Ends are rounded, each
                // in an order of its own, so one may lie behind the next: two CTAs could hold the goal between theirs, or
                // one without weight.)
                const uint32_t with = __ballot_sync(0xffffffffu, own.h > 0.f);
                const uint32_t past = __ballot_sync(0xffffffffu, own.h > 0.f && less(goal, incl));
                const Pair before = of_lane(incl, max(rank - 1, 0));
                if (lane == 0) {
                    find.goal = goal;
                    find.before = rank ? before : Pair{0.f, 0.f};
                    find.here = rank == (past ? __ffs(past) - 1 : 31 - __clz(with));
                    find.none = !(S.h > 0.f);
                }
            }
            __syncwarp();
        }
        parity ^= 1;
        if (!fin) continue;
        __syncthreads();
        if (find.none) {
            if (fell_back || (!with_q && !gone)) break;   // p has no weight
            fell_back = true;
            p_row = -1;
            __syncthreads();
            continue;
        }
        if (!find.here) break;
        // the warp, then the lanes' runs, then the token
        const Pair ws = lane < kVerifyWarps ? warp_sums[lane] : Pair{0.f, 0.f}, wi = lanes_scan<4>(ws, lane);
        const Pair goal = find.goal, start = find.before;
        const uint32_t with = __ballot_sync(0xffffffffu, ws.h > 0.f);
        const uint32_t past = __ballot_sync(0xffffffffu, ws.h > 0.f && less(goal, norm(add(start, wi))));
        // (rounding apart, some warp's end is past the goal)
        if (warp != (past ? __ffs(past) - 1 : 31 - __clz(with))) break;
        const Pair from = warp ? norm(add(start, of_lane(wi, warp - 1))) : start;
        const int32_t run = ((hi - lo) / PER + 31) / 32 * PER, r0 = min(hi, lo + lane * run), r1 = min(hi, r0 + run);
        constexpr int U = 8;
        auto weights = [&](int32_t e, Pair (&w)[U]) {   // of the U elements from e on, in the words' numbering
            float p[U], q[U];
            const int32_t r = e - skew;
#pragma unroll
            for (int u = 0; u < U; ++u) p[u] = e + u < r1 && r + u >= 0 && r + u < a.vocab ? load_prob(rp + r + u) : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                q[u] = with_q && e + u < r1 && r + u >= 0 && r + u < a.vocab ? load_prob(rq + r + u) : 0.f;
            for (uint64_t g = here; g; g &= g - 1) {
                const int32_t x = nodes.token[__ffsll((long long)g) - 1];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u == x) p[u] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; u += 2) {
                Pair2 x = {pack(p[u], p[u + 1]), 0};
                if (with_q) x = residual<false>(x.h, pack(q[u], q[u + 1]), fc);
                const float2 h = unpack(x.h), l = unpack(x.l);
                w[u] = norm({h.x, l.x});
                w[u + 1] = norm({h.y, l.y});
            }
        };
        Pair x = {0.f, 0.f}, w[U];
        for (int32_t e = r0; e < r1; e += U) {
            weights(e, w);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Pair s = two_sum(x.h, w[u].h);
                x = {s.h, __fadd_rn(x.l, __fadd_rn(s.l, w[u].l))};
            }
            x = norm(x);
        }
        const Pair incl = lanes_scan<5>(x, lane);
        // the first lane whose end passes the goal, or the last one with weight
        const uint32_t has = __ballot_sync(0xffffffffu, x.h > 0.f);
        const uint32_t over = __ballot_sync(0xffffffffu, x.h > 0.f && less(goal, norm(add(from, incl))));
        const int32_t pick = over ? __ffs(over) - 1 : 31 - __clz(has);
        const Pair ahead = of_lane(incl, max(pick - 1, 0));
        if (lane == pick) {
            Pair s = pick ? add(from, ahead) : from;
            int32_t token = -1;
            bool found = false;
            for (int32_t e = r0; e < r1 && !found; e += U) {
                weights(e, w);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (found || !(w[u].h > 0.f)) continue;
                    s = norm(add(s, w[u]));
                    token = e + u - skew;
                    found = less(goal, s);
                }
            }
            a.next[i] = token;
        }
        break;
    }
    // (the loop ends after the last exchange of every CTA: none writes to another any more)
    if (rank == 0 && warp == 0) {
        const int32_t kept = walk.kept;
        for (int32_t j = kept + lane; j < nd; j += 32) a.path[i * nd + j] = -1;
        if (lane == 0) a.n_keep[i] = kept;
    }
}

// CTAs per sequence: as many as are resident at once (two an SM), more than 1,024 tokens each.
int verify_cluster(const dendrite_pool* p, int32_t n, int32_t vocab) {
    int cs = 1;
    while (cs < kVerifyCluster && (int64_t)n * cs <= p->sm_count && vocab > 2048 * cs) cs *= 2;
    return cs;
}

template <typename T, typename A>
int launch_verify(const A& tree, const VerifyArgs& a, int32_t n, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)n * a.cluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = a.draft ? kDraftSmem : 0;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    auto go = [&](auto* fn) -> int {
        DENDRITE_CUDA(cudaLaunchKernelEx(&cfg, fn, tree, a));
        return DENDRITE_OK;
    };
    return a.draft ? go(k_verify_draft<T, true, A>) : go(k_verify_draft<T, false, A>);
}

// More than 8 CTAs a cluster, and the shared memory, have to be asked for.
template <typename T, typename A>
int setup_one() {
    auto allow = [](auto* fn, bool draft) -> int {
        DENDRITE_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
        if (draft) DENDRITE_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kDraftSmem));
        return DENDRITE_OK;
    };
    DENDRITE_TRY(allow(k_verify_draft<T, true, A>, true));
    return allow(k_verify_draft<T, false, A>, false);
}
template <typename A>
int setup_types() {
    DENDRITE_TRY((setup_one<float, A>()));
    return setup_one<__nv_bfloat16, A>();
}

struct Span {
    uintptr_t at, end;
};

}  // namespace

namespace dendrite {

int verify_setup() {
    DENDRITE_TRY(setup_types<ParamTree<64>>());
    DENDRITE_TRY(setup_types<ParamTree<kTreeWordsCap>>());
    return setup_types<GlobalTree>();
}

}  // namespace dendrite

extern "C" int dendrite_verify_draft(dendrite_pool* p, int32_t n, int32_t n_draft, const int32_t* parents, int32_t n_trees,
                                     const int32_t* tokens, int32_t vocab, int32_t dtype, const void* target,
                                     int64_t target_stride, const void* draft, int64_t draft_stride, const float* accept,
                                     const float* sample, int32_t* path, int32_t* n_keep, int32_t* next, void* stream) {
    if (!p) return DENDRITE_EINVAL;
    if (p->poisoned) return p->poisoned;
    if (dtype != DENDRITE_FP32 && dtype != DENDRITE_BF16) return DENDRITE_EDTYPE;
    if (n < 0 || vocab < 1) return DENDRITE_EINVAL;
    if (n == 0) return DENDRITE_OK;
    DENDRITE_TRY(check_trees(parents, n_trees, n, n_draft));
    if (!tokens || !target || !accept || !sample || !path || !n_keep || !next) return DENDRITE_EINVAL;
    const uintptr_t e = dtype == DENDRITE_FP32 ? 4 : 2;
    if (((uintptr_t)tokens | (uintptr_t)accept | (uintptr_t)sample | (uintptr_t)path | (uintptr_t)n_keep | (uintptr_t)next) & 3)
        return DENDRITE_EINVAL;
    if (((uintptr_t)target | (uintptr_t)draft) & (e - 1)) return DENDRITE_EINVAL;
    constexpr int64_t kMost = (int64_t)1 << 30;
    if (vocab > kMost) return DENDRITE_ELIMIT;
    if (target_stride < vocab || (draft && draft_stride < vocab)) return DENDRITE_EINVAL;
    if (target_stride > kMost || (draft && draft_stride > kMost)) return DENDRITE_ELIMIT;
    if ((int64_t)n * (1 + n_draft) > INT32_MAX) return DENDRITE_ELIMIT;
    // the outputs: apart from one another and from everything that is read
    const uintptr_t u = n, d = (uintptr_t)n * n_draft;
    auto span = [](const void* x, uintptr_t bytes) { return Span{(uintptr_t)x, (uintptr_t)x + bytes}; };
    const Span outs[3] = {span(path, 4 * d), span(n_keep, 4 * u), span(next, 4 * u)};
    const Span ins[5] = {span(tokens, 4 * d), span(accept, 4 * d), span(sample, 4 * u),
                         span(target, ((u + d - 1) * target_stride + vocab) * e),
                         span(draft, draft ? ((d - 1) * draft_stride + vocab) * e : 0)};
    for (int k = 0; k < 3; ++k) {
        for (const Span& x : ins)
            if (x.at < outs[k].end && outs[k].at < x.end) return DENDRITE_EINVAL;
        for (int m = 0; m < k; ++m)
            if (outs[m].at < outs[k].end && outs[k].at < outs[m].end) return DENDRITE_EINVAL;
    }
    DENDRITE_CUDA(cudaSetDevice(p->device));
    cudaStream_t s = (cudaStream_t)stream;
    DENDRITE_TRY(check_not_capturing(s));
    VerifyArgs a{};
    a.n_draft = n_draft;
    a.vocab = vocab;
    a.one_tree = n_trees == 1;
    a.cluster = verify_cluster(p, n, vocab);
    a.tokens = tokens;
    a.target = target;
    a.draft = draft;
    a.target_stride = target_stride;
    a.draft_stride = draft_stride;
    a.accept = accept;
    a.sample = sample;
    a.path = path;
    a.n_keep = n_keep;
    a.next = next;
    a.meta = p->d_meta;
    const size_t bytes = (size_t)n_trees * n_draft, words = (bytes + 3) / 4;
    auto fill = [&](uint8_t* to) {
        for (size_t k = 0; k < bytes; ++k) to[k] = (uint8_t)(parents[k] + 1);
    };
    auto go = [&](const auto& tree) {
        return dtype == DENDRITE_FP32 ? launch_verify<float>(tree, a, n, s) : launch_verify<__nv_bfloat16>(tree, a, n, s);
    };
    if (words <= 64) {
        ParamTree<64> tree{};
        fill(reinterpret_cast<uint8_t*>(tree.v));
        return go(tree);
    }
    if (words <= (size_t)kTreeWordsCap) {
        ParamTree<kTreeWordsCap> tree{};
        fill(reinterpret_cast<uint8_t*>(tree.v));
        return go(tree);
    }
    char *h, *dv;
    DENDRITE_TRY(p->staging.reserve(bytes, &h, &dv));
    fill(reinterpret_cast<uint8_t*>(h));
    DENDRITE_TRY(p->staging.upload(s, h, bytes));
    DENDRITE_TRY(go(GlobalTree{reinterpret_cast<const uint8_t*>(dv)}));
    return p->staging.release(s);
}
