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
// fp64 adds being 1/64 of the fp32 rate here.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "rows.h"

using namespace dendrite;

namespace {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32, kVerifyCluster = 8;
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

// A sum of two floats, hi + lo.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.h, b.h);
    return two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
// Inclusive sums over the lanes.
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = {__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
        if (lane >= o) x = add(y, x);
    }
    return x;
}
__device__ __forceinline__ Pair lane_of(Pair x, int lane) {
    return {__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}
__device__ __forceinline__ double value(Pair a) { return (double)a.h + (double)a.l; }
__device__ __forceinline__ Pair pair_of(double x) {
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = add(x, Pair{__shfl_xor_sync(0xffffffffu, x.h, o), __shfl_xor_sync(0xffffffffu, x.l, o)});
    return x;
}

// A probability: what is not positive and finite counts as zero.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }
__device__ __forceinline__ float load_prob(const float* p) { return prob(__ldg(p)); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) { return prob(__bfloat162float(__ldg(p))); }

// max(p - c q, 0) to 48 bits: the product's and the difference's errors carried.
__device__ __forceinline__ Pair residual(float p, float q, Pair c) {
    const float ph = __fmul_rn(c.h, q);
    const float pl = __fmaf_rn(c.l, q, __fmaf_rn(c.h, q, -ph));
    Pair d = two_sum(p, -ph);
    d.l = __fsub_rn(d.l, pl);
    return __fadd_rn(d.h, d.l) > 0.f ? d : Pair{0.f, 0.f};
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
__device__ __forceinline__ void store_peer(uint32_t at, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

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
    int32_t status;
    int32_t token[kMaxDraft];   // -1: no such node
    float accept[kMaxDraft], p[kMaxDraft], q[kMaxDraft];
    float sample;
};

// A node's weights: max(p - c q, 0), or p without the refused nodes' tokens.
template <typename T>
struct Weights {
    const T* p;
    const T* q;          // null: c is zero
    Pair c;
    uint64_t refused;    // certain drafts: nodes whose tokens are gone
};

template <typename T, bool DRAFT, typename A>
__global__ void __launch_bounds__(kVerifyThreads, 2) k_verify_draft(const __grid_constant__ A tree, const __grid_constant__ VerifyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ Nodes nodes;
    __shared__ int32_t up[kMaxDraft];
    __shared__ uint32_t kids[kMaxDraft + 1][2];
    __shared__ Pair cta_sum[2][kVerifyCluster];   // every CTA's, of two passes in turn
    __shared__ Pair warp_sums[kVerifyWarps];
    __shared__ struct {
        int32_t done, cur;
        Pair c;
        uint64_t refused;
    } order;
    __shared__ struct {
        int32_t here, none;   // whether the token is in this CTA's share; no weight at all
        double before, goal;
    } find;
    const int32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int32_t cs = a.cluster, nd = a.n_draft;
    const int32_t rank = cs > 1 ? (int32_t)cluster_rank() : 0;
    const int64_t i = blockIdx.x / cs;
    const T* P = static_cast<const T*>(a.target) + i * (1 + nd) * a.target_stride;
    const T* Q = static_cast<const T*>(a.draft) + i * nd * a.draft_stride;
    if (cs > 1) cluster_arrive();   // (the others have to have begun before their memory is written)
    // the nodes: gathered by the first CTA, given to the others
    if (t < 2 * (kMaxDraft + 1)) kids[t >> 1][t & 1] = 0;
    if (t < nd) up[t] = tree((a.one_tree ? 0 : i * nd) + t);
    if (rank == 0) {
        if (t < nd) {
            const int32_t x = __ldg(a.tokens + i * nd + t);
            const bool real = x >= 0 && x < a.vocab;
            nodes.token[t] = real ? x : -1;
            nodes.accept[t] = __ldg(a.accept + i * nd + t);
            nodes.p[t] = real ? load_prob(P + up[t] * a.target_stride + x) : 0.f;
            nodes.q[t] = !real ? 0.f : DRAFT ? load_prob(Q + up[t] * a.draft_stride + x) : 1.f;
        } else if (t == kMaxDraft) {
            nodes.status = a.meta->status;
            const float u = __ldg(a.sample + i);
            nodes.sample = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
        }
    }
    if (cs > 1) {
        cluster_wait();
        __syncthreads();
        if (rank == 0) {
            constexpr int words = sizeof(Nodes) / 4;
            for (int32_t e = t; e < words * (cs - 1); e += kVerifyThreads) {
                const int32_t to = e / words + 1, w = e % words;
                store_peer(peer(reinterpret_cast<const uint32_t*>(&nodes) + w, to), reinterpret_cast<const uint32_t*>(&nodes)[w]);
            }
        }
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (nodes.status) return;   // (all CTAs of the cluster alike)
    if (t < nd && nodes.token[t] >= 0) atomicOr(&kids[up[t]][t >> 5], 1u << (t & 31));
    __syncthreads();

    // this warp's range of every row
    const int32_t share = ((a.vocab + cs * kVerifyWarps - 1) / (cs * kVerifyWarps) + 31) & ~31;
    const int32_t lo = min(a.vocab, (rank * kVerifyWarps + warp) * share), hi = min(a.vocab, lo + share);

    // the walk (warp 0): state of the current node
    int32_t cur = 0, kept = 0, parity = 0;   // cur: row of the current node
    double c = 0.0, S = 1.0;
    bool stale = false;                      // S is not the sum of w yet
    uint64_t refused = 0, left = 0;          // certain drafts: refused nodes; children to try
    if (warp == 0) left = (uint64_t)kids[0][1] << 32 | kids[0][0];
    bool fresh = true;                       // the node has refused none
    bool last = false, fell_back = false;

    for (;;) {
        if (warp == 0) {
            bool pass = false;
            while (!last && left && !pass) {
                const int32_t j = __ffsll((long long)left) - 1;
                if (stale) {   // the sum first
                    pass = true;
                    break;
                }
                left &= left - 1;
                double w = nodes.p[j], asked = (double)nodes.accept[j];
                if (DRAFT) {
                    if (!fresh) w = fmax(w - c * (double)nodes.q[j], 0.0);
                    asked *= (double)nodes.q[j];
                    if (!fresh) asked *= S;
                } else {
                    for (uint64_t r = refused; r; r &= r - 1)
                        if (nodes.token[__ffsll((long long)r) - 1] == nodes.token[j]) w = 0.0;
                    if (!fresh) asked *= S;
                }
                if (w > 0.0 && asked < w) {
                    if (rank == 0 && lane == 0) a.path[i * nd + kept] = j;
                    ++kept;
                    cur = j + 1;
                    left = (uint64_t)kids[cur][1] << 32 | kids[cur][0];
                    c = 0.0;
                    S = 1.0;
                    refused = 0;
                    fresh = true;
                } else {
                    if (DRAFT) c += S;
                    else refused |= 1ull << j;
                    fresh = false;
                    stale = true;
                }
            }
            if (!pass) last = true;
            if (lane == 0) {
                order.done = last;
                order.cur = cur;
                order.c = pair_of(c);
                order.refused = refused;
            }
        }
        __syncthreads();
        const bool fin = order.done != 0;
        Weights<T> W;
        W.p = P + order.cur * a.target_stride;
        W.c = order.c;
        W.q = DRAFT && W.c.h != 0.f ? Q + order.cur * a.draft_stride : nullptr;
        W.refused = order.refused;
        if (fell_back) {
            W.q = nullptr;
            W.refused = 0;
        }
        // refused tokens in this warp's range
        uint64_t mine = 0;
        if (!DRAFT)
            for (uint64_t r = W.refused; r; r &= r - 1) {
                const int32_t x = nodes.token[__ffsll((long long)r) - 1];
                if (x >= lo && x < hi) mine |= r & (0 - r);
            }
        Pair sum = {0.f, 0.f};
        constexpr int U = 8;
        for (int32_t e0 = lo + lane; e0 < hi; e0 += 32 * U) {
            float p[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) p[u] = e0 + 32 * u < hi ? load_prob(W.p + e0 + 32 * u) : 0.f;
            if (DRAFT && W.q) {
#pragma unroll
                for (int u = 0; u < U; ++u) q[u] = e0 + 32 * u < hi ? load_prob(W.q + e0 + 32 * u) : 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Pair w = residual(p[u], q[u], W.c), s = two_sum(sum.h, w.h);
                    sum = {s.h, __fadd_rn(sum.l, __fadd_rn(s.l, w.l))};
                }
            } else {
                if (!DRAFT)
                    for (uint64_t r = mine; r; r &= r - 1) {
                        const int32_t x = nodes.token[__ffsll((long long)r) - 1];
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (e0 + 32 * u == x) p[u] = 0.f;
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Pair s = two_sum(sum.h, p[u]);
                    sum = {s.h, __fadd_rn(sum.l, s.l)};
                }
            }
        }
        sum = warp_sum(two_sum(sum.h, sum.l));
        if (lane == 0) warp_sums[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            Pair x = lane < kVerifyWarps ? warp_sums[lane] : Pair{0.f, 0.f};
            x = warp_sum(x);
            if (lane < cs) {
                const uint32_t at = peer(&cta_sum[parity][rank], lane);
                store_peer(at, __float_as_uint(x.h));
                store_peer(at + 4, __float_as_uint(x.l));
            }
        }
        if (cs > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        // every CTA's sum, added in the same order in every CTA (fp64 by one warp alone)
        if (warp == 0) {
            const Pair incl = warp_scan(lane < cs ? cta_sum[parity][lane] : Pair{0.f, 0.f}, lane);
            S = value(lane_of(incl, 31));
            stale = false;
            const Pair before = lane_of(incl, max(rank - 1, 0)), upto = lane_of(incl, rank);
            if (fin && lane == 0) {
                find.goal = (double)nodes.sample * S;
                find.before = rank ? value(before) : 0.0;
                find.here = find.goal >= find.before && find.goal < value(upto);
                find.none = !(S > 0.0);
            }
        }
        parity ^= 1;
        if (!fin) continue;
        __syncthreads();
        if (find.none) {
            if (fell_back || (!W.q && !W.refused)) {   // p has no weight
                if (rank == 0 && t == 0) a.next[i] = -1;
                break;
            }
            fell_back = true;
            __syncthreads();
            continue;
        }
        if (!find.here) break;
        // the warp, then the lanes' runs, then the token
        const Pair ws = lane < kVerifyWarps ? warp_sums[lane] : Pair{0.f, 0.f}, wi = warp_scan(ws, lane);
        const double goal = find.goal;
        const uint32_t with = __ballot_sync(0xffffffffu, ws.h > 0.f);
        const uint32_t past = __ballot_sync(0xffffffffu, ws.h > 0.f && goal < find.before + value(wi));
        // (rounding apart, some warp's end is past the goal)
        if (warp != (past ? __ffs(past) - 1 : 31 - __clz(with))) break;
        const double from = find.before + (warp ? value(lane_of(wi, warp - 1)) : 0.0);
        const int32_t run = (hi - lo + 31) / 32, r0 = min(hi, lo + lane * run), r1 = min(hi, r0 + run);
        auto weight = [&](int32_t e) {
            const float p = load_prob(W.p + e);
            if (W.q) return residual(p, load_prob(W.q + e), W.c);
            for (uint64_t r = mine; r; r &= r - 1)
                if (nodes.token[__ffsll((long long)r) - 1] == e) return Pair{0.f, 0.f};
            return Pair{p, 0.f};
        };
        Pair x = {0.f, 0.f};
        for (int32_t e = r0; e < r1; ++e) x = add(x, weight(e));
        const Pair incl = warp_scan(x, lane);
        // the first lane whose end passes the goal, or the last one with weight
        const uint32_t has = __ballot_sync(0xffffffffu, x.h > 0.f);
        const uint32_t over = __ballot_sync(0xffffffffu, x.h > 0.f && goal < from + value(incl));
        const int32_t pick = over ? __ffs(over) - 1 : 31 - __clz(has);
        if (lane == pick) {
            const double base = from + (value(incl) - value(x));
            Pair s = {0.f, 0.f};
            int32_t token = -1;
            for (int32_t e = r0; e < r1; ++e) {
                const Pair w = weight(e);
                if (!(w.h > 0.f)) continue;
                s = add(s, w);
                token = e;
                if (goal < base + value(s)) break;
            }
            a.next[i] = token;
        }
        break;
    }
    // (the loop ends after the last exchange of every CTA: none writes to another any more)
    if (rank == 0 && warp == 0) {
        for (int32_t j = kept + lane; j < nd; j += 32) a.path[i * nd + j] = -1;
        if (lane == 0) a.n_keep[i] = kept;
    }
}

// CTAs per sequence: enough for two CTAs an SM, at least 4,096 tokens each.
int verify_cluster(const dendrite_pool* p, int32_t n, int32_t vocab) {
    int cs = 1;
    while (cs < kVerifyCluster && (int64_t)n * cs < 2 * (int64_t)p->sm_count && vocab > 4096 * cs) cs *= 2;
    return cs;
}

template <typename T, typename A>
int launch_verify(const A& tree, const VerifyArgs& a, int32_t n, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)n * a.cluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (a.draft) DENDRITE_CUDA(cudaLaunchKernelEx(&cfg, k_verify_draft<T, true, A>, tree, a));
    else DENDRITE_CUDA(cudaLaunchKernelEx(&cfg, k_verify_draft<T, false, A>, tree, a));
    return DENDRITE_OK;
}

struct Span {
    uintptr_t at, end;
};

}  // namespace

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
