// Rows into and out of the blocks: appends that rotate (rotary positions) or
// quantise (8-bit pools), gathers of stored rows, and the moves that keep an
// accepted draft path; see rows.cu.
#pragma once

#include "dendrite_internal.h"

namespace dendrite {

// 8-bit pools: a (block, kv head) tile is 16 rows of 128 e4m3 codes, the
// 16-byte chunk c of slot s at chunk c ^ (s & 7) (so that the attention
// kernel's loads of eight slots fall in distinct banks), then one exponent
// byte per slot: value = code * 2^(byte - 127), byte 1..247; 255: a row of NaN.
// A slot never written holds byte 0 and codes 0.
constexpr int kFp8Dim = 128;
constexpr int kFp8TileBytes = kBlockSize * kFp8Dim + kBlockSize;
constexpr int kMaxDraft = 64;   // drafted tokens per branch: one mask bit each

// The rows of an append (device pointers; layer y of the input starts y *
// kv_layer / q_layer elements after layer 0).
struct RowsCall {
    const int32_t* branches;
    const int32_t* lens;       // lengths before the append
    int32_t n, n_new;
    int64_t touched;           // (branch, block) pairs the rows land in
    const void* K;
    const void* V;
    const void* Q;             // null: no queries
    void* q_out;
    int32_t n_q_heads;
    int32_t layer0, n_layers_in;
    int64_t kv_layer, q_layer;
    const dendrite_rope* rope; // null: rows are stored as they are
    const uint8_t* depth;      // [n_trees][n_new] draft tree depths; null: token j is at length + j
    int32_t n_trees;
    const dendrite_positions* at;   // positions given with the rows; null: by length (and depth)
};

// The kernel's argument words: how many the caller has to stage (0: they go as
// kernel parameters), the words themselves, and the launch (staged: their device
// copy, or null where none are staged).
size_t staged_rows_words(const RowsCall& c);
void fill_rows_words(const RowsCall& c, int32_t block_size, int32_t* words);
int launch_append_rows(dendrite_pool* p, const RowsCall& c, const int32_t* staged, cudaStream_t s);

// Children forked onto selected rows (one launch; see k_fork_rows).  Child i
// shares the parent's first starts[i] / 16 blocks and owns the rows from there
// to its length starts[i] + counts[i].
struct ForkRows {
    const int32_t *parents, *starts, *counts, *children;
    int32_t n;
    const int32_t* rows;   // device: [sum counts], or [n_layers][sum counts][n_kv] where per_head
    bool per_head;
    int64_t total;         // sum counts
    int64_t blocks;        // blocks taken off the free stack
    int64_t items;         // (child, owned block) pairs and chunks of shared entries
};
constexpr int32_t kShareChunk = 256;   // shared table entries an item copies
int launch_fork_rows(dendrite_pool* p, const ForkRows& c, cudaStream_t s);

// Checks n_trees (1 or n) trees of t drafted tokens (parents[j] in [-1, j)).
int check_trees(const int32_t* parents, int32_t n_trees, int32_t n, int32_t t);
// Each node's depth (0 for a child of the last accepted token).
void tree_depths(const int32_t* parents, int32_t n_trees, int32_t t, std::vector<uint8_t>& depth);

// DENDRITE_EINVAL while the stream is being captured into a graph.
int check_not_capturing(cudaStream_t s);

}  // namespace dendrite
