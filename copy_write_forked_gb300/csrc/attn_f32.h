// Cross attention over fp32 blocks; see attn_f32.cu.
#pragma once

#include "attn_common.cuh"

namespace dendrite {

// Rows per unit: 16, 32, 64 or, for head_dim <= 128 (registers and shared memory), 128.
constexpr int kF32TiledMinRows = 16;
inline int f32_tiled_max_rows(int head_dim) { return head_dim <= 128 ? 128 : 64; }

// Shared memory attributes; resident CTAs per SM of the kernels for 16, 32, 64 and 128 rows.
int attn_f32_tiled_setup(int head_dim, int (&ctas_per_sm)[4]);
inline int attn_f32_tiled_ctas(int rows, const int (&ctas_per_sm)[4]) {
    return ctas_per_sm[rows == 16 ? 0 : rows == 32 ? 1 : rows == 64 ? 2 : 3];
}
int launch_attn_f32_tiled(const AttnArgs& a, cudaStream_t s);

}  // namespace dendrite
