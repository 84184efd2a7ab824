// Cross attention over fp32 blocks; see attn_f32.cu.
#pragma once

#include "attn_common.cuh"

namespace dendrite {

// Rows per unit: 4, 8, 16, 32, 64 or, for head_dim <= 128 (registers and shared memory), 128.
constexpr int kF32TiledMinRows = 4, kF32TiledKernels = 6;
inline int f32_tiled_max_rows(int head_dim) { return head_dim <= 128 ? 128 : 64; }

// Shared memory attributes; resident CTAs per SM of the kernels for 4, 8, .. rows.
int attn_f32_tiled_setup(int head_dim, int (&ctas_per_sm)[kF32TiledKernels]);
inline int attn_f32_tiled_ctas(int rows, const int (&ctas_per_sm)[kF32TiledKernels]) {
    int i = 0;
    while (kF32TiledMinRows << i < rows) ++i;
    return ctas_per_sm[i];
}
int launch_attn_f32_tiled(const AttnArgs& a, cudaStream_t s);

}  // namespace dendrite
