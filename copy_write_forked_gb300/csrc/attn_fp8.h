// Attention partial kernel over 8-bit blocks; see attn_fp8.cu.
#pragma once

#include "attn_common.cuh"

namespace dendrite {

int attn_fp8_setup(int* ctas_per_sm);   // shared memory attributes; resident CTAs per SM
int launch_attn_fp8(const AttnArgs& a, cudaStream_t s);

}  // namespace dendrite
