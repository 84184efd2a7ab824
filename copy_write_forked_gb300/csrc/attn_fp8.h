// Attention partial kernel over 8-bit blocks; see attn_fp8.cu.
#pragma once

#include "attn_common.cuh"

namespace dendrite {

int attn_fp8_setup(int* ctas_per_sm);   // shared memory attributes; resident CTAs per SM
// after_event: the stream's order comes from an event, not from the kernel before.
int launch_attn_fp8(const AttnArgs& a, bool after_event, cudaStream_t s);

}  // namespace dendrite
