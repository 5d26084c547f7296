// Instances of the tiled attention, bf16, heads of up to 128 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_bf16_128(int rows, bool three) { return attn_bf16<128>(rows, three); }

}  // namespace hybrid
