// Instances of the tiled attention, bf16, heads of up to 256 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_bf16_256(int rows) { return attn_bf16<256>(rows, false, false); }

}  // namespace hybrid
