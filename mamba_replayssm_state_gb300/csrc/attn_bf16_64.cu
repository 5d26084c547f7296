// Instances of the tiled attention, bf16, heads of up to 64 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_bf16_64(int rows, bool low) { return attn_bf16<64>(rows, rows <= 16, low); }

}  // namespace hybrid
