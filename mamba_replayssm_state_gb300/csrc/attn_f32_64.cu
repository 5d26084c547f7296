// Instances of the tiled attention, fp32, heads of up to 64 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_f32_64(int rows) { return attn_f32<64>(rows); }

}  // namespace hybrid
