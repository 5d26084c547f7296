// Instances of the tiled attention, fp32, heads of up to 256 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_f32_256(int rows) { return attn_f32<256>(rows); }

}  // namespace hybrid
