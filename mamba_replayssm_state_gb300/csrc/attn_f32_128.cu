// Instances of the tiled attention, fp32, heads of up to 128 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_f32_128(int rows) { return attn_f32<128>(rows); }

}  // namespace hybrid
