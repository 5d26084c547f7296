// Instances of the tiled attention, bf16, heads of up to 128 columns.
#include "attn_instances.cuh"

namespace hybrid {

AttnKernels attn_bf16_128(int rows, bool three, bool low) { return attn_bf16<128>(rows, three, low); }

}  // namespace hybrid
