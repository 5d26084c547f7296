// Instances of the tensor-core prompt kernel.
#include "ssm_tc_kernel.cuh"

namespace ssm {

const void* tc_kernel(int heads, bool lo) {
  if (heads == 2)
    return lo ? reinterpret_cast<const void*>(&ssm_tc_kernel<2, true>) : reinterpret_cast<const void*>(&ssm_tc_kernel<2, false>);
  return lo ? reinterpret_cast<const void*>(&ssm_tc_kernel<1, true>) : reinterpret_cast<const void*>(&ssm_tc_kernel<1, false>);
}

const void* join_kernel() { return reinterpret_cast<const void*>(&ssm_join_kernel); }

}  // namespace ssm
