// The attention kernels over a cache of W4_KV_F16 elements.
#include "kv_attend_mma.cuh"

namespace w4kv {

template <>
AttendKernel attend_kernel_for<W4_KV_F16>(int32_t dim, int32_t group, bool brief) {
  if (group >= least_group(dim) && !brief) return matrix_kernel_for<W4_KV_F16, 8>(dim);
  return plain_kernel_for<W4_KV_F16>(dim, group);
}

}  // namespace w4kv
