// The attention kernels over a cache of W4_KV_BF16 elements.
#include "kv_attend.cuh"

namespace w4kv {

template <>
AttendKernel attend_kernel_for<W4_KV_BF16>(int32_t dim, int32_t group) {
  return plain_kernel_for<W4_KV_BF16>(dim, group);
}

}  // namespace w4kv
