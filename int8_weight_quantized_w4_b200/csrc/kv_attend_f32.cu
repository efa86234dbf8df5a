// The attention kernels over a cache of W4_KV_F32 elements.
#include "kv_attend.cuh"

namespace w4kv {

template <>
AttendKernel attend_kernel_for<W4_KV_F32>(int32_t dim, int32_t group, bool) {
  return plain_kernel_for<W4_KV_F32>(dim, group);
}

}  // namespace w4kv
