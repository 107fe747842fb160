// The paged history attention's kernels for rows of 64 values (k_kv_attn.cuh).
#include "k_kv_attn.cuh"

namespace cvr {
KvAttendKernel kv_attend_kernel_64(int dtype, bool int8, int group) {
  return int8 ? kv::instance<64, kKv8>(dtype, group) : kv::instance<64, kKv16>(dtype, group);
}
}  // namespace cvr
