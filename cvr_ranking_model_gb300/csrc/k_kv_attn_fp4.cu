// The paged history attention's kernels for pools of 4 bits (k_kv_attn.cuh).
#include "k_kv_attn.cuh"

namespace cvr {
KvAttendKernel kv_attend_kernel_fp4(int dtype, int head_dim, int group) {
  return head_dim == 32   ? kv::instance<32, kKv4>(dtype, group)
         : head_dim == 64 ? kv::instance<64, kKv4>(dtype, group)
                          : kv::instance<128, kKv4>(dtype, group);
}
}  // namespace cvr
