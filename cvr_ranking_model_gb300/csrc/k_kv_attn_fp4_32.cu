// The paged history attention's kernels for rows of 32 values in 4 bits (k_kv_attn.cuh).
#include "k_kv_attn.cuh"

namespace cvr {
KvAttendKernel kv_attend_kernel_fp4_32(int dtype, int group) { return kv::instance<32, kKv4>(dtype, group); }
}  // namespace cvr
