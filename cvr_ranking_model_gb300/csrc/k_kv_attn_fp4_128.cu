// The paged history attention's kernels for rows of 128 values in 4 bits (k_kv_attn.cuh).
#include "k_kv_attn.cuh"

namespace cvr {
KvAttendKernel kv_attend_kernel_fp4_128(int dtype, int group) { return kv::instance<128, kKv4>(dtype, group); }
}  // namespace cvr
