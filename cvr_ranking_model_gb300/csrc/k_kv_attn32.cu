// The paged history attention's kernels for rows of 32 values (k_kv_attn.cuh).
#include "k_kv_attn.cuh"

namespace cvr {
KvAttendKernel kv_attend_kernel_32(int dtype, bool int8, int group) { return kv::instance<32>(dtype, int8, group); }
}  // namespace cvr
